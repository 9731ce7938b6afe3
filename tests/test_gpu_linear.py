"""GPU parity of the grouped linear operators against their formulas in 64 bits, over
ragged groups, every activation, odd sizes, and the ways a program calls them."""
import pytest
import torch

import linear_reference as R
import sparse_mixture_experts_26_b200 as moe

pytestmark = pytest.mark.gpu
bf, f32 = torch.bfloat16, torch.float32

# group sizes, K, N: one row, empty experts, one past a tile, long ragged groups, every
# switch between the kernels, K and N that end inside a tile
SHAPES = [
    ((1,), 8, 8), ((0, 1, 0), 64, 40), ((1, 1, 0, 2), 4096, 264), ((3, 0, 5, 16), 136, 200),
    ((17, 31, 0, 1, 8, 0, 0, 9), 256, 384), ((16,) * 8, 520, 1000), ((33, 65), 72, 2056),
    ((128, 129, 127), 512, 256), ((257, 1, 300, 0), 192, 328), ((500,), 4104, 136),
    ((700, 13, 0, 311), 264, 520), ((1025,), 64, 72), ((2, 3, 1) * 10 + (4, 0), 128, 96),
    ((1500, 0, 600), 328, 712), ((300, 280, 290, 310), 1032, 640), ((4097,), 200, 264),
    # reductions cut into many shares, for few tokens and for many
    ((5, 0, 3), 20000, 40), ((100,), 8192, 264), ((250, 6), 5000, 136), ((1496,), 5144, 192),
]


def ids(s):
    return "x".join(map(str, (sum(s[0]), len(s[0])) + s[1:]))


def check_y(y, t, counts, K, name, n):
    z, mag = R.grouped_z(t["x"], t["W"], t["bias"], counts)
    ref = R.act(z, name)
    tol = R.SLOPE_MAX * R.accumulation(K) * mag + R.ACT_ERR * (1 + z.abs())
    if t["residual"] is not None:
        ref = ref + t["residual"][:n].double()
        tol = tol + 2.0 ** -23 * ref.abs()
    u = R.U_BF16 if y.dtype == bf else 2.0 ** -24
    tol = tol + u * (ref.abs() + tol)
    err = (y[:n].double() - ref).abs()
    assert bool((err <= tol).all()), float((err / tol).max())
    # independent roundings of at most u each; the rest is fp32 noise
    assert R.relative(y[:n], ref) <= u + 2.0 ** -15


@pytest.mark.parametrize("dtype,y_dtype", [(bf, bf), (bf, f32), (f32, f32)])
@pytest.mark.parametrize("shape", SHAPES, ids=ids)
def test_forward(shape, dtype, y_dtype):
    counts, K, N = shape
    n, tail = sum(counts), 3
    i = SHAPES.index(shape)
    t = R.inputs(counts, K, N, dtype, 11 + i, bias=i % 3 != 0, residual=i % 2 == 0, tail=tail)
    t["x"][n:] = float("nan")  # rows behind the last group reach nothing
    name = R.ACTS[i % 4]
    y = torch.full((n + tail, N), 7.0, dtype=y_dtype, device="cuda")
    ws = moe.alloc_grouped_linear_workspace(n + tail, K, N, len(counts), dtype)
    off = R.offsets_of(counts)
    for _ in range(2):  # a second call on the same workspace gives the same bits
        before = y.clone()
        moe.moe_grouped_linear(t["x"], off, t["W"], y, ws, bias=t["bias"],
                               residual=t["residual"], act=name)
    assert torch.equal(y, before)
    assert moe.moe_device_status(ws) == 0
    check_y(y, t, counts, K, name, n)
    assert bool((y[n:] == 7).all())


@pytest.mark.parametrize("name", R.ACTS)
@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("residual", [False, True])
def test_forward_every_epilogue(name, bias, residual):
    for counts, K, N in (((5, 0, 20), 128, 136), ((300, 260), 128, 264), ((1100, 900), 128, 264)):
        n = sum(counts)
        t = R.inputs(counts, K, N, bf, 3, bias=bias, residual=residual)
        y = moe.grouped_linear(t["x"], R.offsets_of(counts), t["W"], t["bias"], t["residual"],
                               act=name)
        check_y(y, t, counts, K, name, n)


@pytest.mark.parametrize("rows", [1, 7, 40, 260, 1300])
def test_one_group_without_offsets_equals_one_with(rows):
    t = R.inputs((rows,), 192, 136, bf, 4)
    a = moe.grouped_linear(t["x"], None, t["W"], t["bias"], act="gelu")
    b = moe.grouped_linear(t["x"], R.offsets_of((rows,)), t["W"], t["bias"], act="gelu")
    assert torch.equal(a, b)
    check_y(a, t, (rows,), 192, "gelu", rows)


def test_residual_may_be_the_output():
    for counts in ((3, 9), (700, 800)):
        t = R.inputs(counts, 256, 264, bf, 8, residual=True)
        off = R.offsets_of(counts)
        y = moe.grouped_linear(t["x"], off, t["W"], t["bias"], t["residual"], act="silu")
        inout = t["residual"].clone()
        moe.grouped_linear(t["x"], off, t["W"], t["bias"], inout, act="silu", out=inout)
        assert torch.equal(y, inout)


FAR = [0.0, 2.0 ** -100, 1.0, 5.9375, 20.0, 42.5, 50.0, 100.0, 2.0 ** 13, 2.0 ** 40, 2.0 ** 80,
       2.0 ** 127]


@pytest.mark.parametrize("dtype", [bf, f32])
@pytest.mark.parametrize("name", R.ACTS)
def test_activations_of_far_out_values(name, dtype):
    """z is the bias: huge values of either sign, and infinities and NaN, whose neighbours keep
    their own results."""
    z = torch.tensor([s * v for v in FAR for s in (1, -1)], dtype=torch.float64, device="cuda")
    rows, K, N = 5, 16, 2 * len(FAR) + 8
    special = {1: float("nan"), 4: float("inf"), 11: -float("inf"), 18: float("nan")}
    for with_special in (False, True):
        b = torch.cat([z, z[:8]])
        if with_special:
            for i, v in special.items():
                b[i] = v
        b = b.to(dtype)
        x = torch.zeros(rows, K, dtype=dtype, device="cuda")
        W = torch.ones(1, N, K, dtype=dtype, device="cuda")
        y = moe.grouped_linear(x, None, W, b[None], act=name).double()
        zz = b.double()
        ref = R.act(zz, name)
        if name != "none":  # the limit, where the formula is 0 times infinity
            ref = torch.where(zz == -float("inf"), torch.zeros_like(ref), ref)
        u = R.U_BF16 if dtype == bf else 2.0 ** -23
        nan = zz.isnan()
        assert bool((y.isnan() == nan).all())
        inf = ref.isinf()
        assert bool((y[:, inf] == ref[inf]).all())
        ok = ~nan & ~inf
        # the activation's own error goes with |z| where z is of order one and vanishes far out
        tol = u * ref.abs() + (0 if name in ("none", "relu") else
                               R.ACT_ERR * (1 + zz.abs().clamp(max=10)) * (zz.abs() < 40) + 1e-15)
        assert bool(((y - ref).abs()[:, ok] <= tol[ok]).all())


@pytest.mark.parametrize("name", ["relu", "gelu", "silu"])
@pytest.mark.parametrize("scale", [2.0 ** 8, 2.0 ** 60, 2.0 ** 120])
def test_slopes_of_far_out_values(name, scale):
    """Values of at least 128: the slope is one or zero by the sign."""
    rows, N = 70, 40
    g = torch.Generator(device="cuda").manual_seed(4)
    codes = torch.randint(-128, 128, (rows, N), generator=g, device="cuda", dtype=torch.int8)
    scales = torch.full((rows, 2), scale, device="cuda")
    dy = torch.randint(-8, 9, (rows, N), generator=g, device="cuda").to(bf)
    x, W = torch.zeros(rows, 8, dtype=bf, device="cuda"), torch.zeros(1, N, 8, dtype=bf,
                                                                      device="cuda")
    db = torch.empty(1, N, device="cuda")
    ws = moe.alloc_grouped_linear_backward_workspace(rows, 8, N, 1)
    moe.moe_grouped_linear_backward(dy, x, None, W, ws, db=db, codes=codes, scales=scales, act=name)
    assert bool(((db[0].double() - (dy.double() * (codes >= 0)).sum(0)).abs() <= 1e-12).all())


# ------------------------------------------------------------------------- checkpoint
@pytest.mark.parametrize("dtype", [bf, f32])
@pytest.mark.parametrize("rows,N", [(1, 8), (1, 32), (3, 40), (65, 72), (7, 7168), (1000, 264)])
def test_checkpoint_save_and_restore(rows, N, dtype):
    g = torch.Generator(device="cuda").manual_seed(rows * N)
    v = (torch.randn(rows, N, generator=g, device="cuda")
         * torch.exp(4 * torch.randn(rows, 1, generator=g, device="cuda"))).to(dtype)
    v[rows // 2] = 0
    v[0, : N // 2] *= 2.0 ** -110 if dtype == f32 else 2.0 ** -120
    codes, scales = moe.alloc_checkpoint(rows, N)
    moe.moe_checkpoint_save(v, codes, scales)
    q, s = R.quantise(v)
    assert torch.equal(scales.double(), s)
    if dtype == bf:  # bf16 quotients are never within fp32's rounding of a step
        assert torch.equal(codes, q)
    ok = R.half_step(s, N) * (1 + 2.0 ** -20) + 2.0 ** -100
    assert bool(((R.values(codes, scales) - v.double()).abs() <= ok).all())
    live = s.repeat_interleave(32, 1)[:, :N] > 0
    assert bool(((codes >= 0) == (v >= 0))[live].all())
    for name in R.ACTS:
        for out_dt, u in ((f32, 2.0 ** -22), (bf, R.U_BF16)):
            out = torch.empty(rows, N, dtype=out_dt, device="cuda")
            moe.moe_checkpoint_restore(codes, scales, out, act=name)
            ref = R.act(R.values(codes, scales), name)
            if name == "none" and out_dt == f32:
                assert torch.equal(out.double(), ref.float().double())
            zabs = R.values(codes, scales).abs()
            tol = u * ref.abs() + (0 if name in ("none", "relu") else R.ACT_ERR * (1 + zabs))
            assert bool(((out.double() - ref).abs() <= tol + 1e-40).all())


def test_checkpoint_codes_of_every_bf16_quotient():
    """Every significand of a block's largest value against every bf16 value down to 2^-20 of
    it, both signs: the codes are the floor of the exact quotient."""
    sig = torch.arange(128, 256, device="cuda", dtype=torch.float64)
    vals = (sig[:, None] * 2.0 ** torch.arange(-20, 1, device="cuda")).flatten()
    vals = torch.cat([vals, -vals, torch.zeros(2, device="cuda")])
    for scale in (1.0, 2.0 ** -60, 2.0 ** 90):
        rows = []
        for top in sig.tolist():
            v = vals[vals.abs() <= top]
            v = torch.nn.functional.pad(v, (0, -len(v) % 31)).view(-1, 31)
            rows.append(torch.cat([torch.full((len(v), 1), top, device="cuda"), v], 1))
        v = (torch.cat(rows) * scale).to(bf)
        codes, scales = moe.alloc_checkpoint(*v.shape)
        moe.moe_checkpoint_save(v, codes, scales)
        q, s = R.quantise(v)
        assert torch.equal(scales.double(), s) and torch.equal(codes, q)


def test_checkpoint_blocks_with_infinities_and_nans_come_back_as_such():
    v = torch.ones(4, 96, device="cuda")
    v[0, 5] = float("inf")
    v[1, 40] = float("nan")
    v[2, 70] = -float("inf")
    codes, scales = moe.alloc_checkpoint(4, 96)
    moe.moe_checkpoint_save(v, codes, scales)
    out = torch.empty_like(v)
    moe.moe_checkpoint_restore(codes, scales, out)
    assert not bool(out[0, :32].isfinite().any()) and bool(out[0, 32:].isfinite().all())
    assert not bool(out[1, 32:64].isfinite().any()) and bool(out[1, :32].isfinite().all())
    assert not bool(out[2, 64:].isfinite().any())
    assert bool(out[3].isfinite().all())


@pytest.mark.parametrize("skip", [4, 8])  # floats: a start on a 16- and on a 32-byte boundary
def test_fp32_buffers_on_any_16_byte_boundary(skip):
    rows, N, K = 37, 264, 72
    g = torch.Generator(device="cuda").manual_seed(skip)
    v = torch.randn(skip + rows * N, generator=g, device="cuda")[skip:].view(rows, N)
    codes, scales = moe.alloc_checkpoint(rows, N)
    moe.moe_checkpoint_save(v, codes, scales)
    assert torch.equal(scales.double(), R.quantise(v)[1])
    buf = torch.full((skip + rows * N + 8,), 3.0, device="cuda")
    out = buf[skip:skip + rows * N].view(rows, N)
    moe.moe_checkpoint_restore(codes, scales, out)
    assert torch.equal(out.double(), R.values(codes, scales).float().double())
    assert bool((buf[:skip] == 3).all()) and bool((buf[skip + rows * N:] == 3).all())
    t = R.inputs((rows,), K, N, bf, 31)
    buf.fill_(3)
    moe.grouped_linear(t["x"], None, t["W"], t["bias"], act="silu", out=out)
    check_y(out, t, (rows,), K, "silu", rows)
    assert bool((buf[:skip] == 3).all()) and bool((buf[skip + rows * N:] == 3).all())


@pytest.mark.parametrize("shape", SHAPES, ids=ids)
def test_train_keeps_y_and_the_checkpoint(shape):
    counts, K, N = shape
    n, tail = sum(counts), 2
    i = SHAPES.index(shape)
    t = R.inputs(counts, K, N, bf, 40 + i, bias=i % 2 == 0, residual=i % 3 == 0, tail=tail)
    name = R.ACTS[(i + 1) % 4]
    ws = moe.alloc_grouped_linear_workspace(n + tail, K, N, len(counts))
    off = R.offsets_of(counts)
    y0 = torch.zeros(n + tail, N, dtype=bf, device="cuda")
    y = torch.zeros_like(y0)
    codes, scales = moe.alloc_checkpoint(n + tail, N)
    codes.fill_(99)
    scales.fill_(-3)
    moe.moe_grouped_linear(t["x"], off, t["W"], y0, ws, bias=t["bias"], residual=t["residual"],
                           act=name)
    moe.moe_grouped_linear_train(t["x"], off, t["W"], y, codes, scales, ws, bias=t["bias"],
                                 residual=t["residual"], act=name)
    assert torch.equal(y, y0)
    assert bool((codes[n:] == 99).all()) and bool((scales[n:] == -3).all())
    z, mag = R.grouped_z(t["x"], t["W"], t["bias"], counts)
    tol = R.accumulation(K) * mag
    step = R.half_step(scales[:n], N)
    # half a step, and where the fp32 sum falls on the other side of one, its error
    err = (R.values(codes[:n], scales[:n]) - z).abs()
    assert bool((err <= step * (1 + 2.0 ** -20) + tol + 2.0 ** -100).all())
    top = R.quantise(z)[1] * 128
    got = scales[:n].double() * 128
    block_tol = torch.nn.functional.pad(tol, (0, got.shape[1] * 32 - N)).view(n, -1, 32).amax(2)
    assert bool(((got - top).abs() <= block_tol + 2.0 ** -23 * top).all())


# --------------------------------------------------------------------------- backward
def run_backward(t, counts, name, dw_dtype=bf, tail=0, zhat=None, offsets="given"):
    n, (E, N, K) = sum(counts), t["W"].shape
    rows = n + tail
    codes = scales = None
    if name != "none":
        z = torch.randn(rows, N, device="cuda",
                        generator=torch.Generator(device="cuda").manual_seed(1))
        codes, scales = moe.alloc_checkpoint(rows, N)
        moe.moe_checkpoint_save(z, codes, scales)
        zhat = R.values(codes, scales)
        if tail:
            scales[n:] = float("nan")
    if tail:
        t["dy"][n:] = float("inf")
        t["x"][n:] = float("nan")
    ws = moe.alloc_grouped_linear_backward_workspace(rows, K, N, E)
    dx = torch.full((rows, K), 5.0, dtype=bf, device="cuda")
    dW = torch.full((E, N, K), 5.0, dtype=dw_dtype, device="cuda")
    db = torch.full((E, N), 5.0, device="cuda")
    off = R.offsets_of(counts) if offsets == "given" else None
    args = (t["dy"], t["x"], off, t["W"], ws)
    for _ in range(2):
        old = dx.clone(), dW.clone(), db.clone()
        moe.moe_grouped_linear_backward(*args, dx=dx, dW=dW, db=db, codes=codes, scales=scales,
                                        act=name)
    assert all(torch.equal(a, b) for a, b in zip(old, (dx, dW, db)))  # the same bits again
    assert moe.moe_device_status(ws) == 0
    assert bool((dx[n:] == 5).all())
    return dx, dW, db, zhat, args, codes, scales


def check_gradients(dx, dW, db, t, zhat, name, counts):
    n, (E, N, K) = sum(counts), t["W"].shape
    (rx, rW, rb), dz = R.gradients(t["dy"], t["x"], t["W"], zhat, name, counts)
    # dz: its slope is off by ACT_ERR of numbers of order one, and for the products it is
    # rounded to bf16 (dy itself, without an activation, is one already)
    dz_u = 0.0 if name == "none" else R.U_BF16
    slope_err = 0.0 if name in ("none", "relu") else 2 * R.ACT_ERR
    off_dz = slope_err * t["dy"][:n].double().abs()
    x, W = t["x"][:n].abs(), t["W"].abs()
    mx, mW, mb = R.products(dz.abs(), x, W, counts)
    ox, oW, _ = R.products(dz_u * dz.abs() + off_dz, x, W, counts)
    for got, ref, mag, off, C in ((dx[:n], rx, mx, ox, N), (dW, rW, mW, oW, max(counts))):
        u = R.U_BF16 if got.dtype == bf else 2.0 ** -24
        slack = off + R.accumulation(C) * mag
        err = (got.double() - ref).abs()
        tol = u * (ref.abs() + slack) + slack
        assert bool((err <= tol).all()), float((err - tol).max())
        # independent roundings of dz and of the result, at most u each
        assert R.relative(got, ref) <= dz_u + u + 2.0 ** -15
    tol = (max(counts) + 16) * 2.0 ** -23 * mb + R.products(off_dz, x, W, counts)[2]
    assert bool(((db.double() - rb).abs() <= tol).all())


@pytest.mark.parametrize("dw_dtype", [bf, f32])
@pytest.mark.parametrize("shape", SHAPES, ids=ids)
def test_backward(shape, dw_dtype):
    counts, K, N = shape
    i = SHAPES.index(shape)
    name = R.ACTS[(i + (1 if dw_dtype == bf else 0)) % 4]
    t = R.inputs(counts, K, N, bf, 70 + i, tail=4)
    dx, dW, db, zhat, *_ = run_backward(t, counts, name, dw_dtype, tail=4)
    check_gradients(dx, dW, db, t, zhat, name, counts)
    for e, c in enumerate(counts):
        if c == 0:
            assert not bool(dW[e].any()) and not bool(db[e].any())


# tiles of 64, 128 and 256 inputs, their last one narrower, and rows that lie across lines
@pytest.mark.parametrize("dw_dtype", [bf, f32])
@pytest.mark.parametrize("shape", [((2000,), 520, 1024), ((130, 900), 96, 1320),
                                   ((1000, 24), 176, 392), ((70,), 2056, 2056),
                                   ((257, 0, 640), 1032, 1288), ((3000,), 72, 24)], ids=ids)
def test_backward_tile_widths(shape, dw_dtype):
    counts, K, N = shape
    t = R.inputs(counts, K, N, bf, 300 + K, tail=3)
    dx, dW, db, zhat, *_ = run_backward(t, counts, "silu", dw_dtype, tail=3)
    check_gradients(dx, dW, db, t, zhat, "silu", counts)


@pytest.mark.parametrize("counts", [(5, 0, 20), (300, 260), (1100, 900)])
@pytest.mark.parametrize("name", R.ACTS)
def test_backward_every_activation_and_any_gradient_alone(counts, name):
    t = R.inputs(counts, 264, 328, bf, 12)
    dx, dW, db, zhat, args, codes, scales = run_backward(t, counts, name)
    check_gradients(dx, dW, db, t, zhat, name, counts)
    for key, full in (("dx", dx), ("dW", dW), ("db", db)):
        alone = torch.full_like(full, 3)
        moe.moe_grouped_linear_backward(*args, codes=codes, scales=scales, act=name,
                                        **{key: alone})
        assert torch.equal(alone, full)


@pytest.mark.parametrize("rows", [1, 7, 64, 260, 1300])
@pytest.mark.parametrize("name", ["none", "gelu"])
def test_backward_without_offsets(rows, name):
    t = R.inputs((rows,), 136, 264, bf, 21)
    a = run_backward(t, (rows,), name, offsets="none")
    b = run_backward(t, (rows,), name)
    assert all(torch.equal(p, q) for p, q in zip(a[:3], b[:3]))
    check_gradients(*a[:3], t, a[3], name, (rows,))


def test_backward_of_no_rows_is_zero():
    W = torch.zeros(2, 16, 8, dtype=bf, device="cuda")
    x = torch.empty(0, 8, dtype=bf, device="cuda")
    dy = torch.empty(0, 16, dtype=bf, device="cuda")
    ws = moe.alloc_grouped_linear_backward_workspace(1, 8, 16, 2)
    dW, db = torch.full_like(W, 3), torch.full((2, 16), 3.0, device="cuda")
    moe.moe_grouped_linear_backward(dy, x, torch.zeros(3, dtype=torch.int32, device="cuda"), W, ws,
                                    dx=torch.empty_like(x), dW=dW, db=db)
    assert not bool(dW.any()) and not bool(db.any())


@pytest.mark.parametrize("counts", [(9, 0, 23), (640, 500)])
@pytest.mark.parametrize("name", ["gelu", "silu"])
def test_gradients_against_differences(counts, name):
    """The loss sum(y dy) moves along random directions of x, W and b as the gradients say.
    The checkpoint moves z by at most half a step, so each element's slope by at most
    CURVE_MAX times that."""
    K, N = 128, 264
    t = R.inputs(counts, K, N, bf, 33)
    off, n = R.offsets_of(counts), sum(counts)
    ws = moe.alloc_grouped_linear_workspace(n, K, N, len(counts))
    y = torch.empty(n, N, dtype=bf, device="cuda")
    codes, scales = moe.alloc_checkpoint(n, N)
    moe.moe_grouped_linear_train(t["x"], off, t["W"], y, codes, scales, ws, bias=t["bias"],
                                 act=name)
    bws = moe.alloc_grouped_linear_backward_workspace(n, K, N, len(counts))
    dx, dW = torch.empty_like(t["x"]), torch.empty(t["W"].shape, device="cuda")
    db = torch.empty(len(counts), N, device="cuda")
    moe.moe_grouped_linear_backward(t["dy"], t["x"], off, t["W"], bws, dx=dx, dW=dW, db=db,
                                    codes=codes, scales=scales, act=name)
    g = torch.Generator(device="cuda").manual_seed(2)
    v = {k: torch.randn(t[k].shape, generator=g, device="cuda", dtype=torch.float64)
         for k in ("x", "W", "bias")}
    h = 1e-4

    def loss(x, W, bias):
        return float((R.act(R.grouped_z(x, W, bias, counts)[0], name) * t["dy"].double()).sum())

    base = {k: t[k].double() for k in v}
    for key, grad in (("x", dx), ("W", dW), ("bias", db)):
        up, down = ({k: base[k] + s * h * v[k] if k == key else base[k] for k in v}
                    for s in (1, -1))
        numeric = (loss(**up) - loss(**down)) / (2 * h)
        zero = {k: torch.zeros_like(base[k]) if k != "bias" else None for k in v}
        if key == "bias":
            moved = R.grouped_z(zero["x"], base["W"], v["bias"], counts)[0]
        else:
            pair = (v["x"], base["W"]) if key == "x" else (base["x"], v["W"])
            moved = R.grouped_z(*pair, None, counts)[0]
        # |dy| |moved z| times the slope's error, as independent errors over the elements
        # (six standard deviations), and dz's and the result's roundings likewise
        w = (t["dy"].double() * moved).norm()
        slope_err = R.CURVE_MAX * float(R.half_step(scales, N).max())
        tol = 6 * float(w) * (slope_err + R.SLOPE_MAX * R.U_BF16) \
            + 6 * R.U_BF16 * float((grad.double() * v[key]).norm()) + 1e-4
        assert abs(numeric - float((grad.double() * v[key]).sum())) <= tol


# ------------------------------------------------------------------ as a program calls it
def test_a_two_matrix_expert_trained_between_permute_and_combine():
    """Route, group, two projections with a GELU between them, combine; and back, the second
    projection's input recomputed from the first one's checkpoint."""
    T, d, h, E = 150, 256, 328, 8
    g = torch.Generator(device="cuda").manual_seed(17)
    n = lambda *s, std=1.0: (torch.randn(s, generator=g, device="cuda") * std).to(bf)  # noqa: E731
    x, Wg = n(T, d), n(d, E, std=d ** -0.5)
    A, a = n(E, h, d, std=d ** -0.5), n(E, h, std=0.2)
    B, b = n(E, d, h, std=h ** -0.5), n(E, d, std=0.2)
    i32 = dict(dtype=torch.int32, device="cuda")
    idx, w = torch.empty(T, 2, **i32), torch.empty(T, 2, device="cuda")
    off, pt, inv = torch.empty(E + 1, **i32), torch.empty(2 * T, **i32), torch.empty(T, 2, **i32)
    xp = torch.empty(2 * T, d, dtype=bf, device="cuda")
    lws = moe.alloc_workspace(T, d, h, E)
    moe.moe_route(x, Wg, idx, w)
    moe.moe_permute(idx, x, off, pt, inv, xp, lws, E)
    ws = moe.alloc_grouped_linear_workspace(2 * T, max(d, h), max(d, h), E)
    hid = torch.empty(2 * T, h, dtype=bf, device="cuda")
    codes, scales = moe.alloc_checkpoint(2 * T, h)
    moe.moe_grouped_linear_train(xp, off, A, hid, codes, scales, ws, bias=a, act="gelu")
    out = torch.empty(2 * T, d, device="cuda")  # fp32, as moe_combine reads it
    moe.moe_grouped_linear(hid, off, B, out, ws, bias=b)
    y = torch.empty_like(x)
    moe.moe_combine(out, inv, w, y)

    counts = (off[1:] - off[:-1]).tolist()
    assert sum(counts) == 2 * T
    z1, _ = R.grouped_z(xp, A, a, counts)
    z2, _ = R.grouped_z(R.act(z1, "gelu"), B, b, counts)
    ref = (z2[inv.long()] * w.double()[..., None]).sum(1)
    assert R.relative(y, ref) <= 2 * R.U_BF16  # hid and y are each rounded once

    dout = n(2 * T, d)
    bws = moe.alloc_grouped_linear_backward_workspace(2 * T, max(d, h), max(d, h), E)
    hid2 = torch.empty_like(hid)
    moe.moe_checkpoint_restore(codes, scales, hid2, act="gelu")
    dhid, dxp = torch.empty_like(hid), torch.empty_like(xp)
    dA, dB = torch.empty_like(A), torch.empty(B.shape, device="cuda")
    da, db = torch.empty(E, h, device="cuda"), torch.empty(E, d, device="cuda")
    moe.moe_grouped_linear_backward(dout, hid2, off, B, bws, dx=dhid, dW=dB, db=db)
    moe.moe_grouped_linear_backward(dhid, xp, off, A, bws, dx=dxp, dW=dA, db=da, codes=codes,
                                    scales=scales, act="gelu")
    kept = R.values(codes, scales)
    (rh, rB, rb), _ = R.gradients(dout, R.act(kept, "gelu"), B, None, "none", counts)
    (rx, rA, ra), _ = R.gradients(rh, xp, A, kept, "gelu", counts)
    # roundings on the way: hid2, dB: 1; dhid: 1; dz, dxp, dA: 3; da: 1 (of dhid)
    for got, r, k in ((dB, rB, 1), (dhid, rh, 1), (dxp, rx, 3), (dA, rA, 3), (da, ra, 1)):
        assert R.relative(got, r) <= k * R.U_BF16
    assert R.relative(db, rb) <= 2.0 ** -18
    # and the whole is the derivative of the whole, up to the 8 bits
    (ex, eA, _), _ = R.gradients(rh, xp, A, z1, "gelu", counts)
    assert R.relative(dxp, ex) <= 3 * R.U_BF16 + 2.0 ** -6
    assert R.relative(dA, eA) <= 3 * R.U_BF16 + 2.0 ** -6


@pytest.mark.parametrize("counts", [(4, 0, 7), (90, 0, 210), (1100, 1000)])
def test_captured_and_replayed_with_new_inputs(counts):
    K, N, E, n = 320, 264, len(counts), sum(counts)
    t = R.inputs(counts, K, N, bf, 50)
    off = R.offsets_of(counts)
    ws = moe.alloc_grouped_linear_workspace(n, K, N, E)
    bws = moe.alloc_grouped_linear_backward_workspace(n, K, N, E)
    y = torch.zeros(n, N, dtype=bf, device="cuda")
    codes, scales = moe.alloc_checkpoint(n, N)
    dx, dW, db = torch.zeros_like(t["x"]), torch.zeros_like(t["W"]), torch.zeros(E, N,
                                                                                device="cuda")

    def step():
        moe.moe_grouped_linear_train(t["x"], off, t["W"], y, codes, scales, ws, bias=t["bias"],
                                     act="silu")
        moe.moe_grouped_linear_backward(t["dy"], t["x"], off, t["W"], bws, dx=dx, dW=dW, db=db,
                                        codes=codes, scales=scales, act="silu")

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    # other values, and other group sizes of the same rows
    new = R.inputs(counts, K, N, bf, 51)
    for k in ("x", "dy", "W", "bias"):
        t[k].copy_(new[k])
    other = counts[::-1]
    off.copy_(R.offsets_of(other))
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    got = [v.clone() for v in (y, codes, scales, dx, dW, db)]
    check_y(y, {**t, "residual": None}, other, K, "silu", n)
    step()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, (y, codes, scales, dx, dW, db)))


def test_two_streams_with_a_workspace_each():
    K, N = 512, 264
    counts = (40, 30, 0, 20)
    off = R.offsets_of(counts)
    sets, streams = [], [torch.cuda.Stream() for _ in range(2)]
    for s in range(2):
        t = R.inputs(counts, K, N, bf, 60 + s)
        ws = moe.alloc_grouped_linear_workspace(90, K, N, 4)
        y = torch.empty(90, N, dtype=bf, device="cuda")
        sets.append((t, ws, y))
    torch.cuda.synchronize()
    for _ in range(20):
        for (t, ws, y), st in zip(sets, streams):
            moe.moe_grouped_linear(t["x"], off, t["W"], y, ws, bias=t["bias"], act="gelu",
                                   stream=st)
    torch.cuda.synchronize()
    for t, _, y in sets:
        check_y(y, t, counts, K, "gelu", 90)


def test_allocating_call_on_a_given_stream():
    """The workspace that the call allocates is zeroed, and later handed on, in the order of the
    stream it is used on: the current stream is busy meanwhile, its cached blocks hold ones."""
    K, N = 4096, 1032
    t = R.inputs((3,), K, N, bf, 77)
    need = moe.moe_grouped_linear_workspace_bytes(3, K, N, 1)
    for side in (torch.cuda.Stream(), torch.cuda.Stream().cuda_stream):
        dirty = torch.full((need,), 255, dtype=torch.uint8, device="cuda")
        torch.cuda.synchronize()
        del dirty
        torch.cuda._sleep(50_000_000)  # some 30 ms
        y = moe.grouped_linear(t["x"], None, t["W"], t["bias"], act="gelu", stream=side)
        noise = torch.full((need,), 255, dtype=torch.uint8, device="cuda")
        torch.cuda.synchronize()
        check_y(y, t, (3,), K, "gelu", 3)
        del noise


def test_four_threads_call_at_once():
    """Own streams and workspaces, the first calls of their shapes: equal to serial calls."""
    import threading
    jobs = []
    for i, counts in enumerate([(3, 0, 9), (70, 30, 0), (400, 300, 350), (1, 1, 1)]):
        t = R.inputs(counts, 264, 648 + 8 * i, bf, 90 + i)
        n = sum(counts)
        y = torch.empty(n, t["W"].shape[1], dtype=bf, device="cuda")
        dW = torch.empty_like(t["W"])
        ws = moe.alloc_grouped_linear_workspace(n, 264, y.shape[1], 3)
        bws = moe.alloc_grouped_linear_backward_workspace(n, 264, y.shape[1], 3)
        jobs.append((t, R.offsets_of(counts), y, dW, ws, bws, torch.cuda.Stream()))
    torch.cuda.synchronize()
    errors = []

    def work(t, off, y, dW, ws, bws, stream):
        try:
            for _ in range(5):
                moe.moe_grouped_linear(t["x"], off, t["W"], y, ws, bias=t["bias"], act="gelu",
                                       stream=stream)
                moe.moe_grouped_linear_backward(t["dy"], t["x"], off, t["W"], bws, dW=dW,
                                                stream=stream)
        except Exception as e:  # noqa: BLE001
            errors.append(e)

    threads = [threading.Thread(target=work, args=j) for j in jobs]
    for th in threads:
        th.start()
    for th in threads:
        th.join()
    torch.cuda.synchronize()
    assert not errors
    for t, off, y, dW, ws, bws, _ in jobs:
        y2, dW2 = torch.empty_like(y), torch.empty_like(dW)
        moe.moe_grouped_linear(t["x"], off, t["W"], y2, ws, bias=t["bias"], act="gelu")
        moe.moe_grouped_linear_backward(t["dy"], t["x"], off, t["W"], bws, dW=dW2)
        assert torch.equal(y, y2) and torch.equal(dW, dW2)


def test_offsets_beyond_32_bits():
    """rows x N above 2^31 elements: the last rows and gradients come from their own data."""
    rows, K, N = 150_016, 64, 14336
    assert rows * N > 2 ** 31
    counts = (rows - 3000, 3000)
    t = R.inputs((1,) * 2, K, N, bf, 5, bias=True)  # W and bias for two groups
    g = torch.Generator(device="cuda").manual_seed(6)
    x = torch.randn(rows, K, generator=g, device="cuda").to(bf)
    off = R.offsets_of(counts)
    ws = moe.alloc_grouped_linear_workspace(rows, K, N, 2)
    y = torch.empty(rows, N, dtype=bf, device="cuda")
    codes, scales = moe.alloc_checkpoint(rows, N)
    moe.moe_grouped_linear_train(x, off, t["W"], y, codes, scales, ws, bias=t["bias"], act="silu")
    last = slice(rows - 40, rows)
    z = x[last].double() @ t["W"][1].double().t() + t["bias"][1].double()
    assert R.relative(y[last], R.act(z, "silu")) <= R.U_BF16
    kept = R.values(codes[last], scales[last])
    assert bool(((kept - z).abs() <= R.half_step(scales[last], N) * 1.001 + 1e-4).all())
    del ws
    out = torch.empty_like(y)
    moe.moe_checkpoint_restore(codes, scales, out)
    assert R.relative(out[last], kept) <= R.U_BF16
    again = torch.zeros(rows, N, dtype=torch.int8, device="cuda")
    moe.moe_checkpoint_save(out, again, scales.clone())
    assert torch.equal(again[last], R.quantise(out[last])[0])
    del again, out
    bws = moe.alloc_grouped_linear_backward_workspace(rows, K, N, 2)
    dx, dW = torch.empty_like(x), torch.empty_like(t["W"])
    db = torch.empty(2, N, device="cuda")
    moe.moe_grouped_linear_backward(y, x, off, t["W"], bws, dx=dx, dW=dW, db=db, codes=codes,
                                    scales=scales, act="silu")
    r = slice(rows - 3000, rows)
    dz = y[r].double() * R.slope(R.values(codes[r], scales[r]), "silu")
    assert R.relative(dx[r], dz @ t["W"][1].double()) <= 2 * R.U_BF16
    assert R.relative(dW[1], dz.t() @ x[r].double()) <= 2 * R.U_BF16
    assert R.relative(db[1], dz.sum(0)) <= 2.0 ** -15


def test_one_workspace_serves_smaller_batches():
    K, N, E = 256, 1032, 8
    ws = moe.alloc_grouped_linear_workspace(3000, K, N, E)
    bws = moe.alloc_grouped_linear_backward_workspace(3000, K, N, E)
    for counts in ((400,) * 7 + (200,), (1, 0, 2, 0, 0, 0, 0, 0), (20,) * 8, (375,) * 8):
        n = sum(counts)
        t = R.inputs(counts, K, N, bf, n)
        off = R.offsets_of(counts)
        y = torch.empty(n, N, dtype=bf, device="cuda")
        moe.moe_grouped_linear(t["x"], off, t["W"], y, ws, bias=t["bias"], act="relu")
        check_y(y, t, counts, K, "relu", n)
        dx, dW = torch.empty_like(t["x"]), torch.empty_like(t["W"])
        db = torch.empty(E, N, device="cuda")
        moe.moe_grouped_linear_backward(t["dy"], t["x"], off, t["W"], bws, dx=dx, dW=dW, db=db)
        check_gradients(dx, dW, db, t, None, "none", counts)


def test_one_workspace_serves_other_shapes_and_directions_in_turn():
    """Long groups, whose bias gradients are joined from several chunks, after calls of other
    shapes that fill the same bytes with values."""
    shapes = [((700, 513), 264, 1032), ((300, 0, 500, 90), 1032, 264), ((900,), 136, 2056),
              ((5, 3), 4104, 520), ((1100, 400), 520, 72)]
    bws = torch.zeros(max(moe.moe_grouped_linear_backward_workspace_bytes(sum(c), K, N, len(c))
                          for c, K, N in shapes), dtype=torch.uint8, device="cuda")
    for turn in range(2):
        for i, (counts, K, N) in enumerate(shapes):
            n, E = sum(counts), len(counts)
            t = R.inputs(counts, K, N, bf, 200 + 10 * turn + i)
            off = R.offsets_of(counts)
            y = torch.empty(n, N, dtype=bf, device="cuda")
            codes, scales = moe.alloc_checkpoint(n, N)
            moe.moe_grouped_linear_train(t["x"], off, t["W"], y, codes, scales, bws,
                                         bias=t["bias"], act="relu")
            check_y(y, t, counts, K, "relu", n)
            dx, dW = torch.empty_like(t["x"]), torch.empty_like(t["W"])
            db = torch.full((E, N), 9.0, device="cuda")
            moe.moe_grouped_linear_backward(t["dy"], t["x"], off, t["W"], bws, dx=dx, dW=dW, db=db,
                                            codes=codes, scales=scales, act="relu")
            check_gradients(dx, dW, db, t, R.values(codes, scales), "relu", counts)
    assert moe.moe_device_status(bws) == 0


def test_bias_gradient_with_more_strips_than_counters():
    K, N, counts = 8, 65792, (70, 0, 1) + (0,) * 28 + (129,)
    assert len(counts) * (N // 256) > 8192
    t = R.inputs(counts, K, N, bf, 7, bias=False)
    dx, dW, db, zhat, *_ = run_backward(t, counts, "relu")
    check_gradients(dx, dW, db, t, zhat, "relu", counts)


def test_nothing_is_written_outside_the_outputs():
    guard = 4096

    def fenced(shape, dtype):
        size = torch.empty(0, dtype=dtype).element_size()
        nbytes = size
        for s in shape:
            nbytes *= s
        room = (nbytes + 15) // 16 * 16
        buf = torch.full((guard + room + guard,), 0xA5, dtype=torch.uint8, device="cuda")
        view = buf[guard:guard + nbytes].view(dtype).view(shape)
        return view, lambda: bool((buf[:guard] == 0xA5).all()) and bool(
            (buf[guard + nbytes:] == 0xA5).all())

    for counts, K, N in (((1, 0, 2), 72, 40), ((20, 61), 136, 200), ((600, 700), 264, 136)):
        n, E = sum(counts), len(counts)
        t = R.inputs(counts, K, N, bf, 1)
        off = R.offsets_of(counts)
        need = moe.moe_grouped_linear_workspace_bytes(n, K, N, E)
        bneed = moe.moe_grouped_linear_backward_workspace_bytes(n, K, N, E)
        specs = dict(y=((n, N), bf), codes=((n, N), torch.int8), scales=((n, (N + 31) // 32), f32),
                     dx=((n, K), bf), dW=((E, N, K), bf), db=((E, N), f32),
                     ws=((need,), torch.uint8), bws=((bneed,), torch.uint8))
        v, whole = {}, {}
        for k, (shape, dtype) in specs.items():
            v[k], whole[k] = fenced(shape, dtype)
        v["ws"].zero_()
        v["bws"].zero_()
        moe.moe_grouped_linear_train(t["x"], off, t["W"], v["y"], v["codes"], v["scales"], v["ws"],
                                     bias=t["bias"], act="gelu")
        moe.moe_grouped_linear_backward(t["dy"], t["x"], off, t["W"], v["bws"], dx=v["dx"],
                                        dW=v["dW"], db=v["db"], codes=v["codes"],
                                        scales=v["scales"], act="gelu")
        torch.cuda.synchronize()
        assert all(f() for f in whole.values()), [k for k, f in whole.items() if not f()]
