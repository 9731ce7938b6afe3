"""GPU tests of the grouped linear operators at the values where an activation, its slope or the
checkpoint's codes can go wrong: exact zeros, far tails, steps of the quantisation."""
import math

import pytest
import torch

import linear_reference as R
import sparse_mixture_experts_26_b200 as moe

pytestmark = pytest.mark.gpu
bf, f32 = torch.bfloat16, torch.float32


# ---------------------------------------------------------------- exact zeros under a ReLU
# shares of a long reduction, single SMs, pairs; one group; blocks that end inside 32 features
@pytest.mark.parametrize("counts,K,N", [((5, 0, 20), 128, 136), ((300, 260), 128, 264),
                                        ((1100, 900), 128, 264), ((6, 0, 3), 8192, 40),
                                        ((70,), 64, 8)])
def test_relu_gradient_of_exact_zeros(counts, K, N):
    """z are whole numbers, many of them zero beside live ones: the slope there is 0."""
    n, E = sum(counts), len(counts)
    g = torch.Generator(device="cuda").manual_seed(n + K)

    def whole(*shape, most=2):
        return torch.randint(-most, most + 1, shape, generator=g, device="cuda").to(bf)

    x, W, dy = whole(n, K), whole(E, N, K), whole(n, N, most=8)
    x[::7] = 0            # rows whose z is all zero
    W[:, ::3] = 0         # pruned features
    off = R.offsets_of(counts)
    ws = moe.alloc_grouped_linear_workspace(n, K, N, E)
    bws = moe.alloc_grouped_linear_backward_workspace(n, K, N, E)
    y = torch.empty(n, N, dtype=bf, device="cuda")
    codes, scales = moe.alloc_checkpoint(n, N)
    moe.moe_grouped_linear_train(x, off, W, y, codes, scales, ws, act="relu")
    z, _ = R.grouped_z(x, W, None, counts)
    assert bool((z == 0).any()) and bool((z != 0).any())
    kept = R.values(codes, scales)
    assert bool(((kept > 0) == (z > 0)).all())
    assert bool(((kept - z).abs() <= R.half_step(scales, N) * (1 + 2.0 ** -13)).all())
    dx, dW, db = torch.empty_like(x), torch.empty_like(W), torch.empty(E, N, device="cuda")
    moe.moe_grouped_linear_backward(dy, x, off, W, bws, dx=dx, dW=dW, db=db, codes=codes,
                                    scales=scales, act="relu")
    (rx, rW, rb), _ = R.gradients(dy, x, W, z, "relu", counts)
    # sums of whole numbers below 2^24: exact, up to the one rounding to bf16
    assert torch.equal(db.double(), rb)
    assert torch.equal(dx, rx.to(bf)) and torch.equal(dW, rW.to(bf))
    assert not bool(dW[:, ::3].any())


FAR_SILU = [-float("inf"), -1e30, -2.0 ** 44, -200.0, -104.0, -95.0, -86.5, -70.0, -60.0, -50.0,
            -44.0, -43.5, -43.0, -42.0, -30.0, -17.0, -3.0, -0.5, 0.0, 0.5, 17.0, 30.0, 43.0, 60.0,
            200.0, 1e30]


@pytest.mark.parametrize("dtype,y_dtype", [(bf, bf), (bf, f32), (f32, f32)])
def test_silu_far_below_zero(dtype, y_dtype):
    """z e^z, which goes to 0, relative to itself while e^z is a normal number.  Its argument is
    rounded twice: |z| log2 e 2^-23 ln 2 <= 87 2^-23 < 2^-16; the rest is a few roundings."""
    z = torch.tensor(FAR_SILU, dtype=torch.float64, device="cuda")
    z = torch.cat([z, z.flip(0), z.roll(7)])[:72].to(dtype)  # three neighbourhoods
    x = torch.zeros(3, 16, dtype=dtype, device="cuda")
    W = torch.ones(1, 72, 16, dtype=dtype, device="cuda")
    y = torch.empty(3, 72, dtype=y_dtype, device="cuda")
    moe.grouped_linear(x, None, W, z[None], act="silu", out=y)
    zd = z.double()
    ref = torch.where(zd < 0, zd.clamp(min=-800) * torch.exp(zd.clamp(min=-800)) /
                      (1 + torch.exp(zd)), zd / (1 + torch.exp(-zd)))
    tol = (2.0 ** -15 + (R.U_BF16 if y_dtype == bf else 0)) * ref.abs() + 1e-35
    err = (y.double() - ref).abs()
    assert bool((err <= tol).all()), (err / tol).max()


# -------------------------------------------------------------------- slopes, value by value
def slopes_of(z, name):
    """The kernel's slope at every z [N] (each (q + 1/2) s of one of the blocks' scales)."""
    codes, scales, N = z["codes"], z["scales"], z["codes"].shape[1]
    rows = codes.shape[0]
    db = torch.empty(rows, N, device="cuda")  # a group a row: db is dz itself, in fp32
    off = torch.arange(rows + 1, dtype=torch.int32, device="cuda")
    x = torch.zeros(rows, 8, dtype=bf, device="cuda")
    W = torch.zeros(rows, N, 8, dtype=bf, device="cuda")
    ws = moe.alloc_grouped_linear_backward_workspace(rows, 8, N, rows)
    moe.moe_grouped_linear_backward(torch.ones(rows, N, dtype=bf, device="cuda"), x, off, W, ws,
                                    db=db, codes=codes, scales=scales, act=name)
    return db.double()


def every_code(scales):
    """Rows of all 256 codes, in blocks whose neighbours differ; one scale (exact) a row."""
    q = (torch.arange(256, device="cuda").view(2, 128).t().reshape(1, -1) - 128).to(torch.int8)
    codes = q.repeat(len(scales), 1).contiguous()
    s = torch.tensor(scales, device="cuda")[:, None].repeat(1, 8).contiguous()
    return dict(codes=codes, scales=s, z=R.values(codes, s))


@pytest.mark.parametrize("scale", [0.25, 2.0, 4.0, 8.0, 2.0 ** 10])
def test_silu_slope_beside_far_neighbours(scale):
    """s (1 + z (1 - s)) for every code of a block, whatever stands beside it: 1 for large z.  The
    exponential's argument is rounded twice: |z| log2 e 2^-23 ln 2 <= |z| 2^-23; the rest is a few
    roundings, times the condition of 1 + z (1 - s), at most 8 away from its zero near -1.28."""
    t = every_code([scale])
    z = t["z"]
    got = slopes_of(t, "silu")
    e = torch.exp(-z.abs())  # without the loss of 1 - s in 64 bits
    s, c = torch.where(z > 0, 1.0, e) / (1 + e), torch.where(z > 0, e, 1.0) / (1 + e)
    want = s * (1 + z * c)
    live = z >= -85  # beyond, e^z leaves the normal numbers
    err = (got - want).abs()
    tol = (z.abs().clamp(max=85) + 8) * 2.0 ** -22 * (s * (1 + z.abs() * c))
    assert bool((err <= tol)[live].all()), float((err / tol)[live].max())
    assert bool((err <= 1e-34)[~live].all())


def test_gelu_slope_in_its_tail():
    """z Phi'(z) + Phi(z) for z in [-6, -2], relative to itself.  Phi(-x) comes from Abramowitz and
    Stegun 7.1.26, whose own error is taken from the formula in 64 bits.  The rest is rounding:
    exp(-x^2 / 2) has its argument (up to 26 in log2) rounded twice and two constants by 2^-25, so
    26 (2^-23 + 2^-24) ln 2 < 2^-18; exp2's 2^-22 and five roundings of 2^-24; the sum of the two
    terms has a condition of at most 1.6 here: less than 2^-16 in all."""
    t = every_code([3 / 64, 1 / 32])
    z = t["z"]
    x = z.abs()
    got = slopes_of(t, "gelu")
    tail = 0.5 * torch.erfc(x / math.sqrt(2))
    u = 1 / (1 + 0.3275911 / math.sqrt(2) * x)
    poly = ((((1.061405429 * u - 1.453152027) * u + 1.421413741) * u - 0.284496736) * u
            + 0.254829592) * u
    published = 0.5 * poly * torch.exp(-x * x / 2)
    want = tail + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)  # z < 0
    at = (z >= -6) & (z <= -2)
    assert int(at.sum()) > 100
    tol = (published - tail).abs() + 2.0 ** -16 * want.abs()
    assert bool(((got - want).abs() <= tol)[at].all()), float(((got - want).abs() / tol)[at].max())


@pytest.mark.parametrize("name", ["gelu", "silu"])
def test_fp32_activations_relative_to_themselves(name):
    """The fp32 operator is fp32 throughout: normcdff is within 5 units in the last place and one
    rounding follows; expf is within 2, and so is the quotient, with a sum and a product."""
    z = torch.linspace(-12, 12, 4096, dtype=torch.float64).float().cuda()
    x, W = torch.zeros(2, 8, device="cuda"), torch.ones(1, 4096, 8, device="cuda")
    y = moe.grouped_linear(x, None, W, z[None], act=name).double()
    zd = z.double()
    ref = (zd * 0.5 * torch.erfc(-zd / math.sqrt(2)) if name == "gelu"
           else zd / (1 + torch.exp(-zd)))
    assert bool(((y - ref).abs() <= 6 * 2.0 ** -23 * ref.abs()).all()), float(
        ((y - ref).abs() / ref.abs()).nan_to_num().max())


# --------------------------------------------------------------------- training's codes
@pytest.mark.parametrize("name", ["none", "relu"])
@pytest.mark.parametrize("top", [128.0, 100.0, 255.0, 2.0 ** -90 * 3])
def test_training_codes_around_every_step(top, name):
    """z on each step and one unit in the last place to either side, both signs: the code is the
    exact floor, or within 2^-14 of a step the neighbour nearer zero.  (The reciprocal is short of
    1 / s by 2^-22 and off by 2^-23 and a rounding, and |z / s| <= 128: less than 2^-14.)  Zero has
    the code 0, under a ReLU -1."""
    steps = torch.arange(-127, 128, dtype=torch.float64, device="cuda") * (top / 128)
    near = steps.float()
    inf = torch.full_like(near, float("inf"))
    up, down = torch.nextafter(near, inf), torch.nextafter(near, -inf)
    up[127], down[127] = top * 2.0 ** -40, -top * 2.0 ** -40  # beside the step at 0
    z = torch.cat([near, up, down])
    z = torch.nn.functional.pad(z, (0, -len(z) % 31)).view(-1, 31)
    z = torch.cat([torch.full((len(z), 1), top, device="cuda"), z], 1)  # 32 a block
    N = z.numel()
    # z = x W^T + b exactly, from three bf16 parts of its 24 bits
    parts, rest = [], z.flatten()
    for _ in range(3):
        parts.append(rest.to(bf))
        rest = rest - parts[-1].float()
    assert not bool(rest.any())
    W = torch.zeros(1, N, 8, dtype=bf, device="cuda")
    W[0, :, :2] = torch.stack(parts[:2], 1)
    x = torch.zeros(2, 8, dtype=bf, device="cuda")
    x[:, :2] = 1
    ws = moe.alloc_grouped_linear_workspace(2, 8, N, 1)
    y = torch.empty(2, N, device="cuda")
    codes, scales = moe.alloc_checkpoint(2, N)
    moe.moe_grouped_linear_train(x, None, W, y, codes, scales, ws, bias=parts[2][None],
                                 act=name)
    out = R.act(z.flatten(), name)
    assert torch.equal(y[0], out) and torch.equal(y[1], out)
    v = z.flatten().double() / (top / 128)
    assert bool((scales == top / 128).all())
    floor = v.floor().clamp(-128, 127)
    if name == "relu":
        floor[v == 0] = -1
    for got in codes.double():
        off = got != floor
        nearer = torch.where(v > 0, floor - 1, floor + 1)
        assert bool((got == nearer)[off].all())
        assert bool(((v - v.round()).abs() < 2.0 ** -14)[off].all())
        kept = (got + 0.5 - v).abs()
        assert bool((kept <= 0.5 + 2.0 ** -14).all())
        assert bool(((got >= 0) == (v >= 0))[v != 0].all())


# -------------------------------------------------------------------------- the most rows
def test_weight_gradient_of_the_most_rows():
    """2^30 rows of one group: a single reduction of more than four seconds."""
    rows = 1 << 30
    x = torch.ones(rows, 8, dtype=bf, device="cuda")
    dy = torch.zeros(rows, 8, dtype=bf, device="cuda")
    dy[::4096] = 1
    W = torch.zeros(1, 8, 8, dtype=bf, device="cuda")
    ws = moe.alloc_grouped_linear_backward_workspace(rows, 8, 8, 1)
    dW = torch.empty(1, 8, 8, device="cuda")
    moe.moe_grouped_linear_backward(dy, x, None, W, ws, dW=dW)
    assert moe.moe_device_status(ws) == 0
    assert bool((dW == rows // 4096).all())
    with pytest.raises(moe.MoeError):
        moe.alloc_grouped_linear_backward_workspace(rows + 1, 8, 8, 1)
    del x, dy, ws
    torch.cuda.empty_cache()


@pytest.mark.parametrize("counts,K,N", [((5, 0, 20), 128, 136), ((300, 260), 128, 264),
                                        ((1100, 900), 128, 264), ((5, 0, 3), 8192, 40)])
@pytest.mark.parametrize("name", R.ACTS)
def test_train_with_fp32_output(counts, K, N, name):
    n = sum(counts)
    t = R.inputs(counts, K, N, bf, 19, residual=True)
    off = R.offsets_of(counts)
    ws = moe.alloc_grouped_linear_workspace(n, K, N, len(counts))
    y, y16 = torch.empty(n, N, device="cuda"), torch.empty(n, N, dtype=bf, device="cuda")
    kept, kept16 = moe.alloc_checkpoint(n, N), moe.alloc_checkpoint(n, N)
    for out, ck in ((y, kept), (y16, kept16)):
        moe.moe_grouped_linear_train(t["x"], off, t["W"], out, *ck, ws, bias=t["bias"],
                                     residual=t["residual"], act=name)
    only = moe.grouped_linear(t["x"], off, t["W"], t["bias"], t["residual"], act=name, ws=ws,
                              out=torch.empty_like(y))
    assert torch.equal(y, only) and torch.equal(y.to(bf), y16)
    assert all(torch.equal(a, b) for a, b in zip(kept, kept16))
    z, mag = R.grouped_z(t["x"], t["W"], t["bias"], counts)
    ref = R.act(z, name) + t["residual"].double()
    # fp32 sums, the activation's own error, one rounding each
    tol = R.SLOPE_MAX * R.accumulation(K) * mag + R.ACT_ERR * (1 + z.abs()) + 2.0 ** -23 * ref.abs()
    assert bool(((y.double() - ref).abs() <= tol).all())
