"""Host-side checks of the grouped linear operators: the C ABI's and the binding's
refusals, before anything reaches a GPU, and the oracle's own formulas."""
import ctypes

import pytest
import torch

import linear_reference as R
import sparse_mixture_experts_26_b200 as moe

OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3
F32, BF16 = 0, 1
NONE, GELU = 0, 2
P = 1 << 20  # 16-byte aligned, never dereferenced
BIG = 1 << 60
lib = moe._lib


def forward(x=P, off=P, W=P, bias=None, res=None, rows=5, K=64, N=128, E=8, act=GELU, dt=BF16,
            y_dt=BF16, y=P, ws=P, ws_bytes=BIG):
    return lib.moe_grouped_linear(x, off, W, bias, res, rows, K, N, E, act, dt, y_dt, y, ws,
                                  ws_bytes, None)


def train(codes=P, scales=P, rows=5, K=64, N=128, E=8, act=GELU, dt=BF16, y_dt=BF16,
          ws_bytes=BIG):
    return lib.moe_grouped_linear_train(P, P, P, None, None, rows, K, N, E, act, dt, y_dt, P,
                                        codes, scales, P, ws_bytes, None)


def backward(dy=P, x=P, off=P, W=P, codes=P, scales=P, rows=5, K=64, N=128, E=8, act=GELU,
             dt=BF16, dw_dt=BF16, dx=P, dW=P, db=P, ws=P, ws_bytes=BIG):
    return lib.moe_grouped_linear_backward(dy, x, off, W, codes, scales, rows, K, N, E, act, dt,
                                           dw_dt, dx, dW, db, ws, ws_bytes, None)


@pytest.mark.parametrize("bad,code", [
    (dict(x=None), INVALID), (dict(W=None), INVALID), (dict(y=None), INVALID),
    (dict(ws=None), INVALID), (dict(x=P + 8), INVALID), (dict(bias=P + 2), INVALID),
    (dict(res=P + 4), INVALID), (dict(off=P + 4), INVALID), (dict(off=None), INVALID),
    (dict(rows=-1), INVALID), (dict(K=0), INVALID), (dict(N=-8), INVALID), (dict(E=0), INVALID),
    (dict(act=4), INVALID), (dict(act=-1), INVALID), (dict(dt=2), INVALID), (dict(y_dt=7), INVALID),
    (dict(K=60), UNSUPPORTED), (dict(N=100), UNSUPPORTED), (dict(E=33), UNSUPPORTED),
    (dict(rows=(1 << 30) + 1), UNSUPPORTED), (dict(N=1 << 28), UNSUPPORTED),
    (dict(dt=F32, y_dt=BF16), UNSUPPORTED), (dict(ws_bytes=0), WORKSPACE)])
def test_forward_refusals(bad, code):
    assert forward(**bad) == code


def test_one_byte_less_than_the_workspace_is_refused():
    for rows, K, N, E in ((1, 64, 128, 8), (1000, 256, 128, 4), (5000, 4096, 64, 1)):
        need = lib.moe_grouped_linear_workspace_bytes(rows, K, N, E, BF16)
        assert need > 0
        assert forward(rows=rows, K=K, N=N, E=E, ws_bytes=need - 1) == WORKSPACE
        assert train(rows=rows, K=K, N=N, E=E, ws_bytes=need - 1) == WORKSPACE
        need = lib.moe_grouped_linear_backward_workspace_bytes(rows, K, N, E, BF16)
        assert need > 0
        assert backward(rows=rows, K=K, N=N, E=E, ws_bytes=need - 1) == WORKSPACE


@pytest.mark.parametrize("E", [1, 8])
@pytest.mark.parametrize("fn", ["moe_grouped_linear_workspace_bytes",
                                "moe_grouped_linear_backward_workspace_bytes"])
def test_workspace_size_never_decreases_with_rows(fn, E):
    sizes = [getattr(lib, fn)(rows, 256, 640, E, BF16)
             for rows in list(range(0, 700)) + [1023, 1024, 1025, 2047, 2048, 9000]]
    assert all(a <= b for a, b in zip(sizes, sizes[1:]))
    assert getattr(lib, fn)(8, 60, 64, E, BF16) == 0
    assert getattr(lib, fn)(8, 64, 64, 33, BF16) == 0


@pytest.mark.parametrize("bad,code", [
    (dict(codes=None), INVALID), (dict(scales=None), INVALID), (dict(codes=P + 8), INVALID),
    (dict(dt=F32, y_dt=F32), UNSUPPORTED)])
def test_train_refusals(bad, code):
    assert train(**bad) == code


@pytest.mark.parametrize("bad,code", [
    (dict(dy=None), INVALID), (dict(x=P + 4), INVALID), (dict(W=None), INVALID),
    (dict(codes=None), INVALID), (dict(scales=None), INVALID), (dict(dx=P + 2), INVALID),
    (dict(dW=P + 2), INVALID), (dict(db=P + 4), INVALID), (dict(off=None), INVALID),
    (dict(dw_dt=3), INVALID), (dict(act=9), INVALID), (dict(rows=-3), INVALID),
    (dict(dt=F32), UNSUPPORTED), (dict(K=12), UNSUPPORTED), (dict(ws_bytes=0), WORKSPACE)])
def test_backward_refusals(bad, code):
    assert backward(**bad) == code
    # the gradients' types and the absence of a checkpoint are looked at before the sizes
    assert lib.moe_grouped_linear_backward_workspace_bytes(4, 64, 64, 2, F32) == 0


def test_checkpoint_refusals():
    save, restore = lib.moe_checkpoint_save, lib.moe_checkpoint_restore
    assert save(None, 4, 64, BF16, P, P, None) == INVALID
    assert save(P, 4, 64, BF16, P + 8, P, None) == INVALID
    assert save(P, 4, 60, BF16, P, P, None) == UNSUPPORTED
    assert save(P, -4, 64, BF16, P, P, None) == INVALID
    assert save(P, 4, 64, 3, P, P, None) == INVALID
    assert restore(P, None, 4, 64, NONE, BF16, P, None) == INVALID
    assert restore(P, P, 4, 64, 5, BF16, P, None) == INVALID
    assert restore(P, P, 4, 64, NONE, 2, P, None) == INVALID
    assert restore(P, P, 4, 44, NONE, BF16, P, None) == UNSUPPORTED


def test_no_rows_queue_nothing():
    assert forward(x=None, off=None, W=None, y=None, ws=None, rows=0, ws_bytes=0) == OK
    assert train(codes=None, scales=None, rows=0, ws_bytes=0) == OK
    assert lib.moe_checkpoint_save(None, 0, 64, BF16, None, None, None) == OK
    assert lib.moe_checkpoint_restore(None, None, 0, 64, NONE, BF16, None, None) == OK


bf = torch.bfloat16


def operands(**over):
    t = dict(x=torch.zeros(6, 16, dtype=bf), offsets=torch.zeros(5, dtype=torch.int32),
             W=torch.zeros(4, 40, 16, dtype=bf), y=torch.zeros(6, 40, dtype=bf),
             ws=torch.zeros(8, dtype=torch.uint8), bias=None, residual=None)
    t.update(over)
    return t


@pytest.mark.parametrize("name,bad,err", [
    ("W", torch.zeros(4, 16, 40, dtype=bf), ValueError),
    ("W", torch.zeros(4, 40, 16), TypeError),
    ("offsets", torch.zeros(4, dtype=torch.int32), ValueError),
    ("offsets", torch.zeros(5, dtype=torch.int64), TypeError),
    ("offsets", None, ValueError),
    ("y", torch.zeros(6, 16, dtype=bf), ValueError),
    ("y", torch.zeros(6, 40, dtype=torch.float16), TypeError),
    ("bias", torch.zeros(40, dtype=bf), ValueError),
    ("bias", torch.zeros(4, 40), TypeError),
    ("residual", torch.zeros(5, 40, dtype=bf), ValueError),
    ("residual", torch.zeros(6, 40), TypeError),
    ("ws", torch.zeros(8), TypeError)])
def test_binding_rejects_bad_operands(name, bad, err):
    match = "dtype" if name == "y" and err is TypeError else name
    with pytest.raises(err, match=match):
        moe.moe_grouped_linear(**operands(**{name: bad}))


def test_binding_checks_checkpoint_act_and_devices():
    codes, scales = moe.alloc_checkpoint(6, 40, device="cpu")
    assert scales.shape == (6, 2) and codes.shape == (6, 40)
    t = operands()
    with pytest.raises(ValueError, match="CUDA"):
        moe.moe_grouped_linear(**t)
    with pytest.raises(ValueError, match="scales"):
        moe.moe_grouped_linear_train(t["x"], t["offsets"], t["W"], t["y"], codes, scales[:, :1],
                                     t["ws"])
    with pytest.raises(TypeError, match="codes"):
        moe.moe_grouped_linear_train(t["x"], t["offsets"], t["W"], t["y"], codes.to(torch.uint8),
                                     scales, t["ws"])
    with pytest.raises(ValueError, match="dy"):
        moe.moe_grouped_linear_backward(t["x"], t["x"], t["offsets"], t["W"], t["ws"])
    with pytest.raises(ValueError, match="go together"):
        moe.moe_grouped_linear_backward(t["y"], t["x"], t["offsets"], t["W"], t["ws"],
                                        codes=codes)
    with pytest.raises(TypeError, match="db"):
        moe.moe_grouped_linear_backward(t["y"], t["x"], t["offsets"], t["W"], t["ws"],
                                        db=torch.zeros(4, 40, dtype=bf))
    with pytest.raises(ValueError, match="out"):
        moe.moe_checkpoint_restore(codes, scales, torch.zeros(40))
    with pytest.raises(TypeError, match="dtype"):
        moe.moe_checkpoint_save(torch.zeros(6, 40, dtype=torch.float16), codes, scales)
    with pytest.raises(ValueError, match="CUDA"):
        moe.moe_checkpoint_save(torch.zeros(6, 40), codes, scales)
    assert moe._act("silu") == 3
    with pytest.raises(ValueError, match="act"):
        moe._act("tanh")


# ------------------------------------------------------------------ the oracle's own pins
def test_oracle_slopes_match_differences():
    z = torch.linspace(-6, 6, 241, dtype=torch.float64) + 0.0137
    for name in R.ACTS:
        h = 1e-5
        d = (R.act(z + h, name) - R.act(z - h, name)) / (2 * h)
        assert float((d - R.slope(z, name)).abs().max()) < 1e-9
        assert float(R.slope(z, name).abs().max()) <= R.SLOPE_MAX
        c = (R.slope(z + h, name) - R.slope(z - h, name)) / (2 * h)
        if name != "relu":
            assert float(c.abs().max()) <= R.CURVE_MAX


def test_oracle_checkpoint_bounds():
    g = torch.Generator().manual_seed(3)
    v = torch.randn(17, 72, generator=g, dtype=torch.float64)
    v[3] = 0
    v[4, :32] = 2.0 ** -101
    q, s = R.quantise(v)
    got = R.values(q, s)
    assert bool(((got - v).abs() <= R.half_step(s, 72) * (1 + 1e-12) + 2.0 ** -100).all())
    assert bool(((v >= 0) == (q >= 0))[s.repeat_interleave(32, 1)[:, :72] > 0].all())
    assert int(q.max()) == 127 and int(q.min()) == -128
    assert bool((got[3] == 0).all())


def test_oracle_gradients_match_differences():
    counts, K, N = (3, 0, 2), 16, 24
    t = R.inputs(counts, K, N, torch.float64, 5, device="cpu")
    z, _ = R.grouped_z(t["x"], t["W"], t["bias"], counts)
    for name in ("gelu", "silu", "none"):
        (dx, dW, db), _ = R.gradients(t["dy"], t["x"], t["W"], z, name, counts)

        def loss(x, W, b):
            return float((R.act(R.grouped_z(x, W, b, counts)[0], name) * t["dy"]).sum())

        h = 1e-6
        for key, grad in (("x", dx), ("W", dW), ("bias", db)):
            v = torch.randn(t[key].shape, dtype=torch.float64,
                            generator=torch.Generator().manual_seed(9))
            up, down = ({k: t[k] + sign * h * v if k == key else t[k] for k in ("x", "W", "bias")}
                        for sign in (1, -1))
            num = (loss(*up.values()) - loss(*down.values())) / (2 * h)
            assert abs(num - float((grad * v).sum())) < 1e-6 * (1 + abs(num))
