"""Performance cases of the grouped linear operators: the expert projection with its
bias, activation and residual, its training form with an 8-bit checkpoint of the
pre-activation, the checkpoint's own save and restore, and the backward pass.

Rows are grouped by expert (group e owns rows offsets[e] .. offsets[e+1]-1); for a row r
of expert e

    z_r  = x_r W_e^T + b_e                    y_r = act(z_r) + residual_r
    dz_r = dy_r act'(zhat_r)                  zhat: z as the 8-bit checkpoint holds it
    dx_r = dz_r W_e,  dW_e = sum_r dz_r^T x_r,  db_e = sum_r dz_r

The checkpoint keeps 32 consecutive features of a row as one block: s = amax / 128,
q = floor(z / s) in [-128, 127], and q stands for (q + 1/2) s.

With ``own`` false every case runs in plain torch operations in 32 bits; with ``own``
true it makes the calls of ``sparse_mixture_experts_26_b200``.
"""
import math

import torch

own = False

BLOCK = 32


# ------------------------------------------------------------------------ the cases
def listed():
    return [
        # one token of a chat reply: two experts' up projections are read for two rows
        dict(name="forward_one_token", op="forward", T=1, K=4096, N=14336, E=8, dt="bf16",
             act="gelu", bias=True, residual=False, routing="plain", tail=0),
        # a decode batch through the down projection: every expert's weights, few rows
        dict(name="forward_decode_down", op="forward", T=16, K=14336, N=4096, E=8, dt="bf16",
             act="none", bias=True, residual=False, routing="plain", tail=0),
        # the tiny fp32 layer: latency of one call
        dict(name="forward_tiny_f32", op="forward", T=64, K=128, N=256, E=8, dt="f32",
             act="relu", bias=True, residual=True, routing="plain", tail=0),
        # a prompt of 4096 tokens through the up projection of top-2 routed experts
        dict(name="forward_prefill", op="forward", T=4096, K=4096, N=14336, E=8, dt="bf16",
             act="gelu", bias=True, residual=False, routing="plain", tail=0),
        # a dense (shared) down projection that closes a residual block
        dict(name="forward_dense_residual", op="forward", T=4096, K=14336, N=4096, E=1, dt="bf16",
             act="none", bias=True, residual=True, routing="dense", tail=0),
        # a small ragged training batch: latency, odd group sizes, rows outside the groups
        dict(name="train_small_ragged", op="train", T=37, K=256, N=384, E=8, dt="bf16",
             act="silu", bias=True, residual=True, routing="skew", tail=3),
        # a training batch of a half-width layer
        dict(name="train_half_width", op="train", T=4096, K=2048, N=7168, E=8, dt="bf16",
             act="gelu", bias=True, residual=False, routing="plain", tail=0),
        # any activation kept in 8 bits and read back as it is
        dict(name="checkpoint_round_trip", op="save", T=300, K=64, N=7168, E=8, dt="bf16",
             act="none", bias=False, residual=False, routing="plain", tail=0),
        # the next projection's input recomputed from the checkpoint
        dict(name="checkpoint_restore_gelu", op="restore", T=4096, K=64, N=14336, E=8, dt="bf16",
             act="gelu", bias=False, residual=False, routing="plain", tail=0),
        # fine-tuning on a few tokens: the weight gradients' bytes are the cost
        dict(name="backward_decode", op="backward", T=16, K=4096, N=14336, E=8, dt="bf16",
             act="gelu", bias=True, residual=False, routing="plain", tail=0),
        # a skewed middle-sized batch with empty experts
        dict(name="backward_skew", op="backward", T=300, K=2048, N=7168, E=8, dt="bf16",
             act="relu", bias=True, residual=False, routing="skew", tail=5),
        # a training batch of the full-width layer
        dict(name="backward_prefill", op="backward", T=4096, K=4096, N=14336, E=8, dt="bf16",
             act="silu", bias=True, residual=False, routing="plain", tail=0),
    ]


def _spread(rng, low, high, step=1):
    """A multiple of `step` between low and high, spread over its logarithm."""
    v = math.exp(rng.uniform(math.log(low), math.log(high)))
    return max(low, min(high, int(round(v / step)) * step))


def draw(rng):
    op = rng.choice(["forward", "forward", "forward", "train", "train", "save", "restore",
                     "backward", "backward", "backward"])
    dt = "f32" if op == "forward" and rng.random() < 0.25 else "bf16"
    if dt == "f32":
        T, K, N = _spread(rng, 1, 512), _spread(rng, 64, 1024, 8), _spread(rng, 64, 1024, 8)
    else:
        T, K, N = _spread(rng, 1, 4096), _spread(rng, 64, 14336, 8), _spread(rng, 64, 14336, 8)
    if op in ("save", "restore"):
        K = 64
    E = rng.choice([1, 2, 3, 4, 8, 8, 16, 32])
    while E * N * K > 8 * 4096 * 14336:
        E = max(1, E // 2) if E > 1 else 1
        if E == 1:
            break
    while N * K > 4096 * 14336:
        N = max(64, N // 16 * 8)
    return dict(op=op, T=T, K=K, N=N, E=E, dt=dt,
                act="none" if op == "save" else rng.choice(["none", "relu", "gelu", "silu"]),
                bias=rng.random() < 0.7, residual=op in ("forward", "train") and rng.random() < 0.4,
                routing="dense" if E == 1 else rng.choice(["plain", "plain", "skew"]),
                tail=rng.choice([0, 0, 1, 5, 17]) if E > 1 else 0)


def _sizes(case):
    """rows in groups, and how many experts get any (an expectation for routed rows)."""
    T, E = case["T"], case["E"]
    if case["routing"] == "dense":
        return T, 1.0
    k = min(2, E)
    return T * k, E * (1.0 - (1.0 - k / E) ** T)


def work(case):
    n, touched = _sizes(case)
    K, N = case["K"], case["N"]
    el = 4 if case["dt"] == "f32" else 2
    kept = n * N * (1 + 4 / BLOCK)
    w = touched * N * K * el
    fwd = n * K * el + w + n * N * el * (2 if case["residual"] else 1)
    if case["op"] == "forward":
        return {"bytes": fwd, "flops": 2.0 * n * N * K}
    if case["op"] == "train":  # the checkpoint is written, and read back as bf16 values
        return {"bytes": fwd + 2 * kept + n * N * 2, "flops": 2.0 * n * N * K}
    if case["op"] == "save":   # bf16 in, 8 bits, fp32 values out
        return {"bytes": n * N * 2 + 2 * kept + n * N * 4, "flops": 4.0 * n * N}
    if case["op"] == "restore":
        return {"bytes": kept + n * N * 2, "flops": 8.0 * n * N}
    grads = case["E"] * (N * K * el + 4 * N)
    kept = 0 if case["act"] == "none" else kept
    return {"bytes": n * N * el + kept + 2 * n * K * el + w + grads, "flops": 4.0 * n * N * K}


# ------------------------------------------------------------------------- the inputs
def _quantise(z):
    """8-bit codes and block scales of fp32 rows [rows, N]."""
    rows, N = z.shape
    nb = (N + BLOCK - 1) // BLOCK
    zb = torch.nn.functional.pad(z, (0, nb * BLOCK - N)).view(rows, nb, BLOCK)
    amax = zb.abs().amax(dim=2)
    s = torch.where(amax < 2.0 ** -100, torch.zeros_like(amax), amax / 128)
    q = torch.floor(zb / torch.where(s == 0, torch.ones_like(s), s)[..., None]).clamp(-128, 127)
    return q.view(rows, nb * BLOCK)[:, :N].to(torch.int8).contiguous(), s


def _values(codes, scales):
    """What the codes stand for, in 32 bits."""
    s = scales.repeat_interleave(BLOCK, dim=1)[:, :codes.shape[1]]
    return (codes.float() + 0.5) * s


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed))
    T, K, N, E = case["T"], case["K"], case["N"], case["E"]
    dt = torch.float32 if case["dt"] == "f32" else torch.bfloat16

    def normal(*shape, std=1.0):
        return torch.randn(shape, generator=g, device=dev).mul_(std)

    s = dict(case=case, op=case["op"], act=case["act"], E=E)
    if case["routing"] == "dense":
        counts = [T]
        s["offsets"] = None
    else:
        logits = normal(T, E)
        if case["routing"] == "skew":  # some experts take most rows, the last ones few or none
            logits += torch.linspace(2.0, -4.0, E, device=dev)
        picks = logits.topk(min(2, E), dim=1).indices.flatten()
        counts = torch.bincount(picks, minlength=E).tolist()
        at = [0]
        for c in counts:
            at.append(at[-1] + c)
        s["offsets"] = torch.tensor(at, dtype=torch.int32, device=dev)
    n = sum(counts)
    rows = n + case["tail"]
    s["n"], s["largest"] = n, max(counts)
    # group and place inside it of every grouped row (the plain form's indexing)
    s["group"] = torch.repeat_interleave(torch.arange(E, device=dev),
                                         torch.tensor(counts, device=dev))
    first = torch.tensor([sum(counts[:e]) for e in range(E)], device=dev)
    s["place"] = torch.arange(n, device=dev) - first[s["group"]]
    s["counts"] = counts
    op = case["op"]
    if op in ("forward", "train", "backward"):
        s["x"] = normal(rows, K).to(dt)
        s["W"] = normal(E, N, K, std=K ** -0.5).to(dt)
    if op in ("forward", "train"):
        s["bias"] = normal(E, N, std=0.5).to(dt) if case["bias"] else None
        s["residual"] = normal(rows, N).to(dt) if case["residual"] else None
        s["y"] = torch.zeros(rows, N, dtype=dt, device=dev)
    if op in ("train", "save"):
        s["codes"] = torch.zeros(rows, N, dtype=torch.int8, device=dev)
        s["scales"] = torch.zeros(rows, (N + BLOCK - 1) // BLOCK, device=dev)
        s["values"] = torch.zeros(rows, N, device=dev,
                                  dtype=torch.float32 if op == "save" else torch.bfloat16)
    if op == "save":
        s["z"] = normal(rows, N).to(dt)
    if op == "restore":
        s["codes"], s["scales"] = _quantise(normal(rows, N))
        s["values"] = torch.zeros(rows, N, dtype=torch.bfloat16, device=dev)
    if op == "backward":
        s["dy"] = normal(rows, N).to(dt)
        if case["act"] == "none":
            s["codes"] = s["scales"] = None
        else:
            s["codes"], s["scales"] = _quantise(normal(rows, N))
        s["dx"] = torch.zeros(rows, K, dtype=dt, device=dev)
        s["dW"] = torch.zeros(E, N, K, dtype=dt, device=dev)
        s["db"] = torch.zeros(E, N, device=dev) if case["bias"] else None
    return s


# --------------------------------------------------------------------- the plain forms
def _act(z, act):
    if act == "relu":
        return torch.where(z > 0, z, torch.zeros_like(z))
    if act == "gelu":
        return 0.5 * z * (1 + torch.erf(z * (0.5 ** 0.5)))
    if act == "silu":
        return z / (1 + torch.exp(-z))
    return z


def _act_slope(z, act):
    if act == "relu":
        return (z > 0).to(z.dtype)
    if act == "gelu":
        return (0.5 * (1 + torch.erf(z * (0.5 ** 0.5)))
                + z * torch.exp(-0.5 * z * z) * ((2 * math.pi) ** -0.5))
    if act == "silu":
        p = 1 / (1 + torch.exp(-z))
        return p * (1 + z * (1 - p))
    return torch.ones_like(z)


def _padded(s, rows):
    """Grouped rows as [E, largest group, columns] in 32 bits, zeros behind each group."""
    out = torch.zeros(s["E"], max(1, s["largest"]), rows.shape[1], device=rows.device)
    out[s["group"], s["place"]] = rows[:s["n"]].float()
    return out


def _z(s):
    z = torch.bmm(_padded(s, s["x"]), s["W"].float().transpose(1, 2))
    if s["bias"] is not None:
        z = z + s["bias"].float()[:, None, :]
    return z[s["group"], s["place"]]


def _plain(s):
    op, n = s["op"], s["n"]
    if op in ("forward", "train"):
        z = _z(s)
        y = _act(z, s["act"])
        if s["residual"] is not None:
            y = y + s["residual"][:n].float()
        out = s["y"].clone()
        out[:n] = y.to(out.dtype)
        if op == "forward":
            return out
        values = s["values"].clone()
        values[:n] = _values(*_quantise(z)).to(values.dtype)
        return out, values
    if op == "save":
        return _values(*_quantise(s["z"].float()))
    if op == "restore":
        return _act(_values(s["codes"], s["scales"]), s["act"]).to(s["values"].dtype)
    dz = s["dy"].float()
    if s["codes"] is not None:
        dz = dz * _act_slope(_values(s["codes"], s["scales"]), s["act"])
    dz = _padded(s, dz)
    dx = s["dx"].clone()
    dx[:n] = torch.bmm(dz, s["W"].float())[s["group"], s["place"]].to(dx.dtype)
    dW = torch.bmm(dz.transpose(1, 2), _padded(s, s["x"])).to(s["dW"].dtype)
    return (dx, dW) if s["db"] is None else (dx, dW, dz.sum(dim=1))


# ------------------------------------------------------------------- the framework's
def _own(s):
    import sparse_mixture_experts_26_b200 as moe
    op = s["op"]
    if op in ("forward", "train", "backward") and "ws" not in s:  # kept by the program
        rows, K = s["x"].shape
        alloc = (moe.alloc_grouped_linear_backward_workspace if op == "backward"
                 else moe.alloc_grouped_linear_workspace)
        s["ws"] = alloc(rows, K, s["W"].shape[1], s["E"], s["x"].dtype)
    if op == "forward":
        moe.moe_grouped_linear(s["x"], s["offsets"], s["W"], s["y"], s["ws"], bias=s["bias"],
                               residual=s["residual"], act=s["act"])
        return s["y"]
    if op == "train":
        moe.moe_grouped_linear_train(s["x"], s["offsets"], s["W"], s["y"], s["codes"],
                                     s["scales"], s["ws"], bias=s["bias"],
                                     residual=s["residual"], act=s["act"])
        moe.moe_checkpoint_restore(s["codes"], s["scales"], s["values"])
        return s["y"], s["values"]
    if op == "save":
        moe.moe_checkpoint_save(s["z"], s["codes"], s["scales"])
        moe.moe_checkpoint_restore(s["codes"], s["scales"], s["values"])
        return s["values"]
    if op == "restore":
        moe.moe_checkpoint_restore(s["codes"], s["scales"], s["values"], act=s["act"])
        return s["values"]
    moe.moe_grouped_linear_backward(s["dy"], s["x"], s["offsets"], s["W"], s["ws"], dx=s["dx"],
                                    dW=s["dW"], db=s["db"], codes=s["codes"],
                                    scales=s["scales"], act=s["act"])
    return (s["dx"], s["dW"]) if s["db"] is None else (s["dx"], s["dW"], s["db"])


def run(state):
    return _own(state) if own else _plain(state)


# ------------------------------------------------- the definition, in 64 bits, by expert
def exact(case, seed):
    s = prepare(case, seed)
    act, n, op = case["act"], s["n"], case["op"]

    def f(v):
        if act == "relu":
            return v.clamp(min=0)
        if act == "gelu":
            return v * torch.special.ndtr(v)
        if act == "silu":
            return v * torch.sigmoid(v)
        return v

    def slope(v):
        if act == "relu":
            return (v > 0).double()
        if act == "gelu":
            return torch.special.ndtr(v) + v * torch.exp(-v * v / 2) / math.sqrt(2 * math.pi)
        if act == "silu":
            p = torch.sigmoid(v)
            return p + v * p * (1 - p)
        return torch.ones_like(v)

    def kept(v):
        """v [rows, N] as the 8-bit checkpoint holds it."""
        out = torch.empty_like(v)
        for b in range(0, v.shape[1], BLOCK):
            part = v[:, b:b + BLOCK]
            top = part.abs().max(dim=1, keepdim=True).values
            step = top / 128
            q = torch.floor(part / step).clamp(-128, 127)
            out[:, b:b + BLOCK] = torch.where(top < 2.0 ** -100, torch.zeros_like(q),
                                              (q + 0.5) * step)
        return out

    def held():
        out = s["codes"].double() + 0.5
        for b in range(0, out.shape[1], BLOCK):
            out[:, b:b + BLOCK] *= s["scales"][:, b // BLOCK, None].double()
        return out

    if op == "save":
        return kept(s["z"].double())
    if op == "restore":
        return f(held())
    bounds = [0]
    for c in s["counts"]:
        bounds.append(bounds[-1] + c)
    groups = [(e, slice(bounds[e], bounds[e + 1])) for e in range(case["E"])]
    if op in ("forward", "train"):
        y = torch.zeros(s["y"].shape, dtype=torch.float64, device=s["y"].device)
        values = torch.zeros_like(y) if op == "train" else None
        for e, r in groups:
            z = s["x"][r].double() @ s["W"][e].double().t()
            if s["bias"] is not None:
                z += s["bias"][e].double()
            y[r] = f(z)
            if op == "train":
                values[r] = kept(z)
        if s["residual"] is not None:
            y[:n] += s["residual"][:n].double()
        return y if op == "forward" else (y, values)
    dz = s["dy"].double()
    if s["codes"] is not None:
        dz = dz * slope(held())
    dx = torch.zeros(s["dx"].shape, dtype=torch.float64, device=dz.device)
    dW = torch.empty(s["dW"].shape, dtype=torch.float64, device=dz.device)
    db = torch.empty(s["dW"].shape[:2], dtype=torch.float64, device=dz.device)
    for e, r in groups:
        dx[r] = dz[r] @ s["W"][e].double()
        dW[e] = dz[r].t() @ s["x"][r].double()
        db[e] = dz[r].sum(dim=0)
    return (dx, dW) if s["db"] is None else (dx, dW, db)
