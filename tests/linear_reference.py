"""Grouped linear operators in 64 bits, from their formulas: the tests' oracle.

Tolerances are elementwise bounds.  u(bf16) = 2^-8 and u(fp32) = 2^-24 are half a step
relative to the value; a sum of C products accumulated in fp32 is off by at most
(C + 16) 2^-23 of the sum of the magnitudes (one step instead of half of one per
addition, because a tensor core may truncate)."""
import math

import torch

BLOCK = 32
U_BF16 = 2.0 ** -8
ACTS = ("none", "relu", "gelu", "silu")
# the largest |act'| and |act''| (GELU's slope peaks at 1.129, SiLU's at 1.0998; their
# second derivatives at 0 are 0.798 and 0.5)
SLOPE_MAX = 1.13
CURVE_MAX = 0.8
# fp32 evaluation of an activation or its slope: a few roundings of numbers of order one,
# and __expf's 2^-21
ACT_ERR = 2.0 ** -19


def act(z, name):
    if name == "relu":
        return z.clamp(min=0)
    if name == "gelu":
        return 0.5 * z * (1 + torch.erf(z / math.sqrt(2)))
    if name == "silu":
        return z / (1 + torch.exp(-z))
    return z


def slope(z, name):
    if name == "relu":
        return (z > 0).to(z.dtype)
    if name == "gelu":
        return 0.5 * (1 + torch.erf(z / math.sqrt(2))) + z * torch.exp(-z * z / 2) / math.sqrt(
            2 * math.pi)
    if name == "silu":
        s = 1 / (1 + torch.exp(-z))
        return s * (1 + z * (1 - s))
    return torch.ones_like(z)


def bounds(counts):
    at = [0]
    for c in counts:
        at.append(at[-1] + c)
    return at


def offsets_of(counts, device="cuda"):
    return torch.tensor(bounds(counts), dtype=torch.int32, device=device)


def grouped_z(x, W, bias, counts):
    """z and the sum of the magnitudes that went into it, rows of the groups only."""
    at = bounds(counts)
    z = torch.zeros(at[-1], W.shape[1], dtype=torch.float64, device=x.device)
    mag = torch.zeros_like(z)
    for e in range(len(counts)):
        r = slice(at[e], at[e + 1])
        xe, We = x[r].double(), W[e].double()
        z[r] = xe @ We.t()
        mag[r] = xe.abs() @ We.abs().t()
        if bias is not None:
            z[r] += bias[e].double()
            mag[r] += bias[e].double().abs()
    return z, mag


def quantise(v):
    """Codes and scales of rows [rows, N], and the values they stand for (64 bits)."""
    rows, N = v.shape
    nb = (N + BLOCK - 1) // BLOCK
    p = torch.nn.functional.pad(v.double(), (0, nb * BLOCK - N)).view(rows, nb, BLOCK)
    top = p.abs().amax(dim=2)
    s = torch.where(top < 2.0 ** -100, torch.zeros_like(top), top / 128)
    q = torch.floor(p / torch.where(s == 0, torch.ones_like(s), s)[..., None]).clamp(-128, 127)
    q = torch.where(s[..., None] == 0, torch.zeros_like(q), q)
    return q.view(rows, -1)[:, :N].to(torch.int8), s


def values(codes, scales):
    s = scales.double().repeat_interleave(BLOCK, dim=1)[:, :codes.shape[1]]
    return (codes.double() + 0.5) * s


def half_step(scales, N):
    return scales.double().repeat_interleave(BLOCK, dim=1)[:, :N] / 2


def products(dz, x, W, counts):
    """dz W_e, dz_e^T x_e and the sums of dz over each group, in 64 bits."""
    at = bounds(counts)
    E, N, K = W.shape
    dx = torch.zeros(at[-1], K, dtype=torch.float64, device=W.device)
    dW = torch.zeros(E, N, K, dtype=torch.float64, device=W.device)
    db = torch.zeros(E, N, dtype=torch.float64, device=W.device)
    for e in range(E):
        r = slice(at[e], at[e + 1])
        dx[r] = dz[r] @ W[e].double()
        dW[e] = dz[r].t() @ x[r].double()
        db[e] = dz[r].sum(dim=0)
    return dx, dW, db


def gradients(dy, x, W, zhat, name, counts):
    """(dx, dW, db) and dz; zhat: what the checkpoint holds (None: slope 1)."""
    n = sum(counts)
    dz = dy[:n].double()
    if zhat is not None:
        dz = dz * slope(zhat[:n].double(), name)
    return products(dz, x, W, counts), dz


def accumulation(C):
    return (C + 16) * 2.0 ** -23


def relative(a, b):
    """Frobenius norm of the difference over the reference's."""
    return float((a.double() - b).norm() / b.norm().clamp(min=1e-300))


def inputs(counts, K, N, dtype, seed, bias=True, residual=False, tail=0, device="cuda"):
    g = torch.Generator(device=device)
    g.manual_seed(seed)
    rows, E = sum(counts) + tail, len(counts)

    def normal(*shape, std=1.0):
        return (torch.randn(shape, generator=g, device=device) * std).to(dtype)

    return dict(x=normal(rows, K), W=normal(E, N, K, std=K ** -0.5),
                bias=normal(E, N, std=0.5) if bias else None,
                residual=normal(rows, N) if residual else None, dy=normal(rows, N))
