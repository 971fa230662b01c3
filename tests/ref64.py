"""Plain 64-bit forms of the products with epilogues, the gated block and the gradients, and
bounds on how far the fp32-accumulating kernels may be from them.

Bounds, element by element, with S the sum of the products' magnitudes:
  - rounding a result to fp16: half a step, 2^-11 of the value, or 2^-25 below the normal
    range;
  - the sum: the tensor cores take 16 products at a time into an fp32 accumulator; each of
    the ceil(n / 16) additions may lose one unit of fp32 (2^-23) of a partial sum that is at
    most S, and so may the 16 aligned products themselves; pieces of a split sum and the
    epilogue's own additions are a handful more: (2 ceil(n / 16) + 8) 2^-23 S;
  - an operand rounded to fp16 on the way (dG, dU): 2^-11 of each product, so 2^-11 S, and
    2^-25 of the other operand where it is subnormal;
  - an activation evaluated in fp32 from z: |act'| <= 1.13 of z's error, and 2^-19 of
    max(1, |z|) for its own operations (__expf is good to 2 + |x| units; |x| <= 2.3 |z|^3 / 10
    + 1.6 |z| stays below 64 wherever the result is not negligible).
"""
import math

import torch

ACTS = ["none", "relu", "silu", "gelu", "gelu_tanh"]
HALF = 2.0 ** -11
TINY = 2.0 ** -25


def act(z, name):
    """(act(z), act'(z)) in double."""
    if name == "relu":
        return torch.relu(z), (z > 0).double()
    if name == "silu":
        s = torch.sigmoid(z)
        return z * s, s * (1 + z * (1 - s))
    if name == "gelu":
        p = 0.5 * torch.special.erfc(-z / math.sqrt(2))
        return z * p, p + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    if name == "gelu_tanh":
        c = math.sqrt(2 / math.pi)
        t = torch.tanh(c * (z + 0.044715 * z ** 3))
        return z * (1 + t) / 2, (1 + t) / 2 + z / 2 * (1 - t * t) * c * (1 + 3 * 0.044715 * z * z)
    return z, torch.ones_like(z)


def sum_err(n, S):
    return (2 * math.ceil(n / 16) + 8) * 2.0 ** -23 * S


def act_err(z, dz):
    return 1.13 * dz + 2.0 ** -19 * z.abs().clamp(min=1.0)


def product(X, W):
    """(X W^T, bound on its fp32 sum) for fp16 operands, W already masked."""
    Xd, Wd = X.double(), W.double()
    return Xd @ Wd.T, sum_err(W.shape[1], Xd.abs() @ Wd.abs().T)


def epilogue(z, dz, name, bias=None, residual=None):
    if bias is not None:
        z = z + bias.double()
        dz = dz + 2.0 ** -23 * z.abs()
    a, _ = act(z, name)
    d = act_err(z, dz) if name not in ("none", "relu") else dz
    if residual is not None:
        a = a + residual.double()
        d = d + 2.0 ** -23 * a.abs()
    return a, d + HALF * a.abs() + TINY


def gated(X, Wg, Wu, name):
    """((H, bound), (G, bound), (U, bound))."""
    g, dg = product(X, Wg)
    u, du = product(X, Wu)
    a, _ = act(g, name)
    da = act_err(g, dg) if name not in ("none", "relu") else dg
    h = a * u
    return ((h, da * (u.abs() + du) + a.abs() * du + HALF * h.abs() + TINY),
            (g, dg + HALF * g.abs() + TINY), (u, du + HALF * u.abs() + TINY))


def gate_grads(G, U, dH, name):
    """dG and dU in double and their bounds as fp16 operands."""
    a, slope = act(G.double(), name)
    h, u = dH.double(), U.double()
    exact = name in ("none", "relu")
    ds = 0.0 if exact else 2.0 ** -18 * G.double().abs().clamp(min=1.0)
    dG, dU = h * u * slope, h * a
    return ((dG, (h * u).abs() * ds + 2 * HALF * dG.abs() + TINY),
            (dU, h.abs() * ds + 2 * HALF * dU.abs() + TINY))


def dx(pairs):
    """sum of dY W over (dY, its bound or None, W): (dX, bound)."""
    out = err = S = 0.0
    n = 0
    for dY, e, W in pairs:
        Wd = W.double()
        out = out + dY.double() @ Wd
        S = S + dY.double().abs() @ Wd.abs()
        if e is not None:
            err = err + e @ Wd.abs()
        n += W.shape[0]
    return out, err + sum_err(n, S) + HALF * out.abs() + TINY


def dw(dY, e, X):
    """dY^T X and its bound."""
    Xd = X.double()
    out = dY.double().T @ Xd
    err = sum_err(X.shape[0], dY.double().abs().T @ Xd.abs())
    if e is not None:
        err = err + e.T @ Xd.abs()
    return out, err + HALF * out.abs() + TINY


def packed_order(mask):
    """For each entry of the values section its index in the flattened weight, -1 for filling.

    From the layout's own words: tiles of 64 x 64, strip by strip, column by column, the
    kept rows ascending, filled to a multiple of eight."""
    N, K = mask.shape
    order = []
    m = mask.cpu().numpy()
    for s in range(0, N, 64):
        for k0 in range(0, K, 64):
            n0 = len(order)
            for k in range(k0, min(k0 + 64, K)):
                rows = m[s:s + 64, k].nonzero()[0] + s
                order.extend((rows * K + k).tolist())
            order.extend([-1] * (-(len(order) - n0) % 8))
    return torch.tensor(order, dtype=torch.int64, device=mask.device)


def pack(a, order, fill=0.0):
    flat = torch.cat([a.flatten(), torch.full((1,), fill, dtype=a.dtype, device=a.device)])
    return flat[order]


def assert_within(got, ref, bound, what=""):
    got = got.double()
    assert got.shape == ref.shape, (got.shape, ref.shape)
    bad = ~((got - ref).abs() <= bound)
    if bad.any():
        i = tuple(x[0].item() for x in bad.nonzero(as_tuple=True))
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} off, first at {i}: "
                             f"{got[i].item()} against {ref[i].item()} +- {bound[i].item()}")
