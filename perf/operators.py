"""The products of a pruned linear layer with what surrounds them in a transformer, in plain
torch and as calls of this library, with the cases they are timed and compared on.

Five operators on a masked fp16 weight W (N x K, zero where the mask drops a weight):

  spmv_ep       decode, 1 to 16 rows:  y = act(W x~ + bias) + residual, x~ by the threshold
                rule and the caller's column set
  spmm_ep       prefill, M rows:       Y = act(X W^T + bias) + residual
  spmm_ffn      prefill, gated block:  H = act(X Wg^T) * (X Wu^T), G = X Wg^T and U = X Wu^T
                beside it where a backward pass follows
  ffn_backward  from X, G, U and dH:   dX, and the gradients of the kept weights of Wg and Wu
  spmm_backward from X and dY:         dX, and the gradient of the kept weights of W

A kept weight's gradient stands where the weight stands in the compressed buffer: tiles of 64
rows by 64 columns, strip after strip; inside a tile column by column, the kept rows of a
column in ascending order; every tile filled up with zeros to a multiple of eight values.
"""
import math

import torch

own = False

ACTS = ("none", "relu", "silu", "gelu", "gelu_tanh")
MAX_FLOPS = 7.4e11  # of the largest listed case


def listed():
    return [
        # decode step of Llama-7B: the down projection of one token, its input the activation of
        # the gated block with the smaller half dropped, added to the residual stream
        dict(name="spmv down 7B, 1 token", op="spmv_ep", N=4096, K=11008, M=1, keep=0.5, act="none", bias=False, residual=True, drop=0.5, columns=True),
        # a projection with a bias for a batch of sequences
        dict(name="spmv attn 7B, 4 tokens", op="spmv_ep", N=4096, K=4096, M=4, keep=0.5, act="none", bias=True, residual=False, drop=0.0, columns=False),
        # a ragged layer whose rows need scalar stores, at the decode's largest odd batch
        dict(name="spmv ragged, 15 tokens", op="spmv_ep", N=1111, K=2049, M=15, keep=0.4, act="gelu", bias=True, residual=True, drop=0.3, columns=False),
        # prefill: the down projection onto the residual stream
        dict(name="spmm down 7B, 2048 tokens", op="spmm_ep", N=4096, K=11008, M=2048, keep=0.5, act="none", bias=False, residual=True),
        # an ungated block's first projection at the 13B sizes, 512 tokens
        dict(name="spmm up 13B, 512 tokens", op="spmm_ep", N=13824, K=5120, M=512, keep=0.4, act="gelu_tanh", bias=True, residual=False),
        # a short prompt on a ragged layer
        dict(name="spmm ragged, 77 tokens", op="spmm_ep", N=1001, K=2047, M=77, keep=0.6, act="relu", bias=True, residual=True),
        # the gated block: a long prefill, a short prompt, and the training form of a ragged one
        dict(name="ffn 7B, 4096 tokens", op="spmm_ffn", N=11008, K=4096, M=4096, keep=0.5, act="silu", save=False),
        dict(name="ffn 7B, 100 tokens", op="spmm_ffn", N=11008, K=4096, M=100, keep=0.5, act="silu", save=False),
        dict(name="ffn ragged, 333 tokens, saved", op="spmm_ffn", N=2730, K=1021, M=333, keep=0.3, act="gelu", save=True),
        # fine-tuning of the kept weights: the gated block's gradients, then the down projection's
        dict(name="ffn gradients 7B, 2048 tokens", op="ffn_backward", N=11008, K=4096, M=2048, keep=0.5, act="silu"),
        dict(name="ffn gradients, 250 tokens", op="ffn_backward", N=1377, K=515, M=250, keep=0.5, act="gelu_tanh"),
        dict(name="spmm gradients 7B, 1024 tokens", op="spmm_backward", N=4096, K=11008, M=1024, keep=0.5),
    ]


def draw(rng):
    def size(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(("spmv_ep", "spmm_ep", "spmm_ffn", "ffn_backward", "spmm_backward"))
    while True:
        N, K = size(64, 13824), size(64, 13824)
        M = rng.randint(1, 16) if op == "spmv_ep" else size(1, 4096)
        if rng.random() < 0.5:
            N, K = -(-N // 64) * 64, -(-K // 64) * 64
        case = dict(op=op, N=N, K=K, M=M, keep=round(rng.uniform(0.2, 0.6), 2))
        if op != "spmm_backward":
            case["act"] = rng.choice(ACTS)
        if op in ("spmv_ep", "spmm_ep"):
            case |= dict(bias=rng.random() < 0.5, residual=rng.random() < 0.5)
        if op == "spmv_ep":
            case |= dict(drop=rng.choice((0.0, 0.3, 0.5, 0.7)), columns=rng.random() < 0.5)
        if op == "spmm_ffn":
            case["save"] = rng.random() < 0.5
        # weights up to the largest listed one, each at most 13824 x 5120
        if N * K <= 13824 * 5120 and work(case)["flops"] <= MAX_FLOPS:
            return case


# ------------------------------------------------------------------ inputs

def _inputs(case, seed):
    """The data of a case, from the seed alone: fp16 tensors on the GPU."""
    N, K, M = case["N"], case["K"], case["M"]
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 1000003 + N * 31 + K * 7 + M)

    def normal(*shape, std=1.0):
        return (torch.randn(*shape, generator=g, device="cuda") * std).to(torch.float16)

    def rows(t):  # rows of an odd length sit at a stride that is a multiple of 8 elements
        ld = -(-t.shape[1] // 8) * 8
        return torch.nn.functional.pad(t, (0, ld - t.shape[1]))[:, :t.shape[1]]

    def weight(which):
        """N(0, 0.02) with the smallest magnitudes dropped. What is dropped belongs to the case, as
        a layer's pattern does (the length of its values and of their gradient hangs on it); the
        values are the seed's."""
        p = torch.Generator(device="cuda")
        p.manual_seed(N * 131071 + K * 17 + which)
        W = torch.randn(N, K, generator=p, device="cuda")
        cut = math.sqrt(2.0) * torch.erfinv(torch.tensor(1.0 - case["keep"])).item()
        mask = (W.abs() >= cut).to(torch.uint8)
        sign = torch.randint(0, 2, (N, K), generator=g, device="cuda") * 2 - 1
        size = 0.8 + 0.4 * torch.rand(N, K, generator=g, device="cuda")
        return (W * sign * size * 0.02).to(torch.float16), mask

    op = case["op"]
    d = {"W": weight(0)}
    if op in ("spmm_ffn", "ffn_backward"):
        d["Wu"] = weight(1)
    x = normal(M, K)
    if op == "spmv_ep":
        if case["drop"]:  # SiLU(g) * u, whose small entries the threshold drops
            x = (torch.nn.functional.silu(x.float()) * normal(M, K).float()).to(torch.float16)
            flat = x.float().abs().flatten().sort().values
            d["t"] = flat[int(case["drop"] * (flat.numel() - 1))].item()
        else:
            d["t"] = 0.0
        # the column set: every column that some row keeps, less a tenth of them
        on = ((x != 0) & ~(x.float().abs() < d["t"])).any(0)
        on &= torch.rand(K, generator=g, device="cuda") >= 0.1
        d["columns"] = on if case["columns"] else None
    d["X"] = rows(x)
    if case.get("bias"):
        d["bias"] = normal(N, std=0.5)
    if case.get("residual"):
        d["residual"] = normal(M, N)
    if op == "ffn_backward":
        # the block's own G and U (products of such weights have this spread)
        spread = 0.02 * math.sqrt(K * case["keep"])
        d["G"], d["U"] = normal(M, N, std=spread), normal(M, N, std=spread)
        d["dH"] = normal(M, N)  # a scaled loss: gradients of order one
    if op == "spmm_backward":
        d["dY"] = rows(normal(M, N))
    return d


def _words(on):
    """A column set as 32-bit words, bit k % 32 of word k / 32."""
    pad = torch.nn.functional.pad(on.to(torch.int64), (0, -on.numel() % 32)).view(-1, 32)
    w = (pad << torch.arange(32, device=on.device)).sum(1)
    return torch.where(w >= 2 ** 31, w - 2 ** 32, w).to(torch.int32)


def _packed(mask):
    """Where the kept weights stand in the values of a compressed buffer: (their places there,
    their places in the flattened N x K weight, the number of values with the filling)."""
    N, K = mask.shape
    m = torch.nn.functional.pad(mask, (0, -K % 64, 0, -N % 64)) != 0
    S, T = m.shape[0] // 64, m.shape[1] // 64
    flat = m.view(S, 64, T, 64).permute(0, 2, 3, 1).reshape(S * T, 4096)
    count = flat.sum(1)
    filled = (count + 7) // 8 * 8
    at = flat.reshape(-1).nonzero().squeeze(1)
    tile = at // 4096
    rank = torch.arange(at.numel(), device=mask.device) - (count.cumsum(0) - count)[tile]
    place = (filled.cumsum(0) - filled)[tile] + rank
    row = (tile // T) * 64 + at % 64
    col = (tile % T) * 64 + at % 4096 // 64
    return place, row * K + col, int(filled.sum())


def prepare(case, seed):
    d = _inputs(case, seed)
    s = {"case": case, "t": d.get("t", 0.0)}
    s |= {k: d[k] for k in ("X", "bias", "residual", "G", "U", "dH", "dY") if k in d}
    s["columns"] = _words(d["columns"]) if d.get("columns") is not None else None
    if own:
        import spmm_tiled_column_b200 as spw
        s["lin"] = spw.SparseLinear(*d["W"])
        if "Wu" in d:
            s["ffn"] = spw.SparseFFN(s["lin"], spw.SparseLinear(*d["Wu"]), act=case["act"])
    else:
        s["on"] = d.get("columns")
        s["W"] = d["W"][0] * d["W"][1]
        s["packed"] = _packed(d["W"][1]) if "backward" in case["op"] else None
        if "Wu" in d:
            s["Wu"] = d["Wu"][0] * d["Wu"][1]
            s["packed_u"] = _packed(d["Wu"][1]) if "backward" in case["op"] else None
    return s


# ------------------------------------------------------------------ the operators, plainly

def _act(z, name):
    if name == "relu":
        return torch.where(z > 0, z, torch.zeros_like(z))
    if name == "silu":
        return z / (1 + torch.exp(-z))
    if name == "gelu":
        return 0.5 * z * torch.erfc(-z * math.sqrt(0.5))
    if name == "gelu_tanh":
        return z / (1 + torch.exp(-2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z)))
    return z


def _act_slope(z, name):
    if name == "relu":
        return (z > 0).to(z.dtype)
    if name == "silu":
        s = 1 / (1 + torch.exp(-z))
        return s * (1 + z * (1 - s))
    if name == "gelu":
        return 0.5 * torch.erfc(-z * math.sqrt(0.5)) + z * torch.exp(-0.5 * z * z) * (1 / math.sqrt(2 * math.pi))
    if name == "gelu_tanh":
        c = math.sqrt(2 / math.pi)
        s = 1 / (1 + torch.exp(-2 * c * (z + 0.044715 * z * z * z)))
        return s + z * s * (1 - s) * 2 * c * (1 + 3 * 0.044715 * z * z)
    return torch.ones_like(z)


def _kept(dW, packed):
    place, where, n = packed
    out = torch.zeros(n, dtype=torch.float32, device=dW.device)
    out[place] = dW.flatten()[where]
    return out.to(torch.float16)


def _plain(s):
    case = s["case"]
    op = case["op"]
    x = s["X"].float()
    if op == "spmv_ep":
        keep = (x != 0) & ~(x.abs() < s["t"])
        if s["on"] is not None:
            keep = keep & s["on"]
        x = torch.where(keep, x, torch.zeros_like(x))
    if op in ("spmv_ep", "spmm_ep"):
        y = x @ s["W"].float().T
        if "bias" in s:
            y = y + s["bias"].float()
        y = _act(y, case["act"])
        if "residual" in s:
            y = y + s["residual"].float()
        return y.to(torch.float16)
    if op == "spmm_ffn":
        g, u = x @ s["W"].float().T, x @ s["Wu"].float().T
        h = (_act(g, case["act"]) * u).to(torch.float16)
        return (h, g.to(torch.float16), u.to(torch.float16)) if case["save"] else h
    if op == "ffn_backward":
        g, u, dh = s["G"].float(), s["U"].float(), s["dH"].float()
        dg, du = dh * u * _act_slope(g, case["act"]), dh * _act(g, case["act"])
        dx = dg @ s["W"].float() + du @ s["Wu"].float()
        return dx.to(torch.float16), _kept(dg.T @ x, s["packed"]), _kept(du.T @ x, s["packed_u"])
    dy = s["dY"].float()
    return (dy @ s["W"].float()).to(torch.float16), _kept(dy.T @ x, s["packed"])


def run(s):
    if not own:
        return _plain(s)
    case, lin = s["case"], s["lin"]
    op = case["op"]
    if op == "spmv_ep":
        return lin.spmv_ep(s["X"], s["t"], s["columns"], bias=s.get("bias"), act=case["act"], residual=s.get("residual"))
    if op == "spmm_ep":
        return lin.spmm_ep(s["X"], bias=s.get("bias"), act=case["act"], residual=s.get("residual"))
    if op == "spmm_ffn":
        return s["ffn"].spmm(s["X"], save=case["save"])
    if op == "ffn_backward":
        return s["ffn"].backward(s["X"], s["G"], s["U"], s["dH"])
    return lin.spmm_backward(s["X"], s["dY"])


# ------------------------------------------------------------------ what a pass cannot do without

def work(case):
    N, K, M, op = case["N"], case["K"], case["M"], case["op"]
    # a stored weight: its kept values and one bit for each entry
    weight = N * K * (2 * case["keep"] + 0.125)
    grad = 2 * N * K * case["keep"]
    flops = 2.0 * M * N * K
    if op == "spmv_ep":  # only the kept weights of the columns that take part
        part = (1 - case["drop"]) if M == 1 else 1.0
        return {"bytes": weight * part + 2 * M * (K + N * (1 + case["residual"])), "flops": flops * case["keep"] * part}
    if op == "spmm_ep":
        return {"bytes": weight + 2 * M * (K + N * (1 + case["residual"])), "flops": flops}
    if op == "spmm_ffn":
        return {"bytes": 2 * weight + 2 * M * (K + N * (3 if case["save"] else 1)), "flops": 2 * flops}
    if op == "ffn_backward":
        return {"bytes": 2 * weight + 2 * grad + 2 * M * (2 * K + 3 * N), "flops": 4 * flops}
    return {"bytes": weight + grad + 2 * M * (2 * K + N), "flops": 2 * flops}


# ------------------------------------------------------------------ the definition, in 64 bits

def exact(case, seed):
    d = _inputs(case, seed)
    op, act = case["op"], case.get("act", "none")

    def f(z):  # the activation and its derivative, written with the error function and tanh
        if act == "relu":
            return z.clamp(min=0), (z > 0).double()
        if act == "silu":
            s = torch.sigmoid(z)
            return z * s, s + z * s * (1 - s)
        if act == "gelu":
            p = 0.5 * (1 + torch.special.erf(z / 2 ** 0.5))
            return z * p, p + z * torch.exp(-z * z / 2) / (2 * math.pi) ** 0.5
        if act == "gelu_tanh":
            c = (2 / math.pi) ** 0.5
            t = torch.tanh(c * (z + 0.044715 * z ** 3))
            return z * (1 + t) / 2, (1 + t) / 2 + z / 2 * (1 - t * t) * c * (1 + 0.134145 * z * z)
        return z, torch.ones_like(z)

    def dense(pair):
        return pair[0].double().masked_fill(pair[1] == 0, 0.0)

    def kept(dW, mask):  # tile by tile, through a padded copy in the buffer's order
        N, K = dW.shape
        pad = (0, -K % 64, 0, -N % 64)

        def tiles(a):
            a = torch.nn.functional.pad(a, pad)
            return a.unfold(0, 64, 64).unfold(1, 64, 64).transpose(2, 3).reshape(-1, 4096)

        v, m = tiles(dW), tiles(mask) != 0
        n = m.sum(1)
        to = (m.cumsum(1) - 1 + ((n + 7) // 8 * 8).cumsum(0)[:, None] - ((n + 7) // 8 * 8)[:, None])
        out = torch.zeros(int(((n + 7) // 8 * 8).sum()), dtype=torch.float64, device=dW.device)
        out[to[m]] = v[m]
        return out

    X = d["X"].double()
    if op == "spmv_ep":
        X = X.masked_fill(X.abs() < d["t"], 0.0)
        if d["columns"] is not None:
            X = X * d["columns"].double()
    if op in ("spmv_ep", "spmm_ep"):
        z = torch.einsum("mk,nk->mn", X, dense(d["W"]))
        if "bias" in d:
            z = z + d["bias"].double()
        y = f(z)[0]
        return y + d["residual"].double() if "residual" in d else y
    if op == "spmm_ffn":
        g = torch.einsum("mk,nk->mn", X, dense(d["W"]))
        u = torch.einsum("mk,nk->mn", X, dense(d["Wu"]))
        h = f(g)[0] * u
        return (h, g, u) if case["save"] else h
    if op == "ffn_backward":
        a, slope = f(d["G"].double())
        dU = d["dH"].double() * a
        dG = d["dH"].double() * d["U"].double() * slope
        dX = torch.einsum("mn,nk->mk", dG, dense(d["W"])) + torch.einsum("mn,nk->mk", dU, dense(d["Wu"]))
        return (dX, kept(torch.einsum("mn,mk->nk", dG, X), d["W"][1]),
                kept(torch.einsum("mn,mk->nk", dU, X), d["Wu"][1]))
    dY = d["dY"].double()
    return (torch.einsum("mn,nk->mk", dY, dense(d["W"])),
            kept(torch.einsum("mn,mk->nk", dY, X), d["W"][1]))
