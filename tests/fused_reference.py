"""Plain fp64 implementations of the fused / grouped linears, routing and combination, and the
error bounds that the tests hold the kernels to (derived here, from the formats alone)."""
import math

import torch

NIBBLE = (0, 4, 1, 5, 2, 6, 3, 7)      # nibble of a qweight word that holds its code j

# Half a step of fp16 relative to the value: the output is rounded once, and so is each
# dequantised weight where a kernel multiplies in fp16.
HALF = torch.finfo(torch.float16).eps / 2


def packed(seed, N, K, G, zp, lead=(), scale=0.02, device="cuda"):
    """Random packed weights covering every code and zero point: (qweight, scales, qzeros)."""
    g = torch.Generator().manual_seed(seed)
    ng = K // G
    q = torch.randint(-2 ** 31, 2 ** 31, (*lead, N, K // 8), generator=g, dtype=torch.int64).to(torch.int32)
    s = (scale * (0.5 + torch.rand(*lead, N, ng, generator=g))).half()
    z = torch.randint(0, 16, (*lead, N, (ng + 7) // 8, 8), generator=g)
    z.flatten(-2)[..., ng:] = 0
    zw = (z << torch.arange(0, 32, 4)).sum(-1)
    zw = torch.where(zw >= 2 ** 31, zw - 2 ** 32, zw).to(torch.int32)
    return q.to(device), s.to(device), zw.to(device) if zp else None


def activations(seed, M, K, device="cuda"):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(M, K, generator=g)
    x[:, torch.randperm(K, generator=g)[:max(1, K // 100)]] *= 20
    return x.half().to(device)


def dequantised(w, G):
    """(q - z) * scale in fp64, [..., N, K]."""
    q, s, z = w
    sh = torch.tensor([4 * n for n in NIBBLE], device=q.device, dtype=torch.int32)
    c = ((q.unsqueeze(-1) >> sh) & 15).flatten(-2).unflatten(-1, (-1, G)).double()
    if z is None:
        zz = 8.0
    else:
        zsh = torch.arange(0, 32, 4, device=q.device, dtype=torch.int32)
        zz = ((z.unsqueeze(-1) >> zsh) & 15).flatten(-2)[..., :s.shape[-1]].unsqueeze(-1).double()
    return ((c - zz) * s.double().unsqueeze(-1)).flatten(-2)


def act64(v, name):
    if name == "relu":
        return torch.where(v < 0, 0.0, v)
    if name == "silu":
        return v / (1 + torch.exp(-v))
    if name == "gelu":
        return v * 0.5 * torch.special.erfc(-v / math.sqrt(2))
    if name == "gelu_tanh":
        return 0.5 * v * (1 + torch.tanh(math.sqrt(2 / math.pi) * (v + 0.044715 * v ** 3)))
    return v


def linear64(X, w, G, bias=None, act=None, gated=False, residual=None):
    """(y, bound): the fused linear in fp64 and how far the kernel's fp16 result may be from it.

    bound: every product x w is off by at most HALF |x w| (the weight's rounding) and the fp32
    sum of K terms by at most K 2^-24 sum |x w|; the activations' slopes are at most 1.13; then
    the output's own rounding (and fp16's smallest step)."""
    W = dequantised(w, G)
    K = X.shape[1]
    x = X.double()
    v = x @ W.T
    e = (HALF + K * 2.0 ** -24) * (x.abs() @ W.abs().T)
    if bias is not None:
        v = v + bias.double()
        e = e + 2.0 ** -24 * v.abs()
    if gated:
        f = v.shape[1] // 2
        a, u = act64(v[:, :f], act), v[:, f:]
        ea, eu = 1.13 * e[:, :f] + 2.0 ** -20 * (a.abs() + 2.0 ** -20), e[:, f:]
        y, b = a * u, ea * (u.abs() + eu) + a.abs() * eu
    else:
        y = act64(v, act)
        b = 1.13 * e + 2.0 ** -20 * (y.abs() + 2.0 ** -20)
    if residual is not None:
        y = y + residual.double()
    return y, b + HALF * (y.abs() + b) + 2.0 ** -24


# rms(error) / rms(y): a rounding to fp16 is off by at most half a step, evenly spread: its rms is at
# most HALF / sqrt(3).  The weights' and the output's together: HALF sqrt(2/3); a gated product carries
# two such sums whose factors are uncorrelated (heavy-tailed): four times that.
RMS = HALF * math.sqrt(2 / 3)


def assert_close(y, ref, bound, gated=False, rms=True):
    y = y.double()
    assert torch.isfinite(y).all(), "non-finite outputs"
    err = (y - ref).abs()
    bad = err > bound
    assert not bad.any(), f"{int(bad.sum())} of {y.numel()} out of bounds, worst {float((err / bound).max()):.3g} x"
    if rms and y.numel() >= 64:
        r = float(err.square().mean().sqrt() / ref.square().mean().sqrt().clamp_min(1e-30))
        assert r <= (4 if gated else 1) * RMS, f"rms error {r:.3g}"


def route64(logits, k, scoring="softmax", renormalize=True):
    """Per token, in Python: (weights fp64 [T][k], experts, offsets, rows, positions) as lists."""
    rows_of = [[] for _ in range(logits.shape[1])]
    weights, experts = [], []
    for t, row in enumerate(logits.double().cpu().tolist()):
        live = [e for e, l in enumerate(row) if not math.isnan(l) and l != -math.inf]
        top = sorted(live, key=lambda e: (-row[e], e))[:k]
        cap = 3.4028234663852886e38
        l = [min(v, cap) for v in row]
        m = max((l[e] for e in live), default=0.0)
        if scoring == "sigmoid":
            w = [1 / (1 + math.exp(-l[e])) if l[e] > -700 else 0.0 for e in top]
        else:
            total = sum(math.exp(l[e] - m) for e in live)
            w = [math.exp(l[e] - m) / total for e in top]
        if renormalize and sum(w) > 0:
            w = [v / sum(w) for v in w]
        weights.append(w + [0.0] * (k - len(top)))
        experts.append(top + [-1] * (k - len(top)))
        for e in top:
            rows_of[e].append(t)
    offsets = [0]
    for r in rows_of:
        offsets.append(offsets[-1] + len(r))
    flat = [t for r in rows_of for t in r]
    at = {(t, e): offsets[e] + i for e, r in enumerate(rows_of) for i, t in enumerate(r)}
    positions = [[at[t, e] if e >= 0 else -1 for e in es] for t, es in enumerate(experts)]
    rows = flat + [-1] * (len(experts) * k - len(flat))
    return weights, experts, offsets, rows, positions
