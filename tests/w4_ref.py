"""Plain 64-bit forms of the 4-bit weight and mixture-of-experts operators for
the tests, on whatever device the tensors are on, and the packed layout
written out element by element from its definition."""
from __future__ import annotations

import math

import torch

TYPES = [torch.float16, torch.bfloat16]


def half_step(dtype) -> float:
    """The largest relative error of one rounding to nearest."""
    return torch.finfo(dtype).eps / 2


def word_and_bit(K, device="cpu"):
    """(word, bit) of each element of a packed row."""
    k = torch.arange(K, device=device)
    word = k // 128 * 16 + 4 * (k % 32 // 8) + k % 128 // 32
    e = k % 8
    return word, 4 * (e // 2) + 16 * (e % 2)


def pack(q):
    """int32 words of q [..., K] (values 0 .. 15)."""
    K = q.shape[-1]
    word, bit = word_and_bit(K, q.device)
    out = torch.zeros(q.shape[:-1] + (-(-K // 128) * 16,), dtype=torch.int64, device=q.device)
    out.index_add_(-1, word, q.to(torch.int64) << bit)
    return torch.where(out >= 2 ** 31, out - 2 ** 32, out).to(torch.int32)


def unpack(Q, K):
    word, bit = word_and_bit(K, Q.device)
    return (Q.to(torch.int64)[..., word] >> bit) & 15


def group_of(K, group, device="cpu"):
    return torch.arange(K, device=device) // group


def values(Q, S, Z, K, group):
    """(q - z) * s in 64 bits."""
    g = group_of(K, group, Q.device)
    z = 8 if Z is None else (Z.to(torch.int64) & 15)[..., g]
    return (unpack(Q, K) - z).double() * S.double()[..., g]


def quantize(W, group, zeros):
    """(q, s, z) by the definition, the divisions in fp32 as it says."""
    K, G = W.shape[-1], -(-W.shape[-1] // group)
    q = torch.full(W.shape, 8, dtype=torch.int64)
    s = torch.zeros(W.shape[:-1] + (G,), dtype=W.dtype)
    z = torch.full(s.shape, 8, dtype=torch.int64)
    for g in range(G):
        at = slice(g * group, min(K, (g + 1) * group))
        x = W[..., at].float()
        zero = torch.zeros(())
        lo, hi = torch.minimum(x.amin(-1), zero), torch.maximum(x.amax(-1), zero)
        d = torch.tensor(15.0 if zeros else 7.0)
        s[..., g] = (((hi - lo) if zeros else torch.maximum(hi, -lo)) / d).to(W.dtype)
        odd = ~torch.isfinite(x).all(-1)
        live = (s[..., g].float() > 0) & ~odd
        step = torch.where(live, s[..., g].float(), torch.ones(()))
        r = torch.round(torch.where(live.unsqueeze(-1), x, zero) / step.unsqueeze(-1))
        if zeros:
            zz = torch.where(live, torch.round(-lo / step).clamp(0, 15), torch.full((), 8.0))
            z[..., g] = zz.to(torch.int64)
            q[..., at] = (r + zz.unsqueeze(-1)).clamp(0, 15).to(torch.int64)
        else:
            q[..., at] = r.clamp(-8, 7).to(torch.int64) + 8
        s[..., g] = torch.where(odd, torch.full((), math.nan).to(W.dtype), s[..., g])
    return q, s, z if zeros else None


def random_weight(gen, N, K, group, zeros, dtype, scale=0.02, lead=()):
    """(Q, S, Z) with every word random (padding bits too) and scales in
    (0.5, 1] * scale."""
    def ints(lo, hi, *shape):
        return torch.randint(lo, hi, shape, generator=gen, device=gen.device)
    G = -(-K // group)
    Q = ints(-2 ** 31, 2 ** 31, *lead, N, -(-K // 128) * 16).to(torch.int32)
    S = (torch.rand(lead + (N, G), generator=gen, device=gen.device) * 0.5 + 0.5) * scale
    Z = ints(0, 16, *lead, N, G).to(torch.uint8) if zeros else None
    return Q, S.to(dtype), Z


def moe(X, ids, weights, W13, W2):
    """y in 64 bits for given slots; W13 and W2 in 64 bits, expert by expert."""
    E, H, I = W2.shape
    y = torch.zeros(X.shape, dtype=torch.float64, device=X.device)
    for e in range(E):
        t, j = torch.nonzero(ids == e, as_tuple=True)
        if len(t):
            gu = X[t].double() @ W13[e].double().T
            g = gu[:, :I]
            h = g / (1 + torch.exp(-g)) * gu[:, I:]
            y.index_add_(0, t, h @ W2[e].double().T * weights[t, j].double().unsqueeze(-1))
    return y


def rel(x, ref) -> float:
    """2-norm of the difference over 2-norm of the reference."""
    n = float(ref.double().norm())
    d = float((x.double() - ref.double()).norm())
    return d / n if n else d
