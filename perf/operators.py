"""The measured cases of the 4-bit weight and mixture-of-experts operators.

Three operators, each as a user calls it and in a plain form made of
elementary torch operations in 32 bits (64 for the router's logits, whose
order decides which experts a token gets):

- ``quant``: a weight matrix to 4 bits with one scale (and zero point) per
  group along K, and back to 16 bits;
- ``w4``: D = A . W^T with such a weight, A in fp16 or bfloat16;
- ``moe``: a mixture-of-experts layer, from the tokens to the layer's output:
  router, softmax, the topk largest, and the chosen experts' gated products,
  with weights in 16 or in 4 bits.

A packed weight row is a run of 64-byte blocks of 128 elements.  Element k of
a row sits in block k // 128; inside it, with j = k % 128 // 32,
c = k % 32 // 8 and e = k % 8, in 32-bit word 4 c + j, at bit
4 (e // 2) + 16 (e % 2).  Its value is (q - z) * s with the scale s and zero
point z of group k // group (z = 8 where there are no zero points).
"""
import math

import torch

own = False

DEV = "cuda"
TYPES = {"f16": torch.float16, "bf16": torch.bfloat16}


# ---- cases ------------------------------------------------------------------

def listed():
    return [
        # a small projection's weight, requantised while a model is loaded
        {"name": "quant_1024x1024_f16", "op": "quant", "N": 1024, "K": 1024, "group": 128,
         "zeros": False, "type": "f16"},
        # the largest weight here, small groups and zero points: memory alone
        {"name": "quant_16384x8192_bf16_z", "op": "quant", "N": 16384, "K": 8192, "group": 32,
         "zeros": True, "type": "bf16"},
        # one token through a small projection: latency alone
        {"name": "w4_1x1024x1024_f16", "op": "w4", "M": 1, "N": 1024, "K": 1024, "group": 128,
         "zeros": False, "type": "f16"},
        # one token through a large projection: the weight's bytes
        {"name": "w4_1x16384x8192_bf16_z", "op": "w4", "M": 1, "N": 16384, "K": 8192,
         "group": 128, "zeros": True, "type": "bf16"},
        # a few tokens, nothing a multiple of anything
        {"name": "w4_7x5000x2050_f16_z", "op": "w4", "M": 7, "N": 5000, "K": 2050, "group": 32,
         "zeros": True, "type": "f16"},
        # a decode batch, the shape of the 16-bit skinny product
        {"name": "w4_64x16384x8192_f16", "op": "w4", "M": 64, "N": 16384, "K": 8192,
         "group": 128, "zeros": False, "type": "f16"},
        # a prompt: bound by the matrix units
        {"name": "w4_2048x8192x8192_bf16", "op": "w4", "M": 2048, "N": 8192, "K": 8192,
         "group": 64, "zeros": False, "type": "bf16"},
        # one token, a small layer: latency alone
        {"name": "moe_1_e8k2_1024x1024_f16", "op": "moe", "T": 1, "E": 8, "topk": 2, "H": 1024,
         "I": 1024, "group": 0, "zeros": False, "renorm": True, "type": "f16"},
        # one token, many experts, 4-bit weights
        {"name": "moe_1_e64k8_4096x1536_bf16_w4", "op": "moe", "T": 1, "E": 64, "topk": 8,
         "H": 4096, "I": 1536, "group": 128, "zeros": True, "renorm": True, "type": "bf16"},
        # a few tokens, odd sizes
        {"name": "moe_5_e12k3_1000x700_f16_w4", "op": "moe", "T": 5, "E": 12, "topk": 3,
         "H": 1000, "I": 700, "group": 32, "zeros": False, "renorm": False, "type": "f16"},
        # a decode batch over many small experts
        {"name": "moe_16_e64k6_2048x1024_bf16", "op": "moe", "T": 16, "E": 64, "topk": 6,
         "H": 2048, "I": 1024, "group": 0, "zeros": False, "renorm": False, "type": "bf16"},
        # a decode batch over few large experts: every expert's weights
        {"name": "moe_64_e16k2_4096x4096_bf16", "op": "moe", "T": 64, "E": 16, "topk": 2,
         "H": 4096, "I": 4096, "group": 0, "zeros": False, "renorm": True, "type": "bf16"},
    ]


def _size(rng, lo, hi):
    """Log-uniform over [lo, hi]; one in three is left odd or ragged, the others are multiples
    of 64 where they are large enough."""
    n = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    if rng.random() < 1 / 3 or n < 96:
        return n
    return max(64, n // 64 * 64)


def draw(rng):
    kind = rng.choice(["quant", "w4", "w4", "w4", "moe", "moe", "moe"])
    case = {"op": kind, "type": rng.choice(["f16", "bf16"])}
    group, zeros = rng.choice([32, 64, 128]), rng.random() < 0.5
    if kind == "moe":
        while True:
            e = _size(rng, 4, 64)
            case.update(T=_size(rng, 1, 64), E=e, topk=rng.randint(1, min(8, e)),
                        H=_size(rng, 256, 4096), I=_size(rng, 256, 4096))
            if case["E"] * case["H"] * case["I"] <= 16 * 4096 * 4096:
                break
        if rng.random() < 0.5:
            group, zeros = 0, False
        case["renorm"] = rng.random() < 0.5
    else:
        while True:
            case.update(N=_size(rng, 256, 16384), K=_size(rng, 128, 8192))
            if kind == "w4":
                case["M"] = _size(rng, 1, 2048)
            if case.get("M", 1) * case["N"] * case["K"] <= 2048 * 8192 * 8192:
                break
    case.update(group=group, zeros=zeros)
    return case


# ---- the packed form, in torch ----------------------------------------------

def _quantize(W, group, zeros):
    """(q, s, z) of the 16-bit weight W [..., K]: q and z int32, s in W's type.

    Symmetric: s = max|w| / 7, q = rint(w / s) + 8.  With zero points: the
    range from min(w, 0) to max(w, 0) in 15 steps.  s is rounded to W's type
    first and q goes by the rounded s."""
    K = W.shape[-1]
    x = torch.nn.functional.pad(W.float(), (0, -K % group))
    x = x.view(*x.shape[:-1], -1, group)
    if zeros:
        lo, hi = x.amin(-1).clamp(max=0), x.amax(-1).clamp(min=0)
        s = ((hi - lo) / torch.full_like(lo, 15)).to(W.dtype)
    else:
        top = x.abs().amax(-1)
        s = (top / torch.full_like(top, 7)).to(W.dtype)
    d = torch.where(s > 0, s.float(), torch.full_like(s, torch.inf, dtype=torch.float32))
    r = torch.round(x / d.unsqueeze(-1))
    if zeros:
        z = torch.where(s > 0, torch.round(-lo / d).clamp(0, 15), torch.full_like(lo, 8))
        q = (r + z.unsqueeze(-1)).clamp(0, 15)
    else:
        z, q = None, r.clamp(-8, 7) + 8
    return q.flatten(-2)[..., :K].to(torch.int32), s, None if z is None else z.to(torch.uint8)


def _shifts(dev):
    return torch.tensor([4 * (e // 2) + 16 * (e % 2) for e in range(8)], dtype=torch.int32,
                        device=dev)


def _pack(q):
    """Packed words [..., ceil(K / 128) * 16] of q [..., K]."""
    q = torch.nn.functional.pad(q, (0, -q.shape[-1] % 128))
    q = q.view(*q.shape[:-1], -1, 4, 4, 8)                       # block, j, c, e
    w = (q << _shifts(q.device)).sum(-1, dtype=torch.int32)
    return w.transpose(-1, -2).flatten(-3).contiguous()          # block, c, j


def _values(Q, S, Z, K, group):
    """The weight's values in fp32, from its packed words."""
    w = Q.view(*Q.shape[:-1], -1, 4, 4).transpose(-1, -2).unsqueeze(-1)
    q = ((w >> _shifts(Q.device)) & 15).flatten(-4)[..., :K].float()
    z = 8.0 if Z is None else Z.float().repeat_interleave(group, -1)[..., :K]
    return (q - z) * S.float().repeat_interleave(group, -1)[..., :K]


# ---- inputs -----------------------------------------------------------------

def _inputs(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    t = TYPES[case["type"]]

    def normal(scale, *shape):
        return torch.randn(shape, generator=g, device=DEV, dtype=t) * scale

    def weight(*shape):
        W = normal(0.02, *shape)
        if not case["group"]:
            return W
        q, s, z = _quantize(W, case["group"], case["zeros"])
        return _pack(q), s, z

    if case["op"] == "quant":
        return {"W": normal(0.02, case["N"], case["K"])}
    if case["op"] == "w4":
        return {"A": normal(1.0, case["M"], case["K"]), "W": weight(case["N"], case["K"])}
    E, H, I = case["E"], case["H"], case["I"]
    return {"X": normal(1.0, case["T"], H), "R": normal(2.0 / math.sqrt(H), E, H),
            "W13": weight(E, 2 * I, H), "W2": weight(E, H, I)}


def prepare(case, seed):
    state = {"case": case, **_inputs(case, seed)}
    if own:
        # what a serving program keeps: the weight's or the layer's handle
        from dense_gemm_18_amd import MoeLayer, W4Weight

        def held(W, *shape):
            return W4Weight(*W, shape=shape, group=case["group"]) if case["group"] else W

        if case["op"] == "w4":
            state["w"] = held(state["W"], case["N"], case["K"])
        elif case["op"] == "moe":
            E, H, I = case["E"], case["H"], case["I"]
            state["layer"] = MoeLayer(state["R"], held(state["W13"], E, 2 * I, H),
                                      held(state["W2"], E, H, I), topk=case["topk"],
                                      renormalize=case["renorm"])
    return state


# ---- one pass ---------------------------------------------------------------

def run(state):
    return _own(state) if own else _plain(state)


def _own(state):
    import dense_gemm_18_amd as g18

    case = state["case"]
    if case["op"] == "quant":
        w = g18.quantize_w4(state["W"], group=case["group"], zeros=case["zeros"])
        return [g18.dequantize_w4(w), w.scales] + ([w.zeros] if case["zeros"] else [])
    if case["op"] == "w4":
        return g18.gemm_nt_w4(state["A"], state["w"])
    return state["layer"](state["X"])


def _plain(state):
    case = state["case"]
    t, group = TYPES[case["type"]], case["group"]
    if case["op"] == "quant":
        q, s, z = _quantize(state["W"], group, case["zeros"])
        zf = 8.0 if z is None else z.float().repeat_interleave(group, -1)[..., :case["K"]]
        v = (q.float() - zf) * s.float().repeat_interleave(group, -1)[..., :case["K"]]
        return [v.to(t), s] + ([z] if case["zeros"] else [])
    if case["op"] == "w4":
        W = _values(*state["W"], case["K"], group)
        return (state["A"].float() @ W.T).to(t)
    return _plain_moe(state, case["topk"])


def _plain_moe(state, topk):
    """The chosen experts one slot at a time where they are fewer than all of them; otherwise
    every expert for every token, weighted by 0 where it was not chosen."""
    case, X = state["case"], state["X"]
    (T, H), (E, I) = X.shape, (case["E"], case["I"])
    p = torch.softmax(X.double() @ state["R"].double().T, -1)
    top, ids = torch.sort(p, dim=-1, descending=True, stable=True)
    top, ids = top[:, :topk], ids[:, :topk]
    if case["renorm"]:
        top = top / top.sum(-1, keepdim=True)
    slots = ids.flatten() if T * topk < E else slice(None)

    def values(name, K):
        if not case["group"]:
            return state[name][slots].float()
        return _values(*(None if v is None else v[slots] for v in state[name]), K, case["group"])

    W13, W2 = values("W13", H), values("W2", I)
    if T * topk < E:
        gu = (W13 * X.float().repeat_interleave(topk, 0).unsqueeze(1)).sum(-1).view(-1, 2, I)
        h = gu[:, 0] * torch.sigmoid(gu[:, 0]) * gu[:, 1]
        y = (W2 * h.unsqueeze(1)).sum(-1).view(T, topk, H)
        out = (y * top.float().unsqueeze(-1)).sum(1)
    else:
        share = torch.zeros_like(p).scatter_(1, ids, top).float()
        gu = (X.float() @ W13.view(E * 2 * I, H).T).view(T, E, 2, I)
        h = gu[:, :, 0] * torch.sigmoid(gu[:, :, 0]) * gu[:, :, 1] * share.unsqueeze(-1)
        out = h.view(T, E * I) @ W2.transpose(1, 2).reshape(E * I, H)
    return out.to(X.dtype), ids.to(torch.int32), top.float()


# ---- what a pass cannot do without -------------------------------------------

def work(case):
    group = case["group"]

    def weight_bytes(n, k):
        if not group:
            return 2 * n * k
        return n * (-(-k // 128) * 64 + -(-k // group) * (3 if case["zeros"] else 2))

    if case["op"] == "quant":
        # the weight read, its packed form written and read, its values written
        n, k = case["N"], case["K"]
        return {"bytes": 4 * n * k + 2 * weight_bytes(n, k), "flops": 4 * n * k}
    if case["op"] == "w4":
        m, n, k = case["M"], case["N"], case["K"]
        return {"bytes": 2 * m * k + weight_bytes(n, k) + 2 * m * n, "flops": 2 * m * n * k}
    T, E, H, I, k = (case[x] for x in ("T", "E", "H", "I", "topk"))
    # the distinct experts that T tokens choose, where all are alike
    active = E * (1 - (1 - k / E) ** T)
    return {"bytes": active * (weight_bytes(2 * I, H) + weight_bytes(H, I)) + 2 * E * H
            + 4 * T * H + 8 * T * k,
            "flops": 6 * T * k * H * I + 2 * T * E * H}


# ---- the definition in 64 bits -------------------------------------------------

def _exact_values(W, K, group):
    """The weight's values in 64 bits, element by element from its bytes."""
    Q, S, Z = W
    raw = Q.contiguous().view(torch.uint8)
    k = torch.arange(K, device=Q.device)
    nibble = k % 8 // 2 + 4 * (k % 2)
    byte = (k // 128 * 16 + k % 32 // 8 * 4 + k % 128 // 32) * 4 + nibble // 2
    v = ((raw[..., byte] >> (4 * (nibble % 2)).to(torch.uint8)) & 15).double()
    v -= 8 if Z is None else Z.double()[..., k // group]
    return v * S.double()[..., k // group]


def exact(case, seed):
    x = _inputs(case, seed)
    group = case["group"]
    if case["op"] == "quant":
        W, K = x["W"].double(), case["K"]
        at = torch.arange(K, device=DEV) // group
        where = at.expand(case["N"], K)
        zero = torch.zeros(case["N"], -(-K // group), dtype=torch.float64, device=DEV)
        hi = zero.scatter_reduce(1, where, W, "amax")
        lo = zero.scatter_reduce(1, where, W, "amin")
        top = (hi - lo) / 15 if case["zeros"] else torch.maximum(hi, -lo) / 7
        s = top.to(x["W"].dtype).double()
        safe = torch.where(s > 0, s, torch.ones_like(s))
        if not case["zeros"]:
            q = torch.clamp(torch.round(W / safe[:, at]), -8, 7)
            return [q * s[:, at], s]
        z = torch.clamp(torch.round(-lo / safe), 0, 15)
        q = torch.clamp(torch.round(W / safe[:, at]) + z[:, at], 0, 15)
        z = torch.where(s > 0, z, torch.full_like(z, 8))
        return [(q - z[:, at]) * s[:, at], s, z.to(torch.uint8)]
    if case["op"] == "w4":
        return x["A"].double() @ _exact_values(x["W"], case["K"], group).T
    X, I = x["X"].double(), case["I"]
    logits = X @ x["R"].double().T
    ids = torch.sort(logits, dim=-1, descending=True, stable=True).indices[:, :case["topk"]]
    chosen = logits.gather(1, ids)
    over = chosen if case["renorm"] else logits
    weights = torch.exp(chosen - torch.logsumexp(over, -1, keepdim=True))
    out = torch.zeros_like(X)
    for e in range(case["E"]):
        t, j = torch.nonzero(ids == e, as_tuple=True)
        if not len(t):
            continue
        W13, W2 = ((_exact_values([None if v is None else v[e] for v in x[w]], k, group)
                    if group else x[w][e].double()) for w, k in (("W13", case["H"]), ("W2", I)))
        gate, up = X[t] @ W13[:I].T, X[t] @ W13[I:].T
        out.index_add_(0, t, (gate / (1 + torch.exp(-gate)) * up) @ W2.T * weights[t, j, None])
    return out, ids.to(torch.int32), weights
