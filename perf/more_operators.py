"""The measured cases of the operators around a product: what comes before it (a norm, 8-bit
operands), beside it (low-rank adapters) and between two of them (the choice of experts).

Four operators, each as a user calls it and in a plain form made of elementary torch
operations in 32 bits (64 where the order of two values decides which experts a token gets):

- ``norm``: s = x + residual, y = s / sqrt(mean(s^2) + eps) * weight in 16 bits, or in 8 bits
  with a scale for each row, and s in 16 bits;
- ``fp8``: D = A . B^T of 8-bit operands with a scale for each row of A and of B;
- ``gate``: from the router's logits to the chosen experts and their weights: softmax or
  sigmoid scores, a bias that counts for the choice alone, groups of experts, the topk largest;
- ``lora``: D = X . W^T + scale[a] (X . A[a]^T) . B[a]^T, where a is each row's own adapter (or
  none) and W is held in 16 or in 4 bits.

A packed weight row is a run of 64-byte blocks of 128 elements.  Element k of a row sits in
block k // 128; inside it, with j = k % 128 // 32, c = k % 32 // 8 and e = k % 8, in 32-bit word
4 c + j, at bit 4 (e // 2) + 16 (e % 2).  Its value is (q - z) * s with the scale s and zero
point z of group k // group (z = 8 where there are no zero points).
"""
import math

import torch

own = False

DEV = "cuda"
TYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32,
         "e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
LARGEST = {"e4m3": 448.0, "e5m2": 57344.0}
EPS = 1e-6


# ---- cases ------------------------------------------------------------------

def listed():
    return [
        # one token between two products of a decode step: latency alone
        {"name": "norm_1x4096_f16", "op": "norm", "T": 1, "H": 4096, "residual": True,
         "out": "f16", "type": "f16"},
        # a batch of prompts in front of an 8-bit product: memory alone
        {"name": "norm_16384x8192_bf16_e4m3", "op": "norm", "T": 16384, "H": 8192,
         "residual": True, "out": "e4m3", "type": "bf16"},
        # one token through a small projection
        {"name": "fp8_1x4096x4096_f16", "op": "fp8", "M": 1, "N": 4096, "K": 4096, "a": "e4m3",
         "b": "e4m3", "type": "f16"},
        # a few tokens, nothing a multiple of anything
        {"name": "fp8_33x5000x2050_bf16", "op": "fp8", "M": 33, "N": 5000, "K": 2050,
         "a": "e4m3", "b": "e5m2", "type": "bf16"},
        # a decode batch: the weight's bytes
        {"name": "fp8_64x16384x8192_f16", "op": "fp8", "M": 64, "N": 16384, "K": 8192,
         "a": "e4m3", "b": "e4m3", "type": "f16"},
        # a batch of prompts: bound by the matrix units
        {"name": "fp8_4096x8192x8192_bf16", "op": "fp8", "M": 4096, "N": 8192, "K": 8192,
         "a": "e4m3", "b": "e4m3", "type": "bf16"},
        # one token, few experts: latency alone
        {"name": "gate_1x64_k8_softmax", "op": "gate", "T": 1, "E": 64, "topk": 8,
         "scoring": "softmax", "bias": False, "groups": 1, "kept": 1, "group_top": 1,
         "renorm": True, "scale": 1.0, "type": "f32"},
        # a batch of prompts over many experts in groups, with a bias for balance
        {"name": "gate_16384x256_k8_sigmoid", "op": "gate", "T": 16384, "E": 256, "topk": 8,
         "scoring": "sigmoid", "bias": True, "groups": 8, "kept": 4, "group_top": 2,
         "renorm": True, "scale": 2.5, "type": "f32"},
        # one token with an adapter: latency and the weight's bytes
        {"name": "lora_1x4096x4096_r16_f16", "op": "lora", "M": 1, "N": 4096, "K": 4096,
         "rank": 16, "count": 8, "group": 0, "zeros": False, "runs": False, "type": "f16"},
        # a few tokens of as many requests, odd sizes, a 4-bit projection
        {"name": "lora_13x5000x2050_r12_bf16_w4", "op": "lora", "M": 13, "N": 5000, "K": 2050,
         "rank": 12, "count": 5, "group": 32, "zeros": True, "runs": False, "type": "bf16"},
        # a decode batch over many adapters beside a large projection
        {"name": "lora_64x16384x8192_r16_bf16", "op": "lora", "M": 64, "N": 16384, "K": 8192,
         "rank": 16, "count": 32, "group": 0, "zeros": False, "runs": False, "type": "bf16"},
        # prompts of several requests behind each other: bound by the matrix units
        {"name": "lora_2048x8192x8192_r64_bf16", "op": "lora", "M": 2048, "N": 8192, "K": 8192,
         "rank": 64, "count": 8, "group": 0, "zeros": False, "runs": True, "type": "bf16"},
    ]


def _size(rng, lo, hi):
    """Log-uniform over [lo, hi]; one in three is left odd or ragged, the others are multiples
    of 64 where they are large enough."""
    n = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    if rng.random() < 1 / 3 or n < 96:
        return n
    return max(64, n // 64 * 64)


def draw(rng):
    op = rng.choice(["norm", "fp8", "gate", "lora", "lora"])
    case = {"op": op, "type": rng.choice(["f16", "bf16"])}
    if op == "norm":
        case.update(T=_size(rng, 1, 16384), H=_size(rng, 256, 8192),
                    residual=rng.random() < 2 / 3,
                    out=rng.choice([case["type"], "e4m3", "e5m2"]))
    elif op == "fp8":
        while True:
            case.update(M=_size(rng, 1, 4096), N=_size(rng, 256, 16384), K=_size(rng, 128, 8192))
            if case["M"] * case["N"] * case["K"] <= 4096 * 8192 * 8192:
                break
        case.update(a=rng.choice(["e4m3", "e4m3", "e5m2"]), b=rng.choice(["e4m3", "e4m3", "e5m2"]))
    elif op == "gate":
        groups = rng.choice([1, 1, 2, 4, 8])
        kept = rng.randint(1, groups)
        each = max(2, _size(rng, 8, 256) // groups)
        case.update(T=_size(rng, 1, 16384), E=groups * each, groups=groups, kept=kept,
                    topk=rng.randint(1, min(8, kept * each)), group_top=rng.choice([1, 2]),
                    scoring=rng.choice(["softmax", "sigmoid"]), bias=rng.random() < 0.5,
                    renorm=rng.random() < 0.5, scale=rng.choice([1.0, 2.5]),
                    type=rng.choice(["f32", "f32", "f16", "bf16"]))
    else:
        while True:
            case.update(M=_size(rng, 1, 2048), N=_size(rng, 256, 16384), K=_size(rng, 128, 8192))
            if case["M"] * case["N"] * case["K"] <= 2048 * 8192 * 8192:
                break
        case.update(rank=rng.choice([4, 8, 12, 16, 16, 32, 64]), count=_size(rng, 1, 32),
                    group=rng.choice([0, 0, 32, 64, 128]), zeros=rng.random() < 0.5,
                    runs=rng.random() < 0.5)
        case["zeros"] = case["zeros"] and case["group"] > 0
    return case


# ---- inputs -----------------------------------------------------------------

def _normal(g, dtype, scale, *shape):
    return torch.randn(shape, generator=g, device=DEV, dtype=dtype) * scale


def _eight_bits(x, fmt):
    """(the rows of x in 8 bits, their scales)."""
    scale = (x.abs().amax(-1) / LARGEST[fmt]).clamp(min=1e-30)
    return (x / scale[:, None]).clamp(-LARGEST[fmt], LARGEST[fmt]).to(TYPES[fmt]), scale


def _packed(g, case, N, K):
    """A weight in 4 bits: words, scales, zero points or None."""
    t, group = TYPES[case["type"]], case["group"]
    q = torch.randn((N, K), generator=g, device=DEV) * 2.3 + 8
    q = torch.nn.functional.pad(q.round().clamp(0, 15).to(torch.int32), (0, -K % 128))
    e = torch.arange(8, device=DEV)
    shifts = (4 * (e // 2) + 16 * (e % 2)).to(torch.int32)
    w = (q.view(N, -1, 4, 4, 8) << shifts).sum(-1, dtype=torch.int32)      # block, j, c
    words = w.transpose(-1, -2).flatten(1).contiguous()
    groups = (N, -(-K // group))
    scales = (1 + 0.2 * torch.randn(groups, generator=g, device=DEV)) * (0.02 / 2.3)
    zeros = torch.randint(6, 11, groups, generator=g, device=DEV).to(torch.uint8)
    return words, scales.to(t), zeros if case["zeros"] else None


def _adapter_ids(g, case):
    """An adapter for each row, one in eight without: a draw for each row, or runs of rows
    of one request each, 256 of them on average."""
    M, n = case["M"], case["count"]
    each = torch.randint(0, 8 * n, (M,), generator=g, device=DEV)
    each = torch.where(each < 7 * n, each % n, torch.full_like(each, -1))
    if case["runs"]:
        starts = torch.rand((M,), generator=g, device=DEV) < 1 / 256
        each = each[starts.cumsum(0) % M]
    return each.to(torch.int32)


def _inputs(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    t, op = TYPES[case["type"]], case["op"]
    if op == "norm":
        T, H = case["T"], case["H"]
        return {"x": _normal(g, t, 1.0, T, H),
                "r": _normal(g, t, 3.0, T, H) if case["residual"] else None,
                "w": 1 + _normal(g, t, 0.2, H)}
    if op == "fp8":
        A, sa = _eight_bits(_normal(g, torch.float32, 1.0, case["M"], case["K"]), case["a"])
        B, sb = _eight_bits(_normal(g, torch.float32, 0.02, case["N"], case["K"]), case["b"])
        return {"A": A, "sa": sa, "B": B, "sb": sb}
    if op == "gate":
        return {"logits": _normal(g, torch.float32, 2.0, case["T"], case["E"]).to(t),
                "bias": _normal(g, torch.float32, 0.1, case["E"]) if case["bias"] else None}
    M, N, K, r, n = (case[k] for k in ("M", "N", "K", "rank", "count"))
    return {"X": _normal(g, t, 1.0, M, K),
            "W": _packed(g, case, N, K) if case["group"] else _normal(g, t, 0.02, N, K),
            "A": _normal(g, t, 1 / math.sqrt(K), n, r, K), "B": _normal(g, t, 0.1, n, N, r),
            "s": 0.5 + torch.rand((n,), generator=g, device=DEV),
            "ids": _adapter_ids(g, case)}


def prepare(case, seed):
    state = {"case": case, **_inputs(case, seed)}
    if own and case["op"] == "lora":
        # what a serving program keeps: the handles of the weight and of the adapters
        from dense_gemm_18_amd import LoraAdapters, W4Weight

        state["adapters"] = LoraAdapters(state["A"], state["B"], state["s"])
        if case["group"]:
            state["W"] = W4Weight(*state["W"], shape=(case["N"], case["K"]), group=case["group"])
    return state


# ---- one pass ---------------------------------------------------------------

def run(state):
    return _own(state) if own else _plain(state)


def _own(state):
    import dense_gemm_18_amd as g18

    case = state["case"]
    if case["op"] == "norm":
        if case["out"] == case["type"]:
            return g18.rms_norm(state["x"], state["w"], EPS, residual=state["r"])
        return g18.rms_norm_fp8(state["x"], state["w"], EPS, residual=state["r"],
                                dtype=TYPES[case["out"]])
    if case["op"] == "fp8":
        return g18.gemm_nt(state["A"], state["B"], a_scale=state["sa"], b_scale=state["sb"],
                           dtype=TYPES[case["type"]])
    if case["op"] == "gate":
        return g18.choose_experts(state["logits"], case["topk"], scoring=case["scoring"],
                                  bias=state["bias"], groups=case["groups"],
                                  topk_groups=case["kept"], group_top=case["group_top"],
                                  renormalize=case["renorm"], scale=case["scale"])
    return g18.gemm_nt_lora(state["X"], state["W"], state["adapters"], state["ids"])


def _plain(state):
    return {"norm": _plain_norm, "fp8": _plain_fp8, "gate": _plain_gate,
            "lora": _plain_lora}[state["case"]["op"]](state)


def _plain_norm(state):
    case, t = state["case"], TYPES[state["case"]["type"]]
    s = state["x"].float()
    if case["residual"]:
        s = s + state["r"].float()
    y = s * torch.rsqrt((s * s).mean(-1, keepdim=True) + EPS) * state["w"].float()
    after = [s.to(t)] if case["residual"] else []
    if case["out"] == case["type"]:
        return [y.to(t)] + after if after else y.to(t)
    most = LARGEST[case["out"]]
    scale = y.abs().amax(-1) / most
    q = y / torch.where(scale > 0, scale, torch.ones_like(scale))[:, None]
    return [q.clamp(-most, most).to(TYPES[case["out"]]), scale] + after


def _plain_fp8(state):
    D = state["A"].float() @ state["B"].float().T
    return (D * state["sa"][:, None] * state["sb"]).to(TYPES[state["case"]["type"]])


def _plain_gate(state):
    case, l = state["case"], state["logits"].double()
    score = torch.softmax(l, -1) if case["scoring"] == "softmax" else torch.sigmoid(l)
    choice = score if state["bias"] is None else score + state["bias"].double()
    if case["groups"] > 1:
        T, E, G = case["T"], case["E"], case["groups"]
        inside = torch.sort(choice.view(T, G, E // G), dim=-1, descending=True).values
        value = inside[..., :case["group_top"]].sum(-1)
        best = torch.sort(value, dim=-1, descending=True, stable=True).indices[:, :case["kept"]]
        keep = torch.zeros((T, G), dtype=torch.bool, device=DEV).scatter_(1, best, True)
        choice = choice.masked_fill(~keep.repeat_interleave(E // G, 1), -math.inf)
    ids = torch.sort(choice, dim=-1, descending=True, stable=True).indices[:, :case["topk"]]
    weights = score.gather(1, ids)
    if case["renorm"]:
        weights = weights / weights.sum(-1, keepdim=True)
    return ids.to(torch.int32), (weights * case["scale"]).float()


def _values(W, K, group):
    """A packed weight's values in fp32."""
    Q, S, Z = W
    e = torch.arange(8, device=DEV)
    shifts = (4 * (e // 2) + 16 * (e % 2)).to(torch.int32)
    w = Q.view(Q.shape[0], -1, 4, 4).transpose(-1, -2).unsqueeze(-1)
    q = ((w >> shifts) & 15).flatten(1)[:, :K].float()
    z = 8.0 if Z is None else Z.float().repeat_interleave(group, 1)[:, :K]
    return (q - z) * S.float().repeat_interleave(group, 1)[:, :K]


def _plain_lora(state):
    """Every adapter's first product for every row, those of the others times 0."""
    case, X, ids = state["case"], state["X"].float(), state["ids"]
    n, r = case["count"], case["rank"]
    W = _values(state["W"], case["K"], case["group"]) if case["group"] else state["W"].float()
    U = (X @ state["A"].float().flatten(0, 1).T).view(-1, n, r)
    U = U * ((ids[:, None] == torch.arange(n, device=DEV)) * state["s"]).unsqueeze(-1)
    B = state["B"].float().transpose(1, 2).flatten(0, 1)
    return (X @ W.T + U.flatten(1) @ B).to(TYPES[case["type"]])


# ---- what a pass cannot do without -------------------------------------------

def work(case):
    op = case["op"]
    if op == "norm":
        n = case["T"] * case["H"]
        out = n * 2 if case["out"] == case["type"] else n + 4 * case["T"]
        return {"bytes": 2 * n + (4 * n if case["residual"] else 0) + 2 * case["H"] + out,
                "flops": 5 * n}
    if op == "fp8":
        M, N, K = case["M"], case["N"], case["K"]
        return {"bytes": M * K + N * K + 2 * M * N + 4 * (M + N), "flops": 2 * M * N * K}
    if op == "gate":
        n = case["T"] * case["E"]
        return {"bytes": n * (4 if case["type"] == "f32" else 2) + 8 * case["T"] * case["topk"]
                + (4 * case["E"] if case["bias"] else 0), "flops": 8 * n}
    M, N, K, r, n, group = (case[k] for k in ("M", "N", "K", "rank", "count", "group"))
    weight = 2 * N * K
    if group:
        weight = N * (-(-K // 128) * 64 + -(-K // group) * (3 if case["zeros"] else 2))
    # rows that choose for themselves, and the distinct adapters among them
    asks = max(1, M // 256) if case["runs"] else M
    active = n * (1 - (1 - 0.875 / n) ** asks)
    return {"bytes": 2 * M * (K + N) + weight + active * 2 * r * (K + N) + 4 * M,
            "flops": 2 * M * N * K + 0.875 * 2 * M * r * (K + N)}


# ---- the definition in 64 bits -------------------------------------------------

def exact(case, seed):
    x = _inputs(case, seed)
    return {"norm": _exact_norm, "fp8": _exact_fp8, "gate": _exact_gate,
            "lora": _exact_lora}[case["op"]](case, x)


def _exact_norm(case, x):
    s = x["x"].double()
    if case["residual"]:
        s += x["r"].double()
    length = torch.linalg.vector_norm(s, dim=-1, keepdim=True)
    y = s / torch.sqrt(length ** 2 / case["H"] + EPS) * x["w"].double()
    if case["out"] == case["type"]:
        return [y, s] if case["residual"] else y
    # the scale is held in 32 bits, and the 8-bit values go by what is held
    scale = (torch.maximum(y.amax(-1), -y.amin(-1)) / LARGEST[case["out"]]).float()
    v = (y / scale.double()[:, None]).clamp(-LARGEST[case["out"]], LARGEST[case["out"]])
    # the nearest number of 1 + `bits` binary digits, or multiple of the smallest one, ties
    # to the even one
    bits, least = (3, -9) if case["out"] == "e4m3" else (2, -16)
    step = torch.exp2((torch.frexp(v).exponent.double() - 1 - bits).clamp(min=least))
    return [torch.round(v / step) * step, scale.double()] + ([s] if case["residual"] else [])


def _exact_fp8(case, x):
    return (x["A"].double() * x["sa"].double()[:, None]) @ \
        (x["B"].double() * x["sb"].double()[:, None]).T


def _exact_gate(case, x):
    l, k, G = x["logits"].double(), case["topk"], case["groups"]
    if case["scoring"] == "softmax":
        score = torch.exp(l - torch.logsumexp(l, -1, keepdim=True))
    else:
        score = 1 / (1 + torch.exp(-l))
    choice = score.clone()
    if x["bias"] is not None:
        choice += x["bias"].double()
    if G > 1:
        parts = torch.stack(choice.split(case["E"] // G, dim=1), 1)
        value = torch.topk(parts, case["group_top"], dim=-1).values.sum(-1)
        # a group stays if fewer than `kept` others come before it
        first = (value[:, None, :] > value[:, :, None]) | (
            (value[:, None, :] == value[:, :, None])
            & (torch.arange(G, device=DEV) < torch.arange(G, device=DEV)[:, None]))
        out = first.sum(-1) >= case["kept"]
        choice[out.repeat_interleave(case["E"] // G, 1)] = -math.inf
    ids = torch.empty((case["T"], k), dtype=torch.int64, device=DEV)
    at = torch.arange(case["E"], device=DEV).expand_as(choice)
    for j in range(k):
        most = choice.amax(-1, keepdim=True)
        ids[:, j] = torch.where(choice == most, at, case["E"]).amin(-1)
        choice.scatter_(1, ids[:, j:j + 1], -math.inf)
    weights = score.gather(1, ids) * case["scale"]
    if case["renorm"]:
        weights *= case["scale"] / weights.sum(-1, keepdim=True)
    return ids.to(torch.int32), weights


def _exact_lora(case, x):
    X, ids, K, group = x["X"].double(), x["ids"], case["K"], case["group"]
    if group:
        # element by element from the bytes
        Q, S, Z = x["W"]
        raw = Q.view(torch.uint8)
        k = torch.arange(K, device=DEV)
        nibble = k % 8 // 2 + 4 * (k % 2)
        byte = (k // 128 * 16 + k % 32 // 8 * 4 + k % 128 // 32) * 4 + nibble // 2
        W = ((raw[:, byte] >> (4 * (nibble % 2)).to(torch.uint8)) & 15).double()
        W -= 8 if Z is None else Z.double()[:, k // group]
        W *= S.double()[:, k // group]
    else:
        W = x["W"].double()
    D = X @ W.T
    for a in range(case["count"]):
        t = torch.nonzero(ids == a).squeeze(1)
        if len(t):
            U = X[t] @ x["A"][a].double().T
            D[t] += U @ x["B"][a].double().T * x["s"][a].double()
    return D
