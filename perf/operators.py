"""The 8-bit integer product and the experts' operators, as cases to time and to check.

Kinds of case:
  w8a8      y = x . W_hat^T with x quantized to 8-bit integers a token at a time on the way
  dispatch  tokens sorted by expert, and their rows copied in that order
  combine   the experts' rows brought back to their tokens, weighted and summed
  grad      the gradients of both: of the experts' rows and the router's weights from the
            combined rows', and of the tokens' rows from the sorted rows'
  experts   the experts' 8-bit products over sorted rows
  layer     all of a serving pass: sort, gather and quantize, the experts' products, combine
"""
import math

import numpy as np
import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def listed():
    return [
        # one token of a decode step through an up projection: the weights' bytes set the time
        {"name": "w8a8_decode", "kind": "w8a8", "act": "bf16", "M": 1, "N": 14336, "K": 4096},
        # a few dozen rows of odd sizes, as a small batch through a small layer's head
        {"name": "w8a8_ragged", "kind": "w8a8", "act": "f16", "M": 37, "N": 1001, "K": 2064},
        # a prompt of 1024 tokens through the up projection
        {"name": "w8a8_prompt", "kind": "w8a8", "act": "bf16", "M": 1024, "N": 14336, "K": 4096},
        # the smallest step of serving: four tokens to two of eight experts each
        {"name": "dispatch_decode", "kind": "dispatch", "act": "bf16", "T": 4, "topk": 2, "E": 8, "N": 4096, "pad": 0.0},
        # a batch of prompts, a tenth of it padding that goes to no expert
        {"name": "dispatch_prompt", "kind": "dispatch", "act": "bf16", "T": 8192, "topk": 8, "E": 64, "N": 2048,
         "pad": 0.1},
        # odd sizes with padding, rows that are not whole 16-byte chunks
        {"name": "combine_ragged", "kind": "combine", "act": "f16", "T": 333, "topk": 3, "E": 20, "N": 1001,
         "pad": 0.2},
        # a prompt back from the experts
        {"name": "combine_prompt", "kind": "combine", "act": "bf16", "T": 4096, "topk": 2, "E": 8, "N": 4096,
         "pad": 0.0},
        # a small training step in 32 bits
        {"name": "grad_ragged", "kind": "grad", "act": "f32", "T": 77, "topk": 5, "E": 33, "N": 500, "pad": 0.1},
        # a training step's tokens on one card
        {"name": "grad_train", "kind": "grad", "act": "bf16", "T": 4096, "topk": 8, "E": 64, "N": 2048, "pad": 0.0},
        # a decode step of eight tokens: nearly every expert's weights for a row or two
        {"name": "experts_decode", "kind": "experts", "act": "bf16", "T": 8, "topk": 2, "E": 8, "N": 14336, "K": 4096,
         "pad": 0.0},
        # a prompt of 4096 tokens over eight experts, some of them in more demand
        {"name": "experts_prompt", "kind": "experts", "act": "bf16", "T": 4096, "topk": 2, "E": 8, "N": 14336,
         "K": 4096, "pad": 0.0},
        # a batch of 200 sequences' next tokens through many small experts, from rows to rows
        {"name": "layer_batch", "kind": "layer", "act": "f16", "T": 200, "topk": 8, "E": 64, "N": 1024, "K": 2048,
         "pad": 0.1},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["w8a8", "dispatch", "combine", "grad", "experts", "layer"])
    act = rng.choice(["bf16", "f16", "f32"])
    if kind == "w8a8":
        return {"kind": kind, "act": act, "M": _log(rng, 1, 1200), "N": _log(rng, 30, 14000),
                "K": 16 * _log(rng, 4, 256)}
    E = _log(rng, 2, 128)
    topk = rng.randint(1, min(8, E))
    pad = rng.choice([0.0, 0.0, 0.1, 0.5])
    case = {"kind": kind, "act": act, "T": _log(rng, 1, 4096), "topk": topk, "E": E, "N": _log(rng, 64, 2048),
            "pad": pad}
    if kind in ("experts", "layer"):
        case["K"] = 16 * _log(rng, 4, 128)
    elif rng.random() < 0.6:
        case["N"] = case["N"] // 8 * 8  # most models' widths are whole chunks
    return case


def _weights(g, E, N, K):
    """Random weights of E matrices [N][K], quantized to 8 bits with a scale for each row."""
    codes = torch.empty((E, N, K), dtype=torch.int8, device="cuda")
    scales = torch.empty((E, N), dtype=torch.float32, device="cuda")
    for e in range(E):
        w = torch.randn((N, K), generator=g, device="cuda") * 0.02
        s = w.abs().amax(1) / 127.0
        codes[e] = torch.round(w / s[:, None]).clamp_(-127, 127)
        scales[e] = s
    return codes, scales


def _rows(g, M, K, act):
    """Activations: normal, with a few channels of larger magnitude, as models have them."""
    x = torch.randn((M, K), generator=g, device="cuda")
    loud = torch.rand(K, generator=g, device="cuda") < 0.01
    return torch.where(loud, x * 12.0, x).to(TYPES[act])


def _route(g, T, topk, E, pad):
    """A router's choice: `topk` different experts a token, some experts in more demand, and weights
    that sum to one; padding tokens go to no expert (-1)."""
    logits = torch.randn((T, E), generator=g, device="cuda") + 0.5 * torch.randn(E, generator=g, device="cuda")
    top, ids = torch.topk(logits, topk, dim=1)
    weights = torch.softmax(top, dim=1).contiguous()
    ids = ids.to(torch.int32)
    if pad > 0:
        ids[torch.rand(T, generator=g, device="cuda") < pad] = -1
    return ids.contiguous(), weights


def _sorted(ids, E):
    """Each pair's row when pairs are sorted by expert (pairs of one expert in their own order), -1 for
    a pair with no expert; and the experts' first rows [E + 1]."""
    flat = ids.reshape(-1).long()
    key = torch.where((flat >= 0) & (flat < E), flat, E)
    order = torch.sort(key, stable=True).indices
    pos = torch.empty_like(order)
    pos[order] = torch.arange(flat.numel(), device="cuda")
    pos = torch.where(key < E, pos, -1).to(torch.int32).reshape(ids.shape)
    count = torch.bincount(key, minlength=E + 1)[:E]
    offsets = torch.cat([torch.zeros(1, dtype=torch.int64, device="cuda"), count.cumsum(0)]).to(torch.int32)
    return pos, offsets


def _quantized(x):
    """The 8-bit codes and scales of rows: scale max|x| / 127, codes round(x / scale)."""
    x = x.float()
    a = x.abs().amax(1) / 127.0
    a = torch.where(a == 0, torch.ones_like(a), a)
    return torch.round(x / a[:, None]).clamp_(-127, 127).to(torch.int8), a


def _inputs(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    kind, act = case["kind"], case["act"]
    s = {}
    if kind == "w8a8":
        s["codes"], s["scales"] = (t[0] for t in _weights(g, 1, case["N"], case["K"]))
        s["x"] = _rows(g, case["M"], case["K"], act)
        return s
    T, topk, E, N = case["T"], case["topk"], case["E"], case["N"]
    s["ids"], s["weights"] = _route(g, T, topk, E, case["pad"])
    if kind == "dispatch":
        s["x"] = _rows(g, T, N, act)
        return s
    if kind in ("combine", "grad"):
        s["pos"], s["offsets"] = _sorted(s["ids"], E)
        s["ys"] = _rows(g, T * topk, N, act)
        if kind == "grad":
            s["dy"] = _rows(g, T, N, act)
            s["dxs"] = _rows(g, T * topk, N, act)
        return s
    s["codes"], s["scales"] = _weights(g, E, N, case["K"])
    x = _rows(g, T, case["K"], act)
    if kind == "layer":
        s["x"] = x
        return s
    s["pos"], s["offsets"] = _sorted(s["ids"], E)
    xs = torch.zeros((T * topk, case["K"]), dtype=x.dtype, device="cuda")
    at = s["pos"].reshape(-1).long()
    token = torch.arange(T, device="cuda").repeat_interleave(topk)
    xs[at[at >= 0]] = x[token[at >= 0]]
    s["xq"], s["ascale"] = _quantized(xs)
    return s


def prepare(case, seed):
    s = {"case": case, **_inputs(case, seed)}
    kind, dt = case["kind"], TYPES[case["act"]]
    if not own:
        return s
    import gemm_w4a16_amd as w
    s["act"] = {"bf16": w.W4A16_BF16, "f16": w.W4A16_FP16, "f32": w.W4A16_FP32}[case["act"]]
    fmt = w.W4A16_FMT_W8_ROW_FP32
    if kind == "w8a8":
        s["y"] = torch.empty((case["M"], case["N"]), dtype=dt, device="cuda")
        s["ws"] = w.alloc_w8a8_workspace(fmt, case["M"], case["N"], case["K"])
        return s
    T, topk, E, N = case["T"], case["topk"], case["E"], case["N"]
    if kind in ("dispatch", "layer"):
        s["offsets"], s["pos"], s["src"], s["ws"], s["ws_bytes"] = w.alloc_expert_sort(T, topk, E)
    if kind == "dispatch":
        s["xs"] = torch.zeros((T * topk, N), dtype=dt, device="cuda")
    if kind in ("combine", "layer"):
        s["y"] = torch.empty((T, N), dtype=dt, device="cuda")
    if kind == "grad":
        s["dys"] = torch.zeros((T * topk, N), dtype=dt, device="cuda")
        s["dweights"] = torch.empty((T, topk), dtype=torch.float32, device="cuda")
        s["dx"] = torch.empty((T, N), dtype=dt, device="cuda")
    if kind in ("experts", "layer"):
        s["ys"] = torch.zeros((T * topk, N), dtype=dt, device="cuda")
    if kind == "layer":
        s["xq"] = torch.empty((T * topk, case["K"]), dtype=torch.int8, device="cuda")
        s["ascale"] = torch.empty(T * topk, dtype=torch.float32, device="cuda")
    return s


def run(s):
    return _run_own(s) if own else _run_plain(s)


def _run_own(s):
    import gemm_w4a16_amd as w
    c, act, fmt = s["case"], s["act"], w.W4A16_FMT_W8_ROW_FP32
    kind = c["kind"]
    if kind == "w8a8":
        ws, ws_bytes = s["ws"]
        w.w4a16_matmul_w8a8(fmt, act, s["x"], c["M"], s["codes"], s["scales"], None, c["N"], c["K"], s["y"], ws, ws_bytes)
        return s["y"]
    T, topk, E, N = c["T"], c["topk"], c["E"], c["N"]
    if kind == "dispatch":
        w.w4a16_expert_sort(s["ids"], 32, T, topk, E, s["offsets"], s["pos"], s["src"], s["ws"], s["ws_bytes"])
        w.w4a16_expert_gather(act, s["x"], T, topk, s["pos"], N, s["xs"])
        return s["offsets"], s["pos"], s["src"], s["xs"]
    if kind == "combine":
        w.w4a16_expert_combine(act, s["ys"], T, topk, s["pos"], s["weights"], N, s["y"])
        return s["y"]
    if kind == "grad":
        w.w4a16_expert_combine_backward(act, s["dy"], s["ys"], T, topk, s["pos"], s["weights"], N, s["dys"],
                                        s["dweights"])
        w.w4a16_expert_combine(act, s["dxs"], T, topk, s["pos"], None, N, s["dx"])
        return s["dys"], s["dweights"], s["dx"]
    K, R = c["K"], T * topk
    if kind == "layer":
        w.w4a16_expert_sort(s["ids"], 32, T, topk, E, s["offsets"], s["pos"], s["src"], s["ws"], s["ws_bytes"])
        w.w4a16_expert_gather_i8(act, s["x"], T, topk, s["pos"], K, s["xq"], s["ascale"])
    w.w4a16_gemm_w8a8_experts(fmt, act, s["xq"], s["ascale"], R, s["offsets"], E, s["codes"], s["scales"], None, N, K,
                              s["ys"])
    if kind == "experts":
        return s["ys"]
    w.w4a16_expert_combine(act, s["ys"], T, topk, s["pos"], s["weights"], N, s["y"])
    return s["y"]


def _plain_sort(ids, E):
    flat = ids.reshape(-1)
    hit = torch.arange(E, device="cuda", dtype=flat.dtype)[:, None] == flat  # [E][pairs]
    seen = hit.to(torch.int32).cumsum(1, dtype=torch.int32)
    offsets = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    offsets[1:] = seen[:, -1].cumsum(0, dtype=torch.int32)
    row = ((seen + offsets[:-1, None]) * hit).sum(0, dtype=torch.int32) - 1
    return offsets, row.reshape(ids.shape)


def _plain_product(xq, ascale, codes, scales):
    return (xq.float() @ codes.float().t()) * ascale[:, None] * scales[None, :]


def _plain_experts(xq, ascale, offsets, codes, scales, dt):
    y = torch.zeros((xq.shape[0], codes.shape[1]), dtype=dt, device="cuda")
    first = offsets.tolist()
    for e in range(codes.shape[0]):
        a, b = first[e], first[e + 1]
        if b > a:
            y[a:b] = _plain_product(xq[a:b], ascale[a:b], codes[e], scales[e]).to(dt)
    return y


def _plain_combine(ys, pos, weights, dt):
    part = ys[pos.clamp(min=0).long()].float()  # [T][topk][N]
    part = torch.where(pos[:, :, None] >= 0, part, torch.zeros((), device="cuda"))
    if weights is not None:
        part = part * weights[:, :, None]
    return part.sum(1).to(dt)


def _plain_gather(rows, pos, src_rows, dt):
    """rows[token] (already [T][topk][N] or [T][1][N]) written to their sorted places."""
    out = torch.zeros((src_rows + 1, rows.shape[-1]), dtype=dt, device="cuda")
    at = torch.where(pos >= 0, pos, src_rows).long()  # pairs with no expert share one more row, cut off
    out[at.reshape(-1)] = rows.expand(-1, pos.shape[1], -1).reshape(-1, rows.shape[-1]).to(dt)
    return out[:src_rows]


def _run_plain(s):
    c = s["case"]
    kind, dt = c["kind"], TYPES[c["act"]]
    if kind == "w8a8":
        xq, a = _quantized(s["x"])
        return _plain_product(xq, a, s["codes"], s["scales"]).to(dt)
    T, topk, E = c["T"], c["topk"], c["E"]
    R = T * topk
    if kind == "dispatch":
        offsets, pos = _plain_sort(s["ids"], E)
        src = torch.full((R + 1,), -1, dtype=torch.int32, device="cuda")
        src[torch.where(pos >= 0, pos, R).reshape(-1).long()] = torch.arange(R, dtype=torch.int32, device="cuda")
        src[R] = -1
        return offsets, pos, src[:R], _plain_gather(s["x"][:, None, :], pos, R, dt)
    if kind == "combine":
        return _plain_combine(s["ys"], s["pos"], s["weights"], dt)
    if kind == "grad":
        pos, dy = s["pos"], s["dy"].float()
        dys = _plain_gather(dy[:, None, :] * s["weights"][:, :, None], pos, R, dt)
        dot = (s["ys"][pos.clamp(min=0).long()].float() * dy[:, None, :]).sum(2)
        return dys, torch.where(pos >= 0, dot, torch.zeros_like(dot)), _plain_combine(s["dxs"], pos, None, dt)
    if kind == "experts":
        return _plain_experts(s["xq"], s["ascale"], s["offsets"], s["codes"], s["scales"], dt)
    offsets, pos = _plain_sort(s["ids"], E)
    xq, a = _quantized(s["x"])
    xs = _plain_gather(xq[:, None, :], pos, R, torch.int8)
    ascale = _plain_gather(a[:, None, None], pos, R, torch.float32)[:, 0]
    ys = _plain_experts(xs, ascale, offsets, s["codes"], s["scales"], dt)
    return _plain_combine(ys, pos, s["weights"], dt)


def _exact_quantized(x):
    """Codes and scales by their definition: one IEEE division in 32 bits each, ties to even."""
    x = x.float().cpu().numpy()
    a = np.abs(x).max(1) / np.float32(127.0)
    a[a == 0] = 1
    q = np.clip(np.rint(x / a[:, None]), -127, 127)
    return torch.from_numpy(q).cuda().double(), torch.from_numpy(a).cuda().double()


def exact(case, seed):
    """The same outputs in 64 bits, token by token and expert by expert."""
    s = _inputs(case, seed)
    kind = case["kind"]
    if kind == "w8a8":
        q, a = _exact_quantized(s["x"])
        return torch.mm(q * a[:, None], (s["codes"].double() * s["scales"].double()[:, None]).t())
    T, topk, E, N = case["T"], case["topk"], case["E"], case["N"]
    R = T * topk
    ids = s["ids"].cpu().numpy().reshape(-1)
    pairs = [np.nonzero(ids == e)[0] for e in range(E)]  # each expert's pairs, in their own order
    offsets = np.concatenate([[0], np.cumsum([len(p) for p in pairs])])
    order = np.concatenate(pairs)
    pos = np.full(R, -1)
    pos[order] = np.arange(len(order))
    tok = torch.from_numpy(order // topk).cuda()  # the token of each sorted row
    pair = torch.from_numpy(order).cuda()
    n = len(order)

    def zeros(rows, width):
        return torch.zeros((rows, width), dtype=torch.float64, device="cuda")

    def summed(rows):  # sorted rows added to their tokens
        y = zeros(T, rows.shape[1])
        return y.index_add_(0, tok, rows[:n])

    if kind == "dispatch":
        xs = zeros(R, N)
        xs[:n] = s["x"].double()[tok]
        src = np.full(R, -1)
        src[:n] = order
        return offsets.astype(np.int32), pos.astype(np.int32).reshape(T, topk), src.astype(np.int32), xs
    weight = s["weights"].double().reshape(-1)[pair][:, None]
    if kind == "combine":
        return summed(s["ys"][:n].double() * weight)
    if kind == "grad":
        dy = s["dy"].double()[tok]
        dys, dw = zeros(R, N), zeros(R, 1)
        dys[:n] = dy * weight
        dw[pair] = (s["ys"][:n].double() * dy).sum(1, keepdim=True)
        return dys, dw.reshape(T, topk), summed(s["dxs"].double())
    if kind == "experts":
        q, a = s["xq"].double(), s["ascale"].double()
    else:
        q, a = (t[tok] for t in _exact_quantized(s["x"]))
    ys = zeros(R, N)
    for e in range(E):
        lo, hi = int(offsets[e]), int(offsets[e + 1])
        if hi > lo:
            ys[lo:hi] = torch.mm(q[lo:hi] * a[lo:hi, None], (s["codes"][e].double() * s["scales"][e].double()[:, None]).t())
    if kind == "experts":
        return ys
    return summed(ys[:n] * weight)


def work(case):
    """Bytes that a pass reads and writes at the least, and its operations (a multiply and an add are
    two).  Padding tokens and their rows are left out as expected values; of the experts' weights, those
    of the experts that some row needs (all, where the rows outnumber the experts by far)."""
    kind, b = case["kind"], {"bf16": 2, "f16": 2, "f32": 4}[case["act"]]
    if kind == "w8a8":
        M, N, K = case["M"], case["N"], case["K"]
        return {"bytes": M * K * b + N * K + 4 * N + M * N * b, "flops": 2 * M * N * K}
    T, topk, E, N = case["T"], case["topk"], case["E"], case["N"]
    live_t = T * (1 - case["pad"])
    live = live_t * topk
    if kind == "dispatch":
        return {"bytes": T * topk * 4 * 3 + 4 * (E + 1) + (live_t + live) * N * b, "flops": 0}
    if kind == "combine":
        return {"bytes": T * topk * 8 + (live + T) * N * b, "flops": 2 * live * N}
    if kind == "grad":
        return {"bytes": T * topk * 12 + (live_t + 3 * live + T) * N * b, "flops": 4 * live * N}
    K = case["K"]
    used = E * (1 - (1 - topk / E) ** live_t)
    weights = used * (N * K + 4 * N)
    if kind == "experts":
        return {"bytes": live * (K + 4) + weights + live * N * b, "flops": 2 * live * N * K}
    return {"bytes": T * topk * 8 + live_t * K * b + weights + T * N * b, "flops": 2 * live * N * K}
