"""The norm with a residual, microscaled 4-bit products and the experts' layer of a few tokens, as cases to
time and to check.

Kinds of case:
  norm_i8    a row's sum with its residual, and that sum's RMS norm in 8-bit integers with a scale per row
  norm_grad  a training step's norm: the sum and its norm, and the gradients of rows and weights
  mx4        rows or weights quantized to microscaled 4-bit floating point, and the values that stand for
  w4a4       y = x . W_hat^T with x quantized to that format on the way
  layer      a few tokens' whole pass through their experts: up products, SwiGLU, down products, weighted sums
"""
import math

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
GROUP = 64  # columns of an expert's activations that share a scale
EPS = 1e-5


def listed():
    return [
        # one token of a decode step before a layer's projections
        {"name": "norm_decode", "kind": "norm_i8", "act": "bf16", "T": 1, "N": 4096},
        # a batch of prompts before a layer's projections
        {"name": "norm_prompt", "kind": "norm_i8", "act": "bf16", "T": 8192, "N": 4096},
        # a small training step in 32 bits, rows that are not whole 16-byte units a lane
        {"name": "grad_ragged", "kind": "norm_grad", "act": "f32", "T": 77, "N": 500},
        # a training step's tokens on one card
        {"name": "grad_train", "kind": "norm_grad", "act": "bf16", "T": 4096, "N": 2048},
        # a layer's up projection quantized as it is loaded
        {"name": "mx4_weights", "kind": "mx4", "act": "f32", "weights": True, "M": 14336, "K": 4096},
        # activations of a few hundred tokens
        {"name": "mx4_rows", "kind": "mx4", "act": "f16", "weights": False, "M": 333, "K": 2080},
        # one token of a decode step through an up projection: the weights' bytes set the time
        {"name": "w4a4_decode", "kind": "w4a4", "act": "bf16", "M": 1, "N": 14336, "K": 4096},
        # a few dozen rows of odd sizes
        {"name": "w4a4_ragged", "kind": "w4a4", "act": "f16", "M": 37, "N": 1001, "K": 2080},
        # a prompt of 1024 tokens through the up projection
        {"name": "w4a4_prompt", "kind": "w4a4", "act": "bf16", "M": 1024, "N": 14336, "K": 4096},
        # one token through two of eight large experts
        {"name": "layer_decode", "kind": "layer", "act": "bf16", "T": 1, "topk": 2, "E": 8, "H": 4096, "I": 14336,
         "pad": 0.0},
        # a few tokens, some of them padding, through small experts of odd sizes
        {"name": "layer_ragged", "kind": "layer", "act": "f16", "T": 5, "topk": 3, "E": 20, "H": 1008, "I": 496,
         "pad": 0.2},
        # a batch of sequences' next tokens through many small experts
        {"name": "layer_batch", "kind": "layer", "act": "bf16", "T": 32, "topk": 8, "E": 64, "H": 2048, "I": 1024,
         "pad": 0.0},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["norm_i8", "norm_grad", "mx4", "w4a4", "layer"])
    act = rng.choice(["bf16", "f16", "f32"])
    if kind == "norm_i8":
        return {"kind": kind, "act": act, "T": _log(rng, 1, 4096), "N": 16 * _log(rng, 4, 400)}
    if kind == "norm_grad":
        N = _log(rng, 64, 8000)
        if rng.random() < 0.6:
            N = (N + 7) // 8 * 8  # most models' widths are whole 16-byte units
        return {"kind": kind, "act": act, "T": _log(rng, 1, 2048), "N": N}
    if kind == "mx4":
        weights = rng.random() < 0.4
        return {"kind": kind, "act": "f32" if weights else act, "weights": weights, "M": _log(rng, 1, 6000),
                "K": 32 * _log(rng, 2, 180)}
    if kind == "w4a4":
        return {"kind": kind, "act": act, "M": _log(rng, 1, 1000), "N": _log(rng, 30, 14000), "K": 32 * _log(rng, 2, 128)}
    E = _log(rng, 2, 64)
    # (outputs of 16 bits, as serving has them: an activation next to a rounding border may fall on either side of it)
    return {"kind": kind, "act": rng.choice(["bf16", "f16"]), "T": _log(rng, 1, 32), "topk": rng.randint(1, min(8, E)),
            "E": E, "H": 16 * _log(rng, 8, 160), "I": 16 * _log(rng, 4, 128), "pad": rng.choice([0.0, 0.0, 0.2])}


def _normal(g, *shape):
    return torch.randn(shape, generator=g, device="cuda")


def _rows(g, M, K, act):
    """Activations: normal, with a few channels of larger magnitude, as models have them."""
    x = _normal(g, M, K)
    loud = torch.rand(K, generator=g, device="cuda") < 0.01
    return torch.where(loud, x * 12.0, x).to(TYPES[act])


def _int8_rows(w):
    """8-bit codes of rows and a scale for each: scale max|w| / 127, codes round(w / scale)."""
    w = w.float()
    a = w.abs().amax(-1) / w.new_tensor(127.0)
    a = torch.where(a == 0, torch.ones_like(a), a)
    return torch.round(w / a[..., None]).clamp_(-127, 127).to(torch.int8), a


def _experts(g, E, N, K):
    codes = torch.empty((E, N, K), dtype=torch.int8, device="cuda")
    scales = torch.empty((E, N), dtype=torch.float32, device="cuda")
    for e in range(E):
        codes[e], scales[e] = _int8_rows(_normal(g, N, K) * (1.0 / math.sqrt(K)))
    return codes, scales


def _inputs(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    kind, act = case["kind"], case["act"]
    dt = TYPES[act]
    s = {"dt": dt}
    if kind in ("norm_i8", "norm_grad"):
        T, N = case["T"], case["N"]
        s["x"], s["residual"] = _rows(g, T, N, act), _rows(g, T, N, act)
        s["weight"] = (1.0 + 0.2 * _normal(g, N)).to(dt)
        if kind == "norm_grad":
            s["dy"], s["dh"] = _normal(g, T, N).to(dt), _normal(g, T, N).to(dt)
        return s
    if kind == "mx4":
        s["x"] = _normal(g, case["M"], case["K"]) * 0.02 if case["weights"] else _rows(g, case["M"], case["K"], act)
        return s
    if kind == "w4a4":
        s["w"] = _normal(g, case["N"], case["K"]) * 0.02
        s["x"] = _rows(g, case["M"], case["K"], act)
        return s
    T, topk, E, H, I = (case[k] for k in ("T", "topk", "E", "H", "I"))
    s["up"], s["up_scales"] = _experts(g, E, 2 * I, H)
    s["down"], s["down_scales"] = _experts(g, E, H, I)
    s["xq"], s["ascale"] = _int8_rows(_rows(g, T, H, act))
    logits = _normal(g, T, E) + 0.5 * _normal(g, E)
    top, ids = torch.topk(logits, topk, dim=1)
    s["weights"] = torch.softmax(top, dim=1).contiguous()
    ids = ids.to(torch.int32)
    if case["pad"] > 0:  # padding tokens go to no expert
        ids[torch.rand(T, generator=g, device="cuda") < case["pad"]] = -1
    s["ids"] = ids.contiguous()
    return s


def prepare(case, seed):
    s = {"case": case, **_inputs(case, seed)}
    kind, dt = case["kind"], s["dt"]
    if kind == "w4a4":
        w = s.pop("w")
        if not own:
            s["w"] = _mx4(w)  # the weights' values, in 32 bits
            return s
    if not own:
        return s
    import gemm_w4a16_amd as lib
    act = {"bf16": lib.W4A16_BF16, "f16": lib.W4A16_FP16, "f32": lib.W4A16_FP32}
    s["act"] = act[case["act"]]
    if kind in ("norm_i8", "norm_grad"):
        T, N = case["T"], case["N"]
        s["h"] = torch.empty((T, N), dtype=dt, device="cuda")
        if kind == "norm_i8":
            s["xq"] = torch.empty((T, N), dtype=torch.int8, device="cuda")
            s["ascale"] = torch.empty(T, dtype=torch.float32, device="cuda")
            s["values_act"] = act[_values_type(case)]
            s["values"] = torch.empty((T, N), dtype=TYPES[_values_type(case)], device="cuda")
        else:
            s["y"], s["dx"] = torch.empty_like(s["h"]), torch.empty_like(s["h"])
            s["dweight"] = torch.empty(N, dtype=torch.float32, device="cuda")
            s["ws"] = lib.alloc_add_rmsnorm_backward_workspace(T, N)
    elif kind == "mx4":
        s["codes"], s["scales"], _ = lib.alloc_packed(lib.W4A16_FMT_MX4_B32_E8M0, case["M"], case["K"])
        s["values_act"] = act[_values_type(case)]
        s["values"] = torch.empty((case["M"], case["K"]), dtype=TYPES[_values_type(case)], device="cuda")
    elif kind == "w4a4":
        M, N, K, fmt = case["M"], case["N"], case["K"], lib.W4A16_FMT_MX4_B32_E8M0
        s["codes"], s["scales"], _ = lib.alloc_packed(fmt, N, K)
        lib.w4a16_quantize_pack(fmt, w, N, K, s["codes"], s["scales"], None)
        s["y"] = torch.empty((M, N), dtype=dt, device="cuda")
        s["ws"] = lib.alloc_w4a4_workspace(fmt, M, N, K)
    else:
        T, topk, E, H, I = (case[k] for k in ("T", "topk", "E", "H", "I"))
        s["y"] = torch.empty((T, H), dtype=dt, device="cuda")
        s["ws"] = lib.alloc_expert_layer_workspace(T, topk, I)
    return s


def _values_type(case):
    """The 16-bit type in which the values that 8-bit or 4-bit codes stand for are given."""
    return "bf16" if case["act"] == "f32" else case["act"]


def run(s):
    return _run_own(s) if own else _run_plain(s)


def _run_own(s):
    import gemm_w4a16_amd as lib
    c, act = s["case"], s["act"]
    kind = c["kind"]
    mx4, w8 = lib.W4A16_FMT_MX4_B32_E8M0, lib.W4A16_FMT_W8_ROW_FP32
    if kind == "norm_i8":
        T, N = c["T"], c["N"]
        lib.w4a16_add_rmsnorm_i8(act, s["x"], s["residual"], T, N, s["weight"], EPS, s["h"], s["xq"], s["ascale"])
        lib.w4a16_dequant(w8, s["xq"], s["ascale"], None, T, N, s["values_act"], s["values"])
        return s["h"], s["values"]
    if kind == "norm_grad":
        T, N = c["T"], c["N"]
        lib.w4a16_add_rmsnorm(act, s["x"], s["residual"], T, N, s["weight"], EPS, s["h"], s["y"])
        lib.w4a16_add_rmsnorm_backward(act, s["dy"], s["dh"], s["h"], T, N, s["weight"], EPS, s["dx"], s["dweight"], *s["ws"])
        return s["h"], s["y"], s["dx"], s["dweight"]
    if kind == "mx4":
        M, K = c["M"], c["K"]
        if c["weights"]:
            lib.w4a16_quantize_pack(mx4, s["x"], M, K, s["codes"], s["scales"], None)
        else:
            lib.w4a16_quantize_rows_mx4(act, s["x"], M, K, s["codes"], s["scales"])
        lib.w4a16_dequant(mx4, s["codes"], s["scales"], None, M, K, s["values_act"], s["values"])
        return s["values"]
    if kind == "w4a4":
        lib.w4a16_matmul_w4a4(mx4, act, s["x"], c["M"], s["codes"], s["scales"], None, c["N"], c["K"], s["y"], *s["ws"])
        return s["y"]
    T, topk, E, H, I = (c[k] for k in ("T", "topk", "E", "H", "I"))
    lib.w4a16_expert_layer_w8a8(w8, act, s["xq"], s["ascale"], T, s["ids"], 32, topk, s["weights"], E, s["up"], s["up_scales"],
                                s["down"], s["down_scales"], H, I, s["y"], *s["ws"])
    return s["y"]


def _mx4(x):
    """The values of rows in blocks of 32 with a power of two each and 4-bit elements, in 32 bits."""
    x = x.float()
    b = x.reshape(x.shape[0], -1, 32)
    _, e = torch.frexp(b.abs().amax(2, keepdim=True))
    e = (e - 3).clamp_(min=-127)  # the largest magnitude's exponent less the largest element's
    a = torch.ldexp(b.abs(), -e)
    # the elements' magnitudes 0, 0.5, 1, 1.5, 2, 3, 4, 6: to the nearest, ties to the even code
    q = 0.5 * ((a > 0.25).float() + (a >= 0.75) + (a > 1.25) + (a >= 1.75))
    q = q + (a > 2.5) + (a >= 3.5) + 2.0 * (a > 5.0)
    return torch.ldexp(torch.copysign(q, b), e).reshape(x.shape)


def _plain_products(rows, ids, codes, scales):
    """rows [T or T * topk][K] against the experts' matrices that ids [T][topk] name: [T][topk][N], 32 bits."""
    (T, topk), (E, N, K) = ids.shape, codes.shape
    rows = rows.reshape(T, -1, K).expand(T, topk, K)
    e = ids.clamp(min=0).long()
    if T * topk < E:  # each pair's own matrix
        w = codes[e.reshape(-1)].float()
        y = torch.bmm(w, rows.reshape(-1, K, 1)).reshape(T, topk, N)
    else:  # every matrix, and each pair's outputs of those
        y = (rows.reshape(-1, K) @ codes.reshape(E * N, K).float().t()).reshape(T, topk, E, N)
        y = y.gather(2, e[:, :, None, None].expand(T, topk, 1, N))[:, :, 0]
    return y * scales[e]


def _run_plain(s):
    c = s["case"]
    kind, dt = c["kind"], s["dt"]
    if kind in ("norm_i8", "norm_grad"):
        h = s["x"].float() + s["residual"].float()
        w = s["weight"].float()
        y = h * torch.rsqrt(h.square().mean(1, keepdim=True) + EPS) * w
        if kind == "norm_i8":
            q, a = _int8_rows(y)
            return h.to(dt), (q.float() * a[:, None]).to(TYPES[_values_type(c)])
        stored = h.to(dt)
        h = stored.float()
        r = torch.rsqrt(h.square().mean(1, keepdim=True) + EPS)
        dy = s["dy"].float()
        g = dy * w
        dx = r * (g - h * (r * r * (g * h).mean(1, keepdim=True))) + s["dh"].float()
        return stored, y.to(dt), dx.to(dt), (dy * h * r).sum(0)
    if kind == "mx4":
        return _mx4(s["x"]).to(TYPES[_values_type(c)])
    if kind == "w4a4":
        return (_mx4(s["x"]) @ s["w"].t()).to(dt)
    ids, H, I = s["ids"], c["H"], c["I"]
    up = _plain_products(s["xq"].float(), ids, s["up"], s["up_scales"]) * s["ascale"][:, None, None]
    g, u = up[..., :I], up[..., I:]
    v = g / (1.0 + torch.exp(-g)) * u
    v = torch.nn.functional.pad(v, (0, -I % GROUP)).reshape(*ids.shape, -1, GROUP)
    q, b = _int8_rows(v)
    v = (q.float() * b[..., None]).reshape(*ids.shape, -1)[..., :I]
    o = _plain_products(v.reshape(-1, I), ids, s["down"], s["down_scales"])
    o = torch.where(ids[:, :, None] >= 0, o * s["weights"][:, :, None], torch.zeros((), device="cuda"))
    return o.sum(1).to(dt)


def _exact_mx4(x):
    """Blocks of 32 by their definition in 64 bits: each value's distance to every element, the nearest taken (of
    two the one of even code), elements beyond the largest becoming the largest."""
    b = x.double().reshape(x.shape[0], -1, 32)
    top = b.abs().amax(2)
    e = torch.where(top > 0, torch.floor(torch.log2(torch.where(top > 0, top, torch.ones_like(top)))), top.new_tensor(-200.0))
    e = torch.where(torch.pow(2.0, e) > top, e - 1, e)  # (a logarithm that rounded up to a whole number)
    X = torch.pow(2.0, (e - 2).clamp(min=-127))[:, :, None]
    a = b.abs() / X
    best, far = torch.zeros_like(a), a.clone()
    for code, value in enumerate((0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)):
        d = (a - value).abs()
        take = (d < far) | ((d == far) & (code % 2 == 0))
        best, far = torch.where(take, torch.full_like(a, value), best), torch.where(take, d, far)
    return (torch.sign(b) * best * X).reshape(x.shape)


def _exact_int8(v):
    """8-bit values of the last dimension's rows, in 64 bits."""
    a = v.abs().amax(-1, keepdim=True) / 127.0
    a = torch.where(a == 0, torch.ones_like(a), a)
    return torch.round(v / a).clamp(-127, 127) * a


def exact(case, seed):
    """The same outputs in 64 bits, the layer's token by token and choice by choice."""
    s = _inputs(case, seed)
    kind = case["kind"]
    if kind in ("norm_i8", "norm_grad"):
        total, w, N = s["x"].double() + s["residual"].double(), s["weight"].double(), case["N"]
        y = total / torch.sqrt((total * total).sum(1, keepdim=True) / N + EPS) * w
        if kind == "norm_i8":
            return total, _exact_int8(y)
        h = total.to(s["dt"]).double()  # what the backward pass is given
        dy = s["dy"].double()
        # the norm's Jacobian, applied: with r the norm's factor, d(h r)/dh = r (1 - h h^T r^2 / N)
        r = 1.0 / torch.sqrt((h * h).sum(1, keepdim=True) / N + EPS)
        unit = h * r
        dx = (dy * w - unit * (dy * w * unit).sum(1, keepdim=True) / N) * r + s["dh"].double()
        return total, y, dx, (dy * unit).sum(0)
    if kind == "mx4":
        return _exact_mx4(s["x"])
    if kind == "w4a4":
        return torch.mm(_exact_mx4(s["x"]), _exact_mx4(s["w"]).t())
    T, topk, H, I = (case[k] for k in ("T", "topk", "H", "I"))
    ids = s["ids"].tolist()
    x = s["xq"].double() * s["ascale"].double()[:, None]
    y = torch.zeros((T, H), dtype=torch.float64, device="cuda")
    for e in range(case["E"]):
        pairs = [(t, j) for t in range(T) for j in range(topk) if ids[t][j] == e]
        if not pairs:
            continue
        t = torch.tensor([p[0] for p in pairs], device="cuda")
        j = torch.tensor([p[1] for p in pairs], device="cuda")
        up = s["up"][e].double() * s["up_scales"][e].double()[:, None]
        gu = torch.mm(x[t], up.t())
        v = gu[:, :I] * torch.sigmoid(gu[:, :I]) * gu[:, I:]
        v = torch.cat([_exact_int8(v[:, k:k + GROUP]) for k in range(0, I, GROUP)], 1)
        down = s["down"][e].double() * s["down_scales"][e].double()[:, None]
        y.index_add_(0, t, torch.mm(v, down.t()) * s["weights"].double()[t, j][:, None])
    return y


def work(case):
    """Bytes that a pass reads and writes at the least, and its operations (a multiply and an add are two).  Of 8-bit
    and 4-bit results, the values that they stand for are counted as what is written.  Of the experts' weights, those
    of the experts that some token needs, as an expected value."""
    kind, b = case["kind"], {"bf16": 2, "f16": 2, "f32": 4}[case["act"]]
    if kind == "norm_i8":
        T, N = case["T"], case["N"]
        return {"bytes": T * N * (3 * b + 2) + N * b, "flops": 8 * T * N}
    if kind == "norm_grad":
        T, N = case["T"], case["N"]
        return {"bytes": T * N * 7 * b + N * (b + 4), "flops": 16 * T * N}
    if kind == "mx4":
        return {"bytes": case["M"] * case["K"] * (b + 2), "flops": 0}
    if kind == "w4a4":
        M, N, K = case["M"], case["N"], case["K"]
        return {"bytes": M * K * b + N * K * 17 // 32 + M * N * b, "flops": 2 * M * N * K}
    T, topk, E, H, I = (case[k] for k in ("T", "topk", "E", "H", "I"))
    live = T * (1 - case["pad"])
    used = E * (1 - (1 - topk / E) ** live)
    weights = used * (3 * I * H + 4 * (2 * I + H))
    return {"bytes": weights + T * (H + 4) + T * topk * 8 + T * H * b, "flops": 2 * live * topk * 3 * I * H}
