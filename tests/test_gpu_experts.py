"""The experts' operators on the GPU against plain implementations: the sorted order and the gathered
rows exactly, the sums in 64 bits.

Bounds (u: half a step of the output type, 2^-8 bf16, 2^-11 fp16, 0 for fp32, whose last rounding is
among the fp32 ones):
  combine    topk fused multiply-adds in fp32: topk 2^-24 sum_j |w ys|, then u |y|
  dys        one product in fp32 and one rounding: (u + 2^-24) |dys|
  dweights   a thread adds N / 256 products in a row (one 16-byte unit of 8 at the least), then a tree
             over 64 lanes and 4 waves, below 2^3 levels and 2^2 more: (N / 256 + 32) 2^-24 sum_n |dy ys|
  products   as for the 8-bit product: (u + 4 2^-24) |y|
"""
import numpy as np
import pytest
import torch

import gemm_w4a16_amd as w
from test_gpu_w8a8 import TYPES, W8, check, product, product_on_gpu, quantized, rows, weights

pytestmark = pytest.mark.gpu

F24 = 2.0 ** -24


def route(T, topk, E, seed, pad=0.1, skew=False):
    """Expert numbers of random tokens; some tokens are padding, some numbers out of range, some
    experts get nothing and a token may name one expert twice."""
    g = np.random.default_rng(seed)
    ids = g.integers(0, E, (T, topk))
    if skew:
        ids[g.random((T, topk)) < 0.7] = E // 2
    if pad:
        ids[g.random(T) < pad] = -1
        ids[g.random((T, topk)) < pad / 4] = E
    return ids


def sorted_order(ids, E):
    flat = ids.reshape(-1)
    P = flat.size
    order = np.concatenate([np.nonzero(flat == e)[0] for e in range(E)])
    offsets = np.concatenate([[0], np.cumsum([(flat == e).sum() for e in range(E)])])
    pos = np.full(P, -1)
    pos[order] = np.arange(order.size)
    src = np.full(P, -1)
    src[:order.size] = order
    return offsets.astype(np.int32), pos.astype(np.int32).reshape(ids.shape), src.astype(np.int32)


def gpu_sort(ids, E, bits=32, src=True):
    T, topk = ids.shape
    offsets, pos, s, ws, nb = w.alloc_expert_sort(T, topk, E)
    for t in (offsets, pos, s):
        t.fill_(-77)
    if ws is not None:
        ws.fill_(0xFF)
    d = torch.from_numpy(ids.astype(np.int64 if bits == 64 else np.int32)).cuda()
    w.w4a16_expert_sort(d, bits, T, topk, E, offsets, pos, s if src else None, ws, nb)
    return offsets, pos, s


SORTS = [(1, 1, 1), (1, 2, 8), (4, 2, 8), (7, 3, 5), (64, 1, 64), (65, 8, 64), (1000, 8, 128), (333, 3, 512), (1024, 8, 60),
         (4096, 1, 3), (4097, 1, 3), (8192, 1, 3), (2048, 1, 512), (1025, 1, 2), (4097, 2, 512), (5000, 7, 33), (70000, 4, 256), (3000, 100, 16)]


@pytest.mark.parametrize("T,topk,E", SORTS)
@pytest.mark.parametrize("bits", [32, 64])
def test_sort(T, topk, E, bits):
    for seed, pad, skew in [(1, 0.0, False), (2, 0.3, True)]:
        ids = route(T, topk, E, seed, pad, skew)
        for got, ref in zip(gpu_sort(ids, E, bits), sorted_order(ids, E)):
            np.testing.assert_array_equal(got.cpu().numpy(), ref)


def test_sort_of_numbers_out_of_range():
    """Ids far outside [0, E), also ones whose low 32 bits are inside, and a batch of padding alone."""
    ids = np.array([[0, 2 ** 32], [-2 ** 40, 1], [2 ** 62, -1], [3, 2 ** 31]], dtype=np.int64)
    offsets, pos, src = gpu_sort(ids, 4, 64)
    assert offsets.tolist() == [0, 1, 2, 2, 3] and pos.tolist() == [[0, -1], [-1, 1], [-1, -1], [2, -1]]
    assert src.tolist() == [0, 3, 6, -1, -1, -1, -1, -1]
    for T in (3, 9000):
        offsets, pos, src = gpu_sort(np.full((T, 2), -1), 5)
        assert (offsets == 0).all() and (pos == -1).all() and (src == -1).all()


def test_sort_without_src():
    ids = route(500, 4, 16, 5)
    offsets, pos, src = gpu_sort(ids, 16, src=False)
    ref = sorted_order(ids, 16)
    np.testing.assert_array_equal(offsets.cpu().numpy(), ref[0])
    np.testing.assert_array_equal(pos.cpu().numpy(), ref[1])
    assert (src == -77).all()


ROWS = [(1, 1, 1, 8), (4, 2, 8, 4096), (37, 3, 5, 1), (37, 3, 5, 1001), (200, 8, 64, 520), (513, 5, 16, 72), (9, 20, 30, 24),
        (33, 2, 4, 9000)]
# rows that are not whole 16-byte units: an element past them, one short of them, of many units, of more than 64 MiB
ROWS += [(70, 2, 8, 4), (70, 3, 8, 9), (41, 2, 5, 15), (300, 4, 9, 63), (300, 4, 9, 65), (55, 2, 6, 511), (129, 2, 4, 517), (20, 3, 4, 2049),
         (33, 2, 4, 9001), (4200, 2, 4, 4099)]


def plan(T, topk, E, seed, pad=0.2):
    ids = route(T, topk, E, seed, pad)
    offsets, pos, src = sorted_order(ids, E)
    return pos, int(offsets[-1]), torch.from_numpy(pos).cuda()


@pytest.mark.parametrize("T,topk,E,N", ROWS)
@pytest.mark.parametrize("kind", list(TYPES))
def test_gather(T, topk, E, N, kind):
    act, dt = TYPES[kind][:2]
    pos, n, dpos = plan(T, topk, E, 21)
    x = rows(T, N, dt, 22) if N > 8 else torch.randn((T, N)).to(dt)
    xs = torch.full((T * topk, N), 7.0, dtype=dt, device="cuda")
    w.w4a16_expert_gather(act, x.cuda(), T, topk, dpos, N, xs)
    xs = xs.cpu()
    for t in range(T):
        for j in range(topk):
            if pos[t, j] >= 0:
                assert torch.equal(xs[pos[t, j]], x[t])
    assert (xs[n:] == 7).all()  # rows behind the experts' are left as they were


@pytest.mark.parametrize("T,topk,E,K", [(1, 1, 1, 16), (4, 2, 8, 4096), (37, 3, 5, 1008), (200, 8, 64, 2048), (9, 20, 30, 48), (1500, 3, 7, 1008),
                                        (1026, 2, 4, 4096), (1030, 2, 5, 4112)])
@pytest.mark.parametrize("kind", list(TYPES))
def test_gather_i8(T, topk, E, K, kind):
    act, dt = TYPES[kind][:2]
    pos, n, dpos = plan(T, topk, E, 23)
    x = rows(T, K, dt, 24)
    xq = torch.full((T * topk, K), 99, dtype=torch.int8, device="cuda")
    a = torch.full((T * topk,), -3.0, device="cuda")
    w.w4a16_expert_gather_i8(act, x.cuda(), T, topk, dpos, K, xq, a)
    q, ra = quantized(x)
    t, j = np.nonzero(pos >= 0)
    np.testing.assert_array_equal(xq.cpu().numpy()[pos[t, j]], q[t])
    np.testing.assert_array_equal(a.cpu().numpy()[pos[t, j]], ra[t])
    assert (xq[n:] == 99).all() and (a[n:] == -3).all()


def test_rows_past_32_bit_offsets():
    """More than 2^31 elements of sorted rows, gathered and brought back: the tokens at both ends and around
    the border, and the gradients' rows."""
    T, topk, E, N = 70_001, 8, 16, 4096  # 2.3e9 elements
    ids = torch.randint(0, E, (T, topk), dtype=torch.int32, device="cuda", generator=torch.Generator(device="cuda").manual_seed(7))
    offsets, pos, src, ws, nb = w.alloc_expert_sort(T, topk, E)
    w.w4a16_expert_sort(ids, 32, T, topk, E, offsets, pos, src, ws, nb)
    x = torch.randn((T, N), device="cuda").bfloat16()
    xs = torch.empty((T * topk, N), dtype=torch.bfloat16, device="cuda")
    w.w4a16_expert_gather(w.W4A16_BF16, x, T, topk, pos, N, xs)
    for t in (0, 1, T // 2, T - 1):
        for j in range(topk):
            assert torch.equal(xs[int(pos[t, j])], x[t])
    border = 2 ** 31 // N
    for r in (border - 1, border, border + 1, T * topk - 1):
        assert torch.equal(xs[r], x[int(src[r]) // topk])
    y = torch.empty_like(x)
    w.w4a16_expert_combine(w.W4A16_BF16, xs, T, topk, pos, None, N, y)
    assert torch.equal(y[::997], (x[::997].float() * topk).bfloat16())  # eight equal rows: exact
    dw = torch.empty((T, topk), device="cuda")
    dys = xs  # its rows are written anew
    w.w4a16_expert_combine_backward(w.W4A16_BF16, x, xs.clone(), T, topk, pos, torch.full((T, topk), 0.5, device="cuda"), N, dys, dw)
    for r in (0, border - 1, border, border + 1, T * topk - 1):
        assert torch.equal(dys[r], (x[int(src[r]) // topk].float() * 0.5).bfloat16())
    some = torch.tensor([0, 5, T // 2, T - 1], device="cuda")
    ref = (x[some].double() ** 2).sum(1, keepdim=True)
    assert ((dw[some].double() - ref).abs() <= (N / 256 + 32) * F24 * ref).all()
    xq, a = torch.empty((T * topk, N), dtype=torch.int8, device="cuda"), torch.empty(T * topk, device="cuda")
    w.w4a16_expert_gather_i8(w.W4A16_BF16, x, T, topk, pos, N, xq, a)
    at = torch.tensor([0, border - 1, border, border + 1, T * topk - 1], device="cuda")
    q, ra = quantized(x[src[at].long() // topk].cpu())
    np.testing.assert_array_equal(xq[at].cpu().numpy(), q)
    np.testing.assert_array_equal(a[at].cpu().numpy(), ra)


def combined(ys, pos, wt):
    """sum_j w ys[pos], and the sum of the terms' magnitudes, in 64 bits."""
    ys, live = ys.double(), torch.from_numpy(pos >= 0)
    part = ys[torch.from_numpy(pos).clamp(min=0).long()] * wt.double()[:, :, None]
    part = torch.where(live[:, :, None], part, torch.zeros((), dtype=torch.float64))
    return part.sum(1), part.abs().sum(1)


@pytest.mark.parametrize("T,topk,E,N", ROWS)
@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("weighted", [True, False])
def test_combine(T, topk, E, N, kind, weighted):
    act, dt, u, tiny = TYPES[kind]
    pos, n, dpos = plan(T, topk, E, 31)
    g = torch.Generator().manual_seed(32)
    ys = torch.randn((T * topk, N), generator=g).to(dt)
    ys[n:] = float("nan")  # never read
    wt = torch.rand((T, topk), generator=g) - 0.2
    y = torch.full((T, N), float("nan"), dtype=dt, device="cuda")
    w.w4a16_expert_combine(act, ys.cuda(), T, topk, dpos, wt.cuda() if weighted else None, N, y)
    ref, mag = combined(torch.nan_to_num(ys), pos, wt if weighted else torch.ones_like(wt))
    bound = u * ref.abs() + (1 + u) * topk * F24 * mag + tiny
    assert ((y.cpu().double() - ref).abs() <= bound).all()
    assert (y.cpu()[(pos < 0).all(1)] == 0).all()


def test_combine_ignores_pairs_without_a_row():
    """Weights of NaN and infinity at pairs that go nowhere, rows of NaN that no pair names; a weight of
    zero on an infinite row is NaN, as the formula has it."""
    T, topk, N = 6, 3, 40
    pos = torch.tensor([[0, -1, 1], [-1, -1, -1], [2, 3, -1], [-1, 4, 18], [5, -9, 10 ** 9], [6, 7, -1]], dtype=torch.int32)
    ys = torch.randn((T * topk, N))
    ys[8:] = float("nan")
    ys[7, 0] = float("inf")
    wt = torch.rand((T, topk)) + 0.5
    wt[pos < 0] = float("nan")
    wt[3, 2], wt[4, 2], wt[5, 1] = float("inf"), float("nan"), 0.0
    y = torch.empty((T, N), device="cuda")
    w.w4a16_expert_combine(w.W4A16_FP32, ys.cuda(), T, topk, pos.cuda(), wt.cuda(), N, y)
    y = y.cpu()
    assert y[5, 0].isnan() and not y[5, 1:].isnan().any() and not y[:5].isnan().any() and (y[1] == 0).all()
    assert torch.allclose(y[3], wt[3, 1] * ys[4]) and torch.allclose(y[4], wt[4, 0] * ys[5])


@pytest.mark.parametrize("N", [4, 9, 13, 40, 69, 1003])
@pytest.mark.parametrize("kind", list(TYPES))
def test_infinities_at_the_ends_of_rows(N, kind):
    """An infinity in a row's first or last elements counts once in its dot product and reaches no other row."""
    act, dt = TYPES[kind][:2]
    T, pos = 4, torch.tensor([[0, 1], [2, 3], [4, 5], [6, 7]], dtype=torch.int32, device="cuda")
    dy, ys = torch.ones((T, N), dtype=dt), torch.ones((8, N), dtype=dt)
    ys[0, N - 1], ys[2, N - 2], ys[5, 0], ys[6, N // 2] = float("inf"), -float("inf"), float("inf"), float("inf")
    dw = torch.empty((T, 2), device="cuda")
    w.w4a16_expert_combine_backward(act, dy.cuda(), ys.cuda(), T, 2, pos, None, N, None, dw)
    inf = float("inf")
    assert dw.tolist() == [[inf, N], [-inf, N], [N, inf], [inf, N]]  # (sums of ones are exact)
    y = torch.empty((T, N), dtype=dt, device="cuda")
    w.w4a16_expert_combine(act, ys.cuda(), T, 2, pos, None, N, y)
    assert torch.equal(y.cpu(), ys[0::2] + ys[1::2])


@pytest.mark.parametrize("T,topk,E,N", ROWS)
@pytest.mark.parametrize("kind", list(TYPES))
def test_combine_backward(T, topk, E, N, kind):
    act, dt, u, tiny = TYPES[kind]
    pos, n, dpos = plan(T, topk, E, 41)
    g = torch.Generator().manual_seed(42)
    ys, dy = torch.randn((T * topk, N), generator=g).to(dt), torch.randn((T, N), generator=g).to(dt)
    ys[n:] = float("nan")
    wt = torch.rand((T, topk), generator=g) - 0.2
    P = T * topk
    dys = torch.full((P, N), 7.0, dtype=dt, device="cuda")
    dw = torch.full((T, topk), float("nan"), device="cuda")
    args = (dy.cuda(), ys.cuda(), T, topk, dpos, wt.cuda(), N)
    w.w4a16_expert_combine_backward(act, *args, dys, dw)
    t, j = np.nonzero(pos >= 0)
    at = torch.from_numpy(pos[t, j]).long()
    ref = dy.double()[t] * wt.double()[t, j][:, None]
    assert ((dys.cpu().double()[at] - ref).abs() <= (u + 2 * F24) * ref.abs() + tiny).all()
    assert (dys[n:] == 7).all()
    term = ys.double()[at] * dy.double()[t]
    got = dw.cpu().double()
    assert ((got[t, j] - term.sum(1)).abs() <= (N / 256 + 32) * F24 * term.abs().sum(1)).all()
    assert (got[torch.from_numpy(pos < 0)] == 0).all()
    # each gradient alone, and without weights, is the same
    dys2, dw2 = torch.full_like(dys, 7.0), torch.full_like(dw, float("nan"))
    w.w4a16_expert_combine_backward(act, args[0], None, *args[2:], dys2, None)
    w.w4a16_expert_combine_backward(act, *args, None, dw2)
    assert torch.equal(dys2, dys) and torch.equal(dw2, dw)
    ones = torch.full_like(dys, 7.0)
    w.w4a16_expert_combine_backward(act, args[0], None, T, topk, dpos, None, N, ones, None)
    gathered = torch.full_like(dys, 7.0)
    w.w4a16_expert_gather(act, args[0], T, topk, dpos, N, gathered)
    assert torch.equal(ones, gathered)


def test_gradients_against_differences():
    """combine is linear in the rows and in the weights: its values at two points give the gradients of
    L = sum(y g) up to rounding.  With h a power of two the step itself is exact; a value of L is off
    by at most (topk + 1) 2^-24 times the terms' magnitudes, and so is the gradient over 2 h."""
    T, topk, E, N, h = 5, 3, 4, 24, 0.5
    pos, n, dpos = plan(T, topk, E, 51)
    g = torch.Generator().manual_seed(52)
    ys, dy, wt = (torch.randn(s, generator=g) for s in ((T * topk, N), (T, N), (T, topk)))
    dys, dw = torch.zeros((T * topk, N), device="cuda"), torch.zeros((T, topk), device="cuda")
    w.w4a16_expert_combine_backward(w.W4A16_FP32, dy.cuda(), ys.cuda(), T, topk, dpos, wt.cuda(), N, dys, dw)
    dx = torch.empty((T, N), device="cuda")  # the gather's gradient: of rows that all came from x
    w.w4a16_expert_combine(w.W4A16_FP32, ys.cuda(), T, topk, dpos, None, N, dx)

    def value(ys, wt):
        y = torch.empty((T, N), device="cuda")
        w.w4a16_expert_combine(w.W4A16_FP32, ys.cuda(), T, topk, dpos, wt.cuda(), N, y)
        return y.cpu().double()

    bound = 2 * (topk + 1) * F24 * 60.0 / (2 * h) * N  # |w ys g| of a term below 60 (|randn| < 4)
    for t, j in [(0, 0), (1, 2), (4, 1), (2, 2)]:
        step = torch.zeros_like(wt)
        step[t, j] = h
        diff = ((value(ys, wt + step) - value(ys, wt - step)) * dy.double()).sum() / (2 * h)
        assert abs(diff.item() - dw[t, j].item()) <= bound
    for r, c in [(0, 0), (1, 5), (n - 1, N - 1)]:
        step = torch.zeros_like(ys)
        step[r, c] = h
        diff = ((value(ys + step, wt) - value(ys - step, wt)) * dy.double()).sum() / (2 * h)
        assert abs(diff.item() - dys[r, c].item()) <= bound

    def gathered(x):
        xs = torch.zeros((T * topk, N), device="cuda")
        w.w4a16_expert_gather(w.W4A16_FP32, x.cuda(), T, topk, dpos, N, xs)
        return xs.cpu().double()

    x = torch.randn((T, N), generator=g)
    for t, c in [(0, 0), (3, 7), (4, N - 1)]:
        step = torch.zeros_like(x)
        step[t, c] = h
        diff = ((gathered(x + step) - gathered(x - step)) * ys.double()).sum() / (2 * h)
        assert abs(diff.item() - dx[t, c].item()) <= bound


# ---- the experts' products ----------------------------------------------------------------------

def experts_product(q, a, offsets, codes, scales, E, N):
    K = q.shape[1]
    y = torch.full((q.shape[0], N), float("nan"), dtype=torch.float64)
    c, s = codes.view(E, N, K), scales.view(E, N)
    for e in range(E):
        lo, hi = offsets[e], offsets[e + 1]
        if hi > lo:
            y[lo:hi] = product(q[lo:hi], a[lo:hi], c[e], s[e])
    return y


COUNTS = [  # rows of each expert, rows behind them
    ([1], 0), ([0, 0, 3, 0], 2), ([1, 1, 1, 1, 1, 1, 1, 1], 0), ([16, 17, 0, 15, 1], 5), ([0, 300, 0, 2, 0], 1), ([64, 128, 65, 129], 0),
    ([257, 5, 0, 256], 40), ([0] * 70 + [9] + [0] * 30 + [40], 3), ([2] * 200, 0), ([700, 1, 30], 9)]


@pytest.mark.parametrize("counts,behind", COUNTS)
@pytest.mark.parametrize("N,K,kind", [(61, 48, "bf16"), (256, 528, "f16"), (300, 1040, "f32")])
def test_experts_products(counts, behind, N, K, kind):
    E, n = len(counts), sum(counts)
    R = n + behind
    act, dt = TYPES[kind][:2]
    offsets = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    q, a = quantized(rows(R, K, dt, 61))
    codes, scales = weights(N, K, 62, E)
    y = torch.full((R, N), 7.0, dtype=dt, device="cuda")
    w.w4a16_gemm_w8a8_experts(W8, act, torch.from_numpy(q).cuda(), torch.from_numpy(a).cuda(), R, torch.from_numpy(offsets).cuda(),
                              E, codes.cuda(), scales.cuda(), None, N, K, y)
    check(y[:n], experts_product(q, a, offsets, codes, scales, E, N)[:n], kind)
    assert (y[n:] == 7).all()


WIDE = [([520, 1, 700], 7, 61, 1040), ([2] * 9, 4, 1001, 1040), ([260] * 8, 0, 61, 1040), ([130, 0, 128, 257], 3, 515, 144),
        ([17] * 20, 0, 1001, 1040), ([40] * 32, 11, 520, 1040), ([260] * 8, 1, 1001, 1040), ([1030, 900], 0, 2056, 400),
        ([520, 1, 700], 300, 8200, 1040), ([0, 0, 900, 0, 300, 1], 2, 8200, 144),
        ([1, 0, 2, 1] * 4, 3, 2056, 2064), ([20, 0, 33, 17] * 4, 0, 2056, 2064), ([1] * 512, 0, 64, 80), ([0] * 511 + [3], 1, 64, 80)]


MORE = [([1], 1, 37, 1584), ([2, 1, 0, 2], 0, 917, 18592), ([4, 1, 3, 0, 2, 5], 0, 2648, 4240), ([9, 0, 1, 1, 2, 0, 3, 0] * 2, 4, 3131, 1344),
        ([90, 1, 3, 0, 24, 0, 0, 0], 0, 914, 9584), ([1, 2, 0], 0, 8863, 2528), ([20, 3, 33], 0, 21692, 1056), ([65, 0, 0, 1], 0, 3879, 4400),
        ([24] * 128, 2, 33, 80), ([1] * 50 + [0] * 9 + [9], 0, 833, 48), ([900, 30, 7], 0, 1008, 672), ([62] * 64, 0, 9, 144),
        ([400, 60], 0, 530, 160)]


@pytest.mark.parametrize("counts,behind,N,K", WIDE + MORE)
@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_experts_products_wide(counts, behind, N, K, kind):
    """Each size of tile, with experts that end inside one and rows behind them."""
    E, n = len(counts), sum(counts)
    R = n + behind
    act, dt = TYPES[kind][:2]
    offsets = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    q, a = quantized(rows(R, K, dt, 63))
    codes, scales = weights(N, K, 64, E)
    y = torch.full((R, N), 7.0, dtype=dt, device="cuda")
    w.w4a16_gemm_w8a8_experts(W8, act, torch.from_numpy(q).cuda(), torch.from_numpy(a).cuda(), R, torch.from_numpy(offsets).cuda(),
                              E, codes.cuda(), scales.cuda(), None, N, K, y)
    for e in range(E):
        lo, hi = offsets[e], offsets[e + 1]
        if hi > lo:
            check(y[lo:hi], product_on_gpu(q[lo:hi], a[lo:hi], codes.view(E, N, K)[e], scales.view(E, N)[e]), kind)
    assert (y[n:] == 7).all()


def test_offsets_out_of_range():
    """Offsets that fall, pass R or are negative stay inside the buffers: rows behind R are not written."""
    E, R, N, K = 5, 200, 70, 64
    buf = torch.full((R + 600, N), 7.0, device="cuda")
    xq = torch.ones((R, K), dtype=torch.int8, device="cuda")
    codes, scales = torch.ones((E, N, K), dtype=torch.int8, device="cuda"), torch.ones((E, N), device="cuda")
    for offsets in ([0, 150, 20, 180, 10, 200], [0, 500, 900, 10 ** 9, 10 ** 9, 2 ** 31 - 1], [-5, -1, 30, -2 ** 31, 90, 200],
                    [200, 100, 50, 20, 10, 0]):
        buf.fill_(7.0)
        o = torch.tensor(offsets, dtype=torch.int32, device="cuda")
        w.w4a16_gemm_w8a8_experts(W8, w.W4A16_FP32, xq, torch.ones(R, device="cuda"), R, o, E, codes, scales, None, N, K, buf[:R])
        got = buf.cpu()
        assert (got[R:] == 7).all() and ((got[:R] == 7) | (got[:R] == K)).all()


def test_offsets_that_name_rows_many_times():
    """Every other expert claims all rows: more tiles than any sorted order makes."""
    E, R, N, K = 512, 333, 300, 64
    buf = torch.full((R + 600, N), 7.0, device="cuda")
    xq = torch.ones((R, K), dtype=torch.int8, device="cuda")
    codes, scales = torch.ones((E, N, K), dtype=torch.int8, device="cuda"), torch.ones((E, N), device="cuda")
    o = torch.tensor([R * (e % 2) for e in range(E + 1)], dtype=torch.int32, device="cuda")
    w.w4a16_gemm_w8a8_experts(W8, w.W4A16_FP32, xq, torch.ones(R, device="cuda"), R, o, E, codes, scales, None, N, K, buf[:R])
    got = buf.cpu()
    assert (got[R:] == 7).all() and ((got[:R] == 7) | (got[:R] == K)).all()


def test_no_expert_has_rows():
    y = torch.full((5, 32), 7.0, device="cuda")
    z = torch.zeros(8, dtype=torch.int32, device="cuda")
    w.w4a16_gemm_w8a8_experts(W8, w.W4A16_FP32, torch.zeros((5, 64), dtype=torch.int8, device="cuda"), torch.ones(5, device="cuda"),
                              5, z, 7, torch.zeros((7, 32, 64), dtype=torch.int8, device="cuda"), torch.ones((7, 32), device="cuda"),
                              None, 32, 64, y)
    assert (y == 7).all()


def test_one_expert_is_the_plain_product():
    M, N, K = 77, 200, 512
    q, a = quantized(rows(M, K, torch.float16, 71))
    codes, scales = weights(N, K, 72)
    y = [torch.empty((M, N), dtype=torch.float16, device="cuda") for _ in range(2)]
    d = [torch.from_numpy(t).cuda() for t in (q, a)]
    w.w4a16_gemm_w8a8(W8, w.W4A16_FP16, *d, M, codes.cuda(), scales.cuda(), None, N, K, y[0])
    w.w4a16_gemm_w8a8_experts(W8, w.W4A16_FP16, *d, M, torch.tensor([0, M], dtype=torch.int32, device="cuda"), 1, codes.cuda(),
                              scales.cuda(), None, N, K, y[1])
    assert torch.equal(y[0], y[1])


# ---- a serving pass, and a training step ------------------------------------------------------------

class Layer:
    """sort -> gather and quantize -> experts' products -> combine."""

    def __init__(self, T, topk, E, N, K, kind, seed):
        self.dims, (self.act, self.dt, self.u, self.tiny) = (T, topk, E, N, K), TYPES[kind]
        self.codes, self.scales = weights(N, K, seed, E)
        self.dcodes, self.dscales = self.codes.cuda(), self.scales.cuda()
        self.offsets, self.pos, self.src, self.ws, self.nb = w.alloc_expert_sort(T, topk, E)
        P = T * topk
        self.ids = torch.empty((T, topk), dtype=torch.int64, device="cuda")
        self.x = torch.empty((T, K), dtype=self.dt, device="cuda")
        self.wt = torch.empty((T, topk), device="cuda")
        self.xq = torch.empty((P, K), dtype=torch.int8, device="cuda")
        self.a = torch.empty(P, device="cuda")
        self.ys = torch.empty((P, N), dtype=self.dt, device="cuda")
        self.y = torch.empty((T, N), dtype=self.dt, device="cuda")

    def fill(self, seed):
        T, topk, E, N, K = self.dims
        ids = route(T, topk, E, seed)
        x = rows(T, K, self.dt, seed + 1)
        wt = torch.rand((T, topk), generator=torch.Generator().manual_seed(seed + 2))
        self.ids.copy_(torch.from_numpy(ids))
        self.x.copy_(x)
        self.wt.copy_(wt)
        return ids, x, wt

    def run(self):
        T, topk, E, N, K = self.dims
        w.w4a16_expert_sort(self.ids, 64, T, topk, E, self.offsets, self.pos, self.src, self.ws, self.nb)
        w.w4a16_expert_gather_i8(self.act, self.x, T, topk, self.pos, K, self.xq, self.a)
        w.w4a16_gemm_w8a8_experts(W8, self.act, self.xq, self.a, T * topk, self.offsets, E, self.dcodes, self.dscales, None, N, K,
                                  self.ys)
        w.w4a16_expert_combine(self.act, self.ys, T, topk, self.pos, self.wt, N, self.y)

    def check(self, ids, x, wt):
        T, topk, E, N, K = self.dims
        q, a = quantized(x)
        ref, mag = torch.zeros((T, N), dtype=torch.float64), torch.zeros((T, N), dtype=torch.float64)
        for e in range(E):
            t, j = np.nonzero(ids == e)
            if len(t):
                p = product(q[t], a[t], self.codes.view(E, N, K)[e], self.scales.view(E, N)[e]) * wt.double()[t, j][:, None]
                ref.index_add_(0, torch.from_numpy(t), p)
                mag.index_add_(0, torch.from_numpy(t), p.abs())
        u = self.u
        bound = u * ref.abs() + (1 + u) * (u + (topk + 5) * F24) * mag + (topk + 1) * self.tiny
        assert ((self.y.cpu().double() - ref).abs() <= bound).all()


@pytest.mark.parametrize("T,topk,E,N,K,kind", [(1, 2, 8, 256, 512, "bf16"), (9, 2, 4, 61, 80, "f16"), (200, 8, 64, 136, 272, "f16"),
                                               (700, 2, 3, 260, 400, "f32"), (2500, 4, 16, 100, 64, "bf16")])
def test_serving_pass(T, topk, E, N, K, kind):
    layer = Layer(T, topk, E, N, K, kind, 81)
    inputs = layer.fill(82)
    layer.run()
    layer.check(*inputs)


@pytest.mark.parametrize("T", [5, 2500])
def test_serving_pass_captured(T):
    """A captured pass replayed on other tokens and routes, with eager passes of a second layer, on its
    own workspace, on another stream meanwhile."""
    layer, other = (Layer(T, 4, 16, 132, 256, "f16", s) for s in (91, 92))
    layer.fill(93)
    layer.run()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        layer.run()
    s = torch.cuda.Stream()
    for seed in (94, 104, 114):
        a, b = layer.fill(seed), other.fill(seed + 5)
        torch.cuda.synchronize()
        layer.y.fill_(float("nan"))
        g.replay()
        with torch.cuda.stream(s):
            other.run()
        torch.cuda.synchronize()
        layer.check(*a)
        other.check(*b)


def test_training_step():
    """y = combine(f(gather(x))) with f(v) = v^2, and its gradients by the library's backward calls against
    torch's own in 64 bits."""
    T, topk, E, N = 60, 3, 7, 72
    ids = route(T, topk, E, 131)
    offsets, pos, _ = gpu_sort(ids, E)
    x, wt, dy = (torch.randn(s, generator=torch.Generator().manual_seed(i)) for i, s in ((1, (T, N)), (2, (T, topk)), (3, (T, N))))
    xd = x.cuda()
    xs, dys = torch.zeros((T * topk, N), device="cuda"), torch.zeros((T * topk, N), device="cuda")
    dw, dx, y = torch.empty((T, topk), device="cuda"), torch.empty((T, N), device="cuda"), torch.empty((T, N), device="cuda")
    f32 = w.W4A16_FP32
    w.w4a16_expert_gather(f32, xd, T, topk, pos, N, xs)
    ys = xs * xs
    w.w4a16_expert_combine(f32, ys, T, topk, pos, wt.cuda(), N, y)
    w.w4a16_expert_combine_backward(f32, dy.cuda(), ys, T, topk, pos, wt.cuda(), N, dys, dw)
    w.w4a16_expert_combine(f32, 2 * xs * dys, T, topk, pos, None, N, dx)
    X, Wt = x.double().requires_grad_(), wt.double().requires_grad_()
    live = torch.from_numpy((ids >= 0) & (ids < E)).double()
    Y = (X * X)[:, None, :].mul((Wt * live)[:, :, None]).sum(1)
    Y.backward(dy.double())
    # x^2, the products, and sums of topk (y, dx) or N (dw) terms of either sign
    mag = (x * x).double() * (wt.abs() * live).sum(1)[:, None]
    assert ((y.cpu().double() - Y.detach()).abs() <= (topk + 2) * F24 * mag).all()
    assert ((dx.cpu().double() - X.grad).abs() <= (topk + 4) * F24 * (2 * x.abs() * dy.abs()).double() * (wt.abs() * live).sum(1)[:, None]).all()
    assert ((dw.cpu().double() - Wt.grad).abs() <= (N / 256 + 34) * F24 * ((x * x * dy.abs()).double().sum(1)[:, None])).all()


def test_binding_checks_tensors():
    T, topk, N = 4, 2, 8
    x, pos, xs = torch.zeros((T, N), device="cuda"), torch.zeros((T, topk), dtype=torch.int32, device="cuda"), torch.zeros((T * topk, N), device="cuda")
    for bad in [(x.cpu(), pos, xs), (x, pos[:3], xs), (x, pos, xs[:-1]), (x.t(), pos, xs), (x.half(), pos, xs), (x, pos.long(), xs), (x.double(), pos, xs)]:
        with pytest.raises(w.W4A16Error) as e:
            w.w4a16_expert_gather(w.W4A16_FP32, bad[0], T, topk, bad[1], N, bad[2])
        assert e.value.status == w.W4A16_ERR_INVALID
    o, p, s, ws, nb = w.alloc_expert_sort(T, topk, 3)
    for ids, bits in [(pos.long(), 32), (pos, 64)]:
        with pytest.raises(w.W4A16Error) as e:
            w.w4a16_expert_sort(ids, bits, T, topk, 3, o, p, s, ws, nb)
        assert e.value.status == w.W4A16_ERR_INVALID
