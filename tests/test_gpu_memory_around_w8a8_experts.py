"""Memory around the arrays of the W8A8 and experts' calls.  Every array lies between two margins of bytes of one value:
the margins of outputs and workspaces stay as they were, and those of inputs, which read as NaN or -1, reach no
result."""
import numpy as np
import pytest
import torch

import gemm_w4a16_amd as w
from test_gpu_experts import ROWS, combined, plan, route, sorted_order
from test_gpu_w8a8 import TYPES, W8, check, product_on_gpu, quantized, rows, weights

pytestmark = pytest.mark.gpu

F24 = 2.0 ** -24
MARGIN = 8192  # bytes; more than the widest tile's row of outputs


class Arena:
    """Arrays with margins of 0xFF around them (NaN as bf16, fp16 or fp32, -1 as an integer)."""

    def __init__(self):
        self.held = []

    def _room(self, nbytes):
        buf = torch.full((nbytes + 2 * MARGIN,), 0xFF, dtype=torch.uint8, device="cuda")
        self.held.append((buf, nbytes))
        return buf[MARGIN:MARGIN + nbytes]

    def out(self, shape, dtype):
        """An output, 0xFF all over."""
        n = int(np.prod(shape)) * dtype.itemsize
        return self._room(n).view(dtype).view(shape)

    def put(self, t):
        """An input with a tensor's values."""
        t = torch.as_tensor(t)
        a = self.out(t.shape, t.dtype)
        a.copy_(t)
        return a

    def workspace(self, nbytes):
        return self._room(nbytes) if nbytes else None

    def check(self):
        for buf, n in self.held:
            assert (buf[:MARGIN] == 0xFF).all() and (buf[MARGIN + n:] == 0xFF).all()


def untouched(t):
    return (t.contiguous().view(torch.uint8) == 0xFF).all()


@pytest.mark.parametrize("T,topk,E", [(1, 1, 1), (4, 2, 8), (333, 3, 512), (1024, 4, 60), (4097, 1, 3), (5000, 7, 33), (2048, 3, 512)])
@pytest.mark.parametrize("bits", [32, 64])
def test_sort(T, topk, E, bits):
    m, P = Arena(), T * topk
    ids = route(T, topk, E, 3, 0.2)
    nb = w.w4a16_expert_sort_workspace_bytes(T, topk, E)
    offsets, pos, src = (m.out(s, torch.int32) for s in ((E + 1,), (T, topk), (P,)))
    w.w4a16_expert_sort(m.put(ids.astype(np.int64 if bits == 64 else np.int32)), bits, T, topk, E, offsets, pos, src, m.workspace(nb), nb)
    for got, ref in zip((offsets, pos, src), sorted_order(ids, E)):
        np.testing.assert_array_equal(got.cpu().numpy(), ref)
    m.check()


# with routes that use every sorted row and routes that leave some
@pytest.mark.parametrize("pad", [0.0, 0.2])
@pytest.mark.parametrize("T,topk,E,N", ROWS)
@pytest.mark.parametrize("kind", list(TYPES))
def test_row_movers(T, topk, E, N, kind, pad):
    act, dt, u, tiny = TYPES[kind]
    pos, n, _ = plan(T, topk, E, 21, pad)
    m, P = Arena(), T * topk
    g = torch.Generator().manual_seed(22)
    x, wt = torch.randn((T, N), generator=g).to(dt), torch.rand((T, topk), generator=g) - 0.2
    dx, dpos, dwt = m.put(x), m.put(pos), m.put(wt)
    xs, y, dys, dw = m.out((P, N), dt), m.out((T, N), dt), m.out((P, N), dt), m.out((T, topk), torch.float32)
    w.w4a16_expert_gather(act, dx, T, topk, dpos, N, xs)
    t, j = np.nonzero(pos >= 0)
    at = torch.from_numpy(pos[t, j]).long()
    assert torch.equal(xs.cpu()[at], x[t]) and untouched(xs[n:])
    w.w4a16_expert_combine(act, xs, T, topk, dpos, dwt, N, y)
    ys = torch.nan_to_num(xs.cpu())
    ref, mag = combined(ys, pos, wt)
    assert ((y.cpu().double() - ref).abs() <= u * ref.abs() + (1 + u) * topk * F24 * mag + tiny).all()
    w.w4a16_expert_combine_backward(act, dx, xs, T, topk, dpos, dwt, N, dys, dw)
    ref = x.double()[t] * wt.double()[t, j][:, None]
    assert ((dys.cpu().double()[at] - ref).abs() <= (u + 2 * F24) * ref.abs() + tiny).all() and untouched(dys[n:])
    term = ys.double()[at] * x.double()[t]
    assert ((dw.cpu().double()[t, j] - term.sum(1)).abs() <= (N / 256 + 32) * F24 * term.abs().sum(1)).all()
    m.check()


@pytest.mark.parametrize("T,topk,E,K", [(1, 1, 1, 16), (4, 2, 8, 4096), (37, 3, 5, 1008), (9, 20, 30, 48), (1500, 3, 7, 1008)])
@pytest.mark.parametrize("kind", list(TYPES))
def test_quantized_rows(T, topk, E, K, kind):
    act, dt = TYPES[kind][:2]
    pos, n, _ = plan(T, topk, E, 23)
    m, P = Arena(), T * topk
    x = rows(T, K, dt, 24)
    dx, xq, a = m.put(x), m.out((P, K), torch.int8), m.out((P,), torch.float32)
    w.w4a16_expert_gather_i8(act, dx, T, topk, m.put(pos), K, xq, a)
    q, ra = quantized(x)
    t, j = np.nonzero(pos >= 0)
    np.testing.assert_array_equal(xq.cpu().numpy()[pos[t, j]], q[t])
    np.testing.assert_array_equal(a.cpu().numpy()[pos[t, j]], ra[t])
    assert untouched(xq[n:]) and untouched(a[n:])
    xq, a = m.out((T, K), torch.int8), m.out((T,), torch.float32)
    w.w4a16_quantize_rows_i8(act, dx, T, K, xq, a)
    np.testing.assert_array_equal(xq.cpu().numpy(), q)
    np.testing.assert_array_equal(a.cpu().numpy(), ra)
    m.check()


# in one launch (tiles of 16 x 16, 16 x 32, and 16 x 16 with K over eight waves), in two, in parts of K, and the widest
# tiles; rows of y that are whole 16-byte units and rows that are not
@pytest.mark.parametrize("M,N,K", [(1, 61, 48), (2, 1003, 2064), (2, 4096, 512), (1, 4101, 1040), (2, 9000, 528), (3, 61, 80), (9, 1001, 1040),
                                   (37, 1001, 1024), (40, 259, 2064), (130, 257, 272), (300, 2050, 8208), (200, 1030, 14336), (100, 515, 40000),
                                   (780, 14350, 1040), (1030, 2051, 528), (1030, 14352, 144)])
@pytest.mark.parametrize("kind", list(TYPES))
def test_products(M, N, K, kind):
    act, dt = TYPES[kind][:2]
    m = Arena()
    x = rows(M, K, dt, 31)
    codes, scales = weights(N, K, 32)
    nb = w.w4a16_w8a8_workspace_bytes(W8, M, N, K)
    y = m.out((M, N), dt)
    w.w4a16_matmul_w8a8(W8, act, m.put(x), M, m.put(codes), m.put(scales), None, N, K, y, m.workspace(nb), nb)
    q, a = quantized(x)
    check(y, product_on_gpu(q, a, codes, scales), kind)
    m.check()


@pytest.mark.parametrize("counts,behind,N,K", [([1], 1, 37, 1584), ([16, 17, 0, 15, 1], 5, 61, 48), ([1] * 50 + [0] * 9 + [9], 0, 833, 48),
                                               ([62] * 64, 0, 9, 144), ([520, 1, 700], 300, 8203, 1040), ([0, 0, 900, 0, 300, 1], 0, 8197, 144),
                                               ([9, 0, 1, 1, 2, 0, 3, 0] * 2, 4, 3131, 1344), ([130, 0, 128, 257], 3, 515, 144)])
@pytest.mark.parametrize("kind", list(TYPES))
def test_experts_products(counts, behind, N, K, kind):
    E, n = len(counts), sum(counts)
    R = n + behind
    act, dt = TYPES[kind][:2]
    m = Arena()
    offsets = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    q, a = quantized(rows(R, K, dt, 63))
    codes, scales = weights(N, K, 64, E)
    y = m.out((R, N), dt)
    w.w4a16_gemm_w8a8_experts(W8, act, m.put(q), m.put(a), R, m.put(offsets), E, m.put(codes), m.put(scales), None, N, K, y)
    for e in range(E):
        lo, hi = offsets[e], offsets[e + 1]
        if hi > lo:
            check(y[lo:hi], product_on_gpu(q[lo:hi], a[lo:hi], codes.view(E, N, K)[e], scales.view(E, N)[e]), kind)
    assert untouched(y[n:])
    m.check()


def test_a_token_that_is_not_finite_stays_its_own():
    """A whole pass with an infinity in one token and NaN in another, who share experts with all others."""
    T, topk, E, N, K = 50, 2, 3, 68, 96
    ids = route(T, topk, E, 7, 0.0)
    x = rows(T, K, torch.bfloat16, 8)
    codes, scales = weights(N, K, 9, E)
    wt = torch.rand((T, topk), generator=torch.Generator().manual_seed(10)) + 0.1
    out = []
    for hurt in (False, True):
        m, P = Arena(), T * topk
        if hurt:
            x[11, 5], x[29, K - 1] = float("inf"), float("nan")
        offsets, pos = m.out((E + 1,), torch.int32), m.out((T, topk), torch.int32)
        xq, a = m.out((P, K), torch.int8), m.out((P,), torch.float32)
        ys, y = m.out((P, N), torch.bfloat16), m.out((T, N), torch.bfloat16)
        w.w4a16_expert_sort(m.put(ids), 64, T, topk, E, offsets, pos, None)
        w.w4a16_expert_gather_i8(w.W4A16_BF16, m.put(x), T, topk, pos, K, xq, a)
        w.w4a16_gemm_w8a8_experts(W8, w.W4A16_BF16, xq, a, P, offsets, E, m.put(codes), m.put(scales), None, N, K, ys)
        w.w4a16_expert_combine(w.W4A16_BF16, ys, T, topk, pos, m.put(wt), N, y)
        m.check()
        out.append(y.cpu())
    bad = torch.zeros(T, dtype=torch.bool)
    bad[[11, 29]] = True
    assert out[1][bad].isnan().all() and torch.equal(out[0][~bad], out[1][~bad])
