"""The microscaled 4-bit format on the GPU: rows and weights bit-exact with the definition in 64 bits, values back
exact, and the W4A4 product against exact products of those values.

Bound of a product: K products, exact, are added in fp32 in an order that the matrix instructions choose.  Each
addition is off by at most one rounding, to nearest or toward zero, of a partial sum no larger than the sum of the
magnitudes: K 2^-23 of that sum in all, and the output type's rounding.  A sum below fp32's normal numbers (2^-126) may
be taken as zero.
"""
import numpy as np
import pytest
import torch

import gemm_w4a16_amd as w
from test_gpu_memory_around_w8a8_experts import Arena

pytestmark = pytest.mark.gpu

MX4 = w.W4A16_FMT_MX4_B32_E8M0
F = 2.0 ** -24
TYPES = {"bf16": (w.W4A16_BF16, torch.bfloat16, 2.0 ** -8, 0.0), "f16": (w.W4A16_FP16, torch.float16, 2.0 ** -11, 2.0 ** -25),
         "f32": (w.W4A16_FP32, torch.float32, F, 0.0)}
MAGNITUDES = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])


def rows(M, K, dt, seed):
    """Random rows with what a quantizer can get wrong among the first: zeros, every border between elements, the
    largest magnitudes just below a power of two, the smallest and largest numbers of the type."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((M, K), generator=g)
    if M > 1:
        x[1, :32] = 0
        if K > 32:
            x[1, 32:64] = -0.0
    if M > 2:
        b = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, 7.0, 7.5, 0.24, 0.26, 4.9, 5.1, 0.0, -0.0])
        x[2, :32] = torch.cat([b, -b])
        if K > 32:
            x[2, 32:64] = torch.cat([b, -b]) * 2.0 ** -9
    if M > 3:
        x[3] *= 2.0 ** -12
    if M > 4:
        x[4] *= 2.0 ** torch.randint(-14, 10, (K,), generator=g).float()
    x = x.to(dt)
    if M > 5:
        x[5, :32] = torch.finfo(dt).smallest_normal * torch.randn(32, generator=g).to(dt) / 64
        x[5, 3] = torch.finfo(dt).max if K == 32 else 0
    return x


def quantized(x):
    """The definition in 64 bits: (elements' codes [M][K], blocks' scale bytes [M][K/32])."""
    v = x.double().numpy()
    M, K = v.shape
    b = v.reshape(M, K // 32, 32)
    top = np.abs(b).max(2)
    bad = ~np.isfinite(top)
    e = np.where((top > 0) & ~bad, np.frexp(np.where(bad, 1.0, top))[1] - 1, -1000)  # top = m 2^e with 1 <= m < 2
    e = np.maximum(e - 2, -127)
    a = np.abs(b) * np.exp2(-e.astype(np.float64))[:, :, None]
    a = np.where(bad[:, :, None], 0.0, a)
    d = np.abs(a[..., None] - MAGNITUDES)
    near = d.min(-1, keepdims=True)
    # of two elements equally near, the one of even code
    code = np.where(d == near, np.arange(8) + 100 * (np.arange(8) % 2), 1000).min(-1) % 100
    code = code + 8 * np.signbit(b)
    code = np.where(bad[:, :, None], 0, code)
    return code.reshape(M, K).astype(np.uint8), np.where(bad, 255, e + 127).astype(np.uint8)


def packed(code, scale):
    """The arrays of the format."""
    M, G = scale.shape
    T = (G + 7) // 8
    s = np.zeros(((M + 31) // 32 * 32, T * 8), np.uint8)
    s[:M, :G] = scale
    s = s.reshape(-1, 2, 16, T, 2, 4)  # rows / 32, rows / 16 % 2, rows % 16, blocks / 8, blocks / 4 % 2, blocks % 4
    return code[:, 0::2] | code[:, 1::2] << 4, np.ascontiguousarray(s.transpose(3, 0, 5, 2, 1, 4))


def values(code, scale):
    m = MAGNITUDES[code & 7] * np.where(code & 8, -1.0, 1.0)
    X = np.where(scale == 255, np.nan, np.exp2(scale.astype(np.float64) - 127))
    return torch.from_numpy(m * np.repeat(X, 32, 1))


def on_gpu(x, kind, arena=None):
    """Rows quantized by the library."""
    M, K = x.shape
    xq, xs, _ = w.alloc_packed(MX4, M, K)
    if arena:
        xq, xs = arena.out(xq.shape, torch.uint8), arena.out(xs.shape, torch.uint8)
    w.w4a16_quantize_rows_mx4(TYPES[kind][0], arena.put(x) if arena else x.cuda(), M, K, xq, xs)
    return xq, xs


@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("M,K", [(1, 32), (5, 64), (6, 32), (37, 2080), (300, 4096), (17, 288), (1000, 96), (3, 40000)])
def test_rows_bit_exact(M, K, kind):
    act, dt = TYPES[kind][:2]
    m, x = Arena(), rows(M, K, dt, 1)
    xq, xs = on_gpu(x, kind, m)
    ref = packed(*quantized(x))
    np.testing.assert_array_equal(xq.cpu().numpy(), ref[0])
    np.testing.assert_array_equal(xs.cpu().numpy(), ref[1])
    m.check()
    if kind == "f32":  # weights are quantized the same way
        codes, scales = m.out(xq.shape, torch.uint8), m.out(xs.shape, torch.uint8)
        w.w4a16_quantize_pack(MX4, m.put(x), M, K, codes, scales, None)
        assert torch.equal(codes, xq) and torch.equal(scales, xs)
    for out, t in (("bf16", torch.bfloat16), ("f16", torch.float16), ("f32", torch.float32)):
        v = m.out((M, K), t)
        w.w4a16_dequant(MX4, xq, xs, None, M, K, TYPES[out][0], v)
        want = values(*quantized(x)).float().to(t)  # (exact in fp32, then rounded once)
        assert torch.equal(v.cpu(), want)
    m.check()


@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("M,K", [(2000, 4128), (4200, 4128), (8300, 4128)])
def test_many_rows_as_in_pieces(M, K, kind):
    """The kernels of many rows, and of arrays that pass the caches by: bit for bit those of few."""
    act, dt = TYPES[kind][:2]
    x = rows(M, K, dt, 2).cuda()
    xq, xs, _ = w.alloc_packed(MX4, M, K)
    w.w4a16_quantize_rows_mx4(act, x, M, K, xq, xs)
    v = torch.empty((M, K), dtype=dt, device="cuda")
    w.w4a16_dequant(MX4, xq, xs, None, M, K, act, v)
    scales = xs.reshape((K + 255) // 256, -1, 256)
    for r in range(0, M, 640):
        n = min(640, M - r)
        pq, ps, _ = w.alloc_packed(MX4, n, K)
        w.w4a16_quantize_rows_mx4(act, x[r:r + n].contiguous(), n, K, pq, ps)
        assert torch.equal(pq.reshape(n, -1), xq.reshape(M, -1)[r:r + n])
        assert torch.equal(ps.reshape(scales.shape[0], -1, 256), scales[:, r // 32:(r + n + 31) // 32])
        pv = torch.empty((n, K), dtype=dt, device="cuda")
        w.w4a16_dequant(MX4, pq, ps, None, n, K, act, pv)
        assert torch.equal(pv.nan_to_num(7.0), v[r:r + n].nan_to_num(7.0))


def test_smallest_and_largest_numbers():
    """fp32 from the subnormal numbers to the largest: exponents of blocks over the whole range of their byte."""
    g = torch.Generator().manual_seed(3)
    e = torch.arange(-149, 128).repeat_interleave(32).double()
    mant = 1 + torch.rand(e.shape, generator=g).double()
    x = (mant * torch.exp2(e)).clamp(max=torch.finfo(torch.float32).max).float().reshape(277, 32)
    x = x * torch.where(torch.rand(x.shape, generator=g) < 0.5, -1.0, 1.0)
    x[:, 5:] *= torch.rand((277, 27), generator=g)
    xq, xs = on_gpu(x, "f32")
    code, scale = quantized(x)
    ref = packed(code, scale)
    np.testing.assert_array_equal(xs.cpu().numpy(), ref[1])
    np.testing.assert_array_equal(xq.cpu().numpy(), ref[0])
    assert scale.min() == 0 and scale.max() == 252
    v = torch.empty((277, 32), device="cuda")
    w.w4a16_dequant(MX4, xq, xs, None, 277, 32, w.W4A16_FP32, v)
    assert torch.equal(v.cpu().double(), values(code, scale))


@pytest.mark.parametrize("kind", list(TYPES))
def test_blocks_that_are_not_finite(kind):
    x = rows(9, 160, TYPES[kind][1], 5)
    x[0, 40], x[3, 159], x[7, 0] = float("inf"), float("nan"), float("-inf")
    xq, xs = on_gpu(x, kind)
    code, scale = quantized(x)
    assert (scale == 255).sum() == 3
    ref = packed(code, scale)
    np.testing.assert_array_equal(xq.cpu().numpy(), ref[0])
    np.testing.assert_array_equal(xs.cpu().numpy(), ref[1])
    v = torch.empty((9, 160), device="cuda")
    w.w4a16_dequant(MX4, xq, xs, None, 9, 160, w.W4A16_FP32, v)
    assert torch.equal(v.cpu().double().isnan(), values(code, scale).isnan())


def product(x, wt):
    """(exact product, sum of magnitudes) of the values that rows and weights stand for, on the GPU in 64 bits."""
    a, b = values(*quantized(x)).cuda(), values(*quantized(wt)).cuda()
    return (a @ b.t().contiguous()).cpu(), (a.abs() @ b.abs().t().contiguous()).cpu()


SHAPES = [(1, 1, 32), (1, 4100, 64), (1, 1001, 4096), (2, 61, 96), (3, 300, 2080), (5, 2049, 1056), (8, 512, 288), (16, 700, 4096),
          (17, 1001, 2080), (31, 64, 32), (37, 1001, 2080), (64, 257, 544), (65, 2000, 128), (100, 515, 20000), (129, 130, 256), (200, 1030, 8192),
          (257, 520, 1024), (300, 2050, 1312), (520, 4104, 512), (1030, 1030, 160), (1500, 770, 320), (40, 16400, 96), (4, 8192, 16384), (20, 3000, 1024),
          (33, 70, 512), (130, 515, 256), (8, 1000, 2048), (7, 8200, 1024), (300, 500, 480), (24, 9000, 1056)]


@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_product(M, N, K, kind):
    act, dt, u, tiny = TYPES[kind]
    m = Arena()
    x = rows(M, K, dt, 7)
    if M > 5:
        x[5, 3] = 0  # (the largest number, whose products leave fp16's range)
    wt = torch.randn((N, K), generator=torch.Generator().manual_seed(8)) * 0.05
    codes, scales = on_gpu(wt, "f32", m)
    nb = w.w4a16_w4a4_workspace_bytes(MX4, M, N, K)
    y, dx = m.out((M, N), dt), m.put(x)
    w.w4a16_matmul_w4a4(MX4, act, dx, M, codes, scales, None, N, K, y, m.workspace(nb), nb)
    ref, mag = product(x, wt)
    err = (y.cpu().double() - ref).abs() - (u * ref.abs() + (1 + u) * K * 2 * F * mag + tiny + 2.0 ** -126)
    assert not y.isnan().any() and err.max().item() <= 0
    m.check()
    xq, xs = on_gpu(x, kind, m)
    y2 = m.out((M, N), dt)
    w.w4a16_gemm_w4a4(MX4, act, xq, xs, M, codes, scales, None, N, K, y2)
    assert torch.equal(y, y2)
    m.check()


@pytest.mark.parametrize("M,N,K", SHAPES)
def test_whole_numbers_are_exact(M, N, K):
    """Elements that are whole numbers with scales of 1, 2 and 4: every partial sum is one below 2^24, so any order of
    additions gives it, and a wrong pairing of values or scales does not."""
    rng = np.random.default_rng(9)
    def arrays(R):
        code = rng.choice([0, 0, 2, 4, 10], (R, K)).astype(np.uint8)
        scale = rng.choice([127, 128, 129], (R, K // 32)).astype(np.uint8)
        if K > 8192:
            scale[:] = 127
        q, s = packed(code, scale)
        s[s == 0] = 0xFF  # (what pads the scales is of no effect)
        return torch.from_numpy(q).cuda(), torch.from_numpy(s).cuda(), values(code, scale).cuda()
    xq, xs, xv = arrays(M)
    wq, ws, wv = arrays(N)
    y = torch.empty((M, N), device="cuda")
    w.w4a16_gemm_w4a4(MX4, w.W4A16_FP32, xq, xs, M, wq, ws, None, N, K, y)
    assert (xv.abs() @ wv.abs().t().contiguous()).max() < 2 ** 24
    assert torch.equal(y.double(), xv @ wv.t().contiguous())


# Shapes of the tilings that the shapes above leave out, and of K that ends in the first or second half of a k-tile of 256
# or with it, for each tiling (tests/test_w4a4_plan_cpu.py works out which takes which).
WIDE_SHAPES = [(1043, 7365, 1056), (1201, 6501, 672), (1546, 5061, 768), (520, 7245, 1056), (535, 7241, 928), (645, 6001, 768),
               (3655, 1037, 288), (515, 4100, 1056), (530, 4103, 672), (900, 1501, 1024), (300, 2051, 1024), (301, 2050, 416),
               (205, 1031, 2208)]


@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("M,N,K", WIDE_SHAPES)
def test_tilings(M, N, K, kind):
    """Random elements of every kind with random scales against 64 bits; then whole numbers, exactly: every sum is one
    below 2^24, rounded once to the output type."""
    act, dt, u, tiny = TYPES[kind]
    rng = np.random.default_rng(M + N + K)
    m = Arena()

    def arrays(R, codes, scales):
        code, scale = rng.choice(codes, (R, K)).astype(np.uint8), rng.choice(scales, (R, K // 32)).astype(np.uint8)
        q, s = packed(code, scale)
        s[s == 0] = 0xFF  # (what pads the scales is of no effect)
        return m.put(torch.from_numpy(q)), m.put(torch.from_numpy(s)), values(code, scale).cuda()

    for codes, scales in ((np.arange(16), np.arange(119, 127)), ([0, 2, 4, 10, 12], [127, 128])):
        xq, xs, xv = arrays(M, codes, scales)
        wq, ws, wv = arrays(N, codes, scales)
        y = m.out((M, N), dt)
        w.w4a16_gemm_w4a4(MX4, act, xq, xs, M, wq, ws, None, N, K, y)
        wv = wv.t().contiguous()
        ref, mag = xv @ wv, xv.abs() @ wv.abs()
        if len(codes) == 16:
            err = (y.double() - ref).abs() - (u * ref.abs() + (1 + u) * K * 2 * F * mag + tiny)
            assert not y.isnan().any() and err.max().item() <= 0
        else:
            assert mag.max() < 2 ** 24 and torch.equal(y, ref.to(dt))
        m.check()


@pytest.mark.parametrize("M,N,K", WIDE_SHAPES)
def test_blocks_that_are_not_numbers_in_every_tiling(M, N, K):
    """A row's last block and a column's first: NaN in that row and column, whole numbers elsewhere."""
    rng = np.random.default_rng(5)
    code, scale = [rng.choice([0, 2, 4, 10], (R, K)).astype(np.uint8) for R in (M, N)], [np.full((R, K // 32), 127, np.uint8) for R in (M, N)]
    scale[0][M // 2, -1] = scale[0][M - 1, 3] = scale[1][N // 3, 0] = 255
    (xq, xs), (wq, ws) = ([torch.from_numpy(a).cuda() for a in packed(c, s)] for c, s in zip(code, scale))
    xv, wv = (values(c, s).cuda() for c, s in zip(code, scale))
    y = torch.empty((M, N), device="cuda")
    w.w4a16_gemm_w4a4(MX4, w.W4A16_FP32, xq, xs, M, wq, ws, None, N, K, y)
    bad = torch.zeros((M, N), dtype=torch.bool, device="cuda")
    bad[[M // 2, M - 1]], bad[:, N // 3] = True, True
    ref = xv.nan_to_num() @ wv.nan_to_num().t().contiguous()
    assert y[bad].isnan().all() and torch.equal(y[~bad].double(), ref[~bad])


@pytest.mark.parametrize("M,N", [(1, 17), (2, 40), (7, 33), (20, 70), (130, 50)])
def test_longest_rows(M, N):
    """K of 2^22, the most that a call takes: ones and zeros with scales of one, exactly, and x quantized on the way."""
    K = 1 << 22
    g = torch.Generator(device="cuda").manual_seed(M)
    def ones(R):
        t = torch.rand((R, K // 2), generator=g, device="cuda")  # of each pair of elements the first, the second, or none
        return (t < 0.2).to(torch.uint8) * 2 + (t > 0.9).to(torch.uint8) * 0x20
    def value(q):
        return torch.stack([(q & 15) / 2, (q >> 4) / 2], -1).reshape(q.shape[0], K).float()
    xq, wq = ones(M), ones(N)
    xs, ws = (torch.full(w.alloc_packed(MX4, R, K)[1].shape, 127, dtype=torch.uint8, device="cuda") for R in (M, N))
    y = torch.empty((M, N), device="cuda")
    w.w4a16_gemm_w4a4(MX4, w.W4A16_FP32, xq, xs, M, wq, ws, None, N, K, y)
    xv, wv = value(xq), value(wq)
    ref = torch.zeros((M, N), dtype=torch.float64, device="cuda")
    for k in range(0, K, 1 << 18):
        ref += xv[:, k:k + (1 << 18)].double() @ wv[:, k:k + (1 << 18)].double().t().contiguous()
    assert ref.max() < 2 ** 24 and torch.equal(y.double(), ref)
    z, (room, nb) = torch.empty((M, N), device="cuda"), w.alloc_w4a4_workspace(MX4, M, N, K)
    w.w4a16_matmul_w4a4(MX4, w.W4A16_FP32, xv * 4, M, wq, ws, None, N, K, z, room, nb)
    assert torch.equal(z, y * 4)


@pytest.mark.parametrize("M,N,K", [(1, 61, 96), (9, 300, 288), (37, 130, 544), (300, 2051, 160)])
def test_scales_far_from_one(M, N, K):
    """Scales over the whole range of their byte, whose products are near one, exactly; and products below fp32's
    normal numbers, which may be taken as zero."""
    rng = np.random.default_rng(17)
    code = [rng.choice([0, 2, 4, 10], (R, K)).astype(np.uint8) for R in (M, N)]
    for sx, sw in ((0, 252), (252, 0), (2, 252), (252, 2), (27, 227), (227, 27), (57, 57), (1, 1)):
        a, b = (packed(c, np.full((c.shape[0], K // 32), s, np.uint8)) for c, s in zip(code, (sx, sw)))
        (xq, xs), (wq, ws) = ((torch.from_numpy(q).cuda(), torch.from_numpy(s).cuda()) for q, s in (a, b))
        y = torch.empty((M, N), device="cuda")
        w.w4a16_gemm_w4a4(MX4, w.W4A16_FP32, xq, xs, M, wq, ws, None, N, K, y)
        ones = [values(c, np.full((c.shape[0], K // 32), 127, np.uint8)).cuda() for c in code]
        ref = (ones[0] @ ones[1].t().contiguous()) * 2.0 ** (sx + sw - 254)
        if sx + sw > 200:
            assert torch.equal(y.double(), ref)
        else:
            assert ((y.double() - ref).abs() <= 2.0 ** -126).all()


def test_debug_checks_take_what_the_format_defines(monkeypatch):
    """Weights that are not finite have codes in this format: the quantizer's debug check does not refuse them."""
    N, K = 40, 288
    wt = rows(N, K, torch.float32, 31)
    wt[3, 40], wt[39, 287] = float("inf"), float("nan")
    monkeypatch.setenv("W4A16_DEBUG_CHECKS", "1")
    codes, scales, _ = w.alloc_packed(MX4, N, K)
    w.w4a16_quantize_pack(MX4, wt.cuda(), N, K, codes, scales, None)
    ref = packed(*quantized(wt))
    np.testing.assert_array_equal(codes.cpu().numpy(), ref[0])
    np.testing.assert_array_equal(scales.cpu().numpy(), ref[1])


# weights from 64 MiB on, which few rows read past the caches' usual order
@pytest.mark.parametrize("M,N,K", [(1, 33005, 4096), (2, 20001, 7200), (5, 17008, 8192), (16, 70000, 2080)])
def test_few_rows_of_large_weights(M, N, K):
    test_whole_numbers_are_exact(M, N, K)
    if M < 5:  # quantized in the product
        g = torch.Generator().manual_seed(30)
        x = (torch.randint(-3, 4, (M, K), generator=g) * 2).to(torch.bfloat16)
        code = torch.randint(0, 256, (N, K // 2), generator=g, dtype=torch.uint8).cuda() & 0x22  # zeros and ones
        scales = torch.full(w.alloc_packed(MX4, N, K)[1].shape, 127, dtype=torch.uint8, device="cuda")
        wv = torch.stack([code & 0x0F, code >> 4], -1).reshape(N, K).double() / 2
        y, (ws, nb) = torch.empty((M, N), dtype=torch.bfloat16, device="cuda"), w.alloc_w4a4_workspace(MX4, M, N, K)
        w.w4a16_matmul_w4a4(MX4, w.W4A16_BF16, x.cuda(), M, code, scales, None, N, K, y, ws, nb)
        assert torch.equal(y, (x.cuda().double() @ wv.t().contiguous()).to(torch.bfloat16))


@pytest.mark.parametrize("M,N,K", [(1, 100, 512), (20, 200, 288), (300, 300, 1056)])
def test_a_block_that_is_not_finite_stays_its_rows(M, N, K):
    x = rows(M, K, torch.bfloat16, 11)
    if M > 5:
        x[5, 3] = 0
    wt = torch.randn((N, K), generator=torch.Generator().manual_seed(12)) * 0.05
    out = []
    for hurt in (False, True):
        if hurt:
            x[M // 2, K - 1], wt[N // 3, 5] = float("inf"), float("nan")
        codes, scales = on_gpu(wt, "f32")
        y = torch.empty((M, N), dtype=torch.bfloat16, device="cuda")
        ws, nb = w.alloc_w4a4_workspace(MX4, M, N, K)
        w.w4a16_matmul_w4a4(MX4, w.W4A16_BF16, x.cuda(), M, codes, scales, None, N, K, y, ws, nb)
        out.append(y.cpu())
    bad = torch.zeros((M, N), dtype=torch.bool)
    bad[M // 2], bad[:, N // 3] = True, True
    assert out[1][bad].isnan().all() and torch.equal(out[0][~bad], out[1][~bad])


def test_captured_and_on_another_stream():
    M, N, K = 20, 1001, 2080
    wt = torch.randn((N, K), generator=torch.Generator().manual_seed(13)) * 0.05
    codes, scales = on_gpu(wt, "f32")
    x = torch.empty((M, K), dtype=torch.bfloat16, device="cuda")
    y = torch.empty((M, N), dtype=torch.bfloat16, device="cuda")
    ws, nb = w.alloc_w4a4_workspace(MX4, M, N, K)
    step = lambda stream=None: w.w4a16_matmul_w4a4(MX4, w.W4A16_BF16, x, M, codes, scales, None, N, K, y, ws, nb, stream=stream)
    x.copy_(rows(M, K, torch.bfloat16, 14))
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    s = torch.cuda.Stream()
    for seed in range(4):
        x.copy_(rows(M, K, torch.bfloat16, 20 + seed))
        graph.replay()
        torch.cuda.synchronize()
        got = y.clone()
        y.fill_(0)
        torch.cuda.synchronize()
        step(s)
        s.synchronize()
        assert torch.equal(got, y)


def test_rows_past_32_bit_offsets():
    """More than 2^32 bytes of activations and 2^31 outputs: the last rows are those of a call of their own."""
    K, N = 2048, 1040
    M = (1 << 31) // N + 37
    x = torch.zeros((M, K), dtype=torch.bfloat16, device="cuda")
    x[-40:] = torch.randn((40, K), generator=torch.Generator(device="cuda").manual_seed(1), device="cuda")
    wt = torch.randn((N, K), generator=torch.Generator().manual_seed(15)) * 0.05
    codes, scales = on_gpu(wt, "f32")
    y = torch.empty((M, N), dtype=torch.bfloat16, device="cuda")
    ws, nb = w.alloc_w4a4_workspace(MX4, M, N, K)
    w.w4a16_matmul_w4a4(MX4, w.W4A16_BF16, x, M, codes, scales, None, N, K, y, ws, nb)
    last, y40 = x[-40:].clone(), torch.empty((40, N), dtype=torch.bfloat16, device="cuda")
    w.w4a16_matmul_w4a4(MX4, w.W4A16_BF16, last, 40, codes, scales, None, N, K, y40, ws, nb)
    u, bound = 2.0 ** -8, K * 2 * F
    ref, mag = product(last.cpu(), wt)
    for got in (y[-40:], y40):  # (another tile may add in another order)
        assert ((got.cpu().double() - ref).abs() <= u * ref.abs() + (1 + u) * bound * mag).all()
    assert (y[:-40] == 0).all()
