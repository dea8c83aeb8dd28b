"""W8A8 on the GPU against its definition: int8 rows bit-exact with numpy's fp32 division, and every
product against the exact integer sums in 64 bits.

Bound of a product: the integer sum is exact; it is converted to fp32 and multiplied by the two
scales (three roundings of at most 2^-24 each), and rounded once to the output type (2^-8 bf16,
2^-11 fp16; an fp32 output has no rounding of its own).  Outputs below the type's normal range are
off by at most half its smallest step.
"""
import numpy as np
import pytest
import torch

import gemm_w4a16_amd as w

pytestmark = pytest.mark.gpu

W8 = w.W4A16_FMT_W8_ROW_FP32
TYPES = {"bf16": (w.W4A16_BF16, torch.bfloat16, 2.0 ** -8, 0.0), "f16": (w.W4A16_FP16, torch.float16, 2.0 ** -11, 2.0 ** -25),
         "f32": (w.W4A16_FP32, torch.float32, 0.0, 0.0)}


def rows(M, K, dt, seed):
    """Random rows with the cases a quantizer can get wrong among the first: zero, exact ties, the
    largest magnitude negative, magnitudes near the smallest."""
    x = torch.randn((M, K), generator=torch.Generator().manual_seed(seed))
    if M > 4:
        x[1] = 0
        x[2] = 0
        x[2, :6] = torch.tensor([0.5, 1.5, 2.5, -2.5, 126.5, -0.5])
        x[2, -1] = 127.0
        x[3, 5] = -100.0
        x[4] *= 2.0 ** -20
    return x.to(dt)


def quantized(x):
    """The definition, in numpy's fp32 (its division and rint are IEEE's)."""
    x = x.float().numpy()
    a = np.abs(x).max(1) / np.float32(127)
    a[a == 0] = 1
    return np.clip(np.rint(x / a[:, None]), -127, 127).astype(np.int8), a


def weights(N, K, seed, E=1):
    g = torch.Generator().manual_seed(seed)
    codes = torch.randint(-127, 128, (E * N, K), generator=g, dtype=torch.int8)
    scales = torch.rand(E * N, generator=g) * 0.01 + 1e-4
    return codes, scales


def product(q, a, codes, scales):
    """Exact in 64 bits: integer sums below 2^31, then the two scales."""
    s = torch.from_numpy(q.astype(np.float64)) @ codes.double().t()
    return s * torch.from_numpy(a.astype(np.float64))[:, None] * scales.double()[None]


def check(y, ref, kind):
    _, _, u, tiny = TYPES[kind]
    y, ref = y.cpu().double(), ref
    bound = (u + 4 * 2.0 ** -24) * ref.abs() + tiny
    worst = ((y - ref).abs() - bound).max().item()
    assert not torch.isnan(y).any()
    assert worst <= 0, f"past the bound by {worst:.3e}"


def gpu_product(q, a, codes, scales, kind, stream=None):
    act, dt = TYPES[kind][:2]
    M, K = q.shape
    N = codes.shape[0]
    y = torch.full((M, N), float("nan"), dtype=dt, device="cuda")
    w.w4a16_gemm_w8a8(W8, act, torch.from_numpy(q).cuda(), torch.from_numpy(a).cuda(), M, codes.cuda(), scales.cuda(), None,
                      N, K, y, stream=stream)
    return y


@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("M,K", [(1, 16), (5, 48), (37, 2064), (300, 4096), (6, 20000), (1, 8192), (1500, 1040),
                                 (1027, 4096), (1026, 4112)])
def test_quantize_rows_bit_exact(M, K, kind):
    act, dt = TYPES[kind][:2]
    x = rows(M, K, dt, 11)
    xq = torch.full((M, K), 99, dtype=torch.int8, device="cuda")
    a = torch.full((M,), float("nan"), device="cuda")
    w.w4a16_quantize_rows_i8(act, x.cuda(), M, K, xq, a)
    q, ra = quantized(x)
    np.testing.assert_array_equal(a.cpu().numpy(), ra)
    np.testing.assert_array_equal(xq.cpu().numpy(), q)


@pytest.mark.parametrize("kind", list(TYPES))
def test_quantize_rows_of_extreme_magnitudes(kind):
    """Rows of the type's largest and smallest values (subnormals among them), and rows that hold an
    infinity or NaN, which get the scale NaN and codes 0 and leave the other rows alone."""
    act, dt = TYPES[kind][:2]
    K = 64
    x = torch.zeros((6, K), dtype=dt)
    x[0, 3] = torch.finfo(dt).max
    x[1, :4] = torch.finfo(dt).smallest_normal * torch.tensor([1.0, 0.5, -0.25, 0.75])
    x[2, 7], x[2, 8] = float("inf"), 1
    x[3, 9], x[3, 0] = float("nan"), -2
    x[4] = torch.linspace(-3, 3, K).to(dt)
    x[5, 1] = -float("inf")
    xq = torch.full((6, K), 99, dtype=torch.int8, device="cuda")
    a = torch.zeros(6, device="cuda")
    w.w4a16_quantize_rows_i8(act, x.cuda(), 6, K, xq, a)
    xq, a = xq.cpu().numpy(), a.cpu().numpy()
    ok = [0, 1, 4]
    q, ra = quantized(x[ok])
    np.testing.assert_array_equal(a[ok], ra)
    np.testing.assert_array_equal(xq[ok], q)
    assert np.isnan(a[[2, 3, 5]]).all() and (xq[[2, 3, 5]] == 0).all()


SHAPES = [(1, 1, 16), (1, 256, 4096), (2, 61, 48), (3, 64, 1040), (8, 1000, 512), (16, 132, 4096), (17, 4100, 272), (33, 3, 64),
          (64, 515, 2064), (65, 128, 128), (130, 257, 400), (200, 1001, 1536), (257, 770, 144), (300, 512, 4112)]


@pytest.mark.parametrize("M,N,K", SHAPES)
@pytest.mark.parametrize("kind", list(TYPES))
def test_gemm_w8a8(M, N, K, kind):
    q, a = quantized(rows(M, K, TYPES[kind][1], 21))
    codes, scales = weights(N, K, 22)
    y = gpu_product(q, a, codes, scales, kind)
    check(y, product(q, a, codes, scales), kind)
    assert torch.equal(y, gpu_product(q, a, codes, scales, kind))  # bit for bit again


def product_on_gpu(q, a, codes, scales):
    """product() by torch's fp64 on the GPU, for larger shapes."""
    s = torch.from_numpy(q).cuda().double() @ codes.cuda().double().t()
    return (s * torch.from_numpy(a).cuda().double()[:, None] * scales.cuda().double()[None]).cpu()


# wide products, ragged in every direction: few rows against many columns up to several rounds of the
# largest tiles, rows of y that are whole 16-byte chunks and rows that are not
WIDE = [(17, 2050, 1040), (16, 8200, 1040), (17, 4100, 1040), (40, 8200, 1040), (17, 16500, 1040), (33, 16512, 1040),
        (33, 16500, 144), (65, 16500, 1040), (130, 16512, 144), (200, 16500, 1040), (200, 16512, 400), (780, 14350, 1040),
        (1030, 14352, 144), (515, 14352, 1168), (2050, 3000, 1040), (1030, 2051, 528),
        (16, 16500, 4112), (40, 16500, 4112), (3, 4100, 16400)]  # (weights of more than 64 MiB for one row tile)


@pytest.mark.parametrize("M,N,K", WIDE)
@pytest.mark.parametrize("kind", list(TYPES))
def test_gemm_w8a8_wide(M, N, K, kind):
    q, a = quantized(rows(M, K, TYPES[kind][1], 23))
    codes, scales = weights(N, K, 24)
    y = gpu_product(q, a, codes, scales, kind)
    check(y, product_on_gpu(q, a, codes, scales), kind)
    assert torch.equal(y, gpu_product(q, a, codes, scales, kind))


# weights of more than 64 MiB for one row tile, for each size of tile that they can be read once by
ONCE = [(2, 3380, 19856), (5, 15536, 4320), (12, 35397, 1904), (31, 24763, 2752), (17, 5481, 12256), (34, 22750, 2960), (62, 16026, 4336)]


@pytest.mark.parametrize("M,N,K", ONCE)
@pytest.mark.parametrize("kind", list(TYPES))
def test_gemm_w8a8_weights_once(M, N, K, kind):
    q, a = quantized(rows(M, K, TYPES[kind][1], 27))
    codes, scales = weights(N, K, 28)
    check(gpu_product(q, a, codes, scales, kind), product_on_gpu(q, a, codes, scales), kind)


PARTS = [(128, 4096, 14336), (512, 4096, 14352), (300, 2050, 8208), (2000, 1000, 20000), (200, 1030, 14336), (100, 515, 40000)]


MORE_PARTS = [(365, 1389, 8368), (801, 1244, 7984), (1609, 1153, 10112), (81, 1047, 15792), (263, 979, 8096), (1, 1, 15664), (70, 300, 15664)]


@pytest.mark.parametrize("M,N,K", PARTS + MORE_PARTS)
@pytest.mark.parametrize("kind", list(TYPES))
def test_k_in_parts_is_the_same_product(M, N, K, kind):
    """Few columns and a long K, with a workspace for the sums of K's parts and without: the same bits."""
    act, dt = TYPES[kind][:2]
    q, a = quantized(rows(M, K, dt, 25))
    codes, scales = weights(N, K, 26)
    ws, nb = w.alloc_w8a8_workspace(W8, M, N, K)
    assert nb > (M * K + 4 * M + 4 * M * N)  # there are parts
    ws.fill_(0x5A)
    y = torch.full((M, N), float("nan"), dtype=dt, device="cuda")
    w.w4a16_gemm_w8a8(W8, act, torch.from_numpy(q).cuda(), torch.from_numpy(a).cuda(), M, codes.cuda(), scales.cuda(), None, N, K,
                      y, ws, nb)
    assert torch.equal(y, gpu_product(q, a, codes, scales, kind))
    check(y, product_on_gpu(q, a, codes, scales), kind)


@pytest.mark.parametrize("M", [1, 40, 300])
def test_largest_sums(M):
    """Codes of -128 everywhere at the largest K: sums of 2^14 K, just below 2^31."""
    K, N = (1 << 17) - 16, 70
    q = np.full((M, K), -128, dtype=np.int8)
    codes = torch.full((N, K), -128, dtype=torch.int8)
    codes[1] = 127
    a, scales = np.full(M, 0.5, dtype=np.float32), torch.full((N,), 2.0 ** -20)
    check(gpu_product(q, a, codes, scales, "f32"), product(q, a, codes, scales), "f32")


@pytest.mark.parametrize("M,N,K,kind", [(1, 300, 512, "bf16"), (1, 2048, 8192, "f16"), (3, 61, 80, "f16"), (16, 64, 4096, "f32"),
                                        (70, 260, 1040, "bf16"), (260, 300, 512, "f16"), (1, 1, 16, "f32"),
                                        (2, 5003, 2064, "f32"), (2, 700, 8192, "bf16"), (2, 700, 8208, "bf16"),
                                        (1, 4100, 20000, "f16"), (2, 4099, 1008, "f16"), (1, 100, 12288, "f32"),
                                        (2, 4096, 4096, "bf16"), (3, 8200, 144, "bf16"), (37, 1001, 2064, "f16"),
                                        (16, 4096, 2048, "bf16"), (16, 4100, 2048, "bf16"), (9, 61, 4096, "bf16"),
                                        (8, 700, 4608, "f16"), (40, 1300, 1024, "f32"), (16, 200, 1536, "f32"),
                                        (500, 100, 1040, "bf16"), (1, 16500, 4112, "bf16"), (2, 4090, 16416, "f16"), (17, 33, 48, "f16"), (512, 2048, 8192, "bf16"), (200, 1030, 14336, "f16"), (128, 512, 512, "f32")])
def test_matmul_is_the_two_calls(M, N, K, kind):
    act, dt = TYPES[kind][:2]
    x = rows(M, K, dt, 31)
    codes, scales = weights(N, K, 32)
    ws, nb = w.alloc_w8a8_workspace(W8, M, N, K)
    y = torch.full((M, N), float("nan"), dtype=dt, device="cuda")
    w.w4a16_matmul_w8a8(W8, act, x.cuda(), M, codes.cuda(), scales.cuda(), None, N, K, y, ws, nb)
    q, a = quantized(x)
    check(y, product(q, a, codes, scales), kind)
    assert torch.equal(y, gpu_product(q, a, codes, scales, kind))


@pytest.mark.parametrize("M,N,K", [(20, 130, 256), (2, 5000, 528), (1100, 300, 256), (20, 5000, 256)])
def test_nonfinite_rows_stay_their_own(M, N, K):
    """A row with an infinity or NaN gives NaN outputs; every other row is what it is without it."""
    x = rows(M, K, torch.bfloat16, 41)
    codes, scales = weights(N, K, 42)
    ws, nb = w.alloc_w8a8_workspace(W8, M, N, K)
    y = [torch.empty((M, N), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    args = (codes.cuda(), scales.cuda(), None, N, K)
    w.w4a16_matmul_w8a8(W8, w.W4A16_BF16, x.cuda(), M, *args, y[0], ws, nb)
    hurt = [M // 2, M // 3] if M > 2 else [1]
    x[hurt[0], 3] = float("inf")
    x[hurt[-1], 250] = float("nan")
    w.w4a16_matmul_w8a8(W8, w.W4A16_BF16, x.cuda(), M, *args, y[1], ws, nb)
    bad = torch.zeros(M, dtype=torch.bool, device="cuda")
    bad[hurt] = True
    assert y[1][bad].isnan().all() and torch.equal(y[0][~bad], y[1][~bad])


def test_weights_from_the_quantizer():
    """The W8 arrays as w4a16_quantize_pack writes them, against the fp32 weights' own decode."""
    M, N, K = 9, 96, 512
    W = torch.randn((N, K), generator=torch.Generator().manual_seed(51)) * 0.02
    codes, scales, _ = w.alloc_packed(W8, N, K)
    w.w4a16_quantize_pack(W8, W.cuda(), N, K, codes, scales, None)
    q, a = quantized(rows(M, K, torch.float16, 52))
    y = gpu_product(q, a, codes.cpu(), scales.cpu(), "f16")
    check(y, product(q, a, codes.cpu(), scales.cpu()), "f16")
    assert (codes.cpu().double() * scales.cpu().double()[:, None] - W.double()).abs().max() <= scales.max().item() * 0.5001


@pytest.mark.parametrize("M,N,K", [(1, 516, 1040), (30, 516, 1040), (300, 516, 1040), (300, 2050, 8208)])
def test_captured_and_on_another_stream(M, N, K):
    """Replays of a captured call equal eager calls on the inputs of the moment."""
    codes, scales = weights(N, K, 61)
    codes, scales = codes.cuda(), scales.cuda()
    x = torch.empty((M, K), dtype=torch.float16, device="cuda")
    ws, nb = w.alloc_w8a8_workspace(W8, M, N, K)
    y = torch.empty((M, N), dtype=torch.float16, device="cuda")
    call = lambda out: w.w4a16_matmul_w8a8(W8, w.W4A16_FP16, x, M, codes, scales, None, N, K, out, ws, nb)
    s = torch.cuda.Stream()
    x.copy_(rows(M, K, torch.float16, 62))
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        call(y)
    torch.cuda.current_stream().wait_stream(s)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call(y)
    for seed in (63, 64, 65):
        x.copy_(rows(M, K, torch.float16, seed))
        eager = torch.empty_like(y)
        call(eager)
        torch.cuda.synchronize()
        y.zero_()
        g.replay()
        assert torch.equal(y, eager)


def test_outputs_past_32_bit_offsets():
    """More than 2^31 outputs: the last rows and columns, and some between, against the product of those alone."""
    M, N, K = 150_001, 14_400, 64
    g = torch.Generator(device="cuda").manual_seed(5)
    xq = torch.randint(-127, 128, (M, K), dtype=torch.int8, device="cuda", generator=g)
    a = torch.rand(M, device="cuda", generator=g)
    codes, scales = weights(N, K, 73)
    y = torch.full((M, N), float("nan"), dtype=torch.bfloat16, device="cuda")
    w.w4a16_gemm_w8a8(W8, w.W4A16_BF16, xq, a, M, codes.cuda(), scales.cuda(), None, N, K, y)
    for at in (0, 74_565, 149_131, 149_140, M - 70):  # (2^31 / 14400 = 149130.8)
        rows_ = slice(at, at + 70)
        check(y[rows_], product(xq[rows_].cpu().numpy(), a[rows_].cpu().numpy(), codes, scales), "bf16")


def test_outputs_are_written_exactly():
    """Odd sizes inside larger buffers: nothing before or behind the outputs changes."""
    for M, N, K in [(3, 61, 64), (33, 131, 512), (130, 257, 272)]:
        q, a = quantized(rows(M, K, torch.float32, 71))
        codes, scales = weights(N, K, 72)
        buf = torch.full((M * N + 4096,), 7.0, dtype=torch.bfloat16, device="cuda")
        y = buf[2048:2048 + M * N].view(M, N)
        w.w4a16_gemm_w8a8(W8, w.W4A16_BF16, torch.from_numpy(q).cuda(), torch.from_numpy(a).cuda(), M, codes.cuda(),
                          scales.cuda(), None, N, K, y)
        assert (buf[:2048] == 7).all() and (buf[2048 + M * N:] == 7).all()
        check(y, product(q, a, codes, scales), "bf16")


def test_binding_checks_tensors():
    M, N, K = 4, 8, 32
    xq = torch.zeros((M, K), dtype=torch.int8, device="cuda")
    a, codes = torch.ones(M, device="cuda"), torch.zeros((N, K), dtype=torch.int8, device="cuda")
    scales, y = torch.ones(N, device="cuda"), torch.empty((M, N), device="cuda")
    good = dict(xq=xq, ascale=a, codes=codes, scales=scales, y=y)

    def call(**change):
        t = {**good, **change}
        w.w4a16_gemm_w8a8(W8, w.W4A16_FP32, t["xq"], t["ascale"], M, t["codes"], t["scales"], None, N, K, t["y"])

    call()
    for change in [dict(xq=xq.cpu()), dict(codes=torch.zeros((K, N), dtype=torch.int8, device="cuda").t()),
                   dict(y=y[:3]), dict(scales=scales[:7]), dict(y=y.bfloat16()), dict(xq=xq.float()),
                   dict(xq=torch.zeros((M, 2 * K), dtype=torch.int8, device="cuda")[:, ::2])]:
        with pytest.raises(w.W4A16Error) as e:
            call(**change)
        assert e.value.status == w.W4A16_ERR_INVALID
