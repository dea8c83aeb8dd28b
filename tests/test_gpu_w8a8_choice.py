"""Where w4a16_matmul_w8a8 quantizes activations in the product's own launch and where in one of their own.  Only the
latter writes the codes into the workspace, which shows the choice; the outputs are the two calls' bit for bit
either way."""
import pytest
import torch

import gemm_w4a16_amd as w

pytestmark = pytest.mark.gpu

W8 = w.W4A16_FMT_W8_ROW_FP32
TYPES = {"bf16": (w.W4A16_BF16, torch.bfloat16), "f16": (w.W4A16_FP16, torch.float16), "f32": (w.W4A16_FP32, torch.float32)}


def launches(M, N, K, kind):
    """1 or 2, after a check of the outputs."""
    act, dt = TYPES[kind]
    g = torch.Generator(device="cuda").manual_seed(M + N + K)
    x = torch.randn((M, K), generator=g, device="cuda").to(dt)
    codes = torch.randint(-127, 128, (N, K), generator=g, device="cuda", dtype=torch.int8)
    scales = torch.rand(N, generator=g, device="cuda")
    ws, nb = w.alloc_w8a8_workspace(W8, M, N, K)
    ws.fill_(0x80)  # -128: no code
    y, z = torch.full((M, N), float("nan"), dtype=dt, device="cuda"), torch.empty((M, N), dtype=dt, device="cuda")
    w.w4a16_matmul_w8a8(W8, act, x, M, codes, scales, None, N, K, y, ws, nb)
    xq, a = torch.empty((M, K), dtype=torch.int8, device="cuda"), torch.empty(M, device="cuda")
    w.w4a16_quantize_rows_i8(act, x, M, K, xq, a)
    w.w4a16_gemm_w8a8(W8, act, xq, a, M, codes, scales, None, N, K, z)
    assert torch.equal(y, z)
    written = ws[:M * K] != 0x80
    assert written.all() or not written.any()
    return 2 if written.all() else 1


@pytest.mark.parametrize("M,N,K,kind", [
    (1, 14336, 4096, "bf16"), (2, 14336, 4096, "bf16"), (1, 4096, 16384, "f16"), (1, 8192, 16384, "bf16"), (2, 8192, 8192, "bf16"),
    (2, 28672, 4096, "f32"), (1, 57344, 8192, "bf16"), (3, 4096, 2720, "f16"), (8, 1024, 2048, "bf16"), (16, 4096, 1024, "f32"),
    (37, 1001, 1024, "bf16"), (128, 256, 512, "f32"), (16, 2048, 1360, "f32"), (1, 2048, 32768, "bf16")])
def test_one_launch(M, N, K, kind):
    assert launches(M, N, K, kind) == 1


@pytest.mark.parametrize("M,N,K,kind", [
    # one block a CU at a time, for more than one each
    (2, 14336, 8192, "bf16"), (2, 28672, 8192, "f16"), (1, 14336, 16384, "bf16"), (1, 28672, 9824, "f32"),
    # every CU would quantize more than eight rows
    (2, 57344, 1024, "bf16"), (2, 40000, 2048, "f32"), (1, 131072, 1024, "f32"),
    # more rows that are long, or many activations in all
    (3, 1024, 8192, "f32"), (4, 4096, 4096, "bf16"), (6, 1024, 5456, "bf16"), (8, 4096, 4096, "f16"), (16, 4096, 2048, "bf16"),
    (37, 1360, 1360, "bf16"), (64, 256, 2048, "f16"), (6, 2048, 3264, "f32"),
    # one or two rows past 96 KB
    (1, 1024, 24576, "f32"), (2, 1024, 12288, "f32")])
def test_two_launches(M, N, K, kind):
    assert launches(M, N, K, kind) == 2
