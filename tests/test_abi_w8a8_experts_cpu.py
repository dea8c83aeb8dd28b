"""Refusals of the W8A8 and experts' entry points without a GPU: every call below fails a check on the
host before anything touches a device (the addresses are never dereferenced)."""
import pytest

import gemm_w4a16_amd as w

W8, G128 = w.W4A16_FMT_W8_ROW_FP32, w.W4A16_FMT_G128_ASYM_BF16
BF16, F16, F32 = w.W4A16_BF16, w.W4A16_FP16, w.W4A16_FP32
INVALID, UNSUPPORTED = w.W4A16_ERR_INVALID, w.W4A16_ERR_UNSUPPORTED
A = 0x10000  # an aligned address that no call dereferences
BIG = 1 << 31


def _status(fn, args, **changes):
    args = list(args)
    for k, v in changes.items():
        args[int(k[1:])] = v
    try:
        fn(*args)
    except w.W4A16Error as e:
        return e.status
    return w.W4A16_OK


# argument places, with a good call's values, and (changes, status) for each refusal
CALLS = {
    "quantize_rows": (w.w4a16_quantize_rows_i8, (BF16, A, 4, 32, A, A, 0), [
        ({"a0": 7}, INVALID), ({"a1": None}, INVALID), ({"a1": A + 8}, INVALID), ({"a2": 0}, INVALID),
        ({"a2": BIG}, INVALID), ({"a3": 0}, INVALID), ({"a3": 24}, INVALID), ({"a4": A + 4}, INVALID),
        ({"a5": None}, INVALID), ({"a3": (1 << 22) + 16}, UNSUPPORTED)]),
    "gemm_w8a8": (w.w4a16_gemm_w8a8, (W8, BF16, A, A, 4, A, A, None, 8, 32, A, None, 0, 0), [
        ({"a0": 9}, INVALID), ({"a1": 3}, INVALID), ({"a2": None}, INVALID), ({"a2": A + 1}, INVALID),
        ({"a3": A + 4}, INVALID), ({"a4": 0}, INVALID), ({"a4": -1}, INVALID), ({"a5": A + 8}, INVALID),
        ({"a6": None}, INVALID), ({"a7": A}, INVALID), ({"a8": 0}, INVALID), ({"a9": 40}, INVALID),
        ({"a10": A + 2}, INVALID), ({"a11": A + 8, "a12": 64}, INVALID), ({"a0": G128, "a7": A, "a9": 128}, UNSUPPORTED),
        ({"a9": 1 << 17}, UNSUPPORTED), ({"a8": (1 << 26) + 1}, UNSUPPORTED),
        ({"a4": 1 << 30, "a8": 1 << 26}, UNSUPPORTED)]),
    "matmul_w8a8": (w.w4a16_matmul_w8a8, (W8, F16, A, 4, A, A, None, 8, 32, A, A, 144, 0), [
        ({"a1": 3}, INVALID), ({"a2": A + 2}, INVALID), ({"a3": 0}, INVALID), ({"a10": None}, INVALID),
        ({"a11": 143}, INVALID), ({"a10": A + 4}, INVALID), ({"a6": A}, INVALID), ({"a8": 33}, INVALID),
        ({"a8": 1 << 17, "a11": 1 << 40}, UNSUPPORTED)]),
    "experts": (w.w4a16_gemm_w8a8_experts, (W8, F32, A, A, 6, A, 3, A, A, None, 8, 32, A, 0), [
        ({"a4": 0}, INVALID), ({"a5": None}, INVALID), ({"a5": A + 4}, INVALID), ({"a6": 0}, INVALID),
        ({"a6": w.w4a16_max_experts() + 1}, UNSUPPORTED), ({"a9": A}, INVALID), ({"a11": 8}, INVALID),
        ({"a11": 1 << 17}, UNSUPPORTED), ({"a12": None}, INVALID), ({"a0": G128, "a9": A, "a11": 128}, UNSUPPORTED)]),
    "sort": (w.w4a16_expert_sort, (A, 32, 5, 2, 4, A, A, A, None, 0, 0), [
        ({"a0": None}, INVALID), ({"a1": 16}, INVALID), ({"a2": 0}, INVALID), ({"a3": 0}, INVALID), ({"a4": 0}, INVALID),
        ({"a5": A + 4}, INVALID), ({"a6": None}, INVALID), ({"a7": A + 4}, INVALID),
        ({"a4": w.w4a16_max_experts() + 1}, UNSUPPORTED), ({"a3": w.w4a16_max_experts() + 1}, UNSUPPORTED),
        ({"a2": 1 << 30}, UNSUPPORTED), ({"a2": 100_000}, INVALID), ({"a2": 100_000, "a8": A, "a9": 16}, INVALID)]),
    "gather": (w.w4a16_expert_gather, (BF16, A, 5, 2, A, 7, A, 0), [
        ({"a0": 5}, INVALID), ({"a1": A + 2}, INVALID), ({"a2": -3}, INVALID), ({"a4": None}, INVALID),
        ({"a5": 0}, INVALID), ({"a6": A + 8}, INVALID), ({"a5": (1 << 22) + 1}, UNSUPPORTED)]),
    "gather_i8": (w.w4a16_expert_gather_i8, (BF16, A, 5, 2, A, 16, A, A, 0), [
        ({"a5": 24}, INVALID), ({"a7": None}, INVALID), ({"a0": -1}, INVALID), ({"a6": A + 1}, INVALID)]),
    "combine": (w.w4a16_expert_combine, (F16, A, 5, 2, A, None, 7, A, 0), [
        ({"a5": A + 4}, INVALID), ({"a1": None}, INVALID), ({"a6": 0}, INVALID), ({"a7": A + 2}, INVALID),
        ({"a2": 1 << 29, "a3": 4}, UNSUPPORTED)]),
    "backward": (w.w4a16_expert_combine_backward, (F16, A, A, 5, 2, A, None, 7, A, A, 0), [
        ({"a8": None, "a9": None}, INVALID), ({"a2": None}, INVALID), ({"a1": None}, INVALID), ({"a6": A + 4}, INVALID),
        ({"a8": A + 2}, INVALID), ({"a9": A + 4}, INVALID), ({"a7": -7}, INVALID)]),
}


@pytest.mark.parametrize("call,n", [(c, i) for c in CALLS for i in range(len(CALLS[c][2]))])
def test_refused(call, n):
    fn, good, refusals = CALLS[call]
    changes, status = refusals[n]
    assert _status(fn, good, **changes) == status


def test_workspace_sizes():
    assert w.w4a16_w8a8_workspace_bytes(W8, 4, 8, 32) == 4 * 32 + 16
    # few columns and a long K: room for the sums of K's parts besides
    assert w.w4a16_w8a8_workspace_bytes(W8, 512, 4096, 14336) >= 512 * 14336 + 4 * 512 + 2 * 4 * 512 * 4096
    for bad in [(G128, 4, 8, 128), (W8, 0, 8, 32), (W8, 4, 8, 40), (W8, 4, 0, 32), (W8, 4, 8, 1 << 17),
                (W8, 1 << 30, 1 << 26, 32)]:
        assert w.w4a16_w8a8_workspace_bytes(*bad) == 0
    assert w.w4a16_expert_sort_workspace_bytes(2048, 2, 8) == 0       # 4096 pairs: one block
    assert w.w4a16_expert_sort_workspace_bytes(4097, 1, 8) > 0
    assert w.w4a16_expert_sort_workspace_bytes(8193, 1, w.w4a16_max_experts() + 1) == 0


def test_binding_refuses_host_and_short_tensors():
    """Tensors on the host, and of the wrong extent or strides, before the library is called."""
    import torch
    x = torch.zeros((4, 32))
    assert _status(w.w4a16_quantize_rows_i8, (F32, x, 4, 32, A, A, 0)) == INVALID
