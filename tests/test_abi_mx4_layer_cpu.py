"""Refusals of the 4-bit floating point format's and the experts' layer's entry points without a GPU: every call
below fails a check on the host before anything touches a device (the addresses are never dereferenced)."""
import numpy as np
import pytest
import torch

import gemm_w4a16_amd as w
from test_abi_w8a8_experts_cpu import A, BF16, BIG, F16, F32, G128, INVALID, UNSUPPORTED, W8, _status
from test_binding_types_cpu import ACT, F32 as TF32, I8, I32, I64, SAME_WIDTH, U8, Described

MX4 = w.W4A16_FMT_MX4_B32_E8M0
WIDE = (1 << 22) + 32
TOKENS, PAIRS = w.w4a16_expert_layer_max_tokens(), w.w4a16_expert_layer_max_pairs()

CALLS = {
    "rows": (w.w4a16_quantize_rows_mx4, (BF16, A, 4, 64, A, A, 0), [
        ({"a0": 3}, INVALID), ({"a1": None}, INVALID), ({"a1": A + 8}, INVALID), ({"a2": 0}, INVALID), ({"a2": BIG}, INVALID),
        ({"a3": 0}, INVALID), ({"a3": 48}, INVALID), ({"a4": A + 4}, INVALID), ({"a5": None}, INVALID), ({"a3": WIDE}, UNSUPPORTED)]),
    "pack": (w.w4a16_quantize_pack, (MX4, A, 4, 64, A, A, None, 0), [
        ({"a1": A + 4}, INVALID), ({"a3": 80}, INVALID), ({"a4": None}, INVALID), ({"a5": A + 8}, INVALID), ({"a6": A}, INVALID),
        ({"a2": 0}, INVALID), ({"a2": (1 << 26) + 1}, UNSUPPORTED), ({"a3": WIDE}, UNSUPPORTED)]),
    "dequant": (w.w4a16_dequant, (MX4, A, A, None, 4, 64, BF16, A, 0), [
        ({"a1": A + 4}, INVALID), ({"a3": A}, INVALID), ({"a5": 33}, INVALID), ({"a6": 5}, INVALID), ({"a7": None}, INVALID)]),
    "gemm": (w.w4a16_gemm_w4a4, (MX4, F16, A, A, 4, A, A, None, 8, 64, A, 0), [
        ({"a0": 9}, INVALID), ({"a1": 3}, INVALID), ({"a2": None}, INVALID), ({"a3": A + 4}, INVALID), ({"a4": 0}, INVALID),
        ({"a4": BIG}, INVALID), ({"a5": A + 8}, INVALID), ({"a6": None}, INVALID), ({"a7": A}, INVALID), ({"a8": 0}, INVALID),
        ({"a9": 48}, INVALID), ({"a10": A + 2}, INVALID), ({"a0": W8}, UNSUPPORTED), ({"a0": G128, "a7": A, "a9": 128}, UNSUPPORTED),
        ({"a8": (1 << 26) + 1}, UNSUPPORTED), ({"a9": WIDE}, UNSUPPORTED)]),
    "matmul": (w.w4a16_matmul_w4a4, (MX4, F32, A, 4, A, A, None, 8, 64, A, A, 1 << 20, 0), [
        ({"a1": 3}, INVALID), ({"a2": A + 2}, INVALID), ({"a3": 0}, INVALID), ({"a10": None}, INVALID), ({"a10": A + 4}, INVALID),
        ({"a11": w.w4a16_w4a4_workspace_bytes(MX4, 4, 8, 64) - 1}, INVALID), ({"a6": A}, INVALID), ({"a8": 40}, INVALID),
        ({"a0": W8}, UNSUPPORTED)]),
    # the 16-bit products do not take the format
    "gemv": (w.w4a16_gemv, (MX4, F16, A, 1, A, A, None, 8, 64, A, 0), [({}, UNSUPPORTED), ({"a1": BF16}, UNSUPPORTED), ({"a6": A}, INVALID)]),
    "16 bit gemm": (w.w4a16_gemm, (MX4, F16, A, 70, A, A, None, 8, 64, A, None, 0, 0), [({}, UNSUPPORTED), ({"a9": A + 2}, INVALID)]),
    "16 bit matmul": (w.w4a16_matmul, (MX4, BF16, A, 70, A, A, None, 8, 64, A, None, 0, 0), [({}, UNSUPPORTED), ({"a3": 2}, UNSUPPORTED)]),
    "noalloc": (w.w4a16_matmul_noalloc, (MX4, BF16, A, 1, A, A, None, 8, 64, A, 0), [({}, UNSUPPORTED)]),
    "w8a8": (w.w4a16_gemm_w8a8, (MX4, BF16, A, A, 4, A, A, None, 8, 32, A, None, 0, 0), [({}, UNSUPPORTED)]),
    "layer": (w.w4a16_expert_layer_w8a8, (W8, BF16, A, A, 3, A, 32, 2, A, 8, A, A, A, A, 64, 96, A, A, 1 << 20, 0), [
        ({"a0": 11}, INVALID), ({"a1": 3}, INVALID), ({"a2": None}, INVALID), ({"a2": A + 4}, INVALID), ({"a3": A + 4}, INVALID),
        ({"a4": 0}, INVALID), ({"a4": -1}, INVALID), ({"a5": None}, INVALID), ({"a6": 16}, INVALID), ({"a7": 0}, INVALID),
        ({"a8": None}, INVALID), ({"a8": A + 4}, INVALID), ({"a9": 0}, INVALID), ({"a10": A + 1}, INVALID), ({"a11": None}, INVALID),
        ({"a12": None}, INVALID), ({"a13": A + 4}, INVALID), ({"a14": 0}, INVALID), ({"a14": 40}, INVALID), ({"a15": 0}, INVALID),
        ({"a15": 24}, INVALID), ({"a16": A + 2}, INVALID), ({"a17": None}, INVALID), ({"a17": A + 8}, INVALID),
        ({"a18": w.w4a16_expert_layer_workspace_bytes(3, 2, 96) - 1}, INVALID), ({"a0": MX4}, UNSUPPORTED), ({"a0": G128}, UNSUPPORTED),
        ({"a4": TOKENS + 1, "a18": 1 << 40}, UNSUPPORTED), ({"a7": PAIRS // 3 + 1, "a18": 1 << 40}, UNSUPPORTED),
        ({"a9": w.w4a16_max_experts() + 1}, UNSUPPORTED), ({"a14": 1 << 17}, UNSUPPORTED),
        ({"a15": (1 << 22) + 16, "a18": 1 << 40}, UNSUPPORTED)]),
}


@pytest.mark.parametrize("call,n", [(c, i) for c in CALLS for i in range(len(CALLS[c][2]))])
def test_refused(call, n):
    fn, good, refusals = CALLS[call]
    changes, status = refusals[n]
    assert _status(fn, good, **changes) == status


def test_sizes():
    assert w.w4a16_packed_sizes(MX4, 14336, 4096) == (14336 * 2048, 16 * 448 * 256, 0)
    assert w.w4a16_packed_sizes(MX4, 1, 32) == (16, 256, 0)
    assert w.w4a16_packed_sizes(MX4, 17, 288) == (17 * 144, 2 * 256, 0)
    assert w.w4a16_w4a4_workspace_bytes(MX4, 17, 5, 288) == 17 * 144 + 2 * 256
    for bad in [(W8, 4, 8, 32), (MX4, 0, 8, 32), (MX4, 4, 8, 40), (MX4, 4, 0, 32), (MX4, 4, 8, WIDE)]:
        assert w.w4a16_w4a4_workspace_bytes(*bad) == 0
    assert w.w4a16_gemm_workspace_bytes(MX4, 300, 256, 4096) == 0 and w.w4a16_prepared_bytes(MX4, 8, 64) == 0
    assert w.w4a16_expert_layer_workspace_bytes(3, 2, 80) == 6 * 80 + 6 * 2 * 4
    for bad in [(0, 2, 80), (3, 0, 80), (3, 2, 0), (3, 2, 40), (TOKENS + 1, 1, 80), (3, PAIRS, 80)]:
        assert w.w4a16_expert_layer_workspace_bytes(*bad) == 0
    codes, scales, mins = w.alloc_packed(MX4, 17, 288, device="cpu")
    assert codes.shape == (17, 144) and scales.shape == (2, 1, 4, 16, 2, 2) and mins is None
    assert (codes.numel(), scales.numel()) == w.w4a16_packed_sizes(MX4, 17, 288)[:2]


def test_check_weights():
    wt = np.ones((3, 64), np.float32)
    w.w4a16_check_weights(MX4, wt, 3, 64)
    wt[2, 5] = np.inf
    assert _status(w.w4a16_check_weights, (MX4, wt, 3, 64)) == INVALID


M, N, K = 5, 17, 288
T, P, E, H, I = 3, 6, 4, 32, 80
SCALES = lambda rows, k: (U8, (k + 255) // 256 * ((rows + 31) // 32) * 256)


def calls(a):
    act = ACT[a]
    layer = lambda ids, bits: (w.w4a16_expert_layer_w8a8,
                               [W8, act, (I8, T * H), (TF32, T), T, (ids, P), bits, 2, (TF32, P), E, (I8, 2 * E * H * I), (TF32, 2 * E * I),
                                (I8, E * H * I), (TF32, E * H), H, I, (a, T * H), 0x10000, 1 << 20])
    return {"rows": (w.w4a16_quantize_rows_mx4, [act, (a, M * K), M, K, (U8, M * K // 2), SCALES(M, K)]),
            "gemm": (w.w4a16_gemm_w4a4, [MX4, act, (U8, M * K // 2), SCALES(M, K), M, (U8, N * K // 2), SCALES(N, K), None, N, K, (a, M * N)]),
            "matmul": (w.w4a16_matmul_w4a4, [MX4, act, (a, M * K), M, (U8, N * K // 2), SCALES(N, K), None, N, K, (a, M * N), 0x10000, 1 << 20]),
            "layer32": layer(I32, 32), "layer64": layer(I64, 64)}


WRONG = {**SAME_WIDTH, U8: [I8, torch.bool]}
PLACES = [(name, a, i, wrong) for a in ACT for name, (_, args) in calls(a).items() for i, t in enumerate(args)
          if isinstance(t, tuple) for wrong in WRONG[t[0]] + [None]]


@pytest.mark.parametrize("name,a,place,wrong", PLACES, ids=lambda v: str(v).replace("torch.", ""))
def test_binding_refuses_another_type_or_a_shorter_tensor(name, a, place, wrong):
    """(wrong None: of the right type, an element short)"""
    fn, args = calls(a)[name]
    args = [Described(wrong or t[0], t[1] - (wrong is None), False) if i == place else Described(*t, True) if isinstance(t, tuple) else t
            for i, t in enumerate(args)]
    with pytest.raises(w.W4A16Error) as e:
        fn(*args, stream=0)
    assert e.value.status == INVALID
