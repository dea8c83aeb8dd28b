"""Refusals of the norm's entry points without a GPU: every call below fails a check on the host before anything
touches a device (the addresses are never dereferenced)."""
import pytest
import torch

import gemm_w4a16_amd as w
from test_abi_w8a8_experts_cpu import A, BF16, BIG, F16, F32, INVALID, UNSUPPORTED, _status
from test_binding_types_cpu import ACT, F32 as TF32, I8, SAME_WIDTH, Described

WIDE = (1 << 22) + 16
CALLS = {
    "norm": (w.w4a16_add_rmsnorm, (BF16, A, A, 4, 33, A, 1e-5, A + 64, A, 0), [
        ({"a0": 3}, INVALID), ({"a1": None}, INVALID), ({"a1": A + 8}, INVALID), ({"a2": A + 2}, INVALID), ({"a3": 0}, INVALID),
        ({"a3": BIG}, INVALID), ({"a4": 0}, INVALID), ({"a4": -1}, INVALID), ({"a5": A + 4}, INVALID), ({"a6": -1e-5}, INVALID),
        ({"a6": float("nan")}, INVALID), ({"a6": float("inf")}, INVALID), ({"a7": A + 1}, INVALID), ({"a7": A}, INVALID),
        ({"a8": None}, INVALID), ({"a8": A + 2}, INVALID), ({"a4": WIDE}, UNSUPPORTED)]),
    "norm_i8": (w.w4a16_add_rmsnorm_i8, (F16, A, None, 4, 32, None, 0.0, None, A, A, 0), [
        ({"a0": -1}, INVALID), ({"a1": None}, INVALID), ({"a2": A + 8}, INVALID), ({"a3": -5}, INVALID), ({"a4": 24}, INVALID),
        ({"a5": A + 2}, INVALID), ({"a6": -0.1}, INVALID), ({"a7": A + 8}, INVALID), ({"a8": None}, INVALID),
        ({"a8": A + 1}, INVALID), ({"a9": None}, INVALID), ({"a4": WIDE}, UNSUPPORTED)]),
    "backward": (w.w4a16_add_rmsnorm_backward, (F32, A, None, A, 4, 33, None, 1e-5, A, A, A, 1 << 20, 0), [
        ({"a0": 9}, INVALID), ({"a1": None}, INVALID), ({"a2": A + 4}, INVALID), ({"a3": None}, INVALID), ({"a4": 0}, INVALID),
        ({"a5": 0}, INVALID), ({"a6": A + 8}, INVALID), ({"a7": float("nan")}, INVALID), ({"a8": None, "a9": None}, INVALID),
        ({"a8": A + 4}, INVALID), ({"a9": A + 4}, INVALID), ({"a10": None}, INVALID), ({"a10": A + 8}, INVALID),
        ({"a11": w.w4a16_add_rmsnorm_backward_workspace_bytes(4, 33) - 1}, INVALID), ({"a5": WIDE, "a11": 1 << 60}, UNSUPPORTED)]),
}


@pytest.mark.parametrize("call,n", [(c, i) for c in CALLS for i in range(len(CALLS[c][2]))])
def test_refused(call, n):
    fn, good, refusals = CALLS[call]
    changes, status = refusals[n]
    assert _status(fn, good, **changes) == status


def test_workspace_sizes():
    assert w.w4a16_add_rmsnorm_backward_workspace_bytes(4, 33) == 4 * 33 * 4 + 16
    assert w.w4a16_add_rmsnorm_backward_workspace_bytes(10_000, 2048) == 256 * 2048 * 4 + 40_000
    for bad in [(0, 8), (4, 0), (-1, 8), (BIG, 8), (4, WIDE)]:
        assert w.w4a16_add_rmsnorm_backward_workspace_bytes(*bad) == 0


T, N = 5, 48


def calls(a):
    act = ACT[a]
    rows = (a, T * N)
    return {"norm": (w.w4a16_add_rmsnorm, [act, rows, rows, T, N, (a, N), 1e-5, rows, rows]),
            "norm_i8": (w.w4a16_add_rmsnorm_i8, [act, rows, rows, T, N, (a, N), 1e-5, rows, (I8, T * N), (TF32, T)]),
            "backward": (w.w4a16_add_rmsnorm_backward, [act, rows, rows, rows, T, N, (a, N), 1e-5, rows, (TF32, N), 0x10000, 1 << 20])}


PLACES = [(name, a, i, wrong) for a in ACT for name, (_, args) in calls(a).items() for i, t in enumerate(args)
          if isinstance(t, tuple) for wrong in SAME_WIDTH[t[0]] + [None]]


@pytest.mark.parametrize("name,a,place,wrong", PLACES, ids=lambda v: str(v).replace("torch.", ""))
def test_binding_refuses_another_type_or_a_shorter_tensor(name, a, place, wrong):
    """(wrong None: of the right type, an element short)"""
    fn, args = calls(a)[name]
    args = [Described(wrong or t[0], t[1] - (wrong is None), False) if i == place else Described(*t, True) if isinstance(t, tuple) else t
            for i, t in enumerate(args)]
    with pytest.raises(w.W4A16Error) as e:
        fn(*args, stream=0)
    assert e.value.status == INVALID


def test_binding_refuses_host_and_strided_tensors():
    x = torch.zeros((4, 32))
    assert _status(w.w4a16_add_rmsnorm, (F32, x, None, 4, 32, None, 1e-5, None, A, 0)) == INVALID
