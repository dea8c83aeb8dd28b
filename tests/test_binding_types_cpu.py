"""The W8A8 and experts' calls refuse a tensor of another type than they take it as, also one of the same width,
before the library is called (no GPU needed: the tensors here only describe themselves)."""
import pytest
import torch

import gemm_w4a16_amd as w

W8 = w.W4A16_FMT_W8_ROW_FP32
ACT = {torch.bfloat16: w.W4A16_BF16, torch.float16: w.W4A16_FP16, torch.float32: w.W4A16_FP32}


class Described:
    """A contiguous tensor on a GPU, as far as the binding asks.  Its address is not asked for before every check of
    this argument has passed."""

    def __init__(self, dtype, n, fine):
        self.dtype, self.n, self.fine = dtype, n, fine
        self.nbytes = n * dtype.itemsize

    def get_device(self):
        return 0

    def numel(self):
        return self.n

    def element_size(self):
        return self.dtype.itemsize

    def is_contiguous(self):
        return True

    def data_ptr(self):
        assert self.fine, "taken in spite of its type"
        return 0x10000


I8, I16, I32, I64 = torch.int8, torch.int16, torch.int32, torch.int64
U8, BF16, F16, F32, F64 = torch.uint8, torch.bfloat16, torch.float16, torch.float32, torch.float64
SAME_WIDTH = {I8: [U8, torch.bool], I32: [F32], I64: [F64], BF16: [F16, I16], F16: [BF16, I16], F32: [I32]}

# The call with its tensors' types: ("type", elements) are tensors, the rest plain values.  T = 5 tokens of 2 pairs.
T, P, N, K, E = 5, 10, 8, 32, 3


def calls(a):
    act = ACT[a]
    sizes = lambda *s: list(s)
    return {
        "quantize_rows": (w.w4a16_quantize_rows_i8, sizes(act, (a, T * K), T, K, (I8, T * K), (F32, T))),
        "gemm": (w.w4a16_gemm_w8a8, sizes(W8, act, (I8, T * K), (F32, T), T, (I8, N * K), (F32, N), None, N, K, (a, T * N))),
        "matmul": (w.w4a16_matmul_w8a8, sizes(W8, act, (a, T * K), T, (I8, N * K), (F32, N), None, N, K, (a, T * N), 0x10000, 1 << 20)),
        "experts": (w.w4a16_gemm_w8a8_experts, sizes(W8, act, (I8, P * K), (F32, P), P, (I32, E + 1), E, (I8, E * N * K),
                                                     (F32, E * N), None, N, K, (a, P * N))),
        "sort32": (w.w4a16_expert_sort, sizes((I32, P), 32, T, 2, E, (I32, E + 1), (I32, P), (I32, P))),
        "sort64": (w.w4a16_expert_sort, sizes((I64, P), 64, T, 2, E, (I32, E + 1), (I32, P), (I32, P))),
        "gather": (w.w4a16_expert_gather, sizes(act, (a, T * K), T, 2, (I32, P), K, (a, P * K))),
        "gather_i8": (w.w4a16_expert_gather_i8, sizes(act, (a, T * K), T, 2, (I32, P), K, (I8, P * K), (F32, P))),
        "combine": (w.w4a16_expert_combine, sizes(act, (a, P * N), T, 2, (I32, P), (F32, P), N, (a, T * N))),
        "backward": (w.w4a16_expert_combine_backward, sizes(act, (a, T * N), (a, P * N), T, 2, (I32, P), (F32, P), N, (a, P * N),
                                                            (F32, P))),
    }


PLACES = [(name, a, i, wrong) for a in ACT for name, (_, args) in calls(a).items() for i, t in enumerate(args) if isinstance(t, tuple)
          for wrong in SAME_WIDTH[t[0]]]


@pytest.mark.parametrize("name,a,place,wrong", PLACES, ids=lambda v: str(v).replace("torch.", ""))
def test_refused(name, a, place, wrong):
    fn, args = calls(a)[name]
    args = [Described(wrong if i == place else t[0], t[1], i != place) if isinstance(t, tuple) else t for i, t in enumerate(args)]
    with pytest.raises(w.W4A16Error) as e:
        fn(*args, stream=0)
    assert e.value.status == w.W4A16_ERR_INVALID


@pytest.mark.parametrize("name,a,place", [(n, a, i) for a in ACT for n, (_, args) in calls(a).items() for i, t in enumerate(args)
                                          if isinstance(t, tuple)], ids=lambda v: str(v).replace("torch.", ""))
def test_one_element_short_is_refused(name, a, place):
    fn, args = calls(a)[name]
    args = [Described(t[0], t[1] - (i == place), i != place) if isinstance(t, tuple) else t for i, t in enumerate(args)]
    with pytest.raises(w.W4A16Error) as e:
        fn(*args, stream=0)
    assert e.value.status == w.W4A16_ERR_INVALID
