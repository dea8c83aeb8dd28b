"""Python binding of libw4a16 (MI355X / gfx950 W4A16 matmul).

Argument marshalling only: every function below forwards to the C entry point of the same
name in ``libw4a16.so`` (declared in ``include/w4a16.h``) and does no arithmetic of its own.
PyTorch supplies device memory and the current HIP stream; nothing here falls back to torch or
to the CPU.  If the library has not been built, importing this package fails with an error
that says how to build it.

Array arguments may be torch tensors (their ``data_ptr()`` is passed), plain integers (raw
device pointers) or ``None`` (a NULL pointer).
"""
from __future__ import annotations

import ctypes
from pathlib import Path

_LIB_PATH = Path(__file__).resolve().parent / "libw4a16.so"

W4A16_OK, W4A16_ERR_INVALID, W4A16_ERR_UNSUPPORTED, W4A16_ERR_DEVICE = 0, 1, 2, 3
W4A16_FMT_G128_ASYM_BF16, W4A16_FMT_Q4_B32_SYM_FP16, W4A16_FMT_G128_ZP_FP16, W4A16_FMT_W8_ROW_FP32 = 0, 1, 2, 3
W4A16_FMT_MX4_B32_E8M0 = 4
W4A16_BF16, W4A16_FP16, W4A16_FP32 = 0, 1, 2

# Every symbol include/w4a16.h declares.
EXPORTED = (
    "w4a16_status_string", "w4a16_packed_sizes", "w4a16_quantize_pack", "w4a16_dequant",
    "w4a16_gemv", "w4a16_gemv_max_rows", "w4a16_gemm_workspace_bytes", "w4a16_gemm",
    "w4a16_matmul", "w4a16_matmul_gemv_cutoff", "w4a16_quantize_act_i8", "w4a16_gemm_w4a8",
    "w4a16_matmul_w4a8", "w4a16_check_weights", "w4a16_matmul_noalloc", "w4a16_matmul_noalloc_max_scratch_bytes",
    "w4a16_prepared_bytes", "w4a16_prepare", "w4a16_gemv_prepared",
    "w4a16_quantize_rows_i8", "w4a16_gemm_w8a8", "w4a16_matmul_w8a8", "w4a16_w8a8_workspace_bytes",
    "w4a16_gemm_w8a8_experts", "w4a16_max_experts", "w4a16_expert_sort", "w4a16_expert_sort_workspace_bytes",
    "w4a16_expert_gather", "w4a16_expert_gather_i8", "w4a16_expert_combine", "w4a16_expert_combine_backward",
    "w4a16_add_rmsnorm", "w4a16_add_rmsnorm_i8", "w4a16_add_rmsnorm_backward", "w4a16_add_rmsnorm_backward_workspace_bytes",
    "w4a16_quantize_rows_mx4", "w4a16_gemm_w4a4", "w4a16_matmul_w4a4", "w4a16_w4a4_workspace_bytes",
    "w4a16_expert_layer_w8a8", "w4a16_expert_layer_max_tokens", "w4a16_expert_layer_max_pairs",
    "w4a16_expert_layer_workspace_bytes",
)


class W4A16Error(RuntimeError):
    def __init__(self, status: int, call: str):
        self.status = status
        super().__init__(f"{call}: {status_string(status)} (status {status})")


def _load() -> ctypes.CDLL:
    if not _LIB_PATH.exists():
        raise ImportError(f"{_LIB_PATH} is not built; run `python gemm_w4a16_amd/build.py` "
                          "(hipcc for gfx950). There is no fallback path.")
    # PyTorch ships its own HIP runtime (libamdhip64.so.7).  It must be the one in the process
    # before libw4a16.so is loaded, so that the library's dependency on libamdhip64.so.7 binds to
    # it: loaded first, libw4a16.so would pull in the system runtime and torch would then load a
    # second one, whose streams and allocations the library's runtime does not know (every
    # launch on a torch stream would then fail).
    import torch  # noqa: F401
    L = ctypes.CDLL(str(_LIB_PATH))
    P, I64, I, SZ, F = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_size_t, ctypes.c_float
    L.w4a16_status_string.argtypes, L.w4a16_status_string.restype = [I], ctypes.c_char_p
    L.w4a16_packed_sizes.argtypes = [I, I64, I64, ctypes.POINTER(SZ), ctypes.POINTER(SZ), ctypes.POINTER(SZ)]
    L.w4a16_quantize_pack.argtypes = [I, P, I64, I64, P, P, P, P]
    L.w4a16_dequant.argtypes = [I, P, P, P, I64, I64, I, P, P]
    L.w4a16_check_weights.argtypes = [I, P, I64, I64]
    L.w4a16_gemv.argtypes = [I, I, P, I64, P, P, P, I64, I64, P, P]
    L.w4a16_gemv_max_rows.argtypes, L.w4a16_gemv_max_rows.restype = [], I64
    L.w4a16_gemm_workspace_bytes.argtypes, L.w4a16_gemm_workspace_bytes.restype = [I, I64, I64, I64], SZ
    L.w4a16_gemm.argtypes = [I, I, P, I64, P, P, P, I64, I64, P, P, SZ, P]
    L.w4a16_matmul.argtypes = [I, I, P, I64, P, P, P, I64, I64, P, P, SZ, P]
    L.w4a16_matmul_gemv_cutoff.argtypes, L.w4a16_matmul_gemv_cutoff.restype = [], I64
    L.w4a16_matmul_noalloc.argtypes = [I, I, P, I64, P, P, P, I64, I64, P, P]
    L.w4a16_matmul_noalloc_max_scratch_bytes.argtypes = []
    L.w4a16_matmul_noalloc_max_scratch_bytes.restype = SZ
    L.w4a16_prepared_bytes.argtypes, L.w4a16_prepared_bytes.restype = [I, I64, I64], SZ
    L.w4a16_prepare.argtypes = [I, P, P, P, I64, I64, P, SZ, P]
    L.w4a16_gemv_prepared.argtypes = [I, I, P, I64, P, I64, I64, P, P]
    L.w4a16_quantize_act_i8.argtypes = [P, I64, I64, P, P, P, P]
    L.w4a16_gemm_w4a8.argtypes = [I, P, P, P, I64, P, P, P, I64, I64, P, P]
    L.w4a16_matmul_w4a8.argtypes = [I, P, I64, P, P, P, I64, I64, P, P]
    L.w4a16_quantize_rows_i8.argtypes = [I, P, I64, I64, P, P, P]
    L.w4a16_gemm_w8a8.argtypes = [I, I, P, P, I64, P, P, P, I64, I64, P, P, SZ, P]
    L.w4a16_matmul_w8a8.argtypes = [I, I, P, I64, P, P, P, I64, I64, P, P, SZ, P]
    L.w4a16_w8a8_workspace_bytes.argtypes, L.w4a16_w8a8_workspace_bytes.restype = [I, I64, I64, I64], SZ
    L.w4a16_gemm_w8a8_experts.argtypes = [I, I, P, P, I64, P, I64, P, P, P, I64, I64, P, P]
    L.w4a16_max_experts.argtypes, L.w4a16_max_experts.restype = [], I64
    L.w4a16_expert_sort.argtypes = [P, I64, I64, I64, I64, P, P, P, P, SZ, P]
    L.w4a16_expert_sort_workspace_bytes.argtypes, L.w4a16_expert_sort_workspace_bytes.restype = [I64, I64, I64], SZ
    L.w4a16_expert_gather.argtypes = [I, P, I64, I64, P, I64, P, P]
    L.w4a16_expert_gather_i8.argtypes = [I, P, I64, I64, P, I64, P, P, P]
    L.w4a16_expert_combine.argtypes = [I, P, I64, I64, P, P, I64, P, P]
    L.w4a16_expert_combine_backward.argtypes = [I, P, P, I64, I64, P, P, I64, P, P, P]
    L.w4a16_add_rmsnorm.argtypes = [I, P, P, I64, I64, P, F, P, P, P]
    L.w4a16_add_rmsnorm_i8.argtypes = [I, P, P, I64, I64, P, F, P, P, P, P]
    L.w4a16_add_rmsnorm_backward.argtypes = [I, P, P, P, I64, I64, P, F, P, P, P, SZ, P]
    L.w4a16_add_rmsnorm_backward_workspace_bytes.argtypes = [I64, I64]
    L.w4a16_add_rmsnorm_backward_workspace_bytes.restype = SZ
    L.w4a16_quantize_rows_mx4.argtypes = [I, P, I64, I64, P, P, P]
    L.w4a16_gemm_w4a4.argtypes = [I, I, P, P, I64, P, P, P, I64, I64, P, P]
    L.w4a16_matmul_w4a4.argtypes = [I, I, P, I64, P, P, P, I64, I64, P, P, SZ, P]
    L.w4a16_w4a4_workspace_bytes.argtypes, L.w4a16_w4a4_workspace_bytes.restype = [I, I64, I64, I64], SZ
    L.w4a16_expert_layer_w8a8.argtypes = [I, I, P, P, I64, P, I64, I64, P, I64, P, P, P, P, I64, I64, P, P, SZ, P]
    L.w4a16_expert_layer_max_tokens.argtypes, L.w4a16_expert_layer_max_tokens.restype = [], I64
    L.w4a16_expert_layer_max_pairs.argtypes, L.w4a16_expert_layer_max_pairs.restype = [], I64
    L.w4a16_expert_layer_workspace_bytes.argtypes, L.w4a16_expert_layer_workspace_bytes.restype = [I64, I64, I64], SZ
    for name in ("w4a16_quantize_rows_i8", "w4a16_gemm_w8a8", "w4a16_matmul_w8a8", "w4a16_gemm_w8a8_experts",
                 "w4a16_expert_sort", "w4a16_expert_gather", "w4a16_expert_gather_i8", "w4a16_expert_combine",
                 "w4a16_expert_combine_backward", "w4a16_add_rmsnorm", "w4a16_add_rmsnorm_i8", "w4a16_add_rmsnorm_backward",
                 "w4a16_quantize_rows_mx4", "w4a16_gemm_w4a4", "w4a16_matmul_w4a4", "w4a16_expert_layer_w8a8"):
        getattr(L, name).restype = I
    for name in ("w4a16_packed_sizes", "w4a16_quantize_pack", "w4a16_check_weights", "w4a16_dequant", "w4a16_gemv",
                 "w4a16_gemm", "w4a16_matmul", "w4a16_matmul_noalloc", "w4a16_quantize_act_i8", "w4a16_gemm_w4a8",
                 "w4a16_matmul_w4a8", "w4a16_prepare", "w4a16_gemv_prepared"):
        getattr(L, name).restype = I
    return L


lib = _load()
library_path = str(_LIB_PATH)


def _stream_lookup():
    """(current device, its current stream's handle) lookups: torch's own C functions where this torch has
    them (0.2 us; the Stream object of torch.cuda.current_stream() costs 2.7 us a call)."""
    import torch
    device = getattr(torch._C, "_cuda_getDevice", None)
    stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    if device is None or stream is None:  # another torch, or one without a GPU
        return torch.cuda.current_device, lambda d: torch.cuda.current_stream(d).cuda_stream
    return device, stream


# (for a process that has initialised the GPU: one that holds a tensor there)
_current_device, _current_stream = _stream_lookup()


def _p(a):
    """Device pointer of a torch tensor / raw int / None."""
    if a is None:
        return None
    if isinstance(a, int):
        return a
    return a.data_ptr()


def _stream(stream):
    if stream is None:
        import torch
        torch.cuda.init()  # (returns at once when done)
        return _current_stream(_current_device())
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _ok(status: int, call: str) -> None:
    if status != W4A16_OK:
        raise W4A16Error(status, call)


def status_string(status: int) -> str:
    return lib.w4a16_status_string(int(status)).decode()


w4a16_status_string = status_string


def w4a16_packed_sizes(fmt: int, N: int, K: int):
    c, s, m = ctypes.c_size_t(), ctypes.c_size_t(), ctypes.c_size_t()
    _ok(lib.w4a16_packed_sizes(fmt, N, K, ctypes.byref(c), ctypes.byref(s), ctypes.byref(m)),
        "w4a16_packed_sizes")
    return c.value, s.value, m.value


def w4a16_quantize_pack(fmt: int, W, N: int, K: int, codes, scales, mins, stream=None) -> None:
    _ok(lib.w4a16_quantize_pack(fmt, _p(W), N, K, _p(codes), _p(scales), _p(mins), _stream(stream)),
        "w4a16_quantize_pack")


def w4a16_check_weights(fmt: int, W, N: int, K: int) -> None:
    """Host-side weight check (W: a C-contiguous float32 numpy array or a host address)."""
    addr = W if isinstance(W, int) or W is None else W.ctypes.data
    _ok(lib.w4a16_check_weights(fmt, addr, N, K), "w4a16_check_weights")


def w4a16_dequant(fmt: int, codes, scales, mins, N: int, K: int, out_dtype: int, W_hat, stream=None) -> None:
    _ok(lib.w4a16_dequant(fmt, _p(codes), _p(scales), _p(mins), N, K, out_dtype, _p(W_hat), _stream(stream)),
        "w4a16_dequant")


def w4a16_gemv(fmt: int, act: int, x, M: int, codes, scales, mins, N: int, K: int, y, stream=None) -> None:
    _ok(lib.w4a16_gemv(fmt, act, _p(x), M, _p(codes), _p(scales), _p(mins), N, K, _p(y), _stream(stream)),
        "w4a16_gemv")


def w4a16_gemv_max_rows() -> int:
    return int(lib.w4a16_gemv_max_rows())


def w4a16_gemm_workspace_bytes(fmt: int, M: int, N: int, K: int) -> int:
    return int(lib.w4a16_gemm_workspace_bytes(fmt, M, N, K))


def w4a16_gemm(fmt: int, act: int, x, M: int, codes, scales, mins, N: int, K: int, y, workspace=None,
               workspace_bytes: int = 0, stream=None) -> None:
    _ok(lib.w4a16_gemm(fmt, act, _p(x), M, _p(codes), _p(scales), _p(mins), N, K, _p(y), _p(workspace),
                       workspace_bytes, _stream(stream)), "w4a16_gemm")


def w4a16_matmul(fmt: int, act: int, x, M: int, codes, scales, mins, N: int, K: int, y, workspace=None,
                 workspace_bytes: int = 0, stream=None) -> None:
    _ok(lib.w4a16_matmul(fmt, act, _p(x), M, _p(codes), _p(scales), _p(mins), N, K, _p(y), _p(workspace),
                         workspace_bytes, _stream(stream)), "w4a16_matmul")


def w4a16_matmul_noalloc(fmt: int, act: int, x, M: int, codes, scales, mins, N: int, K: int, y, stream=None) -> None:
    _ok(lib.w4a16_matmul_noalloc(fmt, act, _p(x), M, _p(codes), _p(scales), _p(mins), N, K, _p(y), _stream(stream)),
        "w4a16_matmul_noalloc")


def w4a16_matmul_noalloc_max_scratch_bytes() -> int:
    return int(lib.w4a16_matmul_noalloc_max_scratch_bytes())


def w4a16_prepared_bytes(fmt: int, N: int, K: int) -> int:
    return int(lib.w4a16_prepared_bytes(fmt, N, K))


def w4a16_prepare(fmt: int, codes, scales, mins, N: int, K: int, prepared, prepared_bytes: int, stream=None) -> None:
    _ok(lib.w4a16_prepare(fmt, _p(codes), _p(scales), _p(mins), N, K, _p(prepared), prepared_bytes,
                             _stream(stream)), "w4a16_prepare")


def w4a16_gemv_prepared(fmt: int, act: int, x, M: int, prepared, N: int, K: int, y, stream=None) -> None:
    _ok(lib.w4a16_gemv_prepared(fmt, act, _p(x), M, _p(prepared), N, K, _p(y), _stream(stream)),
        "w4a16_gemv_prepared")


def w4a16_matmul_gemv_cutoff() -> int:
    return int(lib.w4a16_matmul_gemv_cutoff())


def w4a16_quantize_act_i8(x, M: int, K: int, xq, ascale, xsum, stream=None) -> None:
    _ok(lib.w4a16_quantize_act_i8(_p(x), M, K, _p(xq), _p(ascale), _p(xsum), _stream(stream)),
        "w4a16_quantize_act_i8")


def w4a16_gemm_w4a8(fmt: int, xq, ascale, xsum, M: int, codes, scales, mins, N: int, K: int, y,
                    stream=None) -> None:
    _ok(lib.w4a16_gemm_w4a8(fmt, _p(xq), _p(ascale), _p(xsum), M, _p(codes), _p(scales), _p(mins), N, K,
                            _p(y), _stream(stream)), "w4a16_gemm_w4a8")


def w4a16_matmul_w4a8(fmt: int, x, M: int, codes, scales, mins, N: int, K: int, y, stream=None) -> None:
    _ok(lib.w4a16_matmul_w4a8(fmt, _p(x), M, _p(codes), _p(scales), _p(mins), N, K, _p(y), _stream(stream)),
        "w4a16_matmul_w4a8")


# ---- W8A8, the experts' operators, W4A4, norms -----------------------------------------------------
# Tensors given to these must be on one GPU, contiguous, of the type the call takes them as and at least as
# large as it reads or writes (W4A16_ERR_INVALID otherwise); the launch goes to that GPU's current stream,
# whichever GPU is current.  Raw addresses are passed as they are.

import torch  # noqa: E402 (loaded with the library, above)

_I8, _U8, _I32, _F32 = torch.int8, torch.uint8, torch.int32, torch.float32
_ACT = {W4A16_BF16: torch.bfloat16, W4A16_FP16: torch.float16, W4A16_FP32: _F32}.get  # None: the library refuses it
_ID = {32: _I32, 64: torch.int64}.get


def _call(name: str, args, arrays, stream) -> None:
    """lib.<name>(*args, stream): ``arrays`` gives the array arguments' places in ``args``, the elements
    each must hold and their type (None: any, and that many bytes)."""
    device = None
    args = list(args)
    for at, count, dtype in arrays:
        t = args[at]
        if t is None or isinstance(t, int):
            continue
        d = t.get_device()
        if (d != device and (d < 0 or device is not None) or (t.nbytes if dtype is None else t.numel()) < count
                or (dtype is not None and t.dtype is not dtype) or not t.is_contiguous()):
            raise W4A16Error(W4A16_ERR_INVALID, name)
        device = d
        args[at] = t.data_ptr()
    fn = getattr(lib, name)
    if device is None:
        status = fn(*args, _stream(stream))
    elif device == _current_device():
        status = fn(*args, _current_stream(device) if stream is None else _stream(stream))
    else:
        with torch.cuda.device(device):
            status = fn(*args, _stream(stream))
    if status != W4A16_OK:
        raise W4A16Error(status, name)


def w4a16_quantize_rows_i8(act: int, x, M: int, K: int, xq, ascale, stream=None) -> None:
    _call("w4a16_quantize_rows_i8", (act, x, M, K, xq, ascale),
          ((1, M * K, _ACT(act)), (4, M * K, _I8), (5, M, _F32)), stream)


def w4a16_gemm_w8a8(fmt: int, out: int, xq, ascale, M: int, codes, scales, mins, N: int, K: int, y, workspace=None,
                    workspace_bytes: int = 0, stream=None) -> None:
    _call("w4a16_gemm_w8a8", (fmt, out, xq, ascale, M, codes, scales, mins, N, K, y, workspace, workspace_bytes),
          ((2, M * K, _I8), (3, M, _F32), (5, N * K, _I8), (6, N, _F32), (7, 0, None), (10, M * N, _ACT(out)),
           (11, workspace_bytes, None)), stream)


def w4a16_matmul_w8a8(fmt: int, act: int, x, M: int, codes, scales, mins, N: int, K: int, y, workspace,
                      workspace_bytes: int, stream=None) -> None:
    t = _ACT(act)
    _call("w4a16_matmul_w8a8", (fmt, act, x, M, codes, scales, mins, N, K, y, workspace, workspace_bytes),
          ((2, M * K, t), (4, N * K, _I8), (5, N, _F32), (6, 0, None), (9, M * N, t), (10, workspace_bytes, None)), stream)


def w4a16_w8a8_workspace_bytes(fmt: int, M: int, N: int, K: int) -> int:
    return int(lib.w4a16_w8a8_workspace_bytes(fmt, M, N, K))


def w4a16_gemm_w8a8_experts(fmt: int, out: int, xq, ascale, R: int, offsets, E: int, codes, scales, mins, N: int, K: int,
                            y, stream=None) -> None:
    _call("w4a16_gemm_w8a8_experts", (fmt, out, xq, ascale, R, offsets, E, codes, scales, mins, N, K, y),
          ((2, R * K, _I8), (3, R, _F32), (5, E + 1, _I32), (7, E * N * K, _I8), (8, E * N, _F32), (9, 0, None),
           (12, R * N, _ACT(out))), stream)


def w4a16_max_experts() -> int:
    return int(lib.w4a16_max_experts())


def w4a16_expert_sort_workspace_bytes(T: int, topk: int, E: int) -> int:
    return int(lib.w4a16_expert_sort_workspace_bytes(T, topk, E))


def w4a16_expert_sort(ids, id_bits: int, T: int, topk: int, E: int, offsets, pos, src, workspace=None,
                      workspace_bytes: int = 0, stream=None) -> None:
    P = T * topk
    _call("w4a16_expert_sort", (ids, id_bits, T, topk, E, offsets, pos, src, workspace, workspace_bytes),
          ((0, P, _ID(id_bits)), (5, E + 1, _I32), (6, P, _I32), (7, P, _I32), (8, workspace_bytes, None)), stream)


def w4a16_expert_gather(act: int, x, T: int, topk: int, pos, K: int, xs, stream=None) -> None:
    P, t = T * topk, _ACT(act)
    _call("w4a16_expert_gather", (act, x, T, topk, pos, K, xs), ((1, T * K, t), (4, P, _I32), (6, P * K, t)), stream)


def w4a16_expert_gather_i8(act: int, x, T: int, topk: int, pos, K: int, xq, ascale, stream=None) -> None:
    P = T * topk
    _call("w4a16_expert_gather_i8", (act, x, T, topk, pos, K, xq, ascale),
          ((1, T * K, _ACT(act)), (4, P, _I32), (6, P * K, _I8), (7, P, _F32)), stream)


def w4a16_expert_combine(act: int, ys, T: int, topk: int, pos, weights, N: int, y, stream=None) -> None:
    P, t = T * topk, _ACT(act)
    _call("w4a16_expert_combine", (act, ys, T, topk, pos, weights, N, y),
          ((1, P * N, t), (4, P, _I32), (5, P, _F32), (7, T * N, t)), stream)


def w4a16_expert_combine_backward(act: int, dy, ys, T: int, topk: int, pos, weights, N: int, dys, dweights,
                                  stream=None) -> None:
    P, t = T * topk, _ACT(act)
    _call("w4a16_expert_combine_backward", (act, dy, ys, T, topk, pos, weights, N, dys, dweights),
          ((1, T * N, t), (2, P * N, t), (5, P, _I32), (6, P, _F32), (8, P * N, t), (9, P, _F32)), stream)


def w4a16_expert_layer_w8a8(fmt: int, out: int, xq, ascale, T: int, ids, id_bits: int, topk: int, weights, E: int, up_codes,
                            up_scales, down_codes, down_scales, H: int, I: int, y, workspace, workspace_bytes: int,
                            stream=None) -> None:
    P, W = T * topk, E * H * I
    _call("w4a16_expert_layer_w8a8", (fmt, out, xq, ascale, T, ids, id_bits, topk, weights, E, up_codes, up_scales, down_codes,
                                      down_scales, H, I, y, workspace, workspace_bytes),
          ((2, T * H, _I8), (3, T, _F32), (5, P, _ID(id_bits)), (8, P, _F32), (10, 2 * W, _I8), (11, 2 * E * I, _F32),
           (12, W, _I8), (13, E * H, _F32), (16, T * H, _ACT(out)), (17, workspace_bytes, None)), stream)


def w4a16_expert_layer_max_tokens() -> int:
    return int(lib.w4a16_expert_layer_max_tokens())


def w4a16_expert_layer_max_pairs() -> int:
    return int(lib.w4a16_expert_layer_max_pairs())


def w4a16_expert_layer_workspace_bytes(T: int, topk: int, I: int) -> int:
    return int(lib.w4a16_expert_layer_workspace_bytes(T, topk, I))


def _mx4_scale_bytes(rows: int, K: int) -> int:
    return (K + 255) // 256 * ((rows + 31) // 32) * 256


def w4a16_quantize_rows_mx4(act: int, x, M: int, K: int, xq, xscales, stream=None) -> None:
    _call("w4a16_quantize_rows_mx4", (act, x, M, K, xq, xscales),
          ((1, M * K, _ACT(act)), (4, M * K // 2, _U8), (5, _mx4_scale_bytes(M, K), _U8)), stream)


def w4a16_gemm_w4a4(fmt: int, out: int, xq, xscales, M: int, codes, scales, mins, N: int, K: int, y, stream=None) -> None:
    _call("w4a16_gemm_w4a4", (fmt, out, xq, xscales, M, codes, scales, mins, N, K, y),
          ((2, M * K // 2, _U8), (3, _mx4_scale_bytes(M, K), _U8), (5, N * K // 2, _U8), (6, _mx4_scale_bytes(N, K), _U8),
           (7, 0, None), (10, M * N, _ACT(out))), stream)


def w4a16_matmul_w4a4(fmt: int, act: int, x, M: int, codes, scales, mins, N: int, K: int, y, workspace,
                      workspace_bytes: int, stream=None) -> None:
    t = _ACT(act)
    _call("w4a16_matmul_w4a4", (fmt, act, x, M, codes, scales, mins, N, K, y, workspace, workspace_bytes),
          ((2, M * K, t), (4, N * K // 2, _U8), (5, _mx4_scale_bytes(N, K), _U8), (6, 0, None), (9, M * N, t),
           (10, workspace_bytes, None)), stream)


def w4a16_w4a4_workspace_bytes(fmt: int, M: int, N: int, K: int) -> int:
    return int(lib.w4a16_w4a4_workspace_bytes(fmt, M, N, K))


def w4a16_add_rmsnorm(act: int, x, residual, T: int, N: int, weight, eps: float, h, y, stream=None) -> None:
    t, n = _ACT(act), T * N
    _call("w4a16_add_rmsnorm", (act, x, residual, T, N, weight, eps, h, y),
          ((1, n, t), (2, n, t), (5, N, t), (7, n, t), (8, n, t)), stream)


def w4a16_add_rmsnorm_i8(act: int, x, residual, T: int, N: int, weight, eps: float, h, xq, ascale, stream=None) -> None:
    t, n = _ACT(act), T * N
    _call("w4a16_add_rmsnorm_i8", (act, x, residual, T, N, weight, eps, h, xq, ascale),
          ((1, n, t), (2, n, t), (5, N, t), (7, n, t), (8, n, _I8), (9, T, _F32)), stream)


def w4a16_add_rmsnorm_backward(act: int, dy, dh, h, T: int, N: int, weight, eps: float, dx, dweight, workspace=None,
                               workspace_bytes: int = 0, stream=None) -> None:
    t, n = _ACT(act), T * N
    _call("w4a16_add_rmsnorm_backward", (act, dy, dh, h, T, N, weight, eps, dx, dweight, workspace, workspace_bytes),
          ((1, n, t), (2, n, t), (3, n, t), (6, N, t), (8, n, t), (9, N, _F32), (10, workspace_bytes, None)), stream)


def w4a16_add_rmsnorm_backward_workspace_bytes(T: int, N: int) -> int:
    return int(lib.w4a16_add_rmsnorm_backward_workspace_bytes(T, N))


# ---- memory plumbing (torch allocations with the ABI's shapes and dtypes) ------------------------

def alloc_packed(fmt: int, N: int, K: int, device="cuda"):
    """Empty (codes, scales, mins) device tensors for an N x K weight (mins is None for Q4, W8 and MX4;
    the zero points for the zero-point format)."""
    import torch
    w4a16_packed_sizes(fmt, N, K)  # validates the shape
    if fmt == W4A16_FMT_G128_ASYM_BF16:
        # scales/mins: [K/128][N] views of buffers padded to the size w4a16_packed_sizes asks for
        n = K // 128 * N
        padded = n + (n & 1)
        return (torch.empty((K // 8, N), dtype=torch.int32, device=device),
                torch.empty(padded, dtype=torch.int16, device=device)[:n].view(K // 128, N),
                torch.empty(padded, dtype=torch.int16, device=device)[:n].view(K // 128, N))
    if fmt == W4A16_FMT_W8_ROW_FP32:
        return (torch.empty((N, K), dtype=torch.int8, device=device),
                torch.empty(N, dtype=torch.float32, device=device),
                None)
    if fmt == W4A16_FMT_MX4_B32_E8M0:  # (rows' codes and scales as well, with M for N)
        return (torch.empty((N, K // 2), dtype=torch.uint8, device=device),
                torch.empty(((K + 255) // 256, (N + 31) // 32, 4, 16, 2, 2), dtype=torch.uint8, device=device),
                None)
    if fmt == W4A16_FMT_G128_ZP_FP16:
        return (torch.empty((N, K // 8), dtype=torch.int32, device=device),
                torch.empty((N, K // 128), dtype=torch.int16, device=device),
                torch.empty((N, K // 128), dtype=torch.int16, device=device))
    return (torch.empty((N, K // 32, 16), dtype=torch.uint8, device=device),
            torch.empty((N, K // 32), dtype=torch.int16, device=device),
            None)


def alloc_act_i8(M: int, K: int, device="cuda"):
    """Empty (xq int8 [M][K], ascale fp32 [M], xsum fp32 [K/128][M]) for w4a16_quantize_act_i8."""
    import torch
    return (torch.empty((M, K), dtype=torch.int8, device=device),
            torch.empty(M, dtype=torch.float32, device=device),
            torch.empty((K // 128, M), dtype=torch.float32, device=device))


def alloc_workspace(fmt: int, M: int, N: int, K: int, device="cuda"):
    """(tensor or None, bytes) sized for w4a16_gemm / w4a16_matmul on this shape."""
    import torch
    nbytes = w4a16_gemm_workspace_bytes(fmt, M, N, K)
    if nbytes == 0:
        return None, 0
    return torch.empty(nbytes, dtype=torch.uint8, device=device), nbytes


def alloc_w8a8_workspace(fmt: int, M: int, N: int, K: int, device="cuda"):
    """(tensor, bytes) sized for w4a16_matmul_w8a8 (and w4a16_gemm_w8a8) on this shape."""
    import torch
    nbytes = w4a16_w8a8_workspace_bytes(fmt, M, N, K)
    return torch.empty(nbytes, dtype=torch.uint8, device=device), nbytes


def alloc_w4a4_workspace(fmt: int, M: int, N: int, K: int, device="cuda"):
    """(tensor, bytes) sized for w4a16_matmul_w4a4 on this shape."""
    import torch
    nbytes = w4a16_w4a4_workspace_bytes(fmt, M, N, K)
    return torch.empty(nbytes, dtype=torch.uint8, device=device), nbytes


def alloc_expert_sort(T: int, topk: int, E: int, device="cuda"):
    """Empty (offsets [E + 1], pos [T][topk], src [T * topk], workspace or None, its bytes) for
    w4a16_expert_sort."""
    import torch
    nbytes = w4a16_expert_sort_workspace_bytes(T, topk, E)
    i32 = lambda *shape: torch.empty(shape, dtype=torch.int32, device=device)
    return (i32(E + 1), i32(T, topk), i32(T * topk),
            torch.empty(nbytes, dtype=torch.uint8, device=device) if nbytes else None, nbytes)


def alloc_add_rmsnorm_backward_workspace(T: int, N: int, device="cuda"):
    """(tensor, bytes) sized for w4a16_add_rmsnorm_backward."""
    import torch
    nbytes = w4a16_add_rmsnorm_backward_workspace_bytes(T, N)
    return torch.empty(nbytes, dtype=torch.uint8, device=device), nbytes


def alloc_expert_layer_workspace(T: int, topk: int, I: int, device="cuda"):
    """(tensor, bytes) sized for w4a16_expert_layer_w8a8."""
    import torch
    nbytes = w4a16_expert_layer_workspace_bytes(T, topk, I)
    return torch.empty(nbytes, dtype=torch.uint8, device=device), nbytes
