"""Python binding of the FP8 (E4M3) GEMM C ABI (``include/fp8gemm.h``).

Argument marshalling only: every computation runs in the CUDA kernels of
``libfp8g.so`` (built in-tree for sm_103a by ``buildlib.py``).  Tensor arguments
may be torch tensors (their ``data_ptr()`` is passed) or raw integer device
addresses.  ``stream`` defaults to torch's current CUDA stream.  A non-OK
status raises :class:`Fp8gError` carrying the ``fp8g_status`` code.

There is no fallback: if the shared library is missing or cannot be loaded,
the first call raises.
"""
from __future__ import annotations

import ctypes
import os
import threading

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libfp8g.so")

FP8G_OK = 0
FP8G_ERR_INVALID_ARG = 1
FP8G_ERR_ALIGNMENT = 2
FP8G_ERR_UNSUPPORTED_SHAPE = 3
FP8G_ERR_SCALE_FORMAT = 4
FP8G_ERR_CUDA = 5
FP8G_ERR_TIMEOUT = 6
FP8G_ERR_DEVICE = 7

FP8G_OUT_BF16 = 0
FP8G_OUT_F32 = 1
FP8G_E4M3 = 0
FP8G_E5M2 = 1
FP8G_E2M1 = 2
FP8G_E2M3 = 3
FP8G_E3M2 = 4
FP8G_BLOCK32_LITERAL = 33
FP8G_IN_F32 = 0
FP8G_IN_BF16 = 1
FP8G_ACT_NONE = 0
FP8G_ACT_RELU = 1
FP8G_ACT_GELU = 2
FP8G_MAX_EXPERTS = 64
FP8G_QUANT_FUSED = 1
FP8G_MAX_ROUTED_EXPERTS = 256
FP8G_MAX_TOP_K = 16
FP8G_MAX_ROUTED_TOKENS = 262144
FP8G_MOE_MAX_TOKENS = 512
FP8G_MAX_ADAPTERS = 1024
FP8G_MAX_LORA_RANK = 256
FP8G_SCORE_SOFTMAX = 0
FP8G_SCORE_SOFTMAX_TOPK = 1
FP8G_SCORE_SIGMOID = 2
FP8G_SCORE_SIGMOID_NORM = 3
FP8G_GATE_SILU = 0
FP8G_GATE_GELU = 1
FP8G_GATE_RELU = 2
FP8G_NT = 0
FP8G_NN = 1
FP8G_TN = 2

# Every symbol include/fp8gemm.h declares.
EXPORTS = (
    "fp8_gemm", "fp8_gemm_blockscaled", "fp8_gemm_blockscaled_noalloc", "fp8_grouped_gemm", "fp8g_grouped_plan",
    "fp8g_gemm_plan", "fp8g_quantize_e4m3", "fp8g_quantize", "fp8_gemm_fmt",
    "fp8_gemm_blockscaled_fmt", "fp8_grouped_gemm_fmt", "fp8_gemm_ex", "fp8_gemm_blockscaled_ex",
    "fp8_grouped_gemm_ex", "fp8_grouped_gemm_scatter", "fp8_grouped_gemm_quant",
    "fp8g_quantize_rows",
    "fp8_gemm_blockscaled_promote", "fp8g_quantize_nvfp4", "fp8_gemm_nvfp4",
    "fp8_grouped_gemm_nvfp4", "fp8g_wait_selftest",
    "fp8g_kernel_timing_begin", "fp8g_kernel_timing_end",
    "fp8_gemm_status", "fp8g_status_string",
    "fp8g_set_wait_timeout_ms", "fp8g_shutdown", "fp8g_version",
    "fp8g_packed_scale_bytes", "fp8g_pack_scales", "fp8g_moe_route", "fp8_moe_layer",
    "fp8_gemm_lora",
    "fp8g_quantize_block128", "fp8g_quantize_tile128", "fp8g_requantize_block128",
    "fp8_gemm_block128", "fp8_gated_block128", "fp8g_gated_block128_backward",
)


class Fp8gError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = int(status)
        super().__init__(f"{where}: {fp8g_status_string(status)} (status {status})")


_lib = None
_lock = threading.Lock()


def build(force: bool = False) -> str:
    from . import buildlib
    return buildlib.build(force=force)


def load():
    """Load libfp8g.so (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is not None:
            return _lib
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"{LIB_PATH} is missing: build it with "
                              "fp8_block_scaled_06_gb300.build() (nvcc, sm_103a)")
        lib = ctypes.CDLL(LIB_PATH)
        P = ctypes.c_void_p
        i64 = ctypes.c_int64
        i32 = ctypes.c_int32
        st = ctypes.c_int
        lib.fp8_gemm.restype = st
        lib.fp8_gemm.argtypes = [P, P, P, P, P, ctypes.c_int, i64, i64, i64, P]
        lib.fp8_gemm_blockscaled.restype = st
        lib.fp8_gemm_blockscaled.argtypes = [P, P, P, P, P, ctypes.c_int, i64, i64, i64, P]
        lib.fp8_gemm_blockscaled_noalloc.restype = st
        lib.fp8_gemm_blockscaled_noalloc.argtypes = [P, P, P, P, P, ctypes.c_int, i64, i64, i64, P]
        lib.fp8_grouped_gemm.restype = st
        lib.fp8_grouped_gemm.argtypes = [P, P, P, P, P, ctypes.c_int, P, i32, i64, i64, i64, P,
                                         P, P]
        lib.fp8g_grouped_plan.restype = st
        lib.fp8g_grouped_plan.argtypes = [i64, i64, i64, i32, P, P, P, P]
        lib.fp8g_gemm_plan.restype = st
        lib.fp8g_gemm_plan.argtypes = [ctypes.c_int, i64, i64, i64, P, P, P, P, P]
        lib.fp8g_quantize_e4m3.restype = st
        lib.fp8g_quantize_e4m3.argtypes = [P, i64, i64, i32, P, P, P]
        lib.fp8g_quantize.restype = st
        lib.fp8g_quantize.argtypes = [P, i64, i64, i32, i32, P, P, P]
        lib.fp8g_quantize_nvfp4.restype = st
        lib.fp8g_quantize_nvfp4.argtypes = [P, i32, i64, i64, P, P, P, P]
        lib.fp8_gemm_nvfp4.restype = st
        lib.fp8_gemm_nvfp4.argtypes = [P, P, P, P, P, P, P, ctypes.c_int, P, i32, i64, i64, i64,
                                       P]
        lib.fp8_grouped_gemm_nvfp4.restype = st
        lib.fp8_grouped_gemm_nvfp4.argtypes = [P, P, P, P, P, P, P, ctypes.c_int, P, i32, P, i32,
                                               i64, i64, i64, P, P, P]
        lib.fp8_gemm_fmt.restype = st
        lib.fp8_gemm_fmt.argtypes = [P, P, P, P, P, ctypes.c_int, i32, i32, i64, i64, i64, P]
        lib.fp8_gemm_blockscaled_fmt.restype = st
        lib.fp8_gemm_blockscaled_fmt.argtypes = [P, P, P, P, P, ctypes.c_int, i32, i32, i64, i64,
                                                 i64, P]
        lib.fp8_gemm_ex.restype = st
        lib.fp8_gemm_ex.argtypes = [P, P, P, P, P, ctypes.c_int, i32, i32, P, i32, i64, i64, i64,
                                    P]
        lib.fp8_gemm_blockscaled_ex.restype = st
        lib.fp8_gemm_blockscaled_ex.argtypes = [P, P, P, P, P, ctypes.c_int, i32, i32, P, i32, i64,
                                                i64, i64, P]
        lib.fp8_grouped_gemm_ex.restype = st
        lib.fp8_grouped_gemm_ex.argtypes = [P, P, P, P, P, ctypes.c_int, i32, i32, P, i32, P, i32,
                                            i64, i64, i64, P, P, P]
        lib.fp8_grouped_gemm_scatter.restype = st
        lib.fp8_grouped_gemm_scatter.argtypes = [P, P, P, P, P, ctypes.c_int, i32, i32, P, i32, P,
                                                 i32, i64, i64, i64, P, i64, P, P, P]
        lib.fp8_grouped_gemm_quant.restype = st
        lib.fp8_grouped_gemm_quant.argtypes = [P, i32, i64, P, P, P, P, ctypes.c_int, i32, P, i32,
                                               P, i32, i64, i64, i64, P, i64, P, P, P, P, i32, P]
        lib.fp8_gemm_blockscaled_promote.restype = st
        lib.fp8_gemm_blockscaled_promote.argtypes = [P, P, P, P, P, ctypes.c_int, i32, i32, P, i32,
                                                     i64, i64, i64, P]
        lib.fp8g_kernel_timing_begin.restype = st
        lib.fp8g_kernel_timing_begin.argtypes = [i32]
        lib.fp8g_kernel_timing_end.restype = st
        lib.fp8g_kernel_timing_end.argtypes = [P, i32, P]
        lib.fp8g_wait_selftest.restype = st
        lib.fp8g_wait_selftest.argtypes = [ctypes.c_uint32, P]
        lib.fp8g_quantize_rows.restype = st
        lib.fp8g_quantize_rows.argtypes = [P, i32, i64, i64, P, i64, i32, i32, P, P, P]
        lib.fp8_grouped_gemm_fmt.restype = st
        lib.fp8_grouped_gemm_fmt.argtypes = [P, P, P, P, P, ctypes.c_int, i32, i32, P, i32, i64,
                                             i64, i64, P, P, P]
        lib.fp8g_packed_scale_bytes.restype = i64
        lib.fp8g_packed_scale_bytes.argtypes = [i64, i64, i64]
        lib.fp8g_pack_scales.restype = st
        lib.fp8g_pack_scales.argtypes = [P, i64, i64, i64, P, P]
        lib.fp8g_moe_route.restype = st
        lib.fp8g_moe_route.argtypes = [P, i32, i64, i64, i32, i32, i32, ctypes.c_float, P, P, P, P,
                                       P, P]
        lib.fp8_moe_layer.restype = st
        lib.fp8_moe_layer.argtypes = [P, i32, P, P, P, P, P, P, P, ctypes.c_int, i32, i32, i64,
                                      i32, i32, i64, i64, P]
        lib.fp8_gemm_lora.restype = st
        lib.fp8_gemm_lora.argtypes = [P, i32, P, P, i32, P, P, P, P, i32, i32, P, P, ctypes.c_int,
                                      i64, i64, i64, P]
        for name, args in (
                ("fp8g_quantize_block128", [P, i32, i64, i64, i64, i32, P, P, P, P, P]),
                ("fp8g_quantize_tile128", [P, i32, i64, i64, i64, i32, P, P, P]),
                ("fp8g_requantize_block128", [P, i32, P, i64, i64, i32, P, P, P]),
                ("fp8_gemm_block128", [i32, P, P, i32, P, P, i32, P, ctypes.c_int, i32, i64, i64, i64, P]),
                ("fp8_gated_block128", [P, P, i32, P, P, i32, i32, P, P, P, P, i64, i64, i64, P]),
                ("fp8g_gated_block128_backward", [P, i32, P, P, i32, i32, i64, i64, P, P, P, P, P, P, P])):
            getattr(lib, name).restype = st
            getattr(lib, name).argtypes = args
        lib.fp8_gemm_status.restype = st
        lib.fp8_gemm_status.argtypes = [P, P]
        lib.fp8g_status_string.restype = ctypes.c_char_p
        lib.fp8g_status_string.argtypes = [st]
        lib.fp8g_set_wait_timeout_ms.restype = None
        lib.fp8g_set_wait_timeout_ms.argtypes = [ctypes.c_uint32]
        lib.fp8g_shutdown.restype = None
        lib.fp8g_shutdown.argtypes = []
        lib.fp8g_version.restype = ctypes.c_int
        lib.fp8g_version.argtypes = []
        _lib = lib
        return lib


def _ptr(x):
    if x is None:
        return None
    if isinstance(x, int):
        return x
    return x.data_ptr()


_current = None


def _bind_stream():
    """The current stream's raw handle, without a Stream object around it (0.2
    against 2.9 us on the GB300 host, a third of a small call)."""
    global _current
    import torch
    raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    dev = getattr(torch._C, "_cuda_getDevice", None)
    if raw is None or dev is None:
        return torch.cuda.current_stream().cuda_stream
    torch.cuda.current_stream()  # CUDA is set up from here on
    _current = lambda: raw(dev())
    return _current()


def _stream(stream):
    if stream is None:
        return _current() if _current is not None else _bind_stream()
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _check(status: int, where: str):
    if status != FP8G_OK:
        raise Fp8gError(status, where)


def fp8g_status_string(status: int) -> str:
    return load().fp8g_status_string(int(status)).decode()


def fp8_gemm(A, B, scale_a, scale_b, C, out: int, M: int, N: int, K: int, stream=None):
    _check(load().fp8_gemm(_ptr(A), _ptr(B), _ptr(scale_a), _ptr(scale_b), _ptr(C), int(out),
                           M, N, K, _stream(stream)), "fp8_gemm")


def fp8_gemm_blockscaled(A, B, sfa, sfb, C, out: int, M: int, N: int, K: int, stream=None):
    _check(load().fp8_gemm_blockscaled(_ptr(A), _ptr(B), _ptr(sfa), _ptr(sfb), _ptr(C), int(out),
                                       M, N, K, _stream(stream)), "fp8_gemm_blockscaled")


def fp8_gemm_blockscaled_noalloc(A, B, sfa, sfb, C, out: int, M: int, N: int, K: int,
                                 stream=None):
    """Allocation-free fp8_gemm_blockscaled (packed scales in the library's fixed array)."""
    _check(load().fp8_gemm_blockscaled_noalloc(_ptr(A), _ptr(B), _ptr(sfa), _ptr(sfb), _ptr(C),
                                               int(out), M, N, K, _stream(stream)),
           "fp8_gemm_blockscaled_noalloc")


def fp8_grouped_gemm(A, B, sfa, sfb, C, out: int, counts, E: int, N: int, K: int,
                     total_rows: int, offsets_out=None, tile_map_out=None, stream=None):
    _check(load().fp8_grouped_gemm(_ptr(A), _ptr(B), _ptr(sfa), _ptr(sfb), _ptr(C), int(out),
                                   _ptr(counts), E, N, K, total_rows, _ptr(offsets_out),
                                   _ptr(tile_map_out), _stream(stream)), "fp8_grouped_gemm")


def fp8g_grouped_plan(N: int, K: int, total_rows: int, E: int) -> dict:
    BM, BN, G = ctypes.c_int32(), ctypes.c_int32(), ctypes.c_int32()
    T = ctypes.c_int64()
    _check(load().fp8g_grouped_plan(N, K, total_rows, E, ctypes.byref(BM), ctypes.byref(BN),
                                    ctypes.byref(G), ctypes.byref(T)), "fp8g_grouped_plan")
    return {"BM": BM.value, "BN": BN.value, "G": G.value, "max_tiles": T.value}


def fp8g_gemm_plan(block: int, M: int, N: int, K: int) -> dict:
    BM, BN, G, S, grid = (ctypes.c_int32() for _ in range(5))
    _check(load().fp8g_gemm_plan(int(block), M, N, K, ctypes.byref(BM), ctypes.byref(BN),
                                 ctypes.byref(G), ctypes.byref(S), ctypes.byref(grid)),
           "fp8g_gemm_plan")
    return {"BM": BM.value, "BN": BN.value, "G": G.value, "split_k": S.value, "grid": grid.value}


def fp8g_quantize_e4m3(x, rows: int, cols: int, block: int, q, scales, stream=None):
    _check(load().fp8g_quantize_e4m3(_ptr(x), rows, cols, int(block), _ptr(q), _ptr(scales),
                                     _stream(stream)), "fp8g_quantize_e4m3")


def fp8g_quantize(x, rows: int, cols: int, block: int, fmt: int, q, scales, stream=None):
    _check(load().fp8g_quantize(_ptr(x), rows, cols, int(block), int(fmt), _ptr(q),
                                _ptr(scales), _stream(stream)), "fp8g_quantize")


def fp8_gemm_fmt(A, B, scale_a, scale_b, C, out: int, a_fmt: int, b_fmt: int, M: int, N: int,
                 K: int, stream=None):
    _check(load().fp8_gemm_fmt(_ptr(A), _ptr(B), _ptr(scale_a), _ptr(scale_b), _ptr(C), int(out),
                               int(a_fmt), int(b_fmt), M, N, K, _stream(stream)), "fp8_gemm_fmt")


def fp8_gemm_blockscaled_fmt(A, B, sfa, sfb, C, out: int, a_fmt: int, b_fmt: int, M: int,
                             N: int, K: int, stream=None):
    _check(load().fp8_gemm_blockscaled_fmt(_ptr(A), _ptr(B), _ptr(sfa), _ptr(sfb), _ptr(C),
                                           int(out), int(a_fmt), int(b_fmt), M, N, K,
                                           _stream(stream)), "fp8_gemm_blockscaled_fmt")


def fp8_grouped_gemm_fmt(A, B, sfa, sfb, C, out: int, a_fmt: int, b_fmt: int, counts, E: int,
                         N: int, K: int, total_rows: int, offsets_out=None, tile_map_out=None,
                         stream=None):
    _check(load().fp8_grouped_gemm_fmt(_ptr(A), _ptr(B), _ptr(sfa), _ptr(sfb), _ptr(C), int(out),
                                       int(a_fmt), int(b_fmt), _ptr(counts), E, N, K, total_rows,
                                       _ptr(offsets_out), _ptr(tile_map_out), _stream(stream)),
           "fp8_grouped_gemm_fmt")


def fp8_gemm_ex(A, B, scale_a, scale_b, C, out: int, a_fmt: int, b_fmt: int, bias, act: int,
                M: int, N: int, K: int, stream=None):
    _check(load().fp8_gemm_ex(_ptr(A), _ptr(B), _ptr(scale_a), _ptr(scale_b), _ptr(C), int(out),
                              int(a_fmt), int(b_fmt), _ptr(bias), int(act), M, N, K,
                              _stream(stream)), "fp8_gemm_ex")


def fp8_gemm_blockscaled_ex(A, B, sfa, sfb, C, out: int, a_fmt: int, b_fmt: int, bias, act: int,
                            M: int, N: int, K: int, stream=None):
    _check(load().fp8_gemm_blockscaled_ex(_ptr(A), _ptr(B), _ptr(sfa), _ptr(sfb), _ptr(C),
                                          int(out), int(a_fmt), int(b_fmt), _ptr(bias), int(act),
                                          M, N, K, _stream(stream)), "fp8_gemm_blockscaled_ex")


def fp8_grouped_gemm_ex(A, B, sfa, sfb, C, out: int, a_fmt: int, b_fmt: int, bias, act: int,
                        counts, E: int, N: int, K: int, total_rows: int, offsets_out=None,
                        tile_map_out=None, stream=None):
    _check(load().fp8_grouped_gemm_ex(_ptr(A), _ptr(B), _ptr(sfa), _ptr(sfb), _ptr(C), int(out),
                                      int(a_fmt), int(b_fmt), _ptr(bias), int(act), _ptr(counts),
                                      E, N, K, total_rows, _ptr(offsets_out), _ptr(tile_map_out),
                                      _stream(stream)), "fp8_grouped_gemm_ex")


def fp8_grouped_gemm_scatter(A, B, sfa, sfb, C, out: int, a_fmt: int, b_fmt: int, bias,
                             act: int, counts, E: int, N: int, K: int, total_rows: int, c_row_of,
                             c_rows: int, offsets_out=None, tile_map_out=None, stream=None):
    _check(load().fp8_grouped_gemm_scatter(_ptr(A), _ptr(B), _ptr(sfa), _ptr(sfb), _ptr(C),
                                           int(out), int(a_fmt), int(b_fmt), _ptr(bias), int(act),
                                           _ptr(counts), E, N, K, total_rows, _ptr(c_row_of),
                                           c_rows, _ptr(offsets_out), _ptr(tile_map_out),
                                           _stream(stream)), "fp8_grouped_gemm_scatter")


def fp8_grouped_gemm_quant(X, x_dtype: int, x_rows: int, rows, B, sfb, C, out: int, b_fmt: int,
                           bias, act: int, counts, E: int, N: int, K: int, total_rows: int,
                           c_row_of=None, c_rows: int = 0, qa_out=None, sfa_out=None,
                           offsets_out=None, tile_map_out=None, flags: int = 0, stream=None):
    """Grouped GEMM from fp32 / bf16 activations: gather, 1x32 E4M3 quantisation
    (inside the GEMM kernel with flags FP8G_QUANT_FUSED when the plan runs
    single-CTA tiles) and the grouped GEMM with bias / activation and row
    scatter."""
    _check(load().fp8_grouped_gemm_quant(_ptr(X), int(x_dtype), x_rows, _ptr(rows), _ptr(B),
                                         _ptr(sfb), _ptr(C), int(out), int(b_fmt), _ptr(bias),
                                         int(act), _ptr(counts), int(E), N, K, total_rows,
                                         _ptr(c_row_of), c_rows, _ptr(qa_out), _ptr(sfa_out),
                                         _ptr(offsets_out), _ptr(tile_map_out), int(flags),
                                         _stream(stream)), "fp8_grouped_gemm_quant")


def fp8_gemm_blockscaled_promote(A, B, sfa, sfb, C, out: int, a_fmt: int, b_fmt: int, bias,
                                 act: int, M: int, N: int, K: int, stream=None):
    _check(load().fp8_gemm_blockscaled_promote(_ptr(A), _ptr(B), _ptr(sfa), _ptr(sfb), _ptr(C),
                                               int(out), int(a_fmt), int(b_fmt), _ptr(bias),
                                               int(act), M, N, K, _stream(stream)),
           "fp8_gemm_blockscaled_promote")


def fp8g_quantize_nvfp4(x, in_dtype: int, rows: int, cols: int, q, sf, g, stream=None):
    _check(load().fp8g_quantize_nvfp4(_ptr(x), int(in_dtype), rows, cols, _ptr(q), _ptr(sf),
                                      _ptr(g), _stream(stream)), "fp8g_quantize_nvfp4")


def fp8_gemm_nvfp4(A, B, sfa, sfb, ga, gb, C, out: int, bias, act: int, M: int, N: int, K: int,
                   stream=None):
    _check(load().fp8_gemm_nvfp4(_ptr(A), _ptr(B), _ptr(sfa), _ptr(sfb), _ptr(ga), _ptr(gb),
                                 _ptr(C), int(out), _ptr(bias), int(act), M, N, K,
                                 _stream(stream)), "fp8_gemm_nvfp4")


def fp8_grouped_gemm_nvfp4(A, B, sfa, sfb, ga, gb, C, out: int, bias, act: int, counts, E: int,
                           N: int, K: int, total_rows: int, offsets_out=None, tile_map_out=None,
                           stream=None):
    _check(load().fp8_grouped_gemm_nvfp4(_ptr(A), _ptr(B), _ptr(sfa), _ptr(sfb), _ptr(ga),
                                         _ptr(gb), _ptr(C), int(out), _ptr(bias), int(act),
                                         _ptr(counts), E, N, K, total_rows, _ptr(offsets_out),
                                         _ptr(tile_map_out), _stream(stream)),
           "fp8_grouped_gemm_nvfp4")


def quantize_nvfp4(x, stream=None):
    """fp32 or bf16 CUDA tensor [rows, cols] -> (codes uint8 [rows, cols/2],
    E4M3 block-scale codes uint8 [rows, cols/16], tensor scale fp32 [1])."""
    import torch
    assert x.is_cuda and x.dim() == 2 and x.dtype in (torch.float32, torch.bfloat16)
    x = x.contiguous()
    rows, cols = x.shape
    q = torch.empty((rows, cols // 2), dtype=torch.uint8, device=x.device)
    sf = torch.empty((rows, cols // 16), dtype=torch.uint8, device=x.device)
    g = torch.empty((1,), dtype=torch.float32, device=x.device)
    dt = FP8G_IN_BF16 if x.dtype == torch.bfloat16 else FP8G_IN_F32
    fp8g_quantize_nvfp4(x, dt, rows, cols, q, sf, g, stream)
    return q, sf, g


def fp8g_quantize_rows(x, in_dtype: int, x_rows: int, cols: int, rows, n_rows: int, block: int,
                       fmt: int, q, scales, stream=None):
    _check(load().fp8g_quantize_rows(_ptr(x), int(in_dtype), x_rows, cols, _ptr(rows), n_rows,
                                     int(block), int(fmt), _ptr(q), _ptr(scales),
                                     _stream(stream)), "fp8g_quantize_rows")


def fp8g_packed_scale_bytes(matrices: int, rows: int, K: int) -> int:
    return int(load().fp8g_packed_scale_bytes(matrices, rows, K))


def fp8g_pack_scales(sf, matrices: int, rows: int, K: int, packed, stream=None):
    _check(load().fp8g_pack_scales(_ptr(sf), matrices, rows, K, _ptr(packed), _stream(stream)),
           "fp8g_pack_scales")


def fp8g_moe_route(logits, in_dtype: int, ld: int, T: int, E: int, k: int, score: int,
                   scale: float, ids, weights, counts=None, rows=None, slots=None, stream=None):
    _check(load().fp8g_moe_route(_ptr(logits), int(in_dtype), ld, T, int(E), int(k), int(score),
                                 float(scale), _ptr(ids), _ptr(weights), _ptr(counts), _ptr(rows),
                                 _ptr(slots), _stream(stream)), "fp8g_moe_route")


def fp8_moe_layer(x, x_dtype: int, ids, weights, W13, sf13, W2, sf2, out, out_dtype: int,
                  w_fmt: int, gate: int, T: int, k: int, E: int, H: int, F: int, stream=None):
    _check(load().fp8_moe_layer(_ptr(x), int(x_dtype), _ptr(ids), _ptr(weights), _ptr(W13),
                                _ptr(sf13), _ptr(W2), _ptr(sf2), _ptr(out), int(out_dtype),
                                int(w_fmt), int(gate), T, int(k), int(E), H, F, _stream(stream)),
           "fp8_moe_layer")


def fp8_gemm_lora(x, x_dtype: int, W, sfw, w_fmt: int, lora_a, lora_b, alpha, adapter, L: int,
                  r: int, bias, C, out: int, M: int, N: int, K: int, stream=None):
    _check(load().fp8_gemm_lora(_ptr(x), int(x_dtype), _ptr(W), _ptr(sfw), int(w_fmt),
                                _ptr(lora_a), _ptr(lora_b), _ptr(alpha), _ptr(adapter), int(L),
                                int(r), _ptr(bias), _ptr(C), int(out), M, N, K, _stream(stream)),
           "fp8_gemm_lora")


def fp8g_quantize_block128(x, in_dtype: int, ld: int, rows: int, cols: int, fmt: int, q_row=None,
                           s_row=None, q_col=None, s_col=None, stream=None):
    _check(load().fp8g_quantize_block128(_ptr(x), int(in_dtype), ld, rows, cols, int(fmt), _ptr(q_row),
                                         _ptr(s_row), _ptr(q_col), _ptr(s_col), _stream(stream)),
           "fp8g_quantize_block128")


def fp8g_quantize_tile128(x, in_dtype: int, ld: int, rows: int, cols: int, fmt: int, q, s,
                          stream=None):
    _check(load().fp8g_quantize_tile128(_ptr(x), int(in_dtype), ld, rows, cols, int(fmt), _ptr(q),
                                        _ptr(s), _stream(stream)), "fp8g_quantize_tile128")


def fp8g_requantize_block128(q, q_fmt: int, s, rows: int, cols: int, fmt: int, q_col, s_col,
                             stream=None):
    _check(load().fp8g_requantize_block128(_ptr(q), int(q_fmt), _ptr(s), rows, cols, int(fmt),
                                           _ptr(q_col), _ptr(s_col), _stream(stream)),
           "fp8g_requantize_block128")


def fp8_gemm_block128(form: int, A, sfa, a_fmt: int, B, sfb, b_fmt: int, C, out: int, add: int,
                      M: int, N: int, K: int, stream=None):
    _check(load().fp8_gemm_block128(int(form), _ptr(A), _ptr(sfa), int(a_fmt), _ptr(B), _ptr(sfb),
                                    int(b_fmt), _ptr(C), int(out), int(add), M, N, K,
                                    _stream(stream)), "fp8_gemm_block128")


def fp8_gated_block128(x, sfx, x_fmt: int, W13, sf13, w_fmt: int, gate: int, h, sh, gu, sgu, M: int,
                       F: int, K: int, stream=None):
    _check(load().fp8_gated_block128(_ptr(x), _ptr(sfx), int(x_fmt), _ptr(W13), _ptr(sf13), int(w_fmt),
                                     int(gate), _ptr(h), _ptr(sh), _ptr(gu), _ptr(sgu), M, F, K,
                                     _stream(stream)), "fp8_gated_block128")


def fp8g_gated_block128_backward(dh, dh_dtype: int, gu, sgu, gate: int, fmt: int, M: int, F: int, dgu_row,
                                 s_row, dgu_col, s_col, h_col, sh_col, stream=None):
    _check(load().fp8g_gated_block128_backward(_ptr(dh), int(dh_dtype), _ptr(gu), _ptr(sgu), int(gate),
                                               int(fmt), M, F, _ptr(dgu_row), _ptr(s_row), _ptr(dgu_col),
                                               _ptr(s_col), _ptr(h_col), _ptr(sh_col), _stream(stream)),
           "fp8g_gated_block128_backward")


def fp8g_kernel_timing_begin(n: int):
    _check(load().fp8g_kernel_timing_begin(int(n)), "fp8g_kernel_timing_begin")


def fp8g_kernel_timing_end(cap: int) -> list:
    """GEMM-kernel durations (ms) of the calls recorded since begin."""
    ms = (ctypes.c_float * max(int(cap), 1))()
    n = ctypes.c_int32(0)
    _check(load().fp8g_kernel_timing_end(ms, int(cap), ctypes.byref(n)), "fp8g_kernel_timing_end")
    return [float(ms[i]) for i in range(n.value)]


def fp8g_wait_selftest(timeout_us: int, stream=None):
    _check(load().fp8g_wait_selftest(int(timeout_us), _stream(stream)), "fp8g_wait_selftest")


def fp8_gemm_status(stream=None):
    """Returns (status, detail) and clears the device status word."""
    detail = ctypes.c_int32(0)
    st = load().fp8_gemm_status(_stream(stream), ctypes.byref(detail))
    return int(st), int(detail.value)


def fp8g_set_wait_timeout_ms(ms: int):
    load().fp8g_set_wait_timeout_ms(int(ms))


def fp8g_shutdown():
    load().fp8g_shutdown()


def fp8g_version() -> int:
    return int(load().fp8g_version())


# ---------------------------------------------------------------- conveniences
# Allocation helpers over torch (device memory is plumbing); the work is the
# ABI call above.

def packed_cols(cols: int, fmt: int) -> int:
    """Bytes of a row of `cols` codes in format fmt."""
    if fmt == FP8G_E2M1:
        return cols // 2
    if fmt in (FP8G_E2M3, FP8G_E3M2):
        return cols * 3 // 4
    return cols


def quantize(x, block: int = 32, stream=None, fmt: int = FP8G_E4M3):
    """fp32 CUDA tensor [rows, cols] -> (uint8 codes, fp32 scales) in format fmt
    (E2M1: two codes per byte, codes [rows, cols/2]; FP6: four codes per three
    bytes, codes [rows, 3 cols/4])."""
    import torch
    assert x.is_cuda and x.dtype == torch.float32 and x.dim() == 2
    x = x.contiguous()
    rows, cols = x.shape
    qcols = packed_cols(cols, fmt)
    q = torch.empty((rows, qcols), dtype=torch.uint8, device=x.device)
    if block != 0:
        s = torch.empty((rows, cols // 32), dtype=torch.float32, device=x.device)
    else:
        s = torch.empty((1,), dtype=torch.float32, device=x.device)
    fp8g_quantize(x, rows, cols, block, fmt, q, s, stream)
    return q, s


def gemm(A, B, sa, sb, out: str = "bf16", block: bool = True, stream=None):
    """Allocates C and runs fp8_gemm_blockscaled (block) or fp8_gemm (per-tensor)."""
    import torch
    M, K = A.shape
    N = B.shape[0]
    dt = torch.bfloat16 if out == "bf16" else torch.float32
    C = torch.empty((M, N), dtype=dt, device=A.device)
    o = FP8G_OUT_BF16 if out == "bf16" else FP8G_OUT_F32
    if block:
        fp8_gemm_blockscaled(A, B, sa, sb, C, o, M, N, K, stream)
    else:
        fp8_gemm(A, B, sa, sb, C, o, M, N, K, stream)
    return C


def _packed(x, stream):
    """x, packed: a copy is made on the current stream and its memory is that
    stream's, so a call on a `stream` of its own refuses to make one."""
    assert stream is None, "with a stream of its own a call takes packed tensors"
    return x.contiguous()


def _packed_bytes(matrices: int, rows: int, K: int) -> int:
    """fp8g_packed_scale_bytes, without the call."""
    return matrices * (-(-rows // 128)) * (-(-K // 128)) * 512


def pack_scales(sf, stream=None):
    """Block scales fp32 [rows, K/32] or [matrices, rows, K/32] -> the packed
    uint8 [(matrices,) ceil(K/128), ceil(rows/128), 512] that moe_layer and
    gemm_lora take (once per weight)."""
    import torch
    assert sf.is_cuda and sf.dtype == torch.float32 and sf.dim() in (2, 3)
    if not sf.is_contiguous():
        sf = _packed(sf, stream)
    rows, kb = sf.shape[-2:]
    lead = tuple(sf.shape[:-2])
    out = torch.empty(lead + (-(-kb // 4), -(-rows // 128), 512), dtype=torch.uint8,
                      device=sf.device)
    fp8g_pack_scales(sf, lead[0] if lead else 1, rows, 32 * kb, out, stream)
    return out


# The three below are called once a layer for a few tokens, where the host's time
# is what a call costs: torch's names are looked up once, dtypes compared by
# identity and the library's function called at once (on the GB300 host gemm_lora
# takes 18.5 us of which the C call 8 to 12, 20.9 before).  The output is the
# current stream's memory.

_t = None  # torch, its dtypes


def _names():
    global _t
    import torch
    _t = (torch.empty, torch.bfloat16, torch.float32, torch.int32, torch.uint8)
    return _t


def moe_route(logits, k: int, score: int = FP8G_SCORE_SOFTMAX_TOPK, scale: float = 1.0,
              ordered: bool = False, stream=None):
    """fp32 or bf16 logits [T, E] -> (ids int32 [T, k], weights fp32 [T, k]), and
    with `ordered` also (counts [E], rows [T k], slots [T k]), the row order of the
    grouped GEMM (its counts, rows and c_row_of)."""
    empty, bf16, f32, i32, _ = _t or _names()
    dt, dev = logits.dtype, logits.device
    assert logits.is_cuda and (dt is f32 or dt is bf16)
    T, E = logits.shape
    ld, step = logits.stride()
    if T <= 1:
        ld = E
    if E > 1 and step != 1 or ld < E:
        logits, ld = _packed(logits, stream), E
    ids = empty((T, k), dtype=i32, device=dev)
    w = empty((T, k), dtype=f32, device=dev)
    if not ordered:
        st = (_lib or load()).fp8g_moe_route(
            logits.data_ptr(), FP8G_IN_BF16 if dt is bf16 else FP8G_IN_F32, ld, T, E, k, score, scale,
            ids.data_ptr(), w.data_ptr(), None, None, None, _stream(stream))
        if st:
            raise Fp8gError(st, "fp8g_moe_route")
        return ids, w
    counts = empty(E, dtype=i32, device=dev)
    rows = empty(T * k, dtype=i32, device=dev)
    slots = empty(T * k, dtype=i32, device=dev)
    st = (_lib or load()).fp8g_moe_route(
        logits.data_ptr(), FP8G_IN_BF16 if dt is bf16 else FP8G_IN_F32, ld, T, E, k, score, scale,
        ids.data_ptr(), w.data_ptr(), counts.data_ptr(), rows.data_ptr(), slots.data_ptr(), _stream(stream))
    if st:
        raise Fp8gError(st, "fp8g_moe_route")
    return ids, w, counts, rows, slots


def moe_layer(x, ids, weights, W13, sf13, W2, sf2, w_fmt: int = FP8G_E4M3,
              gate: int = FP8G_GATE_SILU, out: str = "bf16", stream=None):
    """Mixture-of-experts layer of a few tokens: x fp32 or bf16 [T, H], ids and
    weights [T, k] from moe_route, W13 [E, 2F, H] and W2 [E, H, F] codes of w_fmt
    (one-byte elements), sf13 / sf2 from pack_scales (sf13 of W13's scales viewed
    as [2E, F, H/32]), all on x's device.  Allocates the output [T, H]."""
    empty, bf16, f32, i32, u8 = _t or _names()
    dt, dev = x.dtype, x.get_device()
    assert dev >= 0 and (dt is bf16 or dt is f32)
    assert ids.get_device() == dev and weights.get_device() == dev and W13.get_device() == dev
    assert W2.get_device() == dev and sf13.get_device() == dev and sf2.get_device() == dev
    assert ids.dtype is i32 and weights.dtype is f32 and W13.itemsize == 1 and W2.itemsize == 1
    assert sf13.dtype is u8 and sf2.dtype is u8, "scales from pack_scales"
    T, H = x.shape
    t, k = ids.shape
    E, F2, c13 = W13.shape
    F = F2 // 2
    assert t == T and weights.shape == ids.shape and c13 == packed_cols(H, w_fmt)
    assert W2.shape == (E, H, packed_cols(F, w_fmt)) and W13.is_contiguous() and W2.is_contiguous()
    assert sf13.numel() == _packed_bytes(2 * E, F, H) and sf2.numel() == _packed_bytes(E, H, F)
    assert sf13.is_contiguous() and sf2.is_contiguous()
    if not (x.is_contiguous() and ids.is_contiguous() and weights.is_contiguous()):
        x, ids, weights = _packed(x, stream), _packed(ids, stream), _packed(weights, stream)
    wide = out != "bf16"
    o = empty((T, H), dtype=f32 if wide else bf16, device=x.device)
    st = (_lib or load()).fp8_moe_layer(
        x.data_ptr(), FP8G_IN_BF16 if dt is bf16 else FP8G_IN_F32, ids.data_ptr(), weights.data_ptr(),
        W13.data_ptr(), sf13.data_ptr(), W2.data_ptr(), sf2.data_ptr(), o.data_ptr(),
        FP8G_OUT_F32 if wide else FP8G_OUT_BF16, w_fmt, gate, T, k, E, H, F, _stream(stream))
    if st:
        raise Fp8gError(st, "fp8_moe_layer")
    return o


def gemm_lora(x, W, sfw, lora_a, lora_b, alpha, adapter, bias=None, w_fmt: int = FP8G_E4M3,
              out: str = "bf16", stream=None):
    """Projection with low-rank adapters: x fp32 or bf16 [M, K], W codes [N, K] of
    w_fmt (one-byte elements), sfw from pack_scales, lora_a bf16 [L, r, K], lora_b
    bf16 [L, N, r], alpha fp32 [L] or None, adapter int32 [M] (negative: none),
    bias fp32 [N] or None, all on x's device.  Allocates C [M, N]."""
    empty, bf16, f32, i32, u8 = _t or _names()
    dt, dev = x.dtype, x.get_device()
    assert dev >= 0 and (dt is bf16 or dt is f32)
    assert W.get_device() == dev and sfw.get_device() == dev and adapter.get_device() == dev
    assert lora_a.get_device() == dev and lora_b.get_device() == dev
    assert lora_a.dtype is bf16 and lora_b.dtype is bf16 and adapter.dtype is i32 and W.itemsize == 1
    assert sfw.dtype is u8, "scales from pack_scales"
    M, K = x.shape
    N, cols = W.shape
    L, r, ka = lora_a.shape
    assert cols == (K if w_fmt < FP8G_E2M1 else packed_cols(K, w_fmt)) and ka == K and lora_b.shape == (L, N, r)
    assert adapter.numel() == M and sfw.numel() == (N + 127) // 128 * ((K + 127) // 128) * 512
    assert alpha is None or (alpha.get_device() == dev and alpha.dtype is f32 and alpha.numel() == L
                             and alpha.is_contiguous())
    assert bias is None or (bias.get_device() == dev and bias.dtype is f32 and bias.numel() == N
                            and bias.is_contiguous())
    assert W.is_contiguous() and sfw.is_contiguous()
    if not (x.is_contiguous() and adapter.is_contiguous() and lora_a.is_contiguous() and lora_b.is_contiguous()):
        x, adapter = _packed(x, stream), _packed(adapter, stream)
        lora_a, lora_b = _packed(lora_a, stream), _packed(lora_b, stream)
    wide = out != "bf16"
    C = empty((M, N), dtype=f32 if wide else bf16, device=x.device)
    st = (_lib or load()).fp8_gemm_lora(
        x.data_ptr(), FP8G_IN_BF16 if dt is bf16 else FP8G_IN_F32, W.data_ptr(), sfw.data_ptr(), w_fmt,
        lora_a.data_ptr(), lora_b.data_ptr(), None if alpha is None else alpha.data_ptr(),
        adapter.data_ptr(), L, r, None if bias is None else bias.data_ptr(), C.data_ptr(),
        FP8G_OUT_F32 if wide else FP8G_OUT_BF16, M, N, K, _stream(stream))
    if st:
        raise Fp8gError(st, "fp8_gemm_lora")
    return C


# Scales for blocks of 128 (fp8_gemm_block128 and the calls around it).  Codes are
# uint8 (or torch's float8 of the format that is named) [R, C]; scales fp32 [ceil(C/128), R] along rows,
# [ceil(R/128), C] along columns, [ceil(R/128), ceil(C/128)] of tiles.

_here = None  # the current device's index


def _on(dev: int, *tensors):
    """The tensors lie on device `dev`, the current one, and are packed."""
    global _here
    if _here is None:
        import torch
        _here = torch._C._cuda_getDevice  # (torch.cuda.current_device without its check for a first use)
    assert dev >= 0 and dev == _here(), "tensors of the current CUDA device"
    for t in tensors:
        assert t.get_device() == dev and t.is_contiguous()


_f8 = None


def _coded(t, fmt: int) -> bool:
    """t holds codes of fmt: bytes, or torch's type of that format."""
    global _f8
    dt = t.dtype
    if dt is (_t or _names())[4]:
        return True
    if _f8 is None:
        import torch
        _f8 = (torch.float8_e4m3fn, torch.float8_e5m2)
    return fmt in (FP8G_E4M3, FP8G_E5M2) and dt is _f8[fmt]


def _source(x, stream):
    """x [R, C] fp32 or bf16 -> (x, rows apart), its columns packed and rows 16-byte aligned."""
    _, bf16, f32, _, _ = _t or _names()
    dt = x.dtype
    assert dt is bf16 or dt is f32
    R, C = x.shape
    ld, step = x.stride()
    if R <= 1:
        ld = C
    if (C > 1 and step != 1) or ld < C or ld * x.itemsize % 16 or x.data_ptr() % 16:
        x, ld = _packed(x, stream), C
        if x.data_ptr() % 16:
            x = x.clone()
    return x, ld


def quantize_block128(x, row: bool = True, col: bool = False, fmt: int = FP8G_E4M3, stream=None):
    """fp32 or bf16 [R, C] -> ((codes, scales) along rows or None, (codes, scales)
    along columns or None), one reading of x."""
    empty, bf16, f32, _, u8 = _t or _names()
    dev = x.device
    _on(x.get_device())
    assert row or col
    x, ld = _source(x, stream)
    R, C = x.shape
    qr = empty((R, C), dtype=u8, device=dev) if row else None
    sr = empty((-(-C // 128), R), dtype=f32, device=dev) if row else None
    qc = empty((R, C), dtype=u8, device=dev) if col else None
    sc = empty((-(-R // 128), C), dtype=f32, device=dev) if col else None
    st = (_lib or load()).fp8g_quantize_block128(
        x.data_ptr(), FP8G_IN_BF16 if x.dtype is bf16 else FP8G_IN_F32, ld, R, C, fmt,
        _ptr(qr), _ptr(sr), _ptr(qc), _ptr(sc), _stream(stream))
    if st:
        raise Fp8gError(st, "fp8g_quantize_block128")
    return (qr, sr) if row else None, (qc, sc) if col else None


def quantize_tile128(x, fmt: int = FP8G_E4M3, stream=None):
    """fp32 or bf16 [R, C] (weights) -> (codes, scales of 128 x 128 tiles)."""
    empty, bf16, f32, _, u8 = _t or _names()
    _on(x.get_device())
    x, ld = _source(x, stream)
    R, C = x.shape
    q = empty((R, C), dtype=u8, device=x.device)
    s = empty((-(-R // 128), -(-C // 128)), dtype=f32, device=x.device)
    fp8g_quantize_tile128(x, FP8G_IN_BF16 if x.dtype is bf16 else FP8G_IN_F32, ld, R, C, fmt, q, s, stream)
    return q, s


def requantize_block128(q, s, fmt: int = FP8G_E4M3, q_fmt: int = FP8G_E4M3, stream=None):
    """Codes [R, C] of q_fmt with scales along rows -> (codes, scales) along columns."""
    empty, _, f32, _, u8 = _t or _names()
    _on(q.get_device(), q, s)
    R, C = q.shape
    assert _coded(q, q_fmt) and s.dtype is f32 and s.shape == (-(-C // 128), R)
    qc = empty((R, C), dtype=u8, device=q.device)
    sc = empty((-(-R // 128), C), dtype=f32, device=q.device)
    st = (_lib or load()).fp8g_requantize_block128(q.data_ptr(), q_fmt, s.data_ptr(), R, C, fmt,
                                                   qc.data_ptr(), sc.data_ptr(), _stream(stream))
    if st:
        raise Fp8gError(st, "fp8g_requantize_block128")
    return qc, sc


_FORMS = {"nt": FP8G_NT, "nn": FP8G_NN, "tn": FP8G_TN}


def gemm_block128(A, sfa, B, sfb, form: str = "nt", a_fmt: int = FP8G_E4M3, b_fmt: int = FP8G_E4M3,
                  out: str = "bf16", add_to=None, stream=None):
    """Product of codes with block-128 scales: "nt" A [M, K] B [N, K]^T (forward), "nn"
    A [M, K] B [K, N] (input gradient), A along rows and B in tiles; "tn" A [K, M]^T
    B [K, N] (weight gradient), both along columns.  Allocates C [M, N], or adds to
    add_to (fp32 [M, N]) and returns it."""
    empty, bf16, f32, _, _ = _t or _names()
    dev = A.get_device()
    _on(dev, A, sfa, B, sfb)
    assert _coded(A, a_fmt) and _coded(B, b_fmt) and sfa.dtype is f32 and sfb.dtype is f32
    a0, a1 = A.shape
    b0, b1 = B.shape
    if form == "tn":
        K, M, N = a0, a1, b1
        kb = -(-K // 128)
        assert b0 == K and sfa.shape == (kb, M) and sfb.shape == (kb, N)
    else:
        M, K = a0, a1
        N, k = (b0, b1) if form == "nt" else (b1, b0)
        assert k == K and sfa.shape == (-(-K // 128), M) and sfb.shape == (-(-b0 // 128), -(-b1 // 128))
    if add_to is not None:
        _on(dev, add_to)
        C, wide = add_to, True
        assert C.dtype is f32 and C.shape == (M, N)
    else:
        wide = out != "bf16"
        C = empty((M, N), dtype=f32 if wide else bf16, device=A.device)
    st = (_lib or load()).fp8_gemm_block128(
        _FORMS[form], A.data_ptr(), sfa.data_ptr(), a_fmt, B.data_ptr(), sfb.data_ptr(), b_fmt, C.data_ptr(),
        FP8G_OUT_F32 if wide else FP8G_OUT_BF16, 0 if add_to is None else 1, M, N, K, _stream(stream))
    if st:
        raise Fp8gError(st, "fp8_gemm_block128")
    return C


def gated_block128(x, sfx, W13, sf13, gate: int = FP8G_GATE_SILU, keep: bool = False,
                   x_fmt: int = FP8G_E4M3, w_fmt: int = FP8G_E4M3, stream=None):
    """h = act(x W13[:F]^T) (x W13[F:]^T): x [M, K] codes with scales along rows, W13
    [2F, K] in tiles -> ((codes, scales) of h along rows, with `keep` (codes, scales)
    of gate and up [M, 2F] along rows, the checkpoint of the backward pass, or None)."""
    empty, _, f32, _, u8 = _t or _names()
    dev = x.device
    _on(x.get_device(), x, sfx, W13, sf13)
    assert _coded(x, x_fmt) and _coded(W13, w_fmt) and sfx.dtype is f32 and sf13.dtype is f32
    M, K = x.shape
    F2, k = W13.shape
    F = F2 // 2
    kb = -(-K // 128)
    assert k == K and F2 == 2 * F and sfx.shape == (kb, M) and sf13.shape == (-(-F2 // 128), kb)
    h = empty((M, F), dtype=u8, device=dev)
    sh = empty((-(-F // 128), M), dtype=f32, device=dev)
    gu = empty((M, F2), dtype=u8, device=dev) if keep else None
    sgu = empty((-(-F2 // 128), M), dtype=f32, device=dev) if keep else None
    st = (_lib or load()).fp8_gated_block128(
        x.data_ptr(), sfx.data_ptr(), x_fmt, W13.data_ptr(), sf13.data_ptr(), w_fmt, gate, h.data_ptr(),
        sh.data_ptr(), _ptr(gu), _ptr(sgu), M, F, K, _stream(stream))
    if st:
        raise Fp8gError(st, "fp8_gated_block128")
    return (h, sh), (gu, sgu) if keep else None


def gated_block128_backward(dh, gu, sgu, gate: int = FP8G_GATE_SILU, fmt: int = FP8G_E4M3, stream=None):
    """dh [M, F] fp32 or bf16 and gated_block128's checkpoint -> (codes, scales) of the
    gradient of gate and up [M, 2F] along rows, the same along columns, and h [M, F]
    along columns (E4M3)."""
    empty, bf16, f32, _, u8 = _t or _names()
    dev = dh.device
    if not dh.is_contiguous():
        dh = _packed(dh, stream)
    _on(dh.get_device(), dh, gu, sgu)
    dt = dh.dtype
    M, F = dh.shape
    assert (dt is bf16 or dt is f32) and _coded(gu, FP8G_E4M3) and gu.shape == (M, 2 * F)
    assert sgu.dtype is f32 and sgu.shape == (-(-2 * F // 128), M)
    mb = -(-M // 128)
    row, col = empty((M, 2 * F), dtype=u8, device=dev), empty((M, 2 * F), dtype=u8, device=dev)
    h = empty((M, F), dtype=u8, device=dev)
    s_row, s_col = empty((-(-2 * F // 128), M), dtype=f32, device=dev), empty((mb, 2 * F), dtype=f32, device=dev)
    s_h = empty((mb, F), dtype=f32, device=dev)
    st = (_lib or load()).fp8g_gated_block128_backward(
        dh.data_ptr(), FP8G_IN_BF16 if dt is bf16 else FP8G_IN_F32, gu.data_ptr(), sgu.data_ptr(), gate, fmt,
        M, F, row.data_ptr(), s_row.data_ptr(), col.data_ptr(), s_col.data_ptr(), h.data_ptr(),
        s_h.data_ptr(), _stream(stream))
    if st:
        raise Fp8gError(st, "fp8g_gated_block128_backward")
    return (row, s_row), (col, s_col), (h, s_h)
