"""Thin ctypes binding over libnvfp4ffn.so (argument marshalling only).

Every function here takes torch tensors, checks dtypes/devices, allocates the
outputs with torch, and forwards raw pointers, sizes and the current CUDA
stream to the C entry point of the same name.  All arithmetic runs in the
library's kernels; there is no CPU or PyTorch fallback, and a missing library
raises.
"""
import ctypes
import os

import torch

from . import build as _build

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libnvfp4ffn.so")

NVFP4_ACT_SILU = 0
NVFP4_ACT_GELU_TANH = 1
NVFP4_SRC_F32 = 0
NVFP4_SRC_BF16 = 1
ROPE_PLAIN = 0
ROPE_LINEAR = 1
ROPE_BASE = 2
ROPE_RAMP = 3

STATUS_NAMES = {0: "NVFP4_OK", 1: "NVFP4_ERR_NULL", 2: "NVFP4_ERR_SHAPE", 3: "NVFP4_ERR_ALIGN",
                4: "NVFP4_ERR_RANGE", 5: "NVFP4_ERR_WORKSPACE", 6: "NVFP4_ERR_CUDA",
                7: "NVFP4_ERR_TIMEOUT", 8: "NVFP4_ERR_ALIAS"}

# Every symbol declared in include/nvfp4ffn.h.
EXPORTS = [
    "nvfp4_quantize_scratch_bytes", "nvfp4_quantize", "nvfp4_repacked_bytes", "nvfp4_repack",
    "nvfp4_repacked_gate_up_bytes", "nvfp4_repack_gate_up", "nvfp4_unpack",
    "nvfp4_gemv_workspace_bytes", "nvfp4_gemv", "ffn_swiglu_nvfp4_workspace_bytes",
    "ffn_swiglu_nvfp4_hidden_offset",
    "ffn_swiglu_nvfp4", "ffn_gate_up_nvfp4_workspace_bytes", "ffn_gate_up_nvfp4",
    "ffn_swiglu_nvfp4_noalloc", "nvfp4_noalloc_status",
    "ffn_swiglu_nvfp4_lora_workspace_bytes", "ffn_swiglu_nvfp4_lora",
    "nvfp4_lora_apply_scratch_bytes", "nvfp4_lora_apply",
    "w8a16_repacked_bytes", "w8a16_repacked_gate_up_bytes", "w8a16_repack",
    "w8a16_repack_gate_up", "w8a16_unpack", "w8a16_gemv_workspace_bytes", "w8a16_gemv",
    "ffn_swiglu_w8a16_workspace_bytes", "ffn_swiglu_w8a16",
    "add_rmsnorm_bf16", "add_rmsnorm_e4m3", "rope_table", "kv8_batch_status", "kv8_append",
    "kv8_read", "kv8_attention_workspace_bytes", "kv8_attention",
    "w4a4_repacked_bytes", "w4a4_repacked_gate_up_bytes", "w4a4_repack", "w4a4_repack_gate_up",
    "w4a4_unpack", "w4a4_rows_bytes", "w4a4_quantize", "w4a4_quantize_routed",
    "w4a4_dequantize",
    "w4a4_gemm_workspace_bytes", "w4a4_gemm", "w4a4_gate_up", "w4a4_experts_gemm",
    "w4a4_experts_gate_up", "ffn_swiglu_w4a4_workspace_bytes", "ffn_swiglu_w4a4", "experts_order",
    "experts_sum", "experts_swiglu_w4a4_workspace_bytes", "experts_swiglu_w4a4",
    "nvfp4_workspace_init", "nvfp4_workspace_status", "nvfp4_status_string",
]
# Every symbol declared in include/nvfp4ffn_testing.h (test hooks).
TESTING_EXPORTS = ["nvfp4_testing_inject_stall", "nvfp4_testing_plan_aligned",
                   "nvfp4_testing_plan_aligned_w8a16"]


class Nvfp4Error(RuntimeError):
    def __init__(self, fn, code, lib):
        name = STATUS_NAMES.get(code, str(code))
        msg = lib.nvfp4_status_string(code).decode()
        super().__init__(f"{fn} failed: {name} ({msg})")
        self.code = code


_lib = None


def load(build_if_missing: bool = False):
    """Load the library (optionally building it first).  Raises if absent."""
    global _lib
    if _lib is not None:
        return _lib
    if build_if_missing:
        _build.build()
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"{LIB_PATH} is missing: run nvfp4_weight_only_gb300.build.build() "
                           "(or __graft_entry__.build()) first")
    L = ctypes.CDLL(LIB_PATH)
    vp, sz, i32, f32 = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int, ctypes.c_float
    i64, f64 = ctypes.c_int64, ctypes.c_double
    sig = {
        "nvfp4_quantize_scratch_bytes": (sz, [i32, i32]),
        "nvfp4_quantize": (i32, [vp, i32, i32, i32, vp, vp, ctypes.POINTER(f32), vp, sz, vp]),
        "nvfp4_repacked_bytes": (sz, [i32, i32]),
        "nvfp4_repack": (i32, [vp, vp, i32, i32, vp, vp]),
        "nvfp4_repacked_gate_up_bytes": (sz, [i32, i32]),
        "nvfp4_repack_gate_up": (i32, [vp, vp, vp, vp, i32, i32, vp, vp]),
        "nvfp4_unpack": (i32, [vp, i32, i32, vp, vp, vp]),
        "nvfp4_gemv_workspace_bytes": (sz, [i32, i32, i32]),
        "nvfp4_gemv": (i32, [vp, i32, i32, vp, f32, i32, vp, vp, sz, vp]),
        "ffn_swiglu_nvfp4_workspace_bytes": (sz, [i32, i32, i32]),
        "ffn_swiglu_nvfp4_hidden_offset": (sz, []),
        "ffn_swiglu_nvfp4": (i32, [vp, i32, i32, i32, vp, f32, f32, vp, f32, i32, vp, vp, sz, vp]),
        "ffn_gate_up_nvfp4_workspace_bytes": (sz, [i32, i32, i32]),
        "ffn_gate_up_nvfp4": (i32, [vp, i32, i32, i32, vp, f32, f32, i32, vp, vp, sz, vp]),
        "ffn_swiglu_nvfp4_noalloc": (i32, [vp, i32, i32, i32, vp, f32, f32, vp, f32, i32, vp, vp]),
        "nvfp4_noalloc_status": (i32, [vp]),
        "ffn_swiglu_nvfp4_lora_workspace_bytes": (sz, [i32, i32, i32, i32]),
        "ffn_swiglu_nvfp4_lora": (i32, [vp, i32, i32, i32, vp, f32, f32, vp, f32, i32, i32,
                                        vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]),
        "nvfp4_lora_apply_scratch_bytes": (sz, [i32, i32]),
        "nvfp4_lora_apply": (i32, [vp, i32, i32, vp, vp, i32, i32, vp, vp, sz, vp]),
        "nvfp4_testing_inject_stall": (i32, [i32, ctypes.c_ulonglong]),
        "nvfp4_testing_plan_aligned": (i32, [i32, i32, i32, i32, i32]),
        "nvfp4_testing_plan_aligned_w8a16": (i32, [i32, i32, i32, i32, i32]),
        "w8a16_repacked_bytes": (sz, [i32, i32]),
        "w8a16_repacked_gate_up_bytes": (sz, [i32, i32]),
        "w8a16_repack": (i32, [vp, vp, i32, i32, vp, vp]),
        "w8a16_repack_gate_up": (i32, [vp, vp, vp, vp, i32, i32, vp, vp]),
        "w8a16_unpack": (i32, [vp, i32, i32, vp, vp, vp]),
        "w8a16_gemv_workspace_bytes": (sz, [i32, i32, i32]),
        "w8a16_gemv": (i32, [vp, i32, i32, vp, i32, vp, vp, sz, vp]),
        "ffn_swiglu_w8a16_workspace_bytes": (sz, [i32, i32, i32]),
        "ffn_swiglu_w8a16": (i32, [vp, i32, i32, i32, vp, vp, i32, vp, vp, sz, vp]),
        "add_rmsnorm_bf16": (i32, [vp, vp, vp, i32, i32, f32, f32, vp, vp, vp]),
        "add_rmsnorm_e4m3": (i32, [vp, vp, vp, i32, i32, f32, f32, vp, vp, vp, vp]),
        "rope_table": (i32, [i32, i32, f64, i32, f64, f64, f64, f64, f64, vp, vp]),
        "kv8_batch_status": (i32, [vp, vp]),
        "kv8_append": (i32, [vp, vp, i32, vp, i64, vp, i64, vp, i64, i32, vp, vp, i32, i32, i32,
                             vp]),
        "kv8_read": (i32, [vp, vp, i32, vp, vp, vp]),
        "kv8_attention_workspace_bytes": (sz, [vp, vp, i32, i32]),
        "kv8_attention": (i32, [vp, i64, i32, i32, vp, vp, f32, i32, i32, vp, vp, vp, sz, vp]),
        "w4a4_repacked_bytes": (sz, [i32, i32, i32]),
        "w4a4_repacked_gate_up_bytes": (sz, [i32, i32, i32]),
        "w4a4_repack": (i32, [vp, vp, i32, i32, i32, vp, vp]),
        "w4a4_repack_gate_up": (i32, [vp, vp, vp, vp, i32, i32, i32, vp, vp]),
        "w4a4_unpack": (i32, [vp, i32, i32, i32, vp, vp, vp]),
        "w4a4_rows_bytes": (sz, [i32, i32, i32]),
        "w4a4_quantize": (i32, [vp, i32, i32, vp, vp, vp]),
        "w4a4_quantize_routed": (i32, [vp, i32, i32, vp, vp, i32, vp, vp, vp]),
        "w4a4_dequantize": (i32, [vp, i32, i32, vp, vp, vp]),
        "w4a4_gemm_workspace_bytes": (sz, [i32, i32, i32, i32]),
        "w4a4_gemm": (i32, [vp, i32, i32, vp, f32, i32, vp, vp, sz, vp]),
        "w4a4_gate_up": (i32, [vp, i32, i32, vp, f32, f32, i32, i32, vp, vp, sz, vp]),
        "w4a4_experts_gemm": (i32, [vp, i32, i32, vp, vp, vp, i32, vp, vp, sz, vp]),
        "w4a4_experts_gate_up": (i32, [vp, i32, i32, vp, vp, vp, vp, i32, i32, vp, vp, sz, vp]),
        "ffn_swiglu_w4a4_workspace_bytes": (sz, [i32, i32, i32]),
        "ffn_swiglu_w4a4": (i32, [vp, i32, i32, i32, vp, f32, f32, vp, f32, i32, vp, vp, sz, vp]),
        "experts_order": (i32, [vp, i32, i32, i32, vp, vp, vp, vp]),
        "experts_sum": (i32, [vp, i32, vp, vp, i32, i32, i32, vp, vp]),
        "experts_swiglu_w4a4_workspace_bytes": (sz, [i32, i32, i32, i32, i32]),
        "experts_swiglu_w4a4": (i32, [vp, i32, i32, i32, vp, vp, i32, i32, vp, vp, vp, vp, vp, i32,
                                      vp, vp, sz, vp]),
        "nvfp4_workspace_init": (i32, [vp, sz, vp]),
        "nvfp4_workspace_status": (i32, [vp, vp]),
        "nvfp4_status_string": (ctypes.c_char_p, [i32]),
    }
    for name, (res, args) in sig.items():
        f = getattr(L, name)
        f.restype = res
        f.argtypes = args
    _lib = L
    return L


def _check(fn, code):
    if code != 0:
        raise Nvfp4Error(fn, code, load())


def _ptr(t):
    return ctypes.c_void_p(t.data_ptr()) if t is not None else ctypes.c_void_p(0)


def _stream(device=None):
    return ctypes.c_void_p(torch.cuda.current_stream(device).cuda_stream)


def _cuda(t, name, dtype=None):
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


# ------------------------------------------------------------------ quantise / repack

def nvfp4_quantize(w: torch.Tensor):
    """W fp32/bf16 [N, K] (CUDA) -> (codes u8 [N, K/2], scales u8 [N, K/16], scale2 float)."""
    _cuda(w, "w")
    if w.dtype not in (torch.float32, torch.bfloat16):
        raise ValueError("w must be float32 or bfloat16")
    N, K = w.shape
    L = load()
    codes = torch.empty((N, K // 2), dtype=torch.uint8, device=w.device)
    scales = torch.empty((N, K // 16), dtype=torch.uint8, device=w.device)
    nscr = L.nvfp4_quantize_scratch_bytes(N, K)
    scratch = torch.empty(nscr, dtype=torch.uint8, device=w.device)
    s2 = ctypes.c_float(0.0)
    dt = NVFP4_SRC_BF16 if w.dtype == torch.bfloat16 else NVFP4_SRC_F32
    _check("nvfp4_quantize", L.nvfp4_quantize(_ptr(w), dt, N, K, _ptr(codes), _ptr(scales),
                                              ctypes.byref(s2), _ptr(scratch), nscr,
                                              _stream(w.device)))
    return codes, scales, s2.value


def nvfp4_repack(codes: torch.Tensor, scales: torch.Tensor, N: int, K: int) -> torch.Tensor:
    _cuda(codes, "codes", torch.uint8)
    _cuda(scales, "scales", torch.uint8)
    L = load()
    out = torch.empty(L.nvfp4_repacked_bytes(N, K), dtype=torch.uint8, device=codes.device)
    _check("nvfp4_repack", L.nvfp4_repack(_ptr(codes), _ptr(scales), N, K, _ptr(out),
                                          _stream(codes.device)))
    return out


def nvfp4_repack_gate_up(gate_codes, gate_scales, up_codes, up_scales, I: int, H: int):
    for n, t in (("gate_codes", gate_codes), ("gate_scales", gate_scales),
                 ("up_codes", up_codes), ("up_scales", up_scales)):
        _cuda(t, n, torch.uint8)
    L = load()
    out = torch.empty(L.nvfp4_repacked_gate_up_bytes(I, H), dtype=torch.uint8,
                      device=gate_codes.device)
    _check("nvfp4_repack_gate_up",
           L.nvfp4_repack_gate_up(_ptr(gate_codes), _ptr(gate_scales), _ptr(up_codes),
                                  _ptr(up_scales), I, H, _ptr(out), _stream(gate_codes.device)))
    return out


def nvfp4_unpack(packed: torch.Tensor, N: int, K: int):
    _cuda(packed, "packed", torch.uint8)
    L = load()
    codes = torch.empty((N, K // 2), dtype=torch.uint8, device=packed.device)
    scales = torch.empty((N, K // 16), dtype=torch.uint8, device=packed.device)
    _check("nvfp4_unpack", L.nvfp4_unpack(_ptr(packed), N, K, _ptr(codes), _ptr(scales),
                                          _stream(packed.device)))
    return codes, scales


# ------------------------------------------------------------------ GEMV / FFN

def nvfp4_gemv_workspace_bytes(M: int, N: int, K: int) -> int:
    return load().nvfp4_gemv_workspace_bytes(M, N, K)


def ffn_swiglu_nvfp4_workspace_bytes(M: int, H: int, I: int) -> int:
    return load().ffn_swiglu_nvfp4_workspace_bytes(M, H, I)


def workspace(nbytes: int, device) -> torch.Tensor:
    """A zero-filled workspace buffer of at least `nbytes` (torch allocation)."""
    return torch.zeros(max(int(nbytes), 256), dtype=torch.uint8, device=device)


def nvfp4_gemv(x: torch.Tensor, packed_w: torch.Tensor, scale2: float, N: int,
               ws: torch.Tensor = None, out: torch.Tensor = None) -> torch.Tensor:
    """y bf16 [M, N] = one NVFP4 projection of x bf16 [M, K]."""
    _cuda(x, "x", torch.bfloat16)
    _cuda(packed_w, "packed_w", torch.uint8)
    M, K = x.shape
    L = load()
    if ws is None:
        ws = workspace(L.nvfp4_gemv_workspace_bytes(M, N, K), x.device)
    if out is None:
        out = torch.empty((M, N), dtype=torch.bfloat16, device=x.device)
    _cuda(out, "out", torch.bfloat16)
    _check("nvfp4_gemv", L.nvfp4_gemv(_ptr(x), M, K, _ptr(packed_w), float(scale2), N, _ptr(out),
                                      _ptr(ws), ws.numel(), _stream(x.device)))
    return out


def ffn_swiglu_nvfp4(x: torch.Tensor, gate_up_packed: torch.Tensor, gate_scale2: float,
                     up_scale2: float, down_packed: torch.Tensor, down_scale2: float, I: int,
                     act: int = NVFP4_ACT_SILU, ws: torch.Tensor = None,
                     out: torch.Tensor = None) -> torch.Tensor:
    """out bf16 [M, H] = down(act(gate(x)) * up(x)) for x bf16 [M, H]."""
    _cuda(x, "x", torch.bfloat16)
    _cuda(gate_up_packed, "gate_up_packed", torch.uint8)
    _cuda(down_packed, "down_packed", torch.uint8)
    M, H = x.shape
    L = load()
    if ws is None:
        ws = workspace(L.ffn_swiglu_nvfp4_workspace_bytes(M, H, I), x.device)
    if out is None:
        out = torch.empty((M, H), dtype=torch.bfloat16, device=x.device)
    _cuda(out, "out", torch.bfloat16)
    _check("ffn_swiglu_nvfp4",
           L.ffn_swiglu_nvfp4(_ptr(x), M, H, I, _ptr(gate_up_packed), float(gate_scale2),
                              float(up_scale2), _ptr(down_packed), float(down_scale2), int(act),
                              _ptr(out), _ptr(ws), ws.numel(), _stream(x.device)))
    return out


def ffn_swiglu_nvfp4_noalloc(x: torch.Tensor, gate_up_packed: torch.Tensor, gate_scale2: float,
                             up_scale2: float, down_packed: torch.Tensor, down_scale2: float,
                             I: int, act: int = NVFP4_ACT_SILU,
                             out: torch.Tensor = None) -> torch.Tensor:
    """ffn_swiglu_nvfp4 on the library's fixed device workspace (for callers that
    cannot allocate one); only the output is allocated here, and only when `out`
    is not given."""
    _cuda(x, "x", torch.bfloat16)
    _cuda(gate_up_packed, "gate_up_packed", torch.uint8)
    _cuda(down_packed, "down_packed", torch.uint8)
    M, H = x.shape
    L = load()
    if out is None:
        out = torch.empty((M, H), dtype=torch.bfloat16, device=x.device)
    _cuda(out, "out", torch.bfloat16)
    _check("ffn_swiglu_nvfp4_noalloc",
           L.ffn_swiglu_nvfp4_noalloc(_ptr(x), M, H, I, _ptr(gate_up_packed), float(gate_scale2),
                                      float(up_scale2), _ptr(down_packed), float(down_scale2),
                                      int(act), _ptr(out), _stream(x.device)))
    return out


def ffn_swiglu_nvfp4_lora(x: torch.Tensor, gate_up_packed: torch.Tensor, gate_scale2: float,
                          up_scale2: float, down_packed: torch.Tensor, down_scale2: float, I: int,
                          act: int = NVFP4_ACT_SILU, gate=None, up=None, down=None,
                          ws: torch.Tensor = None, out: torch.Tensor = None) -> torch.Tensor:
    """The FFN with the LoRA overlay; gate/up/down = (A, B) bf16 pairs or None."""
    _cuda(x, "x", torch.bfloat16)
    M, H = x.shape
    pairs = [gate, up, down]
    rank = next((p[0].shape[0] for p in pairs if p is not None), 1)
    for p in pairs:
        if p is not None:
            _cuda(p[0], "lora A", torch.bfloat16)
            _cuda(p[1], "lora B", torch.bfloat16)
    L = load()
    if ws is None:
        ws = workspace(L.ffn_swiglu_nvfp4_lora_workspace_bytes(M, H, I, rank), x.device)
    if out is None:
        out = torch.empty((M, H), dtype=torch.bfloat16, device=x.device)
    _cuda(out, "out", torch.bfloat16)
    ptrs = []
    for p in pairs:
        ptrs += [_ptr(p[0]), _ptr(p[1])] if p is not None else [_ptr(None), _ptr(None)]
    _check("ffn_swiglu_nvfp4_lora",
           L.ffn_swiglu_nvfp4_lora(_ptr(x), M, H, I, _ptr(gate_up_packed), float(gate_scale2),
                                   float(up_scale2), _ptr(down_packed), float(down_scale2),
                                   int(act), rank, *ptrs, _ptr(out), _ptr(ws), ws.numel(),
                                   _stream(x.device)))
    return out


def nvfp4_lora_apply(v: torch.Tensor, a: torch.Tensor, b: torch.Tensor,
                     base: torch.Tensor) -> torch.Tensor:
    """base [M, N] = bf16(base + bf16(b bf16(a v))) in place (returns base)."""
    for n, t in (("v", v), ("a", a), ("b", b), ("base", base)):
        _cuda(t, n, torch.bfloat16)
    M, K = v.shape
    rank = a.shape[0]
    N = b.shape[0]
    L = load()
    scratch = workspace(L.nvfp4_lora_apply_scratch_bytes(M, rank), v.device)
    _check("nvfp4_lora_apply",
           L.nvfp4_lora_apply(_ptr(v), M, K, _ptr(a), _ptr(b), rank, N, _ptr(base),
                              _ptr(scratch), scratch.numel(), _stream(v.device)))
    return base


def ffn_gate_up_nvfp4_workspace_bytes(M: int, H: int, I: int) -> int:
    return load().ffn_gate_up_nvfp4_workspace_bytes(M, H, I)


def ffn_gate_up_nvfp4(x: torch.Tensor, gate_up_packed: torch.Tensor, gate_scale2: float,
                      up_scale2: float, I: int, act: int = NVFP4_ACT_SILU,
                      ws: torch.Tensor = None, h: torch.Tensor = None) -> torch.Tensor:
    """h bf16 [M, I] = act(gate(x)) * up(x) for x bf16 [M, H]."""
    _cuda(x, "x", torch.bfloat16)
    _cuda(gate_up_packed, "gate_up_packed", torch.uint8)
    M, H = x.shape
    L = load()
    if ws is None:
        ws = workspace(L.ffn_gate_up_nvfp4_workspace_bytes(M, H, I), x.device)
    if h is None:
        h = torch.empty((M, I), dtype=torch.bfloat16, device=x.device)
    _cuda(h, "h", torch.bfloat16)
    _check("ffn_gate_up_nvfp4",
           L.ffn_gate_up_nvfp4(_ptr(x), M, H, I, _ptr(gate_up_packed), float(gate_scale2),
                               float(up_scale2), int(act), _ptr(h), _ptr(ws), ws.numel(),
                               _stream(x.device)))
    return h


def ffn_hidden_view(ws: torch.Tensor, M: int, I: int) -> torch.Tensor:
    """The bf16 activation h [M, I] that ffn_swiglu_nvfp4 leaves in its workspace."""
    off = load().ffn_swiglu_nvfp4_hidden_offset()
    return ws[off:off + M * I * 2].view(torch.bfloat16).view(M, I)


def nvfp4_workspace_init(ws: torch.Tensor) -> None:
    _check("nvfp4_workspace_init",
           load().nvfp4_workspace_init(_ptr(ws), ws.numel(), _stream(ws.device)))


def nvfp4_workspace_status(ws: torch.Tensor) -> int:
    """Synchronise, read and clear the device status word (0 = OK, 7 = timeout)."""
    return load().nvfp4_workspace_status(_ptr(ws), _stream(ws.device))


def nvfp4_noalloc_status(device=None) -> int:
    """Status of the fixed-workspace FFN calls (0 = OK, 7 = timeout, after which
    the library has zero-filled its array again)."""
    return load().nvfp4_noalloc_status(_stream(device))


# ------------------------------------------------------------------ block-scaled FP8 (w8a16)

def _fp8_projection(codes, grid, name):
    _cuda(codes, f"{name} codes", torch.uint8)
    _cuda(grid, f"{name} grid", torch.float32)
    N, K = codes.shape
    if tuple(grid.shape) != ((N + 127) // 128, (K + 127) // 128):
        raise ValueError(f"{name} grid must be [ceil(N/128), ceil(K/128)], got {tuple(grid.shape)}")
    return N, K


def w8a16_repack(codes: torch.Tensor, grid: torch.Tensor) -> torch.Tensor:
    """E4M3 bytes [N, K] + fp32 block grid -> the kernel layout (uint8 blob)."""
    N, K = _fp8_projection(codes, grid, "w8a16_repack")
    L = load()
    out = torch.empty(L.w8a16_repacked_bytes(N, K), dtype=torch.uint8, device=codes.device)
    _check("w8a16_repack", L.w8a16_repack(_ptr(codes), _ptr(grid), N, K, _ptr(out),
                                          _stream(codes.device)))
    return out


def w8a16_repack_gate_up(gate_codes, gate_grid, up_codes, up_grid) -> torch.Tensor:
    I, H = _fp8_projection(gate_codes, gate_grid, "gate")
    if _fp8_projection(up_codes, up_grid, "up") != (I, H):
        raise ValueError("gate and up must have the same shape")
    L = load()
    out = torch.empty(L.w8a16_repacked_gate_up_bytes(I, H), dtype=torch.uint8,
                      device=gate_codes.device)
    _check("w8a16_repack_gate_up",
           L.w8a16_repack_gate_up(_ptr(gate_codes), _ptr(gate_grid), _ptr(up_codes),
                                  _ptr(up_grid), I, H, _ptr(out), _stream(gate_codes.device)))
    return out


def w8a16_unpack(packed: torch.Tensor, N: int, K: int):
    _cuda(packed, "packed", torch.uint8)
    L = load()
    codes = torch.empty((N, K), dtype=torch.uint8, device=packed.device)
    grid = torch.empty(((N + 127) // 128, (K + 127) // 128), dtype=torch.float32,
                       device=packed.device)
    _check("w8a16_unpack", L.w8a16_unpack(_ptr(packed), N, K, _ptr(codes), _ptr(grid),
                                          _stream(packed.device)))
    return codes, grid


def w8a16_gemv(x: torch.Tensor, packed_w: torch.Tensor, N: int, ws: torch.Tensor = None,
               out: torch.Tensor = None) -> torch.Tensor:
    """y bf16 [M, N] = one block-scaled FP8 projection of x bf16 [M, K]."""
    _cuda(x, "x", torch.bfloat16)
    _cuda(packed_w, "packed_w", torch.uint8)
    M, K = x.shape
    L = load()
    if ws is None:
        ws = workspace(L.w8a16_gemv_workspace_bytes(M, N, K), x.device)
    if out is None:
        out = torch.empty((M, N), dtype=torch.bfloat16, device=x.device)
    _cuda(out, "out", torch.bfloat16)
    _check("w8a16_gemv", L.w8a16_gemv(_ptr(x), M, K, _ptr(packed_w), N, _ptr(out), _ptr(ws),
                                      ws.numel(), _stream(x.device)))
    return out


def ffn_swiglu_w8a16(x: torch.Tensor, gate_up_packed: torch.Tensor, down_packed: torch.Tensor,
                     I: int, act: int = NVFP4_ACT_SILU, ws: torch.Tensor = None,
                     out: torch.Tensor = None) -> torch.Tensor:
    """out bf16 [M, H] = down(act(gate(x)) * up(x)) on block-scaled FP8 weights."""
    _cuda(x, "x", torch.bfloat16)
    _cuda(gate_up_packed, "gate_up_packed", torch.uint8)
    _cuda(down_packed, "down_packed", torch.uint8)
    M, H = x.shape
    L = load()
    if ws is None:
        ws = workspace(L.ffn_swiglu_w8a16_workspace_bytes(M, H, I), x.device)
    if out is None:
        out = torch.empty((M, H), dtype=torch.bfloat16, device=x.device)
    _cuda(out, "out", torch.bfloat16)
    _check("ffn_swiglu_w8a16",
           L.ffn_swiglu_w8a16(_ptr(x), M, H, I, _ptr(gate_up_packed), _ptr(down_packed), int(act),
                              _ptr(out), _ptr(ws), ws.numel(), _stream(x.device)))
    return out


# ------------------------------------------------------------------ attention side of a layer
#
# A decode step makes these calls for microseconds of GPU work, so their checks
# read each tensor attribute once and pass plain numbers.

_BF16, _U8, _F32, _I32 = torch.bfloat16, torch.uint8, torch.float32, torch.int32
_current_device = torch._C._cuda_getDevice
_current_raw_stream = torch._C._cuda_getCurrentRawStream


def _raw_stream(device):
    """The current stream's handle (without a Stream object) on `device`, which has to be the
    current one: the library launches there."""
    if device != _current_device():
        raise ValueError(f"tensors on device {device} need it as the current device, but the "
                         f"current device is {_current_device()}")
    return _current_raw_stream(device)


def _plain(t, name, dtype, shape, device):
    """Checks a contiguous tensor of `shape` (a tuple) on CUDA device `device`; its address."""
    if t.dtype is not dtype or t.shape != shape or not t.is_contiguous() or \
            t.get_device() != device or device < 0:
        raise ValueError(f"{name} must be a contiguous {dtype} CUDA tensor {list(shape)} on device "
                         f"{device}, got {t.dtype} {list(t.shape)} on {t.device}")
    return t.data_ptr()


def _rows(t, name, tokens, heads, dim, device):
    """Checks a bf16 [tokens, heads, head_dim] view with contiguous heads: (address, token
    stride)."""
    if t.dtype is not _BF16 or t.shape != (tokens, heads, dim) or t.get_device() != device:
        raise ValueError(f"{name} must be a bfloat16 CUDA tensor {[tokens, heads, dim]} on device "
                         f"{device}, got {t.dtype} {list(t.shape)} on {t.device}")
    row, head, one = t.stride()
    if one != 1 or (head != dim and heads > 1):
        raise ValueError(f"{name} must have contiguous heads")
    return t.data_ptr(), (row if tokens > 1 else heads * dim)


def _norm_inputs(x, weight, residual, sum_out):
    """(M, H, device, addresses of residual, weight, sum_out)."""
    if x.dtype is not _BF16 or x.dim() != 2 or not x.is_cuda or not x.is_contiguous():
        raise ValueError(f"x must be a contiguous bfloat16 CUDA matrix, got {x.dtype} "
                         f"{list(x.shape)} on {x.device}")
    shape, device = x.shape, x.get_device()
    return (shape, device,
            None if residual is None else _plain(residual, "residual", _BF16, shape, device),
            _plain(weight, "weight", _BF16, shape[1:], device),
            None if sum_out is None else _plain(sum_out, "sum_out", _BF16, shape, device))


def add_rmsnorm_bf16(x: torch.Tensor, weight: torch.Tensor, eps: float,
                     residual: torch.Tensor = None, sum_out: torch.Tensor = None,
                     weight_bias: float = 0.0, out: torch.Tensor = None) -> torch.Tensor:
    """bf16 norm of x + residual; the sum goes to sum_out (which may be residual) when given."""
    shape, device, res, w, total = _norm_inputs(x, weight, residual, sum_out)
    if out is None:
        out = torch.empty_like(x)
    code = (_lib or load()).add_rmsnorm_bf16(
        x.data_ptr(), res, w, shape[0], shape[1], eps, weight_bias, total,
        _plain(out, "out", _BF16, shape, device), _raw_stream(device))
    if code:
        _check("add_rmsnorm_bf16", code)
    return out


def add_rmsnorm_e4m3(x: torch.Tensor, weight: torch.Tensor, eps: float,
                     residual: torch.Tensor = None, sum_out: torch.Tensor = None,
                     weight_bias: float = 0.0, codes: torch.Tensor = None,
                     scales: torch.Tensor = None):
    """(codes u8 [M, H], scales fp32 [M, ceil(H/128)]) of the norm of x + residual."""
    shape, device, res, w, total = _norm_inputs(x, weight, residual, sum_out)
    groups = (shape[0], (shape[1] + 127) // 128)
    if codes is None:
        codes = torch.empty(shape, dtype=_U8, device=x.device)
    if scales is None:
        scales = torch.empty(groups, dtype=_F32, device=x.device)
    code = (_lib or load()).add_rmsnorm_e4m3(
        x.data_ptr(), res, w, shape[0], shape[1], eps, weight_bias, total,
        _plain(codes, "codes", _U8, shape, device), _plain(scales, "scales", _F32, groups, device),
        _raw_stream(device))
    if code:
        _check("add_rmsnorm_e4m3", code)
    return codes, scales


def rope_table(positions: int, rot_dim: int, base: float, device, scaling: int = ROPE_PLAIN,
               factor: float = 1.0, context: float = 1.0, slow: float = 1.0, fast: float = 32.0,
               magnitude: float = 1.0) -> torch.Tensor:
    """fp32 [positions, rot_dim/2, 2] rotations (cos, sin) for kv8_append."""
    table = torch.empty((positions, rot_dim // 2, 2), dtype=_F32, device=device)
    if not table.is_cuda:
        raise ValueError("device must be a CUDA device")
    _check("rope_table", load().rope_table(positions, rot_dim, base, scaling, factor, context, slow,
                                           fast, magnitude, table.data_ptr(),
                                           _raw_stream(table.get_device())))
    return table


class _CacheStruct(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("k_codes", "v_codes", "k_scales", "v_scales")] + [
        (n, ctypes.c_int) for n in ("pages", "kv_heads", "page", "head_dim")]


class _BatchStruct(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("q_start", "kv_len", "page_table", "status")] + [
        (n, ctypes.c_int) for n in ("batch", "table_width")]


class Kv8Cache:
    """The paged E4M3 cache (kv8_cache): codes u8 [pages, kv_heads, page, head_dim] and fp32 scales
    [pages, kv_heads] for k and v.  Holds the tensors and their description."""

    def __init__(self, k_codes, v_codes, k_scales, v_scales):
        if k_codes.dim() != 4:
            raise ValueError("k_codes must be [pages, kv_heads, page, head_dim]")
        shape, self.device = k_codes.shape, k_codes.get_device()
        self.struct = _CacheStruct(
            _plain(k_codes, "k_codes", _U8, shape, self.device),
            _plain(v_codes, "v_codes", _U8, shape, self.device),
            _plain(k_scales, "k_scales", _F32, shape[:2], self.device),
            _plain(v_scales, "v_scales", _F32, shape[:2], self.device), *shape)
        self.k_codes, self.v_codes, self.k_scales, self.v_scales = (k_codes, v_codes, k_scales,
                                                                    v_scales)
        self.pages, self.kv_heads, self.page, self.head_dim = shape
        self.ref = ctypes.addressof(self.struct)

    @classmethod
    def empty(cls, pages, kv_heads, page, head_dim, device):
        """A cache whose pages hold nothing yet."""
        codes = [torch.empty((pages, kv_heads, page, head_dim), dtype=_U8, device=device)
                 for _ in "kv"]
        scales = [torch.ones((pages, kv_heads), dtype=_F32, device=device) for _ in "kv"]
        return cls(*codes, *scales)


class Kv8Batch:
    """The sequences of one step (kv8_batch): q_start int32 [batch + 1], kv_len int32 [batch] and
    page_table int32 [batch, table_width], all read on the device when a call runs, so a program
    may advance them in place.  Owns a status word, which kv8_batch_status reads."""

    def __init__(self, q_start, kv_len, page_table):
        if page_table.dim() != 2:
            raise ValueError("page_table must be [batch, table_width]")
        batch, width = page_table.shape
        self.device = kv_len.get_device()
        addresses = (_plain(q_start, "q_start", _I32, (batch + 1,), self.device),
                     _plain(kv_len, "kv_len", _I32, (batch,), self.device),
                     _plain(page_table, "page_table", _I32, (batch, width), self.device))
        self.q_start, self.kv_len, self.page_table = q_start, kv_len, page_table
        self.status = torch.zeros(1, dtype=_I32, device=kv_len.device)
        self.struct = _BatchStruct(*addresses, self.status.data_ptr(), batch, width)
        self.ref = ctypes.addressof(self.struct)


def _same_device(cache, batch):
    if cache.device != batch.device:
        raise ValueError("cache and batch must be on the same device")
    return cache.device


def kv8_batch_status(batch: Kv8Batch) -> int:
    """Synchronise, read and clear the batch's status word (0 = OK, 4 = an index out of range)."""
    return load().kv8_batch_status(batch.ref, _raw_stream(batch.device))


def kv8_append(cache: Kv8Cache, batch: Kv8Batch, k: torch.Tensor, v: torch.Tensor,
               q: torch.Tensor = None, q_out: torch.Tensor = None, rope: torch.Tensor = None,
               interleaved: bool = False):
    """Write k, v [tokens, kv_heads, head_dim] into the cache, k rotated by the rope table; with
    q [tokens, heads, head_dim] given, return it rotated (contiguous, in q_out when given)."""
    device, dim = _same_device(cache, batch), cache.head_dim
    T = k.shape[0]
    k_at, k_stride = _rows(k, "k", T, cache.kv_heads, dim, device)
    v_at, v_stride = _rows(v, "v", T, cache.kv_heads, dim, device)
    q_at = out_at = rope_at = None
    heads = q_stride = positions = rot = 0
    if q is not None:
        if q.dim() != 3:
            raise ValueError("q must be [tokens, heads, head_dim]")
        shape = q.shape
        heads = shape[1]
        q_at, q_stride = _rows(q, "q", T, heads, dim, device)
        if q_out is None:
            q_out = torch.empty(shape, dtype=_BF16, device=q.device)
        out_at = _plain(q_out, "q_out", _BF16, shape, device)
    if rope is not None:
        shape = rope.shape
        if len(shape) != 3 or shape[2] != 2:
            raise ValueError("rope must be [positions, rot_dim/2, 2]")
        rope_at = _plain(rope, "rope", _F32, shape, device)
        positions, rot = shape[0], 2 * shape[1]
    code = (_lib or load()).kv8_append(
        cache.ref, batch.ref, T, k_at, k_stride, v_at, v_stride, q_at, q_stride, heads, out_at,
        rope_at, positions, rot, 1 if interleaved else 0, _raw_stream(device))
    if code:
        _check("kv8_append", code)
    return q_out


def kv8_read(cache: Kv8Cache, batch: Kv8Batch, k_out: torch.Tensor, v_out: torch.Tensor):
    """Read the batch's tokens back: k_out, v_out bf16 [tokens, kv_heads, head_dim]."""
    device = _same_device(cache, batch)
    T = k_out.shape[0]
    shape = (T, cache.kv_heads, cache.head_dim)
    code = (_lib or load()).kv8_read(cache.ref, batch.ref, T,
                                     _plain(k_out, "k_out", _BF16, shape, device),
                                     _plain(v_out, "v_out", _BF16, shape, device),
                                     _raw_stream(device))
    if code:
        _check("kv8_read", code)
    return k_out, v_out


def kv8_attention_workspace_bytes(cache: Kv8Cache, batch: Kv8Batch, tokens: int, heads: int) -> int:
    return load().kv8_attention_workspace_bytes(cache.ref, batch.ref, tokens, heads)


def kv8_attention_workspace_size(kv_heads: int, head_dim: int, sequences: int, tokens: int,
                                 heads: int) -> int:
    """The same from sizes, before there is a cache."""
    cache = _CacheStruct(pages=1, kv_heads=kv_heads, page=16, head_dim=head_dim)
    batch = _BatchStruct(batch=sequences, table_width=1)
    return load().kv8_attention_workspace_bytes(ctypes.addressof(cache), ctypes.addressof(batch),
                                                tokens, heads)


def kv8_attention(q: torch.Tensor, cache: Kv8Cache, batch: Kv8Batch, softmax_scale: float,
                  window: int = 0, sinks: int = 0, ws: torch.Tensor = None,
                  out: torch.Tensor = None, lse: torch.Tensor = None) -> torch.Tensor:
    """out bf16 [tokens, heads, head_dim]: attention of q over the cache, which already holds the
    batch's tokens; log-sum-exps go to lse fp32 [tokens, heads] when given."""
    if q.dim() != 3:
        raise ValueError("q must be [tokens, heads, head_dim]")
    device, shape = _same_device(cache, batch), q.shape
    T, heads, _ = shape
    q_at, q_stride = _rows(q, "q", T, heads, cache.head_dim, device)
    if ws is None:
        ws = workspace(kv8_attention_workspace_bytes(cache, batch, T, heads), q.device)
    if out is None:
        out = torch.empty(shape, dtype=_BF16, device=q.device)
    code = (_lib or load()).kv8_attention(
        q_at, q_stride, T, heads, cache.ref, batch.ref, softmax_scale, window, sinks,
        _plain(out, "out", _BF16, shape, device),
        None if lse is None else _plain(lse, "lse", _F32, (T, heads), device),
        _plain(ws, "ws", _U8, ws.shape, device), ws.numel(), _raw_stream(device))
    if code:
        _check("kv8_attention", code)
    return out


# ------------------------------------------------------------------ 4-bit activations (w4a4)

class _GroupsStruct(ctypes.Structure):
    _fields_ = [("start", ctypes.c_void_p), ("experts", ctypes.c_int)]


def _matrix(x, name):
    """(rows, width, device) of a contiguous bf16 CUDA matrix."""
    if x.dtype is not _BF16 or x.dim() != 2 or not x.is_cuda or not x.is_contiguous():
        raise ValueError(f"{name} must be a contiguous bfloat16 CUDA matrix, got {x.dtype} "
                         f"{list(x.shape)} on {x.device}")
    return (*x.shape, x.get_device())


def _stacked(codes, scales, name):
    """Checks codes u8 [N, K/2] or [experts, N, K/2] and their scales: (experts, N, K, device,
    addresses)."""
    if codes.dim() not in (2, 3):
        raise ValueError(f"{name} codes must be [N, K/2] or [experts, N, K/2]")
    shape, device = codes.shape, codes.get_device()
    at = _plain(codes, f"{name} codes", _U8, shape, device)
    scales_at = _plain(scales, f"{name} scales", _U8, (*shape[:-1], shape[-1] // 8), device)
    return (shape[0] if len(shape) == 3 else 1), shape[-2], 2 * shape[-1], device, at, scales_at


def w4a4_repack(codes: torch.Tensor, scales: torch.Tensor) -> torch.Tensor:
    """NVFP4 codes [N, K/2] and scales [N, K/16], or those of experts stacked in front, -> the
    layout of the products on 4-bit activations."""
    experts, N, K, device, at, scales_at = _stacked(codes, scales, "w4a4_repack")
    L = load()
    out = torch.empty(L.w4a4_repacked_bytes(experts, N, K), dtype=_U8, device=codes.device)
    _check("w4a4_repack", L.w4a4_repack(at, scales_at, experts, N, K, out.data_ptr(),
                                        _raw_stream(device)))
    return out


def w4a4_repack_gate_up(gate_codes, gate_scales, up_codes, up_scales) -> torch.Tensor:
    """Gate and up projections [I, H] (experts stacked in front) into one blob."""
    experts, I, H, device, gate, gate_s = _stacked(gate_codes, gate_scales, "gate")
    if up_codes.shape != gate_codes.shape or up_codes.get_device() != device:
        raise ValueError("gate and up must have the same shape and device")
    *_, up, up_s = _stacked(up_codes, up_scales, "up")
    L = load()
    out = torch.empty(L.w4a4_repacked_gate_up_bytes(experts, I, H), dtype=_U8,
                      device=gate_codes.device)
    _check("w4a4_repack_gate_up",
           L.w4a4_repack_gate_up(gate, gate_s, up, up_s, experts, I, H, out.data_ptr(),
                                 _raw_stream(device)))
    return out


def w4a4_unpack(packed: torch.Tensor, N: int, K: int, experts: int = None):
    """Inverse of w4a4_repack; codes and scales have experts in front when it is given."""
    L, n = load(), experts or 1
    device = packed.get_device()
    at = _plain(packed, "packed", _U8, (L.w4a4_repacked_bytes(n, N, K),), device)
    front = () if experts is None else (experts,)
    codes = torch.empty((*front, N, K // 2), dtype=_U8, device=packed.device)
    scales = torch.empty((*front, N, K // 16), dtype=_U8, device=packed.device)
    _check("w4a4_unpack", L.w4a4_unpack(at, n, N, K, codes.data_ptr(), scales.data_ptr(),
                                        _raw_stream(device)))
    return codes, scales


class W4a4Rows:
    """M rows of K values in 4 bits, as w4a4_quantize writes them; with start int32 [experts + 1]
    (rows start[e] .. start[e+1] - 1 belong to expert e, read on the device when a call runs)
    they are an expert product's."""

    def __init__(self, data, M, K, start=None):
        self.data, self.M, self.K, self.start = data, M, K, start
        self.device = data.get_device()
        self.experts = 1 if start is None else start.numel() - 1
        size = load().w4a4_rows_bytes(M, K, self.experts)
        if size == 0:
            raise ValueError(f"no rows of M={M}, K={K}, experts={self.experts}")
        self.at = _plain(data, "data", _U8, (size,), self.device)
        self.struct = self.groups = None
        if start is not None:
            self.struct = _GroupsStruct(_plain(start, "start", _I32, (self.experts + 1,),
                                               self.device), self.experts)
            self.groups = ctypes.addressof(self.struct)

    @classmethod
    def empty(cls, M, K, device, start=None):
        """Rows that nothing has been written to."""
        experts = 1 if start is None else start.numel() - 1
        size = load().w4a4_rows_bytes(M, K, experts)
        return cls(torch.empty(size, dtype=_U8, device=device), M, K, start)


def _rows_for(out, M, K, start, like):
    """Rows to write M quantised rows of K to: `out`, checked, or new ones."""
    if out is None:
        return W4a4Rows.empty(M, K, like.device, start)
    if start is not None and start is not out.start:
        raise ValueError("start is not that of out")
    if out.M != M or out.K != K or out.device != like.get_device():
        raise ValueError(f"out holds {out.M} rows of {out.K} on device {out.device}, "
                         f"got {M} of {K} on {like.device}")
    return out


def w4a4_quantize(x: torch.Tensor, start: torch.Tensor = None, out: W4a4Rows = None) -> W4a4Rows:
    """x bf16 [M, K] in 4 bits.  With start (see W4a4Rows) the rows are an expert product's."""
    M, K, device = _matrix(x, "x")
    out = _rows_for(out, M, K, start, x)
    code = (_lib or load()).w4a4_quantize(x.data_ptr(), M, K, out.groups, out.at,
                                          _raw_stream(device))
    if code:
        _check("w4a4_quantize", code)
    return out


def w4a4_quantize_routed(x: torch.Tensor, ids: torch.Tensor, place: torch.Tensor,
                         start: torch.Tensor = None, out: W4a4Rows = None) -> W4a4Rows:
    """The rows of a routed batch: x bf16 [tokens, K], each token quantised once and written to the
    rows of its choices; ids, place int32 [tokens, choices] and start as experts_order has them."""
    T, K, device = _matrix(x, "x")
    shape = ids.shape
    if len(shape) != 2 or shape[0] != T:
        raise ValueError(f"ids must be [{T}, choices], got {list(shape)}")
    out = _rows_for(out, T * shape[1], K, start, x)
    if out.groups is None:
        raise ValueError("routed rows need start")
    code = (_lib or load()).w4a4_quantize_routed(
        x.data_ptr(), T, K, _plain(ids, "ids", _I32, shape, device),
        _plain(place, "place", _I32, shape, device), shape[1], out.groups, out.at,
        _raw_stream(device))
    if code:
        _check("w4a4_quantize_routed", code)
    return out


def w4a4_dequantize(rows: W4a4Rows, out: torch.Tensor = None) -> torch.Tensor:
    """The values that rows stand for, bf16 [M, K] (rows of no expert are left as they were)."""
    if out is None:
        out = torch.zeros((rows.M, rows.K), dtype=_BF16, device=rows.data.device)
    _check("w4a4_dequantize",
           load().w4a4_dequantize(rows.at, rows.M, rows.K, rows.groups,
                                  _plain(out, "out", _BF16, (rows.M, rows.K), rows.device),
                                  _raw_stream(rows.device)))
    return out


def w4a4_gemm_workspace_bytes(M: int, N: int, K: int, experts: int = 1) -> int:
    return load().w4a4_gemm_workspace_bytes(M, N, K, experts)


def _w4a4_buffers(rows, N, packed, size, ws, out, name):
    """Checks a product's buffers, allocates those not given: (out, its address, ws, its address)."""
    if ws is None:
        ws = workspace(load().w4a4_gemm_workspace_bytes(rows.M, N, rows.K, rows.experts),
                       rows.data.device)
    if out is None:
        out = torch.empty((rows.M, N), dtype=_BF16, device=rows.data.device)
    return (out, _plain(out, name, _BF16, (rows.M, N), rows.device), ws,
            _plain(ws, "ws", _U8, ws.shape, rows.device),
            _plain(packed, "packed weight", _U8, (size,), rows.device))


def _per_expert(scale, name, rows):
    return _plain(scale, name, _F32, (rows.experts,), rows.device)


def w4a4_gemm(rows: W4a4Rows, packed_w: torch.Tensor, scale2, N: int, ws: torch.Tensor = None,
              out: torch.Tensor = None) -> torch.Tensor:
    """y bf16 [M, N]: quantised rows by a weight of w4a4_repack.  Rows with experts take each
    expert's weight, scale2 is then fp32 [experts] on the device, and rows of no expert are left
    as they were."""
    L = _lib or load()
    out, out_at, ws, ws_at, w = _w4a4_buffers(
        rows, N, packed_w, L.w4a4_repacked_bytes(rows.experts, N, rows.K), ws, out, "out")
    if rows.groups is None:
        code = L.w4a4_gemm(rows.at, rows.M, rows.K, w, scale2, N, out_at, ws_at, ws.numel(),
                           _raw_stream(rows.device))
    else:
        code = L.w4a4_experts_gemm(rows.at, rows.M, rows.K, rows.groups, w,
                                   _per_expert(scale2, "scale2", rows), N, out_at, ws_at,
                                   ws.numel(), _raw_stream(rows.device))
    if code:
        _check("w4a4_gemm", code)
    return out


def w4a4_gate_up(rows: W4a4Rows, gate_up_packed: torch.Tensor, gate_scale2, up_scale2, I: int,
                 act: int = NVFP4_ACT_SILU, ws: torch.Tensor = None,
                 h: torch.Tensor = None) -> torch.Tensor:
    """h bf16 [M, I] = act(gate(x)) * up(x) for quantised rows; scales as for w4a4_gemm."""
    L = _lib or load()
    h, h_at, ws, ws_at, w = _w4a4_buffers(
        rows, I, gate_up_packed, L.w4a4_repacked_gate_up_bytes(rows.experts, I, rows.K), ws, h, "h")
    if rows.groups is None:
        code = L.w4a4_gate_up(rows.at, rows.M, rows.K, w, gate_scale2, up_scale2, I, act, h_at,
                              ws_at, ws.numel(), _raw_stream(rows.device))
    else:
        code = L.w4a4_experts_gate_up(rows.at, rows.M, rows.K, rows.groups, w,
                                      _per_expert(gate_scale2, "gate_scale2", rows),
                                      _per_expert(up_scale2, "up_scale2", rows), I, act, h_at,
                                      ws_at, ws.numel(), _raw_stream(rows.device))
    if code:
        _check("w4a4_gate_up", code)
    return h


def ffn_swiglu_w4a4_workspace_bytes(M: int, H: int, I: int) -> int:
    return load().ffn_swiglu_w4a4_workspace_bytes(M, H, I)


def ffn_swiglu_w4a4(x: torch.Tensor, gate_up_packed: torch.Tensor, gate_scale2: float,
                    up_scale2: float, down_packed: torch.Tensor, down_scale2: float, I: int,
                    act: int = NVFP4_ACT_SILU, ws: torch.Tensor = None,
                    out: torch.Tensor = None) -> torch.Tensor:
    """out bf16 [M, H] = down(act(gate(x)) * up(x)) on quantised activations, any number of rows."""
    M, H, device = _matrix(x, "x")
    L = _lib or load()
    if ws is None:
        ws = workspace(L.ffn_swiglu_w4a4_workspace_bytes(M, H, I), x.device)
    if out is None:
        out = torch.empty_like(x)
    code = L.ffn_swiglu_w4a4(
        x.data_ptr(), M, H, I,
        _plain(gate_up_packed, "gate_up_packed", _U8, (L.w4a4_repacked_gate_up_bytes(1, I, H),),
               device), gate_scale2, up_scale2,
        _plain(down_packed, "down_packed", _U8, (L.w4a4_repacked_bytes(1, H, I),), device),
        down_scale2, act, _plain(out, "out", _BF16, x.shape, device),
        _plain(ws, "ws", _U8, ws.shape, device), ws.numel(), _raw_stream(device))
    if code:
        _check("ffn_swiglu_w4a4", code)
    return out


def experts_order(ids: torch.Tensor, experts: int, start: torch.Tensor = None,
                  source: torch.Tensor = None, place: torch.Tensor = None):
    """ids int32 [tokens, choices] sorted by expert: (start [experts + 1], source [tokens *
    choices], place [tokens, choices]), int32."""
    shape, device = ids.shape, ids.get_device()
    if len(shape) != 2:
        raise ValueError("ids must be [tokens, choices]")
    at = _plain(ids, "ids", _I32, shape, device)
    pairs = shape[0] * shape[1]
    # lists made here need no checks
    if start is None:
        start = torch.empty(experts + 1, dtype=_I32, device=ids.device)
    else:
        _plain(start, "start", _I32, (experts + 1,), device)
    if source is None:
        source = torch.empty(pairs, dtype=_I32, device=ids.device)
    else:
        _plain(source, "source", _I32, (pairs,), device)
    if place is None:
        place = torch.empty(shape, dtype=_I32, device=ids.device)
    else:
        _plain(place, "place", _I32, shape, device)
    code = (_lib or load()).experts_order(at, shape[0], shape[1], experts, start.data_ptr(),
                                          source.data_ptr(), place.data_ptr(),
                                          _raw_stream(device))
    if code:
        _check("experts_order", code)
    return start, source, place


def experts_sum(y: torch.Tensor, place: torch.Tensor, weights: torch.Tensor,
                out: torch.Tensor = None) -> torch.Tensor:
    """out bf16 [tokens, H] = each token's sum of weights fp32 [tokens, choices] times the rows of
    y bf16 [rows, H] at place int32 [tokens, choices] (below 0: none)."""
    rows, H, device = _matrix(y, "y")
    shape = place.shape
    if len(shape) != 2:
        raise ValueError("place must be [tokens, choices]")
    if out is None:
        out = torch.empty((shape[0], H), dtype=_BF16, device=y.device)
    code = (_lib or load()).experts_sum(
        y.data_ptr(), rows, _plain(place, "place", _I32, shape, device),
        _plain(weights, "weights", _F32, shape, device), shape[0], shape[1], H,
        _plain(out, "out", _BF16, (shape[0], H), device), _raw_stream(device))
    if code:
        _check("experts_sum", code)
    return out


def experts_swiglu_w4a4_workspace_bytes(tokens: int, choices: int, experts: int, H: int,
                                        I: int) -> int:
    return load().experts_swiglu_w4a4_workspace_bytes(tokens, choices, experts, H, I)


def experts_swiglu_w4a4(x: torch.Tensor, ids: torch.Tensor, weights: torch.Tensor,
                        gate_up_packed: torch.Tensor, gate_scale2: torch.Tensor,
                        up_scale2: torch.Tensor, down_packed: torch.Tensor,
                        down_scale2: torch.Tensor, I: int, act: int = NVFP4_ACT_SILU,
                        ws: torch.Tensor = None, out: torch.Tensor = None) -> torch.Tensor:
    """The experts' FFN of a routed batch: x bf16 [tokens, H], ids int32 and weights fp32 [tokens,
    choices], experts' weights stacked (w4a4_repack), their scales fp32 [experts] on the device."""
    T, H, device = _matrix(x, "x")
    shape, experts = ids.shape, gate_scale2.numel()
    if len(shape) != 2 or shape[0] != T:
        raise ValueError(f"ids must be [{T}, choices], got {list(shape)}")
    L = _lib or load()
    if ws is None:
        ws = workspace(L.experts_swiglu_w4a4_workspace_bytes(T, shape[1], experts, H, I), x.device)
    if out is None:
        out = torch.empty_like(x)
    scales = [_plain(t, f"{n}_scale2", _F32, (experts,), device)
              for t, n in ((gate_scale2, "gate"), (up_scale2, "up"), (down_scale2, "down"))]
    code = L.experts_swiglu_w4a4(
        x.data_ptr(), T, H, I, _plain(ids, "ids", _I32, shape, device),
        _plain(weights, "weights", _F32, shape, device), shape[1], experts,
        _plain(gate_up_packed, "gate_up_packed", _U8,
               (L.w4a4_repacked_gate_up_bytes(experts, I, H),), device), scales[0], scales[1],
        _plain(down_packed, "down_packed", _U8, (L.w4a4_repacked_bytes(experts, H, I),), device),
        scales[2], act, _plain(out, "out", _BF16, x.shape, device),
        _plain(ws, "ws", _U8, ws.shape, device), ws.numel(), _raw_stream(device))
    if code:
        _check("experts_swiglu_w4a4", code)
    return out
