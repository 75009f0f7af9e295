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
# The current stream's handle by device index, without a Stream object.
_raw_stream = torch._C._cuda_getCurrentRawStream


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
