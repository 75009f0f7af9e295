"""Calls on tensors of a device that is not the current one are refused before any launch (no GPU
needed): a launch goes to the current device, where those addresses are nobody's."""
import pytest
import torch

from nvfp4_weight_only_gb300 import ffi

BF, U8, F32, I32 = torch.bfloat16, torch.uint8, torch.float32, torch.int32


class OnDeviceOne:
    """What the binding reads of a tensor, on device 1 (its address is never used)."""
    is_cuda, device = True, torch.device("cpu")

    def __init__(self, dtype, *shape):
        self.dtype, self.shape = dtype, torch.Size(shape)

    def dim(self):
        return len(self.shape)

    def numel(self):
        return self.shape.numel()

    def is_contiguous(self):
        return True

    def get_device(self):
        return 1

    def data_ptr(self):
        return 1 << 36


T = OnDeviceOne


def rows(M, K, start=None):
    size = ffi.load().w4a4_rows_bytes(M, K, 1 if start is None else start.numel() - 1)
    return ffi.W4a4Rows(T(U8, size), M, K, start)


def calls():
    L = ffi.load(build_if_missing=True)
    ws = T(U8, 1 << 30)
    packed = T(U8, L.w4a4_repacked_bytes(1, 64, 64))
    gu, egu = [T(U8, L.w4a4_repacked_gate_up_bytes(n, 64, 64)) for n in (1, 2)]
    epacked, es, start = T(U8, L.w4a4_repacked_bytes(2, 64, 64)), T(F32, 2), T(I32, 3)
    x, ids, weights = T(BF, 4, 64), T(I32, 4, 2), T(F32, 4, 2)
    codes, scales = T(U8, 64, 32), T(U8, 64, 4)
    return {
        "repack": lambda: ffi.w4a4_repack(codes, scales),
        "repack_gate_up": lambda: ffi.w4a4_repack_gate_up(codes, scales, codes, scales),
        "unpack": lambda: ffi.w4a4_unpack(packed, 64, 64),
        "quantize": lambda: ffi.w4a4_quantize(x, out=rows(4, 64)),
        "quantize_routed": lambda: ffi.w4a4_quantize_routed(x, ids, ids, out=rows(8, 64, start)),
        "dequantize": lambda: ffi.w4a4_dequantize(rows(4, 64), out=x),
        "gemm": lambda: ffi.w4a4_gemm(rows(4, 64), packed, 1.0, 64, ws=ws, out=x),
        "gate_up": lambda: ffi.w4a4_gate_up(rows(4, 64), gu, 1.0, 1.0, 64, ws=ws, h=x),
        "experts_gemm": lambda: ffi.w4a4_gemm(rows(4, 64, start), epacked, es, 64, ws=ws, out=x),
        "experts_gate_up": lambda: ffi.w4a4_gate_up(rows(4, 64, start), egu, es, es, 64, ws=ws, h=x),
        "ffn": lambda: ffi.ffn_swiglu_w4a4(x, gu, 1.0, 1.0, packed, 1.0, 64, ws=ws, out=x),
        "order": lambda: ffi.experts_order(ids, 2, start, T(I32, 8), T(I32, 4, 2)),
        "sum": lambda: ffi.experts_sum(T(BF, 8, 64), ids, weights, out=x),
        "experts": lambda: ffi.experts_swiglu_w4a4(x, ids, weights, egu, es, es, epacked, es, 64,
                                                   ws=ws, out=x),
        "norm": lambda: ffi.add_rmsnorm_bf16(x, T(BF, 64), 1e-6, out=x),
    }


@pytest.mark.parametrize("name", list(calls()))
def test_refused(monkeypatch, name):
    monkeypatch.setattr(ffi, "_current_device", lambda: 0, raising=False)
    with pytest.raises(ValueError, match="device 1 .*current device is 0"):
        calls()[name]()
