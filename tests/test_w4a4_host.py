"""Refusals of the calls on 4-bit activations, found on the host before any launch (no GPU
needed), and their size queries."""
import ctypes

import pytest
import torch

from nvfp4_weight_only_gb300 import ffi


@pytest.fixture(scope="module")
def lib():
    return ffi.load(build_if_missing=True)


def P(n):
    return n << 36  # distinct addresses far apart, never dereferenced


NULL, SHAPE, ALIGN, RANGE, WORKSPACE, ALIAS = 1, 2, 3, 4, 5, 8
TILE = 18432


def groups(**kw):
    f = dict(start=P(20), experts=4)
    f.update(kw)
    return ffi._GroupsStruct(**f)


def test_sizes(lib):
    assert lib.w4a4_repacked_bytes(1, 5120, 17408) == 5120 * 17408 * 9 // 16
    assert lib.w4a4_repacked_bytes(3, 257, 272) == 3 * 4 * 2 * TILE
    assert lib.w4a4_repacked_gate_up_bytes(1, 17408, 5120) == 2 * 17408 * 5120 * 9 // 16
    assert lib.w4a4_repacked_gate_up_bytes(2, 16, 16) == 2 * 2 * TILE
    assert lib.w4a4_rows_bytes(1, 256, 1) == TILE + 4
    assert lib.w4a4_rows_bytes(129, 272, 1) == 2 * 2 * TILE + 129 * 4
    assert lib.w4a4_rows_bytes(129, 256, 5) == (2 + 5) * TILE + 129 * 4
    for bad in ((0, 16, 16), (1025, 16, 16), (1, 0, 16), (1, 16, 8), (1, 16, 24), (1, 16, 65552),
                (1, (1 << 20) + 1, 16)):
        assert lib.w4a4_repacked_bytes(*bad) == 0
    assert lib.w4a4_repacked_gate_up_bytes(1, 24, 16) == 0
    assert lib.w4a4_rows_bytes(0, 16, 1) == lib.w4a4_rows_bytes((1 << 22) + 1, 16, 1) == 0
    assert lib.w4a4_gemm_workspace_bytes(0, 16, 16, 1) == 0
    assert lib.w4a4_gemm_workspace_bytes(1, 16, 16, 1) > lib.w4a4_gemm_workspace_bytes(1, 16, 16, 2)
    assert lib.w4a4_gemm_workspace_bytes(1, 16, 16, 2) > 1 << 17
    assert lib.ffn_swiglu_w4a4_workspace_bytes(1, 16, 24) == 0
    assert lib.ffn_swiglu_w4a4_workspace_bytes(70, 256, 512) > 70 * 512 * 2
    assert lib.experts_swiglu_w4a4_workspace_bytes(4, 65, 80, 256, 512) == 0
    assert lib.experts_swiglu_w4a4_workspace_bytes(1 << 20, 5, 8, 256, 512) == 0
    assert lib.experts_swiglu_w4a4_workspace_bytes(4, 2, 8, 256, 512) > 8 * 256 * 2


@pytest.mark.parametrize("kw,code", [
    (dict(codes=None), NULL), (dict(scales=None), NULL), (dict(packed=None), NULL),
    (dict(experts=0), SHAPE), (dict(N=0), SHAPE), (dict(K=24), SHAPE), (dict(K=0), SHAPE),
    (dict(packed=P(3) + 8), ALIGN)])
def test_repack(lib, kw, code):
    f = dict(codes=P(1), scales=P(2), packed=P(3), experts=2, N=32, K=32)
    f.update(kw)
    assert lib.w4a4_repack(f["codes"], f["scales"], f["experts"], f["N"], f["K"], f["packed"],
                           None) == code
    assert lib.w4a4_unpack(f["packed"], f["experts"], f["N"], f["K"], f["codes"], f["scales"],
                           None) == code
    assert lib.w4a4_repack_gate_up(f["codes"], f["scales"], P(4), P(5), f["experts"], f["N"], f["K"],
                                   f["packed"], None) == code


def test_repack_gate_up(lib):
    assert lib.w4a4_repack_gate_up(P(1), P(2), None, P(5), 1, 32, 32, P(3), None) == NULL
    assert lib.w4a4_repack_gate_up(P(1), P(2), P(4), P(5), 1, 24, 32, P(3), None) == SHAPE


@pytest.mark.parametrize("kw,code", [
    (dict(x=None), NULL), (dict(rows=None), NULL), (dict(M=0), RANGE), (dict(M=(1 << 22) + 1), RANGE),
    (dict(K=8), SHAPE), (dict(K=65552), SHAPE), (dict(x=P(1) + 8), ALIGN), (dict(rows=P(2) + 4), ALIGN),
    (dict(rows=P(1)), ALIAS), (dict(rows=P(1) + 30 * 64), ALIAS),
    (dict(g=groups(start=None)), NULL), (dict(g=groups(experts=0)), RANGE),
    (dict(g=groups(experts=1025)), RANGE), (dict(g=groups(start=P(20) + 2)), ALIGN)])
def test_quantize(lib, kw, code):
    f = dict(x=P(1), rows=P(2), M=31, K=32, g=None)
    f.update(kw)
    g = ctypes.addressof(f["g"]) if f["g"] else None
    assert lib.w4a4_quantize(f["x"], f["M"], f["K"], g, f["rows"], None) == code
    assert lib.w4a4_dequantize(f["rows"], f["M"], f["K"], g, f["x"], None) == code


@pytest.mark.parametrize("kw,code", [
    (dict(x=None), NULL), (dict(ids=None), NULL), (dict(place=None), NULL), (dict(g=None), NULL),
    (dict(rows=None), NULL), (dict(T=0), RANGE), (dict(k=0), RANGE), (dict(k=65), RANGE),
    (dict(T=1 << 20, k=5), RANGE), (dict(g=groups(experts=2000)), RANGE), (dict(K=20), SHAPE),
    (dict(ids=P(4) + 2), ALIGN), (dict(rows=P(2) + 8), ALIGN), (dict(rows=P(5)), ALIAS),
    (dict(rows=P(1)), ALIAS)])
def test_quantize_routed(lib, kw, code):
    f = dict(x=P(1), rows=P(2), ids=P(4), place=P(5), T=9, k=3, K=64, g=groups())
    f.update(kw)
    g = ctypes.addressof(f["g"]) if f["g"] else None
    assert lib.w4a4_quantize_routed(f["x"], f["T"], f["K"], f["ids"], f["place"], f["k"], g,
                                    f["rows"], None) == code


PRODUCTS = [
    (dict(rows=None), NULL), (dict(w=None), NULL), (dict(out=None), NULL), (dict(ws=None), NULL),
    (dict(M=0), RANGE), (dict(M=(1 << 22) + 1), RANGE), (dict(N=0), SHAPE), (dict(K=24), SHAPE),
    (dict(N=(1 << 20) + 16), SHAPE), (dict(rows=P(1) + 8), ALIGN), (dict(w=P(2) + 8), ALIGN),
    (dict(out=P(3) + 8), ALIGN), (dict(ws=P(4) + 8), ALIGN)]


@pytest.mark.parametrize("kw,code", PRODUCTS)
def test_products(lib, kw, code):
    f = dict(rows=P(1), w=P(2), out=P(3), ws=P(4), M=40, N=64, K=64, bytes=1 << 30)
    f.update(kw)
    a = (f["rows"], f["M"], f["K"])
    end = (f["out"], f["ws"], f["bytes"], None)
    assert lib.w4a4_gemm(*a, f["w"], 1.0, f["N"], *end) == code
    assert lib.w4a4_gate_up(*a, f["w"], 1.0, 1.0, f["N"], 0, *end) == code
    g = groups()
    at = ctypes.addressof(g)
    assert lib.w4a4_experts_gemm(*a, at, f["w"], P(6), f["N"], *end) == code
    assert lib.w4a4_experts_gate_up(*a, at, f["w"], P(6), P(7), f["N"], 0, *end) == code


def test_products_own_arguments(lib):
    a, end = (P(1), 40, 64), (P(3), P(4), 1 << 30, None)
    g = groups()
    at = ctypes.addressof(g)
    assert lib.w4a4_gate_up(*a, P(2), 1.0, 1.0, 24, 0, *end) == SHAPE
    assert lib.w4a4_gate_up(*a, P(2), 1.0, 1.0, 32, 2, *end) == RANGE
    assert lib.w4a4_experts_gemm(*a, None, P(2), P(6), 64, *end) == NULL
    assert lib.w4a4_experts_gemm(*a, at, P(2), None, 64, *end) == NULL
    assert lib.w4a4_experts_gemm(*a, at, P(2), P(6) + 1, 64, *end) == ALIGN
    assert lib.w4a4_experts_gate_up(*a, at, P(2), P(6), None, 64, 0, *end) == NULL
    bad = groups(experts=0)
    assert lib.w4a4_experts_gemm(*a, ctypes.addressof(bad), P(2), P(6), 64, *end) == RANGE


@pytest.mark.parametrize("kw,code", [
    (dict(x=None), NULL), (dict(gu=None), NULL), (dict(dn=None), NULL), (dict(out=None), NULL),
    (dict(ws=None), NULL), (dict(M=0), RANGE), (dict(act=7), RANGE), (dict(H=8), SHAPE),
    (dict(I=40), SHAPE), (dict(x=P(1) + 2), ALIGN), (dict(dn=P(3) + 8), ALIGN)])
def test_ffn(lib, kw, code):
    f = dict(x=P(1), gu=P(2), dn=P(3), out=P(4), ws=P(5), M=100, H=64, I=64, act=0, ids=P(8),
             wt=P(9), k=2, E=4)
    f.update(kw)
    assert lib.ffn_swiglu_w4a4(f["x"], f["M"], f["H"], f["I"], f["gu"], 1.0, 1.0, f["dn"], 1.0,
                               f["act"], f["out"], f["ws"], 1 << 30, None) == code
    assert lib.experts_swiglu_w4a4(f["x"], f["M"], f["H"], f["I"], f["ids"], f["wt"], f["k"], f["E"],
                                   f["gu"], P(10), P(11), f["dn"], P(12), f["act"], f["out"],
                                   f["ws"], 1 << 30, None) == code


@pytest.mark.parametrize("kw,code", [
    (dict(ids=None), NULL), (dict(wt=None), NULL), (dict(gs=None), NULL), (dict(ds=None), NULL),
    (dict(k=0), RANGE), (dict(k=65), RANGE), (dict(E=0), RANGE), (dict(E=1025), RANGE),
    (dict(ids=P(8) + 2), ALIGN), (dict(gs=P(10) + 2), ALIGN)])
def test_experts_ffn(lib, kw, code):
    f = dict(ids=P(8), wt=P(9), k=2, E=4, gs=P(10), ds=P(12))
    f.update(kw)
    assert lib.experts_swiglu_w4a4(P(1), 10, 64, 64, f["ids"], f["wt"], f["k"], f["E"], P(2), f["gs"],
                                   P(11), P(3), f["ds"], 0, P(4), P(5), 1 << 30, None) == code


@pytest.mark.parametrize("kw,code", [
    (dict(ids=None), NULL), (dict(start=None), NULL), (dict(source=None), NULL),
    (dict(place=None), NULL), (dict(T=0), RANGE), (dict(k=0), RANGE), (dict(k=65), RANGE),
    (dict(E=0), RANGE), (dict(E=1025), RANGE), (dict(T=1 << 20, k=5), RANGE),
    (dict(ids=P(1) + 2), ALIGN), (dict(place=P(4) + 1), ALIGN), (dict(source=P(1)), ALIAS),
    (dict(place=P(3) + 8), ALIAS), (dict(start=P(4)), ALIAS)])
def test_order(lib, kw, code):
    f = dict(ids=P(1), start=P(2), source=P(3), place=P(4), T=9, k=3, E=5)
    f.update(kw)
    assert lib.experts_order(f["ids"], f["T"], f["k"], f["E"], f["start"], f["source"], f["place"],
                             None) == code


@pytest.mark.parametrize("kw,code", [
    (dict(y=None), NULL), (dict(place=None), NULL), (dict(wt=None), NULL), (dict(out=None), NULL),
    (dict(rows=0), RANGE), (dict(T=0), RANGE), (dict(k=65), RANGE), (dict(H=24), SHAPE),
    (dict(H=0), SHAPE), (dict(y=P(1) + 8), ALIGN), (dict(wt=P(3) + 2), ALIGN), (dict(out=P(1)), ALIAS),
    (dict(out=P(2)), ALIAS)])
def test_sum(lib, kw, code):
    f = dict(y=P(1), place=P(2), wt=P(3), out=P(4), rows=27, T=9, k=3, H=64)
    f.update(kw)
    assert lib.experts_sum(f["y"], f["rows"], f["place"], f["wt"], f["T"], f["k"], f["H"], f["out"],
                           None) == code


def test_the_binding_refuses_host_tensors_and_wrong_shapes():
    bf, u8 = torch.bfloat16, torch.uint8
    with pytest.raises(ValueError):
        ffi.w4a4_quantize(torch.zeros(2, 32, dtype=bf))
    with pytest.raises(ValueError):
        ffi.w4a4_repack(torch.zeros(2, 16, dtype=u8), torch.zeros(2, 2, dtype=u8))
    with pytest.raises(ValueError):
        ffi.experts_order(torch.zeros(4, dtype=torch.int32), 2)
    with pytest.raises(ValueError):
        ffi.ffn_swiglu_w4a4(torch.zeros(2, 32, dtype=torch.float32), None, 1.0, 1.0, None, 1.0, 32)
    with pytest.raises(ValueError):
        ffi.W4a4Rows.empty(0, 32, "cpu")
