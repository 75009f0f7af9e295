"""Refusals of the attention-side calls, found on the host before any launch (no GPU needed)."""
import ctypes

import pytest
import torch

import kv8_reference as ref
from nvfp4_weight_only_gb300 import ffi


@pytest.fixture(scope="module")
def lib():
    return ffi.load(build_if_missing=True)


def P(n):
    return n << 32  # distinct addresses far apart, never dereferenced


NULL, SHAPE, ALIGN, RANGE, WORKSPACE, ALIAS = 1, 2, 3, 4, 5, 8


def cache(**kw):
    f = dict(k_codes=P(1), v_codes=P(2), k_scales=P(3), v_scales=P(4), pages=10, kv_heads=2, page=64,
             head_dim=128)
    f.update(kw)
    return ffi._CacheStruct(**f)


def batch(**kw):
    f = dict(q_start=P(5), kv_len=P(6), page_table=P(7), status=P(8), batch=2, table_width=4)
    f.update(kw)
    return ffi._BatchStruct(**f)


CACHES = [(dict(k_codes=None), NULL), (dict(v_scales=None), NULL), (dict(pages=0), SHAPE),
          (dict(kv_heads=0), SHAPE), (dict(head_dim=96), SHAPE), (dict(page=48), SHAPE),
          (dict(page=8), SHAPE), (dict(page=512), SHAPE), (dict(k_codes=P(1) + 8), ALIGN),
          (dict(v_scales=P(4) + 2), ALIGN)]
BATCHES = [(dict(q_start=None), NULL), (dict(kv_len=None), NULL), (dict(page_table=None), NULL),
           (dict(batch=0), RANGE), (dict(batch=1025), RANGE), (dict(table_width=0), SHAPE),
           (dict(table_width=2 ** 26), SHAPE), (dict(kv_len=P(6) + 1), ALIGN)]


def attention(lib, c=None, b=None, q=P(10), q_stride=512, tokens=3, heads=4, scale=0.1, window=0,
              sinks=0, out=P(11), lse=P(12), ws=P(13), ws_bytes=1 << 30):
    c, b = c or cache(), b or batch()
    return lib.kv8_attention(q, q_stride, tokens, heads, ctypes.addressof(c), ctypes.addressof(b),
                             scale, window, sinks, out, lse, ws, ws_bytes, None)


def append(lib, c=None, b=None, tokens=3, k=P(10), ks=256, v=P(11), vs=256, q=P(12), qs=512, heads=4,
           q_out=P(13), rope=P(14), positions=100, rot=128, inter=0):
    c, b = c or cache(), b or batch()
    return lib.kv8_append(ctypes.addressof(c), ctypes.addressof(b), tokens, k, ks, v, vs, q, qs,
                          heads, q_out, rope, positions, rot, inter, None)


@pytest.mark.parametrize("kw,code", CACHES)
def test_caches(lib, kw, code):
    c = cache(**kw)
    assert attention(lib, c) == append(lib, c) == code
    b = batch()
    assert lib.kv8_read(ctypes.addressof(c), ctypes.addressof(b), 3, P(10), P(11), None) == code


@pytest.mark.parametrize("kw,code", BATCHES)
def test_batches(lib, kw, code):
    b = batch(**kw)
    assert attention(lib, b=b) == append(lib, b=b) == code
    c = cache()
    assert lib.kv8_read(ctypes.addressof(c), ctypes.addressof(b), 3, P(10), P(11), None) == code


@pytest.mark.parametrize("kw,code", [
    (dict(q=None), NULL), (dict(out=None), NULL), (dict(ws=None), NULL), (dict(tokens=0), RANGE),
    (dict(heads=3), SHAPE), (dict(heads=0), SHAPE), (dict(q_stride=504), SHAPE),
    (dict(tokens=2 ** 30), RANGE),
    (dict(q_stride=516), SHAPE), (dict(window=-1), RANGE), (dict(sinks=-1), RANGE),
    (dict(scale=float("nan")), RANGE), (dict(scale=float("inf")), RANGE),
    (dict(q=P(10) + 2), ALIGN), (dict(out=P(11) + 8), ALIGN), (dict(lse=P(12) + 2), ALIGN),
    (dict(ws=P(13) + 4), ALIGN), (dict(out=P(10) + 1024), ALIAS), (dict(lse=P(11) + 16), ALIAS)])
def test_attention(lib, kw, code):
    assert attention(lib, **kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(k=None), NULL), (dict(v=None), NULL), (dict(q=None), NULL), (dict(q_out=None), NULL),
    (dict(tokens=-1), RANGE), (dict(ks=128), SHAPE), (dict(vs=260), SHAPE), (dict(qs=256), SHAPE),
    (dict(heads=0), SHAPE), (dict(rot=130), SHAPE), (dict(rot=144), SHAPE), (dict(rot=0), SHAPE),
    (dict(positions=0), SHAPE), (dict(rope=P(14) + 4), ALIGN), (dict(k=P(10) + 2), ALIGN),
    (dict(q_out=P(13) + 8), ALIGN), (dict(q_out=P(12) + 512), ALIAS),
    (dict(q_out=P(12), qs=1024), ALIAS), (dict(q_out=P(10)), ALIAS)])
def test_append(lib, kw, code):
    assert append(lib, **kw) == code


def test_read_and_status(lib):
    c, b = cache(), batch()
    read = lambda *a: lib.kv8_read(ctypes.addressof(c), ctypes.addressof(b), *a, None)  # noqa: E731
    assert read(3, None, P(11)) == NULL
    assert read(0, P(10), P(11)) == RANGE
    assert read(3, P(10) + 4, P(11)) == ALIGN
    assert read(3, P(10), P(10) + 512) == ALIAS
    assert lib.kv8_read(None, ctypes.addressof(b), 3, P(10), P(11), None) == NULL
    assert lib.kv8_batch_status(None, None) == NULL
    assert lib.kv8_batch_status(ctypes.addressof(batch(status=None)), None) == NULL


def test_workspace_query(lib):
    c, b = cache(), batch()
    a = ctypes.addressof
    assert lib.kv8_attention_workspace_bytes(a(c), a(b), 3, 4) > 256
    assert lib.kv8_attention_workspace_bytes(None, a(b), 3, 4) == 0
    assert lib.kv8_attention_workspace_bytes(a(c), a(b), 0, 4) == 0
    assert lib.kv8_attention_workspace_bytes(a(c), a(b), 3, 0) == 0


def norm(lib, name, x=P(1), residual=P(2), weight=P(3), M=4, H=256, eps=1e-6, total=P(4), out=P(5),
         scales=P(6)):
    if name == "bf16":
        return lib.add_rmsnorm_bf16(x, residual, weight, M, H, eps, 0.0, total, out, None)
    return lib.add_rmsnorm_e4m3(x, residual, weight, M, H, eps, 0.0, total, out, scales, None)


@pytest.mark.parametrize("name", ["bf16", "e4m3"])
@pytest.mark.parametrize("kw,code", [
    (dict(x=None), NULL), (dict(weight=None), NULL), (dict(out=None), NULL), (dict(M=0), SHAPE),
    (dict(H=8), SHAPE), (dict(H=250), SHAPE), (dict(H=32784), SHAPE), (dict(eps=-1.0), RANGE),
    (dict(eps=float("nan")), RANGE), (dict(x=P(1) + 2), ALIGN), (dict(residual=P(2) + 8), ALIGN),
    (dict(out=P(5) + 4), ALIGN), (dict(total=P(2) + 16), ALIAS), (dict(out=P(4)), ALIAS),
    (dict(out=P(1) + 16), ALIAS), (dict(total=P(3)), ALIAS)])
def test_norm(lib, name, kw, code):
    assert norm(lib, name, **kw) == code


def test_norm_e4m3_buffers(lib):
    assert norm(lib, "e4m3", scales=None) == NULL
    assert norm(lib, "e4m3", scales=P(6) + 2) == ALIGN
    assert norm(lib, "e4m3", scales=P(5) + 16) == ALIAS
    assert norm(lib, "e4m3", out=P(1)) == ALIAS


@pytest.mark.parametrize("a,code", [
    ((10, 64, 1e4, 0, 1.0, 1.0, 1.0, 32.0, 1.0, None), NULL),
    ((0, 64, 1e4, 0, 1.0, 1.0, 1.0, 32.0, 1.0, P(1)), SHAPE),
    ((10, 24, 1e4, 0, 1.0, 1.0, 1.0, 32.0, 1.0, P(1)), SHAPE),
    ((10, 512, 1e4, 0, 1.0, 1.0, 1.0, 32.0, 1.0, P(1)), SHAPE),
    ((10, 64, 1.0, 0, 1.0, 1.0, 1.0, 32.0, 1.0, P(1)), RANGE),
    ((10, 64, 1e4, 4, 1.0, 1.0, 1.0, 32.0, 1.0, P(1)), RANGE),
    ((10, 64, 1e4, 1, 0.0, 1.0, 1.0, 32.0, 1.0, P(1)), RANGE),
    ((10, 64, 1e4, 3, 2.0, 0.0, 1.0, 32.0, 1.0, P(1)), RANGE),
    ((10, 64, 1e4, 3, 2.0, 1.0, 32.0, 32.0, 1.0, P(1)), RANGE),
    ((10, 64, 1e4, 0, 1.0, 1.0, 1.0, 32.0, 1.0, P(1) + 8), ALIGN)])
def test_rope_table(lib, a, code):
    assert lib.rope_table(*a, None) == code


def test_binding_refuses_what_the_library_cannot_see():
    x = torch.zeros((2, 256), dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        ffi.add_rmsnorm_bf16(x, x[0], 1e-6)  # not on a GPU
    with pytest.raises(ValueError):
        ffi.Kv8Cache(*[torch.zeros((2, 1, 16, 64), dtype=torch.uint8)] * 2,
                     *[torch.zeros((2, 1))] * 2)
    with pytest.raises(ValueError):
        ffi.Kv8Batch(*[torch.zeros(2, dtype=torch.int32)] * 2,
                     torch.zeros((2, 2), dtype=torch.int32))


def test_reference_rounding():
    """The tests' own E4M3 rounding against torch's conversion, ties and both ends included."""
    x = torch.cat((torch.linspace(-500, 500, 40001), torch.linspace(-0.02, 0.02, 40001)))
    want = x.clamp(-448, 448).to(ref.E4M3).view(torch.uint8)
    assert torch.equal(ref.round_e4m3(x), want)
    assert int(ref.round_e4m3(torch.tensor([float("nan")]))[0]) & 0x7F == 0x7F
