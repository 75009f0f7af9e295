"""Workspace queries of kv8_attention: from the sizes alone, and 0 for what the call refuses (no GPU
needed)."""
import ctypes

import pytest

from nvfp4_weight_only_gb300 import ffi


@pytest.fixture(scope="module")
def lib():
    return ffi.load(build_if_missing=True)


def query(lib, tokens=3, heads=4, pages=10, kv_heads=2, page=64, head_dim=128, batch=2, width=4):
    c = ffi._CacheStruct(pages=pages, kv_heads=kv_heads, page=page, head_dim=head_dim)
    b = ffi._BatchStruct(batch=batch, table_width=width)
    return lib.kv8_attention_workspace_bytes(ctypes.addressof(c), ctypes.addressof(b), tokens, heads)


@pytest.mark.parametrize("kw", [dict(), dict(tokens=100), dict(head_dim=64), dict(head_dim=256),
                                dict(batch=1024), dict(page=16), dict(heads=64, tokens=2 ** 24)])
def test_sizes_alone_answer(lib, kw):
    assert query(lib, **kw) > 256


@pytest.mark.parametrize("kw", [
    dict(heads=3), dict(heads=0), dict(tokens=0), dict(head_dim=96), dict(head_dim=0), dict(page=48),
    dict(page=8), dict(pages=0), dict(kv_heads=0), dict(batch=0), dict(batch=1025), dict(width=0),
    dict(width=2 ** 26), dict(tokens=2 ** 30)])
def test_sizes_that_the_call_refuses(lib, kw):
    assert query(lib, **kw) == 0
