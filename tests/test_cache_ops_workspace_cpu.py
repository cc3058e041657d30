"""mla_mha_decode_workspace_bytes refuses what mla_mha_decode_paged refuses, before any CUDA work."""
import ctypes

import pytest

from paged_fp8_kv_mla_b200 import _lib, build


@pytest.fixture(scope="module")
def lib():
    build.build()
    return _lib.load()


def query(lib, element_bytes=2, tokens=1, cached=64, **kw):
    base = dict(batch=2, num_q_heads=16, head_dim=64, v_dim=64, num_blocks=16, kv_dim=2, num_layers=1, page_size=16, num_kv_heads=4,
                num_scale_blocks=16, head_dim_granularity=1, max_pages=8)
    n = ctypes.c_uint64(7)
    st = lib.mla_mha_decode_workspace_bytes(tokens, cached, element_bytes, ctypes.byref(_lib.PagedShape(**{**base, **kw})),
                                            ctypes.byref(n))
    return st, n.value


@pytest.mark.parametrize("want,kw", [
    (1, dict(element_bytes=0)), (1, dict(element_bytes=3)), (1, dict(element_bytes=-1)), (1, dict(element_bytes=2 ** 31 - 1)),
    (2, dict(head_dim=96)), (2, dict(page_size=24)), (1, dict(kv_dim=1)), (2, dict(num_kv_heads=257, num_q_heads=257)),
    (2, dict(head_dim_granularity=2)), (1, dict(num_blocks=0)), (1, dict(batch=-1)),
    (1, dict(batch=0, element_bytes=0)), (2, dict(batch=0, head_dim=96)),
    (1, dict(num_q_heads=6)), (1, dict(tokens=0)), (1, dict(cached=128)),
])
def test_query_refuses(lib, want, kw):
    assert query(lib, **kw) == (want, 0)


@pytest.mark.parametrize("kw", [dict(num_q_heads=6), dict(tokens=0), dict(cached=128)])
def test_query_of_an_empty_batch_refuses_what_the_call_refuses(lib, kw):
    assert query(lib, batch=0, **kw) == (1, 0)


def test_query_of_an_empty_batch(lib):
    assert query(lib, batch=0) == (0, 0) and query(lib, batch=0, element_bytes=1) == (0, 0)
