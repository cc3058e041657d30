"""Refusals of the cache operators: the Python binding's checks on CPU tensors (all fire before the device
check) and the C ABI's checks (all fire before any CUDA work)."""
import ctypes

import pytest
import torch

import paged_fp8_kv_mla_b200 as M
from paged_fp8_kv_mla_b200 import _lib, build


@pytest.fixture(scope="module")
def lib():
    build.build()
    return _lib.load()


def z(*shape, dtype=torch.int32):
    return torch.zeros(shape, dtype=dtype)


F32, BF16, U8 = torch.float32, torch.bfloat16, torch.uint8


# ---------------------------------------------------------------- binding
def _weights(B=2, T=1, H=8, **over):
    a = dict(q=z(B, T, H, 576, dtype=BF16), lse=z(B, T, H, dtype=F32), blocks=z(8, 1, 1, 16, 1, 576, dtype=U8),
             scales=z(8, 1, 1, 16, 1, 1, dtype=F32), cache_lengths=z(B), lookup_table=z(B, 4), scales_lookup_table=None,
             max_prompt_length=T, max_cache_length=40, layer_idx=0, softmax_scale=0.1, scores=z(B, 41, dtype=F32))
    a.update(over)
    return M.accumulate_weights(**a)


@pytest.mark.parametrize("over,msg", [
    (dict(q=z(2, 1, 8, 576, dtype=F32)), "q must have dtype"),
    (dict(q=z(2, 1, 8, 512, dtype=BF16)), "last dim 576"),
    (dict(lse=z(2, 1, 8, dtype=torch.float64)), "lse must have dtype"),
    (dict(lse=z(2, 1, 7, dtype=F32)), "lse must be"),
    (dict(blocks=z(8, 1, 1, 16, 576, dtype=U8)), "blocks must be 6-D"),
    (dict(scales=z(8, 1, 1, 16, 1, 1, dtype=BF16)), "scales must have dtype"),
    (dict(scales=z(8, 1, 1, 32, 1, 1, dtype=F32)), "scales must match blocks"),
    (dict(scales=z(9, 1, 1, 16, 1, 1, dtype=F32)), "as many blocks"),
    (dict(cache_lengths=z(3)), "one per request"),
    (dict(cache_lengths=z(2, dtype=torch.int64)), "cache_lengths must have dtype"),
    (dict(scales_lookup_table=z(2, 5)), "shape of lookup_table"),
    (dict(max_prompt_length=2), "number of tokens"),
    (dict(scores=z(2, 40, dtype=F32)), "scores must be"),
    (dict(scores=z(2, 41, dtype=torch.float64)), "scores must have dtype"),
    (dict(scores=z(82, dtype=F32).as_strided((2, 41), (1, 2))), "contiguous rows"),
    (dict(out=z(2, 41, dtype=F32).expand(2, 41)[:1].expand(2, 41)), "do not overlap"),
    (dict(workspace=z(100, dtype=F32)), "workspace must have dtype"),
    (dict(), "CUDA tensors"),
])
def test_accumulate_weights_refuses(over, msg):
    with pytest.raises(ValueError, match=msg):
        _weights(**over)


def _select(**over):
    a = dict(scores=z(2, 50, dtype=F32), lengths=z(2), max_length=50, budget=20, num_recent=4, num_sink=1)
    a.update(over)
    return M.select_keys(**a)


@pytest.mark.parametrize("over,msg", [
    (dict(lengths=z(2, dtype=F32)), "lengths must have dtype"),
    (dict(scores=z(3, 50, dtype=F32)), "scores must be"),
    (dict(max_length=51), "scores must be"),
    (dict(kept=z(2, 19)), "kept must be"),
    (dict(kept=z(2, 20, dtype=torch.int64)), "kept must have dtype"),
    (dict(kept_lengths=z(3)), "kept_lengths must be"),
    (dict(), "CUDA tensors"),
])
def test_select_keys_refuses(over, msg):
    with pytest.raises(ValueError, match=msg):
        _select(**over)


def _compact(**over):
    a = dict(kept=z(2, 20), kept_lengths=z(2), lookup_table=z(2, 4), scales_lookup_table=None, layer_idx=0,
             blocks=z(8, 1, 1, 16, 1, 576, dtype=U8), scales=z(8, 1, 1, 16, 1, 1, dtype=F32))
    a.update(over)
    return M.compact_cache(**a)


@pytest.mark.parametrize("over,msg", [
    (dict(kept=z(2, 20, dtype=torch.int64)), "kept must have dtype"),
    (dict(kept=z(3, 20)), "kept must be"),
    (dict(lookup_table=z(3, 4)), "one per request"),
    (dict(blocks=z(8, 1, 1, 16, 1, 576, dtype=F32)), "blocks must have dtype"),
    (dict(scales=z(8, 2, 1, 16, 1, 1, dtype=F32)), "scales must match"),
    (dict(scales=z(7, 1, 1, 16, 1, 1, dtype=F32)), "as many blocks"),
    (dict(scores=z(3, 20, dtype=F32)), "scores must be"),
    (dict(), "CUDA tensors"),
])
def test_compact_cache_refuses(over, msg):
    with pytest.raises(ValueError, match=msg):
        _compact(**over)


def _attend(**over):
    a = dict(q=z(2, 1, 8, 64, dtype=BF16), blocks=z(8, 2, 1, 16, 2, 64, dtype=BF16), scales=None, cache_lengths=z(2),
             lookup_table=z(2, 4), scales_lookup_table=None, max_prompt_length=1, max_cache_length=40, layer_idx=0,
             softmax_scale=0.1)
    a.update(over)
    return M.mha_decode(**a)


@pytest.mark.parametrize("over,msg", [
    (dict(q=z(2, 1, 8, 64, dtype=F32)), "q must have dtype"),
    (dict(q=z(2, 8, 64, dtype=BF16)), "4-D"),
    (dict(q=z(2, 1, 8, 128, dtype=BF16)), "blocks hold"),
    (dict(blocks=z(8, 2, 1, 16, 2, 64, dtype=F32)), "blocks must have dtype"),
    (dict(scales=z(8, 2, 1, 16, 2, 1, dtype=F32)), "takes no scales"),
    (dict(blocks=z(8, 2, 1, 16, 2, 64, dtype=U8)), "scales is required"),
    (dict(blocks=z(8, 2, 1, 16, 2, 64, dtype=U8), scales=z(8, 2, 1, 16, 2, 4, dtype=F32)), "scales must be"),
    (dict(cache_lengths=z(3)), "one per request"),
    (dict(max_prompt_length=2), "number of tokens"),
    (dict(out=z(2, 1, 8, 32, dtype=BF16)), "out must be"),
    (dict(lse=z(2, 1, 4, dtype=F32)), "lse must be"),
    (dict(), "CUDA tensors"),
])
def test_mha_decode_refuses(over, msg):
    with pytest.raises(ValueError, match=msg):
        _attend(**over)


@pytest.mark.parametrize("over,msg", [
    (dict(k=z(2, 1, 2, 64, dtype=F32)), "k must have dtype"),
    (dict(v=z(2, 1, 2, 128, dtype=BF16)), "same shape"),
    (dict(blocks=z(8, 2, 1, 16, 4, 64, dtype=BF16)), "blocks hold"),
    (dict(), "CUDA tensors"),
])
def test_mha_kv_store_refuses(over, msg):
    a = dict(k=z(2, 1, 2, 64, dtype=BF16), v=z(2, 1, 2, 64, dtype=BF16), cache_lengths=z(2), lookup_table=z(2, 4),
             scales_lookup_table=None, layer_idx=0, blocks=z(8, 2, 1, 16, 2, 64, dtype=BF16))
    a.update(over)
    with pytest.raises(ValueError, match=msg):
        M.mha_kv_store(**a)


# ---------------------------------------------------------------- C ABI
FAKE = 0x10000          # aligned, never dereferenced: the checks come first


def shape(**kw):
    base = dict(batch=2, num_q_heads=16, head_dim=576, v_dim=512, num_blocks=16, kv_dim=1, num_layers=1, page_size=16,
                num_kv_heads=1, num_scale_blocks=16, head_dim_granularity=1, max_pages=8)
    base.update(kw)
    return ctypes.byref(_lib.PagedShape(**base))


def _abi_weights(lib, shp, q=FAKE, lse=FAKE, T=1, maxc=64, scale=0.1, scores=FAKE, ss=200, out=FAKE, os=200, ws=FAKE, n=1 << 30):
    return lib.mla_accumulate_weights_fp8(q, lse, FAKE, FAKE, FAKE, FAKE, None, T, maxc, 0, scale, shp, scores, ss, out, os, ws, n,
                                          None)


def test_abi_accumulate(lib):
    ok = shape()
    assert _abi_weights(lib, None) == 1
    assert _abi_weights(lib, ok, q=None) == 1 and _abi_weights(lib, ok, lse=None) == 1 and _abi_weights(lib, ok, out=None) == 1
    assert _abi_weights(lib, ok, q=FAKE + 8) == 1 and _abi_weights(lib, ok, out=FAKE + 2) == 1
    assert _abi_weights(lib, ok, os=64) == 1 and _abi_weights(lib, ok, ss=64) == 1
    assert _abi_weights(lib, ok, scale=float("nan")) == 1
    assert _abi_weights(lib, ok, maxc=200) == 1                    # the page table is too narrow
    assert _abi_weights(lib, shape(head_dim_granularity=9)) == 2
    assert _abi_weights(lib, shape(head_dim=512)) == 2
    assert _abi_weights(lib, shape(batch=0)) == 0                  # no-op before any CUDA call
    n = ctypes.c_uint64(0)
    f = lib.mla_accumulate_workspace_bytes
    assert f(1, shape(), ctypes.byref(n)) == 0 and n.value == 2 * 16 * (2 * 576 + 8)
    assert f(0, shape(), ctypes.byref(n)) == 1 and f(1, None, ctypes.byref(n)) == 1
    assert f(100000, shape(num_q_heads=128), ctypes.byref(n)) == 0 and n.value <= 256 << 20


def test_abi_select(lib):
    f = lambda **k: lib.mla_select_keys(*[{**dict(scores=FAKE, ss=100, lengths=FAKE, batch=2, maxl=100, budget=10, recent=2, sink=1,  # noqa: E731
                                                  kept=FAKE, ks=10, kl=FAKE, st=None), **k}[x]
                                          for x in ("scores", "ss", "lengths", "batch", "maxl", "budget", "recent", "sink", "kept",
                                                    "ks", "kl", "st")])
    assert f(batch=0) == 0
    assert f(batch=-1) == 1 and f(recent=-1) == 1 and f(sink=-1) == 1 and f(budget=0) == 1
    assert f(recent=8, sink=3) == 1 and "exceed the budget" in lib.mla_last_error_string().decode()
    assert f(recent=2 ** 31 - 1, sink=2 ** 31 - 1, budget=2 ** 31 - 1) == 1
    assert f(scores=None) == 1 and f(kept=None) == 1 and f(kl=None) == 1 and f(lengths=None) == 1
    assert f(ss=99) == 1 and f(ks=9) == 1
    assert f(maxl=1 << 30, ss=1 << 31) == 2


def test_abi_compact(lib):
    def f(shp=None, **k):
        a = dict(kept=FAKE, ks=10, mk=10, kl=FAKE, lut=FAKE, slut=None, layer=0, eb=1, blocks=FAKE, scales=FAKE, scores=FAKE, ss=10, sc=10)
        a.update(k)
        return lib.mla_compact_paged(a["kept"], a["ks"], a["mk"], a["kl"], a["lut"], a["slut"], a["layer"], a["eb"],
                                     shp or shape(), a["blocks"], a["scales"], a["scores"], a["ss"], a["sc"], None)
    assert f(shape(batch=0)) == 0
    assert f(kept=None) == 1 and f(blocks=None) == 1 and f(lut=None) == 1 and f(kl=None) == 1
    assert f(blocks=FAKE + 4) == 1 and f(scales=FAKE + 1) == 1
    assert f(mk=0) == 1 and f(mk=11) == 1 and f(eb=4) == 1 and f(layer=1) == 1
    assert f(sc=11) == 1 and f(sc=0) == 1
    assert f(shape(head_dim=24)) == 2 and f(shape(batch=70000)) == 2
    assert f(shape(num_blocks=0)) == 1


def test_abi_mha(lib):
    ok = dict(head_dim=64, v_dim=64, kv_dim=2, num_kv_heads=4)

    def store(eb=2, scales=None, T=1, k=FAKE, blocks=FAKE, layer=0, **s):
        return lib.mla_mha_kv_store(k, FAKE, FAKE, FAKE, None, T, layer, eb, shape(**{**ok, **s}), blocks, scales, None)
    assert store(batch=0) == 0 and store(T=0) == 0
    assert store(k=None) == 1 and store(k=FAKE + 8) == 1 and store(blocks=None) == 1 and store(layer=1) == 1
    assert store(eb=1) == 1 and store(eb=2, scales=FAKE) == 1 and store(eb=3) == 1
    assert store(head_dim=96) == 2 and store(page_size=24) == 2 and store(kv_dim=1) == 1 and store(num_kv_heads=257) == 2
    assert store(eb=1, scales=FAKE, head_dim_granularity=2) == 2

    def attend(q=FAKE, out=FAKE, scale=0.1, T=1, maxc=64, eb=2, scales=None, ws=FAKE, **s):
        return lib.mla_mha_decode_paged(q, FAKE, scales, FAKE, FAKE, None, T, maxc, 0, scale, eb, shape(**{**ok, **s}), out, None,
                                        ws, 0, None)
    assert attend(batch=0) == 0
    assert attend(q=None) == 1 and attend(out=None) == 1 and attend(q=FAKE + 2) == 1 and attend(ws=FAKE + 4) == 1
    assert attend(scale=float("nan")) == 1
    assert attend(batch=0, num_q_heads=6) == 1 and attend(batch=0, T=0) == 1 and attend(batch=0, maxc=128) == 1
    n = ctypes.c_uint64(7)
    f = lib.mla_mha_decode_workspace_bytes
    assert f(1, 64, 2, shape(**ok, batch=0), ctypes.byref(n)) == 0 and n.value == 0
    assert f(1, 64, 2, None, ctypes.byref(n)) == 1


def test_workspace_size_of_the_binding():
    assert M.accumulate_workspace_bytes(2, 1, 16) == 2 * 16 * (2 * 576 + 8)
    with pytest.raises(M.MlaError):
        M.accumulate_workspace_bytes(2, 0, 16)


def test_abi_refuses_partial_overlap(lib):
    """kept_lengths may be lengths, not a shifted view of it; out must not touch q anywhere."""
    def select(kl):
        return lib.mla_select_keys(FAKE, 100, FAKE, 4, 100, 10, 2, 1, FAKE, 10, kl, None)
    for off in (-12, -4, 4, 12):
        assert select(FAKE + off) == 1 and "kept_lengths" in lib.mla_last_error_string().decode()
    nbytes = 2 * 2 * 1 * 16 * 64                                   # of q: batch 2, 16 heads of 64

    def attend(out):
        return lib.mla_mha_decode_paged(FAKE, FAKE, None, FAKE, FAKE, None, 1, 64, 0, 0.1, 2,
                                        shape(head_dim=64, v_dim=64, kv_dim=2, num_kv_heads=4), out, None, FAKE, 0, None)
    for off in (16 - nbytes, -16, 0, 16, nbytes - 16):
        assert attend(FAKE + off) == 1 and "overlap" in lib.mla_last_error_string().decode()
