"""Numbers that the C types of the cache operators' calls do not hold are refused, not wrapped: 2**32 + 20 keys to keep
is not 20.  (CPU tensors: without the check the call goes on to the test of the device.)"""
import pytest
import torch

import paged_fp8_kv_mla_b200 as M
from tests.test_cache_ops_cpu import BF16, U8, _attend, _compact, _select, _weights, z

WIDE = [2 ** 31, 2 ** 32, 2 ** 32 + 20, 2 ** 63, -2 ** 31 - 1, -2 ** 32 + 20]


@pytest.mark.parametrize("value", WIDE)
@pytest.mark.parametrize("call,name", [
    (_weights, "layer_idx"), (_attend, "layer_idx"), (_attend, "max_cache_length"), (_compact, "layer_idx"),
    (_select, "budget"), (_select, "num_recent"), (_select, "num_sink"),
])
def test_wide_numbers_are_refused(call, name, value):
    extra = dict(kept=z(2, 50), max_length=50) if call is _select else {}
    with pytest.raises(ValueError, match=name):
        call(**{name: value, **extra})


@pytest.mark.parametrize("value", [-2 ** 32 + 20, -2 ** 31 - 1])
@pytest.mark.parametrize("call,name", [(_weights, "max_cache_length"), (_select, "max_length")])
def test_lengths_that_no_row_bounds_are_refused(call, name, value):
    with pytest.raises(ValueError, match=name):
        call(**{name: value})


@pytest.mark.parametrize("value", WIDE)
def test_store_refuses_a_wide_layer(value):
    k = z(2, 1, 2, 64, dtype=BF16)
    with pytest.raises(ValueError, match="layer_idx"):
        M.mha_kv_store(k, k, z(2), z(2, 4), None, value, z(8, 2, 1, 16, 2, 64, dtype=U8).view(torch.float8_e4m3fn),
                       z(8, 2, 1, 16, 2, 1, dtype=torch.float32))


def test_numbers_that_fit_go_on():
    for call, name in ((_select, "budget"), (_select, "num_recent"), (_attend, "max_cache_length"), (_compact, "layer_idx")):
        for value in (0, -1, 2 ** 31 - 1):                        # left to the library, which says what is wrong with them
            extra = dict(kept=z(2, 50)) if call is _select else {}
            with pytest.raises(ValueError, match="CUDA tensors"):
                call(**{name: value, **extra})


@pytest.mark.parametrize("value", WIDE)
def test_workspace_query_refuses(value):
    for sizes, name in (((value, 1, 16), "batch"), ((2, value, 16), "max_prompt_length"), ((2, 1, value), "num_q_heads")):
        with pytest.raises(ValueError, match=name):
            M.accumulate_workspace_bytes(*sizes)
