"""Multi-head decode: a query row's result is right whatever the rows beside it hold.

The rows that share a kv head (tokens of a step and heads of a group) are computed side by side in one
warp.  Tolerances are those of test_gpu_mha.check, whose terms are the row's own."""
import pytest
import torch

import paged_fp8_kv_mla_b200 as M
from tests.test_gpu_mha import check, make, run

pytestmark = pytest.mark.gpu

# lengths, T, H, HKV, D, page: 4, 8, 16 and 24 rows a kv head, steps of 16, 32 and 64 keys, requests cut in pieces
SHAPES = [([60, 33], 1, 8, 2, 64, 16), ([300, 40], 1, 16, 2, 128, 64), ([700, 90], 2, 16, 2, 64, 64), ([500, 31], 2, 16, 2, 128, 32),
          ([6000, 5], 3, 16, 2, 128, 64), ([5000], 2, 8, 8, 64, 128), ([200], 12, 2, 1, 128, 16)]


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("lengths,T,H,HKV,D,page", SHAPES)
def test_non_finite_rows_stay_by_themselves(lengths, T, H, HKV, D, page, fp8):
    cache, q = make(lengths, T, H, HKV, D, page, fp8, seed=61)
    bad = torch.zeros(q.shape[:3], dtype=torch.bool)
    bad[0, T - 1, 1] = bad[0, 0, H - 1] = True
    dirty = q.clone()
    dirty[0, T - 1, 1, 5] = float("nan")
    dirty[0, 0, H - 1, D - 1] = float("inf")
    if T > 1:                                                     # a token that was never written
        bad[-1, T - 1] = True
        dirty[-1, T - 1] = float("nan")
    clean, clean_lse = run(cache, q, lengths, D ** -0.5)
    out, lse = run(cache, dirty, lengths, D ** -0.5)
    gone = bad.cuda()
    assert out[gone].isnan().all() and lse[gone].isnan().all()
    out[gone], lse[gone] = clean[gone], clean_lse[gone]           # (check wants every row)
    check(cache, q, lengths, D ** -0.5, out, lse)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("power", [24, 40, 100])
@pytest.mark.parametrize("lengths,T,H,HKV,D,page", SHAPES[1:5])
def test_rows_beside_much_larger_ones(lengths, T, H, HKV, D, page, power, fp8):
    """Every third row 2^power times the others: those lose nothing by it.  (The scores of the large ones are
    known to no digit at the larger powers: their tolerance says so.)"""
    cache, q = make(lengths, T, H, HKV, D, page, fp8, seed=62)
    rows = q.view(-1, D)
    rows[::3] *= 2.0 ** power
    out, lse = run(cache, q, lengths, D ** -0.5)
    check(cache, q, lengths, D ** -0.5, out, lse)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("lengths,T,H,HKV,D,page", [([0], 300, 4, 1, 64, 16), ([70, 3], 130, 16, 2, 128, 64)])
def test_prompts(lengths, T, H, HKV, D, page, fp8):
    """More rows than a CTA takes: several row groups, whose masks end in different tiles."""
    cache, q = make(lengths, T, H, HKV, D, page, fp8, seed=63)
    out, lse = run(cache, q, lengths, D ** -0.5)
    check(cache, q, lengths, D ** -0.5, out, lse)
    assert M.device_status() == 0
