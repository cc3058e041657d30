"""Accumulated weights on inputs whose products are exact, so that the tolerance is that of the score's last steps.

Every query head has one element that meets non-zero codes: its product with a key's code has 12 significant bits
and its sum over the dims is exact in fp32, whatever the order.  What is left, with z = x - lse the exponent:
the score's factor softmax_scale * s_t is held in two terms, whose sum is exact; two fused multiply-adds (the
score's terms onto -lse), the product with log2 e and the rounding of log2 e itself are at most 2^-24 |z| each,
or, of the first, 2^-24 of what the second term then moves (2^-24 |x|): 2^-48 |x|; the exponential 2^-22; a
key's sum of T * H weights and its old value (T * H + 2) 2^-24 of itself.  Scores are 500 to 1000 here: a
factor, or a score, rounded to 24 bits before it meets the lse is off by 3 to 6e-5 in the weight, 20 times
the tolerance."""
import pytest
import torch

import paged_fp8_kv_mla_b200 as M
from tests.cache_ref import LatentCache, rows_of

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
SCALE = float(torch.tensor(192.0 ** -0.5))


def build(n, H, seed, power=0, depth=0, top=1000):
    """One request of n keys, one new token; scores of half of top to top.  power: q is 2^power, the scales 2^-power times the usual.  depth: each
    row also holds an element 2^depth (in exponents) above the one that counts, where all codes are zero."""
    gen = torch.Generator().manual_seed(seed)
    cache = LatentCache([n], 64, seed=seed)
    blk, slot = rows_of(cache.table, 0, n, 64)
    dims = (torch.arange(H) * 37 + 5) % 575 + 1                  # dim 0 is the large element's
    codes = torch.randint(0x70, 0x7F, (n, 576), generator=gen).to(torch.uint8)   # 128 .. 448
    codes[:, dims] = 0x7E                                         # 448
    codes[:, 0] = 0
    cache.blocks[blk, 0, 0, slot, 0] = codes
    a = (1 + torch.randint(0, 128, (H,), generator=gen) / 128).double()          # 8 significant bits
    s = top / (2 * 448 * SCALE) * (1 + 0.004 * (2 * torch.rand(n, generator=gen) - 1))
    cache.scales[blk, 0, 0, slot, 0, 0] = (s.double() * 2.0 ** -power).float()
    q = torch.zeros((1, 1, H, 576), dtype=torch.float64)
    q[0, 0, torch.arange(H), dims] = a * 2.0 ** power
    if depth:
        q[0, 0, :, 0] = 2.0 ** (power + depth)
    q16 = q.bfloat16()
    assert torch.equal(q16.double(), q)
    return cache, q16, gen


def run(cache, q, lse, n, scores):
    blocks, scales, table, _ = cache.cuda()
    got = M.accumulate_weights(q.cuda(), lse.cuda(), blocks, scales, torch.tensor([n - 1], dtype=torch.int32).cuda(), table, None, 1,
                               n - 1, 0, SCALE, scores.cuda())
    assert M.device_status() == 0
    return got.cpu().double()


@pytest.mark.parametrize("H", [8, 20, 40])
@pytest.mark.parametrize("power,depth", [(0, 0), (100, 0), (-100, 0), (0, 6), (0, 10), (0, 13), (60, 13)])
def test_weights_of_exact_products(H, power, depth):
    n = 300
    cache, q, gen = build(n, H, 7 + H + depth, power, depth)
    keys = cache.keys(0, n)                                       # fp32 codes * scales, in 64 bits
    x = torch.einsum("hd,kd->hk", q[0, 0].double(), keys) * SCALE
    lse = x.amax(1).float() + 0.5
    z = x - lse.double()[:, None]
    w = torch.exp(z)
    rel = 4 * U * z.abs() + 2.0 ** -48 * x.abs() + 2.0 ** -22
    scores = torch.rand((1, n), generator=gen)
    old = scores[0].double().clone()
    old[n - 1] = 0
    total = w.sum(0) + old
    tol = (w * 1.01 * rel).sum(0) + (H + 2) * U * total
    got = run(cache, q, lse[None, None], n, scores)[0]
    bad = ~((got - total).abs() <= tol)
    assert not bad.any(), (bad.nonzero()[:5].T, got[bad][:5], total[bad][:5], tol[bad][:5])


@pytest.mark.parametrize("depth", [14, 16, 18])
def test_elements_far_below_their_rows_largest(depth):
    """An element below 2^-13 of its row's largest is off by at most 2^-21 of that.  With scores of 0.015 to 0.03 this
    moves a weight by 0.02 % (2^-14) to 0.4 % (2^-18); an element that is lost moves it by 3 %."""
    n, H = 200, 16
    cache, q, gen = build(n, H, 40 + depth, 0, depth, top=0.03)
    x = torch.einsum("hd,kd->hk", q[0, 0].double(), cache.keys(0, n)) * SCALE
    lse = torch.full((H,), 0.5)
    z = x - lse.double()[:, None]
    w = torch.exp(z)
    a = q[0, 0].double().abs().sort(1).values[:, -2:-1]           # the element that counts
    rel = 4 * U * z.abs() + 2.0 ** -22 + 2.0 ** (depth - 21) * x.abs() / a
    scores = torch.rand((1, n), generator=gen)
    old = scores[0].double().clone()
    old[n - 1] = 0
    total = w.sum(0) + old
    tol = (w * 1.01 * rel).sum(0) + (H + 2) * U * total
    got = run(cache, q, lse[None, None], n, scores)[0]
    bad = ~((got - total).abs() <= tol)
    assert not bad.any(), (bad.nonzero()[:5].T, got[bad][:5], total[bad][:5], tol[bad][:5])


@pytest.mark.parametrize("value", [float("nan"), float("inf"), float("-inf")])
def test_a_row_whose_lse_is_minus_infinity_adds_nothing_whatever_it_holds(value):
    """A padded query token: q was never written, and its lse says that it attends to nothing."""
    n, H = 200, 16
    cache, q, gen = build(n, H, 3)
    lse = torch.full((1, 1, H), 1000.0)
    scores = torch.rand((1, n), generator=gen)
    lse[0, 0, 4] = lse[0, 0, 9] = float("-inf")
    want = run(cache, q, lse, n, scores)
    q[0, 0, 4, 7] = value
    q[0, 0, 9] = value
    assert torch.equal(run(cache, q, lse, n, scores), want)
