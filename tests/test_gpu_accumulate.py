"""Accumulated attention weights of the latent cache against the definition in 64 bits.

Tolerance, per key, from the roundings of one weight exp(x - lse): the fp32 sum of 576 products (at
most 576 + 8 roundings of 2^-24 of the sum of magnitudes A), the roundings of the exponent's terms
(|x|, |lse|: 4 of 2^-24 each), q elements below 2^-10 of their row's largest (off by 2^-17 of it
against 2^-10: counted as 2^-17 max|q| sum |k|), 2^-21 for the exponential itself; then one rounding
of 2^-24 per addend of the key's sum.  The exponential flushes results below the smallest normal number
to 0, so each of the T * H addends may lack up to 2^-126."""
import pytest
import torch

import paged_fp8_kv_mla_b200 as M
from tests.cache_ref import LatentCache, latent_scores

pytestmark = pytest.mark.gpu

SCALE = float(torch.tensor(192.0 ** -0.5))
U = 2.0 ** -24


def make(lengths, T, H, page, seed=0, q_mul=1.0, **kw):
    cache = LatentCache([n + T for n in lengths], page, seed=seed, **kw)
    gen = torch.Generator().manual_seed(seed + 100)
    q = (torch.randn((len(lengths), T, H, 576), generator=gen) * q_mul).bfloat16()
    width = max(lengths) + T
    scores = torch.rand((len(lengths), width), generator=gen)
    return cache, q, scores


def reference(cache, q, scores, lengths, lse=None):
    """(lse, out, tolerance) in 64 bits; entries behind a request's keys are NaN."""
    B, T, H, _ = q.shape
    out, tol = torch.full(scores.shape, float("nan")).double(), torch.full(scores.shape, float("nan")).double()
    lses = torch.zeros((B, T, H)) if lse is None else lse
    for b, L in enumerate(lengths):
        n = L + T
        k = cache.keys(b, n)
        x = latent_scores(q[b], k, L, SCALE)
        if lse is None:
            lses[b] = x.logsumexp(-1).float()
        ls = lses[b].double()[..., None]
        w = torch.exp(x - ls)
        w[ls.expand_as(w) == float("-inf")] = 0
        amp = torch.einsum("thd,kd->thk", q[b].double().abs(), k.abs()) * SCALE
        small = q[b].double().abs().amax(-1)[..., None] * k.abs().sum(-1) * SCALE * 2.0 ** -17
        xx = x.masked_fill(x == float("-inf"), 0.0).abs()
        rel = (584 * U * amp + small + 8 * U * (xx + ls.abs().nan_to_num(posinf=0)) + 2.0 ** -21)
        total = w.sum((0, 1))
        old = torch.zeros(n).double()
        old[:L] = scores[b, :L].double()
        out[b, :n] = total + old
        tol[b, :n] = (w * rel).sum((0, 1)) + (T * H + 2) * U * (total + old.abs()) + T * H * 2.0 ** -126
    return lses, out, tol


def run(cache, q, lse, lengths, scores, out=None, **kw):
    blocks, scales, table, stable = cache.cuda()
    T = q.shape[1]
    got = M.accumulate_weights(q.cuda(), lse.cuda(), blocks, scales, torch.tensor(lengths, dtype=torch.int32).cuda(), table,
                               stable, T, max(lengths), cache.layer, SCALE, scores, out=out, **kw)
    assert M.device_status() == 0
    return got


def check(got, want, tol, before):
    got = got.cpu().double()
    past = want.isnan()
    assert torch.equal(got[past].float(), before[past])            # behind the request's keys: as it was
    bad = ~((got - want).abs() <= tol) & ~past
    assert not bad.any(), (bad.nonzero()[:5], got[bad][:5], want[bad][:5], tol[bad][:5])


@pytest.mark.parametrize("lengths,T,H,page", [
    ([0], 1, 1, 16), ([1], 1, 8, 16), ([36, 63], 1, 16, 16), ([127], 1, 128, 64), ([128], 1, 128, 64), ([126, 255, 0, 17], 2, 128, 64),
    ([300, 5, 700], 1, 20, 48), ([1000], 3, 100, 32), ([2047, 1], 1, 136, 64), ([513, 64, 200], 2, 300, 128), ([40, 900], 5, 7, 80),
    ([130, 1, 2], 140, 16, 64),
])
def test_against_64_bits(lengths, T, H, page):
    cache, q, scores = make(lengths, T, H, page)
    lse, want, tol = reference(cache, q, scores, lengths)
    out = torch.full(scores.shape, -7.0)
    check(run(cache, q, lse, lengths, scores.cuda(), out=out.cuda()), want, tol, out)


@pytest.mark.parametrize("kw", [dict(layers=3, layer=1), dict(kv_dim=2), dict(own_scale_pages=True), dict(spread=6.0)])
def test_cache_layouts(kw):
    lengths = [200, 77, 390]
    cache, q, scores = make(lengths, 1, 32, 32, seed=3, **kw)
    lse, want, tol = reference(cache, q, scores, lengths)
    check(run(cache, q, lse, lengths, scores.cuda()), want, tol, scores)   # in place


@pytest.mark.parametrize("q_mul", [1e-30, 1e-3, 30.0, 1e30])
def test_q_of_any_size(q_mul):
    """q's rows are scaled by a power of two each: sizes far from 1 lose nothing.  (Every row's softmax is
    then one-hot or uniform; the lse is the formula's.)"""
    lengths = [150, 260]
    cache, q, scores = make(lengths, 1, 16, 64, seed=5, q_mul=q_mul)
    if q_mul > 1e3:   # scores near 1e30: compare on keys' own terms with an lse that keeps exp finite
        lse = torch.full((2, 1, 16), float("inf"))
        want = reference(cache, q, scores, lengths, lse=lse)[1]
        got = run(cache, q, lse, lengths, scores.cuda()).cpu()
        ok = ~want.isnan()
        assert torch.equal(got[ok].double(), want[ok])
        return
    lse, want, tol = reference(cache, q, scores, lengths)
    check(run(cache, q, lse, lengths, scores.cuda()), want, tol, scores)


def test_rows_of_mixed_size_in_q():
    """A row whose elements span many powers of two, and an all-zero row."""
    lengths = [140]
    cache, q, scores = make(lengths, 1, 16, 64, seed=6)
    q[0, 0, 3] = (q[0, 0, 3].float() * torch.exp2(torch.arange(576) % 24 - 20.0)).bfloat16()
    q[0, 0, 4] = 0
    lse, want, tol = reference(cache, q, scores, lengths)
    check(run(cache, q, lse, lengths, scores.cuda()), want, tol, scores)


def test_empty_rows_and_no_scores():
    """A row with lse = -inf adds nothing; scores=None starts every key at 0."""
    lengths = [140, 33]
    cache, q, scores = make(lengths, 2, 24, 16, seed=7)
    lse, _, _ = reference(cache, q, scores, lengths)
    lse[0, 1] = float("-inf")
    lse[1, :, 5] = float("-inf")
    zero = torch.zeros_like(scores)
    _, want, tol = reference(cache, q, zero, lengths, lse=lse)
    check(run(cache, q, lse, lengths, None), want, tol, zero)


def test_non_finite_values_stay_where_they_belong():
    lengths = [140, 90]
    cache, q, scores = make(lengths, 1, 16, 16, seed=8)
    lse, want, tol = reference(cache, q, scores, lengths)
    blk, slot = cache.table[0, 37 // 16], 37 % 16
    cache.blocks[blk, 0, 0, slot, 0, 100] = 127                    # a NaN code: its own key only
    got = run(cache, q, lse, lengths, scores.cuda()).cpu()
    assert got[0, 37].isnan() and int(got.isnan().sum()) == 1
    want[0, 37] = tol[0, 37] = float("nan")
    got[0, 37] = scores[0, 37]
    check(got, want, tol, scores)
    cache.blocks[blk, 0, 0, slot, 0, 100] = 0
    q[1, 0, 2, 9] = float("inf")                                   # a non-finite q row: its own request
    got = run(cache, q, lse, lengths, scores.cuda()).cpu()
    assert got[1, :91].isnan().all() and not got[0].isnan().any()


def test_strided_scores_and_a_longer_launch_bound():
    """Rows of a wider buffer, and max_cache_length above every length."""
    lengths = [100, 333, 1]
    cache, q, scores = make(lengths, 1, 64, 64, seed=9)
    lse, want, tol = reference(cache, q, scores, lengths)
    wide = torch.full((3, 700), -3.0)
    wide[:, 50:50 + scores.shape[1]] = scores
    dev = wide.cuda()
    blocks, scales, table, stable = cache.cuda()
    view = dev[:, 50:400]
    M.accumulate_weights(q.cuda(), lse.cuda(), blocks, scales, torch.tensor(lengths, dtype=torch.int32).cuda(), table, stable, 1,
                         340, 0, SCALE, view)
    assert M.device_status() == 0
    got = dev.cpu()
    keep = got.clone()
    keep[:, 50:50 + scores.shape[1]] = -3.0
    assert (keep == -3.0).all()
    check(got[:, 50:50 + scores.shape[1]], want, tol, scores)


def test_same_result_every_time_and_with_the_decode():
    """Deterministic; with the scale-folding decode's lse the weights of a row sum to 1."""
    lengths = [1500, 3, 800]
    cache, q, scores = make(lengths, 1, 128, 64, seed=10)
    blocks, scales, table, stable = cache.cuda()
    lens = torch.tensor(lengths, dtype=torch.int32).cuda()
    _, lse = M.decode(q.cuda(), blocks, scales, lens, table, stable, 1, 1500, 0, SCALE, fold_scales=True)
    args = (q.cuda(), lse, blocks, scales, lens, table, stable, 1, 1500, 0, SCALE)
    first = M.accumulate_weights(*args)
    for _ in range(5):
        assert torch.equal(M.accumulate_weights(*args), first)
    assert M.device_status() == 0
    assert (first.double().sum(1).cpu() - 128).abs().max() < 128 * 1e-4


def test_bad_page_and_length_are_flagged_and_skipped():
    lengths = [200, 100]
    cache, q, scores = make(lengths, 1, 16, 64, seed=11)
    lse, want, tol = reference(cache, q, scores, lengths)
    cache.table[0, 1] = 100000
    blocks, scales, table, stable = cache.cuda()
    out = torch.full(scores.shape, -7.0)
    got = M.accumulate_weights(q.cuda(), lse.cuda(), blocks, scales, torch.tensor(lengths, dtype=torch.int32).cuda(), table,
                               stable, 1, 200, 0, SCALE, scores.cuda(), out=out.cuda())
    assert M.device_status() == 6
    want[0, 64:128] = float("nan")
    check(got, want, tol, out)
    got = M.accumulate_weights(q.cuda(), lse.cuda(), blocks, scales, torch.tensor([63, 300], dtype=torch.int32).cuda(), table,
                               stable, 1, 100, 0, SCALE, scores.cuda(), out=out.cuda())
    assert M.device_status() == 6                                  # 300 is read as 100
    check(got[1:], want[1:], tol[1:], out[1:])


def test_graph_capture_and_another_stream():
    lengths = [700, 260]
    cache, q, scores = make(lengths, 1, 128, 64, seed=12)
    lse, want, tol = reference(cache, q, scores, lengths)
    blocks, scales, table, stable = cache.cuda()
    lens, qd, ld, sd = torch.tensor(lengths, dtype=torch.int32).cuda(), q.cuda(), lse.cuda(), scores.cuda()
    out = torch.full(scores.shape, -7.0).cuda()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    M.accumulate_weights(qd, ld, blocks, scales, lens, table, stable, 1, 700, 0, SCALE, sd, out=out, stream=side)
    side.synchronize()
    check(out, want, tol, torch.full(scores.shape, -7.0))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        M.accumulate_weights(qd, ld, blocks, scales, lens, table, stable, 1, 700, 0, SCALE, sd, out=out)
    out.fill_(-7.0)
    graph.replay()
    torch.cuda.synchronize()
    check(out, want, tol, torch.full(scores.shape, -7.0))


def test_a_step_of_many_tokens_runs_in_several_launches():
    """More split query tokens than the workspace holds at once (256 MB): the sums carry on from launch to
    launch.  64-bit sums on the GPU."""
    lengths, T, H = [40, 0, 130, 300, 7, 260, 90, 129], 300, 128
    assert M.accumulate_workspace_bytes(8, T, H) < 8 * T * H * (2 * 576 + 8)
    cache, q, scores = make(lengths, T, H, 64, seed=13)
    blocks, scales, table, stable = cache.cuda()
    lse = torch.empty((8, T, H)).cuda()
    want, tol = torch.zeros(scores.shape).double(), torch.zeros(scores.shape).double()
    for b, L in enumerate(lengths):
        k, qq = cache.keys(b, L + T).cuda(), q[b].double().cuda()
        x = torch.einsum("thd,kd->thk", qq, k) * SCALE
        late = torch.arange(L + T, device="cuda")[None] > L + torch.arange(T, device="cuda")[:, None]
        x = x.masked_fill(late[:, None], float("-inf"))
        lse[b] = x.logsumexp(-1)
        w = torch.exp(x - lse[b].double()[..., None])
        amp = torch.einsum("thd,kd->thk", qq.abs(), k.abs()) * SCALE
        rel = 584 * U * amp + 8 * U * (x.masked_fill(late[:, None], 0).abs() + lse[b].abs()[..., None]) + 2.0 ** -20
        rel = rel + qq.abs().amax(-1)[..., None] * k.abs().sum(-1) * SCALE * 2.0 ** -17
        want[b, :L + T] = w.sum((0, 1)).cpu()
        want[b, :L] += scores[b, :L].double()
        tol[b, :L + T] = (w * rel).sum((0, 1)).cpu() + (T * H + 2) * U * want[b, :L + T] + T * H * 2.0 ** -126
    got = M.accumulate_weights(q.cuda(), lse, blocks, scales, torch.tensor(lengths, dtype=torch.int32).cuda(), table, stable, T,
                               max(lengths), 0, SCALE, scores.cuda(), out=torch.zeros(scores.shape).cuda()).cpu().double()
    assert M.device_status() == 0
    assert ((got - want).abs() <= tol).all()


def test_out_beside_scores_and_overlaps_refused():
    """out and scores as column ranges of one buffer; a partial overlap is refused, an empty batch is fine."""
    lengths = [50, 20]
    cache, q, scores = make(lengths, 1, 8, 16, seed=14)
    lse, want, tol = reference(cache, q, scores, lengths)
    wide = torch.zeros((2, 110)).cuda()
    wide[:, :51] = scores.cuda()
    wide[:, 51:] = -7.0
    run(cache, q, lse, lengths, wide[:, :51], out=wide[:, 51:102])
    check(wide[:, 51:102], want, tol, torch.full((2, 51), -7.0))
    assert torch.equal(wide[:, :51].cpu(), scores) and (wide[:, 102:] == -7.0).all()
    with pytest.raises(ValueError, match="overlap"):
        run(cache, q, lse, lengths, wide[:, :51], out=wide[:, 30:81])
    blocks, scales, table, stable = cache.cuda()
    none = M.accumulate_weights(q[:0].cuda(), lse[:0].cuda(), blocks, scales, torch.zeros(0, dtype=torch.int32).cuda(), table[:0],
                                stable, 1, 50, 0, SCALE)
    assert none.shape == (0, 51)
