"""Key selection and cache compaction: exact results against the definitions, one key and one row at a time."""
import pytest
import torch

import paged_fp8_kv_mla_b200 as M
from tests.cache_ref import LatentCache, MhaCache, rows_of, select_reference

pytestmark = pytest.mark.gpu


def weights(B, n, seed, kind):
    gen = torch.Generator().manual_seed(seed)
    x = torch.exp(2 * torch.randn((B, n), generator=gen))
    if kind == "ties":
        x = (x * 4).round() / 4
    elif kind == "equal":
        x = torch.full((B, n), 0.25)
    elif kind == "zeros":
        x = torch.where(torch.rand((B, n), generator=gen) < 0.9, torch.zeros(()), x)
        x = torch.where(torch.rand((B, n), generator=gen) < 0.5, -x, x)      # -0 among them, and negative numbers
    elif kind == "odd":
        r = torch.rand((B, n), generator=gen)
        x = torch.where(r < 0.2, torch.tensor(float("nan")), x)
        x = torch.where((r > 0.2) & (r < 0.3), torch.tensor(float("inf")), x)
        x = torch.where((r > 0.3) & (r < 0.4), torch.tensor(float("-inf")), x)
        x = torch.where((r > 0.4) & (r < 0.5), torch.tensor(1e-42), x)
    return x


@pytest.mark.parametrize("kind", ["plain", "ties", "equal", "zeros", "odd"])
@pytest.mark.parametrize("lengths,budget,recent,sink", [
    ([1], 1, 0, 0), ([0, 1, 2, 3], 2, 1, 1), ([5, 9, 33], 8, 3, 1), ([700, 40, 2047, 1024], 256, 64, 4), ([4096, 4097], 1000, 0, 0),
    ([300, 301], 300, 0, 300), ([300, 301], 300, 300, 0), ([9000, 20000, 1], 4096, 1000, 4), ([2049], 2048, 0, 0), ([513], 1, 0, 0),
])
def test_select(lengths, budget, recent, sink, kind):
    top = max(lengths)
    x = weights(len(lengths), top, 17 + top, kind)
    kept = torch.full((len(lengths), budget), -5, dtype=torch.int32).cuda()
    got, count = M.select_keys(x.cuda(), torch.tensor(lengths, dtype=torch.int32).cuda(), top, budget, recent, sink, kept=kept)
    assert M.device_status() == 0
    assert got.data_ptr() == kept.data_ptr()
    got = got.cpu()
    for b, n in enumerate(lengths):
        want = select_reference(x[b].tolist(), n, budget, recent, sink)
        assert int(count[b]) == len(want) == min(n, budget)
        assert got[b, :len(want)].tolist() == want
        assert (got[b, len(want):] == -5).all()


def test_select_more_keys_than_a_cluster_holds():
    """Past some 300 000 keys a CTA reads part of its keys again instead of holding them."""
    n, budget = 400_001, 100_000
    x = weights(1, n, 3, "ties")
    got, count = M.select_keys(x.cuda(), torch.tensor([n], dtype=torch.int32).cuda(), n, budget, 7, 3)
    assert M.device_status() == 0 and int(count) == budget
    order = torch.sort(x[0, 3:n - 7], descending=True, stable=True).indices[:budget - 10] + 3
    want = torch.cat([torch.arange(3), order.sort().values, torch.arange(n - 7, n)])
    assert torch.equal(got[0].cpu().long(), want)


@pytest.mark.parametrize("B,n", [(1, 700_001), (9, 330_000), (7, 66_000), (8, 66_000)])
def test_select_long_requests(B, n):
    """Clusters of 8 and 16, with all keys held and with some read again."""
    x = weights(B, n, 5, "ties")
    lengths = torch.tensor([n - 17 * b for b in range(B)], dtype=torch.int32)
    got, count = M.select_keys(x.cuda(), lengths.cuda(), n, n // 3, 9, 2)
    assert M.device_status() == 0 and (count == n // 3).all()
    for b, m in enumerate(lengths.tolist()):
        order = torch.sort(x[b, 2:m - 9], descending=True, stable=True).indices[:n // 3 - 11] + 2
        want = torch.cat([torch.arange(2), order.sort().values, torch.arange(m - 9, m)])
        assert torch.equal(got[b].cpu().long(), want)


def test_select_strided_rows_many_requests_and_a_long_length():
    B = 300
    x = weights(B, 200, 5, "ties")
    lengths = torch.randint(1, 150, (B,), generator=torch.Generator().manual_seed(1), dtype=torch.int32)
    lengths[7] = 180                                             # above max_length: read as 160, flagged
    wide_kept = torch.full((B, 90), -1, dtype=torch.int32).cuda()
    got, count = M.select_keys(x.cuda()[:, 20:], lengths.cuda(), 160, 40, 8, 2, kept=wide_kept[:, 10:60])
    assert M.device_status() == 6
    whole = wide_kept.cpu()
    assert (whole[:, :10] == -1).all() and (whole[:, 50:] == -1).all()
    for b in range(B):
        want = select_reference(x[b, 20:].tolist(), min(int(lengths[b]), 160), 40, 8, 2)
        assert whole[b, 10:10 + len(want)].tolist() == want and int(count[b]) == len(want)


@pytest.mark.parametrize("top", [300, 5000, 70000])
def test_select_writes_the_lengths_in_place(top):
    """kept_lengths may be lengths itself, for clusters of every size; a batch of nothing is fine."""
    lengths = [top, 5, top // 2, top - 1]
    x = weights(4, top, 9, "plain")
    lens = torch.tensor(lengths, dtype=torch.int32).cuda()
    for _ in range(3):
        now = lens.clone()
        kept, same = M.select_keys(x.cuda(), now, top, 100, 10, 2, kept_lengths=now)
        assert same is now and M.device_status() == 0
        for b, n in enumerate(lengths):
            want = select_reference(x[b].tolist(), n, 100, 10, 2)
            assert kept[b, :int(now[b])].tolist() == want
    kept, count = M.select_keys(x.cuda()[:0], lens[:0], top, 100)
    assert kept.shape == (0, 100) and count.shape == (0,)
    kept, count = M.select_keys(torch.zeros((2, 0)).cuda(), torch.zeros(2, dtype=torch.int32).cuda(), 0, 8)
    assert count.tolist() == [0, 0] and M.device_status() == 0


def check_compact(cache, kept, scores, **call):
    """Moves on the GPU and compares every byte of the pool with the definition."""
    blocks, scales = cache.blocks.clone(), None if cache.scales is None else cache.scales.clone()
    stable = cache.table if cache.stable is None else cache.stable
    want_scores = scores.clone()
    for b, ks in enumerate(kept):
        if not ks:
            continue
        dst = list(range(len(ks)))
        for store, before, table in ((blocks, cache.blocks, cache.table), (scales, cache.scales, stable)):
            if store is not None:
                blk, slot = rows_of(table, b, max(ks) + 1, cache.page)
                store[blk[dst], :, cache.layer, slot[dst]] = before[blk[ks], :, cache.layer, slot[ks]]
        want_scores[b, dst] = scores[b, ks]
    width = max(1, max(len(ks) for ks in kept))
    kt = torch.full((len(kept), width), 12345678, dtype=torch.int32)
    for b, ks in enumerate(kept):
        kt[b, :len(ks)] = torch.tensor(ks, dtype=torch.int32)
    db, ds, table, st = cache.cuda()
    sc = scores.cuda()
    M.compact_cache(kt.cuda(), torch.tensor([len(ks) for ks in kept], dtype=torch.int32).cuda(), table, st, cache.layer, db, ds, sc)
    assert M.device_status() == 0
    as_bytes = lambda t: t.contiguous().view(torch.uint8)  # noqa: E731 (NaN scales compare as bytes)
    assert torch.equal(as_bytes(db.cpu()), as_bytes(blocks))
    if scales is not None:
        assert torch.equal(as_bytes(ds.cpu()), as_bytes(scales))
    assert torch.equal(as_bytes(sc.cpu()), as_bytes(want_scores))


def pick(n, k, seed):
    return sorted(torch.randperm(n, generator=torch.Generator().manual_seed(seed))[:k].tolist())


@pytest.mark.parametrize("lengths,keep,page,kw", [
    ([1], 1, 16, {}), ([2, 40, 17], 1, 16, {}), ([300, 20, 5], 100, 48, dict(layers=2, layer=1)), ([1000, 1500], 700, 64, dict(kv_dim=2)),
    ([5000], 3000, 32, dict(own_scale_pages=True)), ([2000] * 20, 1000, 64, {}), ([64] * 40, 63, 16, dict(own_scale_pages=True, layers=3, layer=2)),
])
def test_compact_latent(lengths, keep, page, kw):
    cache = LatentCache(lengths, page, seed=sum(lengths), **kw)
    if kw.get("kv_dim"):
        cache.blocks[:, 1] = torch.randint(0, 256, cache.blocks[:, 1].shape, generator=torch.Generator().manual_seed(1)).to(torch.uint8)
    kept = [pick(n, min(n, keep), 31 + b) for b, n in enumerate(lengths)]
    check_compact(cache, kept, torch.rand((len(lengths), max(lengths)), generator=torch.Generator().manual_seed(2)))


def test_compact_edge_lists():
    """Nothing kept, everything kept, only the tail, only the head, every second key."""
    cache = LatentCache([777, 777, 777, 777, 777], 16, seed=4)
    kept = [[], list(range(777)), list(range(700, 777)), list(range(50)), list(range(1, 777, 2))]
    check_compact(cache, kept, torch.rand((5, 777), generator=torch.Generator().manual_seed(2)))


@pytest.mark.parametrize("fp8,heads,dim", [(False, 2, 64), (False, 8, 128), (True, 1, 64), (True, 5, 64), (True, 8, 128)])
def test_compact_multi_head(fp8, heads, dim):
    lengths = [600, 33, 250]
    cache = MhaCache(lengths, 32, heads, dim, fp8, seed=6, layers=2, layer=1, own_scale_pages=True)
    check_compact(cache, [pick(n, n // 2 + 1, 7) for n in lengths], torch.rand((3, 600), generator=torch.Generator().manual_seed(2)))


def test_compact_without_scales_or_scores():
    cache = LatentCache([100], 16, seed=8)
    db, ds, table, _ = cache.cuda()
    kept = torch.arange(1, 100, 2, dtype=torch.int32)[None].cuda()
    n = torch.tensor([50], dtype=torch.int32).cuda()
    before = ds.clone()
    M.compact_cache(kept, n, table, None, 0, db, None)
    assert M.device_status() == 0
    assert torch.equal(ds.view(torch.int32), before.view(torch.int32))
    blk, slot = rows_of(cache.table, 0, 100, 16)
    assert torch.equal(db.cpu()[blk[:50], 0, 0, slot[:50]], cache.blocks[blk[1::2], 0, 0, slot[1::2]])


def test_compact_bad_lists_are_flagged_and_skipped():
    """Sources without a page, below their position, or past the weights' row; the other rows move."""
    cache = LatentCache([100], 16, seed=9)
    db, ds, table, _ = cache.cuda()
    scores = torch.arange(80.0)[None].cuda()
    kept = torch.tensor([[3, 0, 5, 90, 100000, -4, 99]], dtype=torch.int32).cuda()
    M.compact_cache(kept, torch.tensor([7], dtype=torch.int32).cuda(), table, None, 0, db, ds, scores)
    assert M.device_status() == 6
    blk, slot = rows_of(cache.table, 0, 100, 16)
    got, old = db.cpu()[blk, 0, 0, slot], cache.blocks[blk, 0, 0, slot]
    for j, src in enumerate([3, 1, 5, 90, 4, 5, 99]):
        assert torch.equal(got[j], old[src]), j
    assert scores[0, :7].tolist() == [3, 1, 5, 3, 4, 5, 6]
    M.compact_cache(kept, torch.tensor([8], dtype=torch.int32).cuda(), table, None, 0, db, ds)   # more than kept has
    assert M.device_status() == 6
