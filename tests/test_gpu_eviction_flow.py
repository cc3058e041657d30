"""The cache operators as a serving loop uses them: store, attend, accumulate, and now and then select and
compact, with the attention over what was kept checked against 64 bits after every step."""
import pytest
import torch

import paged_fp8_kv_mla_b200 as M
from tests.cache_ref import E4M3, MhaCache, latent_scores, mha_reference, page_table, rows_of, select_reference

pytestmark = pytest.mark.gpu

SCALE = float(torch.tensor(192.0 ** -0.5))


@pytest.mark.parametrize("own_scale_pages", [False, True])
def test_latent_cache_under_a_budget(own_scale_pages):
    B, H, page, layers, budget, recent, sink = 3, 16, 16, 2, 96, 16, 4
    lengths = [70, 130, 5]
    gen = torch.Generator().manual_seed(1)
    room = [n + 12 for n in lengths]
    table, nb = page_table(room, page, 3, gen)
    stable, nsb = page_table(room, page, 5, gen) if own_scale_pages else (None, nb)
    blocks = torch.full((nb, 1, layers, page, 1, 576), 127, dtype=torch.uint8).cuda()
    scales = torch.full((nsb, 1, layers, page, 1, 1), float("nan")).cuda()
    td, sd = table.cuda(), None if stable is None else stable.cuda()
    width = max(room)
    scores = [torch.full((B, width), float("nan")).cuda() for _ in range(layers)]
    lens = torch.zeros(B, dtype=torch.int32).cuda()

    def rows(b, n, layer):
        blk, slot = rows_of(table, b, n, page)
        sblk = blk if stable is None else rows_of(stable, b, n, page)[0]
        return E4M3[blocks.cpu()[blk, 0, layer, slot, 0].int()] * scales.cpu()[sblk, 0, layer, slot, 0].double()

    # the prompts, written in one step of as many tokens as the longest, shorter ones on top of themselves
    for layer in range(layers):
        for b, n in enumerate(lengths):
            x = torch.randn((1, n, 576), generator=gen).bfloat16().cuda()
            M.kv_store(x, lens[b:b + 1], td[b:b + 1], None if sd is None else sd[b:b + 1], layer, blocks, scales)
    have = list(lengths)
    keys = [[rows(b, have[b], layer) for b in range(B)] for layer in range(layers)]
    sums = [[torch.zeros(have[b]).double() for b in range(B)] for _ in range(layers)]
    for s in scores:
        s[:, :] = 0.0
    lens = torch.tensor(have, dtype=torch.int32).cuda()
    for step in range(10):
        for layer in range(layers):
            x = torch.randn((B, 1, 576), generator=gen).bfloat16().cuda()
            q = torch.randn((B, 1, H, 576), generator=gen).bfloat16()
            M.kv_store(x, lens, td, sd, layer, blocks, scales)
            out, lse = M.decode(q.cuda(), blocks, scales, lens, td, sd, 1, max(have), layer, SCALE, fold_scales=True)
            M.accumulate_weights(q.cuda(), lse, blocks, scales, lens, td, sd, 1, max(have), layer, SCALE, scores[layer])
            assert M.device_status() == 0
            for b in range(B):
                n = have[b] + 1
                now = rows(b, n, layer)
                assert torch.equal(now[:-1], keys[layer][b])       # what was kept, in order, and one more
                keys[layer][b] = now
                ref = latent_scores(q[b], now, have[b], SCALE)
                p = torch.softmax(ref, -1)
                want = torch.einsum("thk,kd->thd", p, now[:, :512])
                err = (out[b].cpu().double() - want).abs().max()
                assert err <= 2e-2 * want.abs().max() + 1e-2, (step, b, err)   # the decode's own bar
                sums[layer][b] = torch.cat([sums[layer][b], torch.zeros(1)]) + p.sum((0, 1))
                got = scores[layer][b, :n].cpu().double()
                # fp32 scores and lse of sizes below 2^5: errors below 2^-14 of a weight, and of their sums
                assert ((got - sums[layer][b]).abs() <= 2.0 ** -13 * (sums[layer][b] + 2.0 ** -100)).all()
        have = [n + 1 for n in have]
        lens += 1
        if step % 3 == 2:
            for layer in range(layers):
                kept, count = M.select_keys(scores[layer], lens, max(have), budget, recent, sink)
                for b in range(B):
                    want = select_reference(scores[layer][b].tolist(), have[b], budget, recent, sink)
                    assert kept[b, :int(count[b])].tolist() == want
                    keys[layer][b] = keys[layer][b][want]
                    sums[layer][b] = sums[layer][b][want]
                M.compact_cache(kept, count, td, sd, layer, blocks, scales, scores[layer])
            lens = count.clone()
            have = count.tolist()
            assert M.device_status() == 0 and max(have) <= budget
    for layer in range(layers):
        for b in range(B):
            assert torch.equal(rows(b, have[b], layer), keys[layer][b])


@pytest.mark.parametrize("fp8", [False, True])
def test_multi_head_cache_stored_attended_and_compacted(fp8):
    B, H, HKV, D, page = 2, 12, 4, 128, 32
    lengths = [90, 400]
    cache = MhaCache([n + 8 for n in lengths], page, HKV, D, fp8, seed=3, layers=2, layer=1)
    blocks, scales, table, _ = cache.cuda()
    gen = torch.Generator().manual_seed(4)
    have = list(lengths)
    for step in range(3):
        k, v, q = (torch.randn((B, 2, h, D), generator=gen).bfloat16() for h in (HKV, HKV, H))
        lens = torch.tensor(have, dtype=torch.int32).cuda()
        M.mha_kv_store(k.cuda(), v.cuda(), lens, table, None, 1, blocks, scales)
        out, lse = M.mha_decode(q.cuda(), blocks, scales, lens, table, None, 2, max(have), 1, 0.1)
        assert M.device_status() == 0
        cache.blocks, cache.scales = blocks.cpu(), None if scales is None else scales.cpu()
        for b in range(B):
            ro, rl, mag, _ = mha_reference(cache, b, q[b], have[b], 0.1)
            assert ((out[b].cpu().double() - ro).abs() <= 2.0 ** -7 * (mag + ro.abs())).all()   # two bf16 roundings and room
            assert (lse[b].cpu().double() - rl).abs().max() < 1e-4
        have = [n + 2 for n in have]
        if step == 1:                                              # keep the first and last, drop some between
            kept = [sorted(set(range(20)) | set(range(50, n, 2)) | set(range(n - 9, n))) for n in have]
            table_k = torch.zeros((B, max(map(len, kept))), dtype=torch.int32)
            for b, ks in enumerate(kept):
                table_k[b, :len(ks)] = torch.tensor(ks, dtype=torch.int32)
            M.compact_cache(table_k.cuda(), torch.tensor([len(x) for x in kept], dtype=torch.int32).cuda(), table, None, 1, blocks,
                            scales)
            have = [len(x) for x in kept]
    assert M.device_status() == 0
