"""Multi-head cache: the KV-store step bit for bit, the decode against 64 bits.

Tolerances.  Scores: fp32 sums of D products, (D + 8) 2^-24 of the sum of magnitudes A, plus the
exponent's roundings; an error e of every score moves a weight by at most a factor exp(2 e).  Weights
are two bf16 terms (half a step, 2^-8, of half a step) for a bf16 cache, rounded to f16 (2^-11, and 2^-25 of V's scale bound
below its normal range: at most twice the largest scale, times 448, per key) for an e4m3 cache; the
output is rounded to bf16 (2^-8).  The log-sum-exp has the scores' error and its own fp32 roundings."""
import pytest
import torch

import paged_fp8_kv_mla_b200 as M
from tests.cache_ref import MhaCache, mha_reference, quantise, rows_of

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


def run(cache, q, lengths, scale, top=None, **kw):
    blocks, scales, table, stable = cache.cuda()
    out, lse = M.mha_decode(q.cuda(), blocks, scales, torch.tensor(lengths, dtype=torch.int32).cuda(), table, stable, q.shape[1],
                            max(lengths) if top is None else top, cache.layer, scale, **kw)
    assert M.device_status() == 0
    return out, lse


def check(cache, q, lengths, scale, out, lse, only=None):
    for b, L in enumerate(lengths):
        if only is not None and b not in only:
            continue
        ro, rl, mag, amp = mha_reference(cache, b, q[b], L, scale)
        n, D = L + q.shape[1], q.shape[-1]
        e = (D + 8) * U * amp + 8 * U * (rl.abs() + amp) + 2.0 ** -21
        weight = 2.0 ** -11 if cache.fp8 else 2.0 ** -16
        tol = mag * (weight + 2 * e[..., None] + (n + 64) * U) + ro.abs() * 2.0 ** -8
        if cache.fp8:
            # f16 weights below the normal range: 2^-25 of V's scale bound per key, times the code (448)
            tol = tol + n * 2.0 ** -25 * 2 * float(cache.rows(1, b, n).abs().max())
        g = out[b].cpu().double()
        bad = ~((g - ro).abs() <= tol)
        assert not bad.any(), (b, bad.nonzero()[:4], g[bad][:4], ro[bad][:4], tol[bad][:4])
        if lse is not None:
            tl = e + (n + 64) * U * 1.0 + U * rl.abs()
            bad = ~((lse[b].cpu().double() - rl).abs() <= tl)
            assert not bad.any(), (b, bad.nonzero()[:4], lse[b].cpu()[bad][:4], rl[bad][:4])


def make(lengths, T, H, HKV, D, page, fp8, seed=0, **kw):
    cache = MhaCache([n + T for n in lengths], page, HKV, D, fp8, seed=seed, **kw)
    q = torch.randn((len(lengths), T, H, D), generator=torch.Generator().manual_seed(seed + 50)).bfloat16()
    return cache, q


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("lengths,T,H,HKV,D,page", [
    ([0], 1, 1, 1, 64, 16), ([36, 63], 1, 16, 4, 64, 16), ([15, 16, 17], 1, 8, 8, 128, 16), ([500, 1, 130], 1, 32, 8, 128, 64),
    ([1000], 1, 8, 1, 128, 48), ([700, 900, 40], 2, 28, 4, 64, 32), ([2100, 5], 1, 20, 5, 64, 64), ([300, 77], 4, 16, 2, 128, 128),
    ([3000], 1, 64, 1, 64, 64), ([260, 1030], 3, 48, 1, 128, 80), ([640, 3], 1, 11, 11, 128, 64), ([400], 2, 140, 2, 64, 16),
    ([150, 600], 9, 16, 1, 128, 64), ([5000, 4, 4000], 1, 24, 3, 128, 64), ([90, 200], 1, 40, 40, 64, 32),
])
def test_decode_against_64_bits(lengths, T, H, HKV, D, page, fp8):
    cache, q = make(lengths, T, H, HKV, D, page, fp8, seed=len(lengths) + H)
    scale = D ** -0.5
    out, lse = run(cache, q, lengths, scale)
    check(cache, q, lengths, scale, out, lse)


@pytest.mark.parametrize("fp8", [False, True])
def test_decode_many_requests_and_splits(fp8):
    """More items than SMs, lengths from nothing to long: pieces of every kind."""
    gen = torch.Generator().manual_seed(2)
    lengths = [int(x) for x in torch.exp(torch.rand(70, generator=gen) * 8).long() - 1]
    cache, q = make(lengths, 1, 12, 3, 128, 32, fp8, seed=4)
    out, lse = run(cache, q, lengths, 0.1)
    check(cache, q, lengths, 0.1, out, lse)


def test_decode_layers_scale_pages_and_value_sizes():
    """e4m3 scales paged apart and of very different sizes; one layer of three."""
    lengths = [900, 333]
    cache, q = make(lengths, 1, 16, 2, 128, 64, True, seed=9, layers=3, layer=1, own_scale_pages=True, value_spread=3.0)
    out, lse = run(cache, q, lengths, 0.09)
    check(cache, q, lengths, 0.09, out, lse)


@pytest.mark.parametrize("mul", [1e-30, 1e-6, 50.0])
@pytest.mark.parametrize("fp8", [False, True])
def test_decode_q_of_any_size(fp8, mul):
    lengths = [300, 31]
    cache, q = make(lengths, 1, 8, 2, 64, 16, fp8, seed=11)
    q = (q.float() * mul).bfloat16()
    out, lse = run(cache, q, lengths, 0.125)
    check(cache, q, lengths, 0.125, out, lse)


def test_decode_scale_zero_and_negative():
    """softmax_scale 0: the mean of the visible values; negative: the least alike keys win."""
    lengths = [200, 700]
    cache, q = make(lengths, 2, 8, 2, 64, 16, False, seed=12)
    for scale in (0.0, -0.2):
        out, lse = run(cache, q, lengths, scale)
        check(cache, q, lengths, scale, out, lse)


def test_decode_without_lse_preallocated_and_deterministic():
    lengths = [1700, 20, 3000]
    cache, q = make(lengths, 1, 32, 8, 128, 64, True, seed=13)
    out, lse = run(cache, q, lengths, 0.09)
    again = torch.empty_like(out)
    got, none = run(cache, q, lengths, 0.09, out=again, want_lse=False)
    assert none is None and got.data_ptr() == again.data_ptr()
    assert torch.equal(again, out)
    long, _ = run(cache, q, lengths, 0.09, top=3007)              # a longer bound changes nothing that is read
    check(cache, q, lengths, 0.09, long, None)


def test_decode_bad_page_is_left_out_and_flagged():
    lengths = [200, 100]
    cache, q = make(lengths, 1, 8, 2, 64, 16, False, seed=14)
    blocks, scales, table, stable = cache.cuda()
    table[0, 3] = 99999
    out, lse = M.mha_decode(q.cuda(), blocks, None, torch.tensor(lengths, dtype=torch.int32).cuda(), table, None, 1, 200, 0, 0.125)
    assert M.device_status() == 6
    check(cache, q, lengths, 0.125, out, lse, only=[1])
    keep = [t for t in range(201) if not 48 <= t < 64]
    k, v = cache.rows(0, 0, 201)[keep], cache.rows(1, 0, 201)[keep]
    x = torch.einsum("grd,kgd->grk", q[0, 0].double().reshape(2, 4, 64), k) * 0.125
    want = torch.einsum("grk,kgd->grd", torch.softmax(x, -1), v).reshape(8, 64)
    assert (out[0, 0].cpu().double() - want).abs().max() < 0.03   # 2^-8 of sums of |values| below 4


def test_decode_two_streams_and_a_graph():
    """Calls that overlap have a workspace each; a captured call replays with new inputs."""
    lengths = [2500, 900, 4100]
    cases = [make(lengths, 1, 16, 4, 128, 64, fp8, seed=20 + fp8) for fp8 in (False, True)]
    lens = torch.tensor(lengths, dtype=torch.int32).cuda()
    on = [c.cuda() for c, _ in cases]
    qs = [q.cuda() for _, q in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    results = []
    for _ in range(4):
        for i, s in enumerate(streams):
            results.append(M.mha_decode(qs[i], on[i][0], on[i][1], lens, on[i][2], on[i][3], 1, 4100, 0, 0.09, stream=s))
    torch.cuda.synchronize()
    assert M.device_status() == 0
    for n, (out, lse) in enumerate(results):
        check(cases[n % 2][0], cases[n % 2][1], lengths, 0.09, out, lse)
    graphs, outs = [], []
    for i in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(M.mha_decode(qs[i], on[i][0], on[i][1], lens, on[i][2], on[i][3], 1, 4100, 0, 0.09))
        graphs.append(g)
    new = [torch.randn(q.shape, generator=torch.Generator().manual_seed(77)).bfloat16() for _, q in cases]
    for i in range(2):
        qs[i].copy_(new[i])
    torch.cuda.synchronize()
    for i, s in enumerate(streams):                               # both graphs at the same time
        with torch.cuda.stream(s):
            graphs[i].replay()
    torch.cuda.synchronize()
    for i in range(2):
        check(cases[i][0], new[i], lengths, 0.09, outs[i][0], outs[i][1])


def test_decode_refuses_out_on_q_and_takes_an_empty_batch():
    cache, q = make([30, 40], 1, 8, 2, 64, 16, False, seed=41)
    blocks, scales, table, stable = cache.cuda()
    lens, qd = torch.tensor([30, 40], dtype=torch.int32).cuda(), q.cuda()
    with pytest.raises(M.MlaError, match="out must not be q"):
        M.mha_decode(qd, blocks, scales, lens, table, stable, 1, 40, 0, 0.1, out=qd)
    out, lse = M.mha_decode(qd[:0], blocks, scales, lens[:0], table[:0], stable, 1, 40, 0, 0.1)
    assert out.shape == (0, 1, 8, 64) and lse.shape == (0, 1, 8)
    with pytest.raises(M.MlaError, match="workspace"):
        big, bq = make([3000], 1, 8, 2, 64, 16, False, seed=42)
        b = big.cuda()
        M.mha_decode(bq.cuda(), b[0], None, torch.tensor([3000], dtype=torch.int32).cuda(), b[2], None, 1, 3000, 0, 0.1,
                     workspace=torch.empty(64, dtype=torch.uint8).cuda())


@pytest.mark.parametrize("lengths,T,HKV,D,page,kw", [
    ([0], 1, 1, 64, 16, {}), ([5, 0, 30], 1, 8, 128, 16, {}), ([10, 100], 37, 3, 64, 48, dict(layers=2, layer=1)),
    ([63, 1], 200, 5, 128, 64, dict(own_scale_pages=True)),
])
@pytest.mark.parametrize("fp8", [False, True])
def test_store_is_exact(lengths, T, HKV, D, page, kw, fp8):
    cache = MhaCache([n + T for n in lengths], page, HKV, D, fp8, seed=30, **kw)
    gen = torch.Generator().manual_seed(31)
    k, v = (torch.randn((len(lengths), T, HKV, D), generator=gen).bfloat16() for _ in range(2))
    k[0, 0, 0] = 0                                                # an all-zero row: scale 1
    k[-1, -1, -1] *= 1e-30
    v[0, 0, 0, 3] = 3e38
    blocks, scales = cache.blocks.clone(), None if cache.scales is None else cache.scales.clone()
    stable = cache.table if cache.stable is None else cache.stable
    for b, L in enumerate(lengths):
        blk, slot = rows_of(cache.table, b, L + T, page)
        sblk = rows_of(stable, b, L + T, page)[0]
        for i, x in ((0, k[b]), (1, v[b])):
            if fp8:
                codes, s = quantise(x)
                blocks[blk[L:], i, cache.layer, slot[L:]] = codes
                scales[sblk[L:], i, cache.layer, slot[L:]] = s
            else:
                blocks[blk[L:], i, cache.layer, slot[L:]] = x
    db, ds, table, st = cache.cuda()
    M.mha_kv_store(k.cuda(), v.cuda(), torch.tensor(lengths, dtype=torch.int32).cuda(), table, st, cache.layer, db, ds)
    assert M.device_status() == 0
    assert torch.equal(db.cpu().view(torch.uint8), blocks.view(torch.uint8))
    if fp8:
        assert torch.equal(ds.cpu().view(torch.int32), scales.view(torch.int32))


def test_store_scale_of_every_bf16_maximum():
    """amax / 448 rounds like the IEEE quotient for every positive finite bf16 value."""
    top = torch.arange(1, 0x7F80, dtype=torch.int32).to(torch.int16).view(torch.bfloat16)
    n = top.numel()
    cache = MhaCache([n], 64, 1, 64, True, seed=34)
    k = torch.zeros((1, n, 1, 64), dtype=torch.bfloat16)
    k[0, :, 0, 17] = -top
    db, ds, table, _ = cache.cuda()
    M.mha_kv_store(k.cuda(), k.cuda(), torch.tensor([0], dtype=torch.int32).cuda(), table, None, 0, db, ds)
    assert M.device_status() == 0
    blk, slot = rows_of(cache.table, 0, n, 64)
    assert torch.equal(ds.cpu()[blk, 0, 0, slot, 0, 0], top.float() / 448.0)


def test_store_bad_page_is_skipped_and_flagged():
    cache = MhaCache([20, 20], 16, 2, 64, True, seed=33)
    db, ds, table, _ = cache.cuda()
    table[0, 1] = 4000
    k = torch.ones((2, 4, 2, 64), dtype=torch.bfloat16).cuda()
    M.mha_kv_store(k, k, torch.tensor([16, 30000], dtype=torch.int32).cuda(), table, None, 0, db, ds)
    assert M.device_status() == 6
    assert torch.equal(db.cpu(), cache.blocks)
    M.mha_kv_store(k[:, :0], k[:, :0], torch.tensor([16, 16], dtype=torch.int32).cuda(), table, None, 0, db, ds)
    assert M.device_status() == 0


@pytest.mark.parametrize("page", [256, 512, 1024])
@pytest.mark.parametrize("HKV,D,fp8", [(1, 64, True), (1, 64, False), (2, 128, True)])
def test_decode_large_pages(page, HKV, D, fp8):
    """Pages of more rows than a copy's box, tiles of more keys than either."""
    lengths = [1500, 255, 700]
    cache, q = make(lengths, 1, 8 * HKV, HKV, D, page, fp8, seed=page)
    out, lse = run(cache, q, lengths, 0.1)
    check(cache, q, lengths, 0.1, out, lse)


@pytest.mark.parametrize("first", [True, False])
@pytest.mark.parametrize("D", [64, 128])
def test_decode_zero_value_rows_among_small_ones(D, first):
    """An all-zero row of V has scale 1, a million times that of its neighbours here; what it may cost them is
    f16's absolute step at 2^9 times the weight: 2^-34 of V's scale bound (2) per key, times the code, over the
    sum of the weights, which is at least exp(lse - largest score)."""
    lengths, HKV, H = [40, 900], 2, 8
    cache, q = make(lengths, 1, H, HKV, D, 64, True, seed=77)
    gen = torch.Generator().manual_seed(78)
    codes = []
    for b, L in enumerate(lengths):
        n = L + 1
        blk, slot = rows_of(cache.table, b, n, 64)
        x = torch.randn((n, HKV, D), generator=gen) * 2e-4
        x[0 if first else n - 2] = 0
        c, s = quantise(x.bfloat16())
        cache.blocks[blk, 1, 0, slot] = c
        cache.scales[blk, 1, 0, slot] = s
        codes.append((cache.rows(1, b, n) / s.double()).abs().sum(0))          # [HKV, D]
    out, lse = run(cache, q, lengths, D ** -0.5)
    for b, L in enumerate(lengths):
        ro, rl, mag, amp = mha_reference(cache, b, q[b], L, D ** -0.5)
        k = cache.rows(0, b, L + 1)
        x = torch.einsum("grd,kgd->grk", q[b, 0].double().reshape(HKV, H // HKV, D), k) * D ** -0.5
        total = torch.exp(rl[0] - x.amax(-1).reshape(H))
        step = codes[b].repeat_interleave(H // HKV, 0) * 2.0 ** -33 / total[:, None]
        e = (D + 8) * U * amp + 8 * U * (rl.abs() + amp) + 2.0 ** -21
        tol = mag * (2.0 ** -11 + 2 * e[..., None] + (L + 65) * U) + ro.abs() * 2.0 ** -8 + step
        bad = ~((out[b].cpu().double() - ro).abs() <= tol)
        assert not bad.any(), (b, int(bad.sum()), out[b].cpu().double()[bad][:4], ro[bad][:4], tol[bad][:4])
