"""Paged caches and 64-bit plain forms for the tests of the cache operators (torch float64, any device).

Pages are drawn from a permuted pool; whatever a kernel must not use is poisoned: page-table entries
behind a request's pages are 0xFFFFFFFF, and rows behind its last key hold NaN codes (or infinities)
and NaN scales."""
import torch

E4M3 = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double()   # value of each code (NaN: 127, 255)


def page_table(stored, page, extra, gen, width=0):
    pages = [-(-n // page) for n in stored]
    pool = torch.randperm(sum(pages) + extra, generator=gen).tolist()
    table = torch.full((len(stored), max(max(pages), 1) + width), -1, dtype=torch.int32)
    for b, k in enumerate(pages):
        for j in range(k):
            table[b, j] = pool.pop()
    return table, sum(pages) + extra


def rows_of(table, b, n, page):
    """(block, slot) of positions 0 .. n - 1 of request b."""
    t = torch.arange(n)
    return table[b, t // page].long(), t % page


def quantise(x):
    amax = x.float().abs().amax(-1, keepdim=True)
    scale = torch.where(amax > 0, amax / 448.0, torch.ones_like(amax))
    return (x.float() / scale).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8), scale


class LatentCache:
    """blocks uint8 [NB, KVD, NL, P, 1, 576], scales fp32 [NSB, KVD, NL, P, 1, 1]; the keys of `layer` are
    random, everything else is poison."""

    def __init__(self, stored, page, seed=0, layers=1, layer=0, kv_dim=1, own_scale_pages=False, spread=1.0):
        gen = torch.Generator().manual_seed(seed)
        self.stored, self.page, self.layer = stored, page, layer
        self.table, nb = page_table(stored, page, 3, gen, width=1)
        self.blocks = torch.full((nb, kv_dim, layers, page, 1, 576), 127, dtype=torch.uint8)
        self.stable, nsb = page_table(stored, page, 5, gen, width=1) if own_scale_pages else (None, nb)
        self.scales = torch.full((nsb, kv_dim, layers, page, 1, 1), float("nan"))
        for b, n in enumerate(stored):
            if n == 0:
                continue
            x = torch.randn((n, 576), generator=gen) * torch.exp(spread * torch.randn((n, 1), generator=gen) * 0.3)
            codes, scale = quantise(x.bfloat16())
            blk, slot = rows_of(self.table, b, n, page)
            sblk = blk if self.stable is None else rows_of(self.stable, b, n, page)[0]
            self.blocks[blk, 0, layer, slot, 0] = codes
            self.scales[sblk, 0, layer, slot, 0] = scale

    def keys(self, b, n):
        blk, slot = rows_of(self.table, b, n, self.page)
        sblk = blk if self.stable is None else rows_of(self.stable, b, n, self.page)[0]
        return E4M3[self.blocks[blk, 0, self.layer, slot, 0].int()] * self.scales[sblk, 0, self.layer, slot, 0].double()

    def cuda(self):
        t = lambda x: None if x is None else x.cuda()  # noqa: E731
        return t(self.blocks), t(self.scales), t(self.table), t(self.stable)


class MhaCache:
    """Keys in kv plane 0, values in plane 1; bf16, or e4m3 with a scale per token and head."""

    def __init__(self, stored, page, heads, dim, fp8, seed=0, layers=1, layer=0, own_scale_pages=False, value_spread=0.0):
        gen = torch.Generator().manual_seed(seed)
        self.stored, self.page, self.layer, self.fp8 = stored, page, layer, fp8
        self.table, nb = page_table(stored, page, 3, gen, width=1)
        self.stable, nsb = page_table(stored, page, 5, gen, width=1) if own_scale_pages and fp8 else (None, nb)
        shape = (nb, 2, layers, page, heads, dim)
        if fp8:
            self.blocks = torch.full(shape, 255, dtype=torch.uint8)
            self.scales = torch.full((nsb,) + shape[1:5] + (1,), float("nan"))
        else:
            self.blocks = torch.full(shape, float("inf"), dtype=torch.bfloat16)
            self.scales = None
        for b, n in enumerate(stored):
            blk, slot = rows_of(self.table, b, n, page)
            sblk = blk if self.stable is None else rows_of(self.stable, b, n, page)[0]
            for plane in (0, 1):
                x = torch.randn((n, heads, dim), generator=gen)
                if plane:
                    x = x * torch.exp(value_spread * torch.randn((n, heads, 1), generator=gen))
                x = x.bfloat16()
                if fp8:
                    codes, scale = quantise(x)
                    self.blocks[blk, plane, layer, slot] = codes
                    self.scales[sblk, plane, layer, slot] = scale
                else:
                    self.blocks[blk, plane, layer, slot] = x

    def rows(self, plane, b, n):
        blk, slot = rows_of(self.table, b, n, self.page)
        if not self.fp8:
            return self.blocks[blk, plane, self.layer, slot].double()
        sblk = blk if self.stable is None else rows_of(self.stable, b, n, self.page)[0]
        return E4M3[self.blocks[blk, plane, self.layer, slot].int()] * self.scales[sblk, plane, self.layer, slot].double()

    def cuda(self):
        t = lambda x: None if x is None else x.cuda()  # noqa: E731
        return t(self.blocks), t(self.scales), t(self.table), t(self.stable)


def latent_scores(q, keys, cached, scale):
    """x [T, H, n] with -inf where a key is not visible; q [T, H, 576]."""
    T, n = q.shape[0], keys.shape[0]
    x = torch.einsum("thd,kd->thk", q.double(), keys) * scale
    late = torch.arange(n)[None] > cached + torch.arange(T)[:, None]
    return x.masked_fill(late[:, None], float("-inf"))


def mha_reference(cache, b, q, cached, scale):
    """(out, lse, sum of |weight * value|, largest sum of |q k|) of request b in 64 bits; q [T, H, D]."""
    T, H, D = q.shape
    n = cached + T
    k, v = cache.rows(0, b, n), cache.rows(1, b, n)
    G = H // k.shape[1]
    qg = q.double().reshape(T, k.shape[1], G, D)
    x = torch.einsum("tgrd,kgd->tgrk", qg, k) * scale
    late = torch.arange(n)[None] > cached + torch.arange(T)[:, None]
    x = x.masked_fill(late[:, None, None], float("-inf"))
    lse = x.logsumexp(-1)
    p = torch.exp(x - lse[..., None])
    out = torch.einsum("tgrk,kgd->tgrd", p, v).reshape(T, H, D)
    mag = torch.einsum("tgrk,kgd->tgrd", p, v.abs()).reshape(T, H, D)
    amp = (torch.einsum("tgrd,kgd->tgrk", qg.abs(), k.abs()) * abs(scale)).amax(-1).reshape(T, H)
    return out, lse.reshape(T, H), mag, amp


def select_reference(scores, n, budget, recent, sink):
    """Kept indices of one request, from the definition: one key at a time."""
    if n <= budget:
        return list(range(n))
    value = [float("-inf") if s != s else s for s in scores[:n]]
    nan = [s != s for s in scores[:n]]
    middle = sorted(range(sink, n - recent), key=lambda i: (nan[i], -value[i], i))
    return sorted(list(range(sink)) + middle[:budget - sink - recent] + list(range(n - recent, n)))
