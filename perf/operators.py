"""Timed cases of the cache-eviction and multi-head paged-attention operators.

Two sets that work on the paged caches between and within decode steps:

  eviction by accumulated attention weight (latent FP8 cache)
    weights   accumulate_weights: add each cached key's softmax weight, summed over heads and new tokens
    select    select_keys: the keys to keep per request (first ones, last ones, largest sums)
    compact   compact_cache: move the kept rows to the front of their pages, in order
  attention with separate keys and values over the same paged layout (bf16 or e4m3 + scales)
    attend    mha_decode: grouped-query attention of the new tokens over the paged cache
    store     mha_kv_store: write the step's keys and values into their pages

`run` computes a case in plain torch operations, or, where `own` is set, with the framework's calls.
"""
import math
import random

import torch

own = False

LATENT = 576           # 512 latent + 64 rope values per cached token
MLA_SCALE = 1.0 / math.sqrt(192.0)
E4M3_MAX = 448.0
NO_PAGE = -1           # unused page-table entries (0xFFFFFFFF)


def listed():
    return [
        # the tiny two-request decode step (latency of one call)
        {"name": "weights_tiny_b2_h16", "op": "weights", "batch": 2, "q_len": 1, "heads": 16, "page": 16,
         "kind": "uniform", "lo": 36, "hi": 63, "layers": 1, "layer": 0, "own_scale_pages": False},
        # speculative step of two tokens, ragged requests from one token to long ones, scales paged apart
        {"name": "weights_ragged_b64_t2_h128", "op": "weights", "batch": 64, "q_len": 2, "heads": 128, "page": 64,
         "kind": "loguniform", "lo": 1, "hi": 32768, "layers": 1, "layer": 0, "own_scale_pages": True},
        # steady-state serving step, 128 requests of 8k cached tokens
        {"name": "weights_steady_b128_l8k", "op": "weights", "batch": 128, "q_len": 1, "heads": 128, "page": 64,
         "kind": "fixed", "lo": 8192, "hi": 8192, "layers": 1, "layer": 0, "own_scale_pages": False},
        # moderate batch trimmed to 1024 keys each; requests shorter than that keep everything
        {"name": "select_b32_l1k-4k_keep1k", "op": "select", "batch": 32, "kind": "uniform", "lo": 700, "hi": 4096,
         "keep": 1024, "recent": 128, "sink": 4},
        # long contexts cut to a quarter
        {"name": "select_b4_l128k_keep32k", "op": "select", "batch": 4, "kind": "fixed", "lo": 131072, "hi": 131072,
         "keep": 32768, "recent": 1024, "sink": 4},
        # moderate batch, layer 1 of 2, after its selection of 1024 keys
        {"name": "compact_b32_l1k-4k_keep1k", "op": "compact", "batch": 32, "page": 64, "kind": "uniform", "lo": 700,
         "hi": 4096, "layers": 2, "layer": 1, "own_scale_pages": False, "keep": 1024, "recent": 128, "sink": 4},
        # the steady-state cache halved
        {"name": "compact_b128_l8k_keep4k", "op": "compact", "batch": 128, "page": 64, "kind": "fixed", "lo": 8192,
         "hi": 8192, "layers": 1, "layer": 0, "own_scale_pages": True, "keep": 4096, "recent": 256, "sink": 4},
        # smallest grouped-query step (latency of one call)
        {"name": "attend_tiny_b2_h16_kv4_d64", "op": "attend", "batch": 2, "q_len": 1, "heads": 16, "kv_heads": 4,
         "dim": 64, "page": 16, "fp8": False, "kind": "uniform", "lo": 36, "hi": 63, "layers": 1, "layer": 0},
        # speculative step of two tokens over ragged bf16 caches
        {"name": "attend_ragged_b64_t2_h32_kv8_d128", "op": "attend", "batch": 64, "q_len": 2, "heads": 32,
         "kv_heads": 8, "dim": 128, "page": 64, "fp8": False, "kind": "loguniform", "lo": 1, "hi": 32768,
         "layers": 1, "layer": 0},
        # steady-state serving step over an e4m3 cache with one scale per token and head
        {"name": "attend_steady_b128_h64_kv8_d128_fp8", "op": "attend", "batch": 128, "q_len": 1, "heads": 64,
         "kv_heads": 8, "dim": 128, "page": 64, "fp8": True, "kind": "fixed", "lo": 8192, "hi": 8192,
         "layers": 1, "layer": 0},
        # one decode step's keys and values into a bf16 cache
        {"name": "store_step_b128_t1_kv8_d128", "op": "store", "batch": 128, "q_len": 1, "kv_heads": 8, "dim": 128,
         "page": 64, "fp8": False, "kind": "uniform", "lo": 0, "hi": 500, "layers": 2, "layer": 1},
        # prompts of 4096 tokens quantised into an e4m3 cache
        {"name": "store_prompt_b16_t4096_kv8_d128_fp8", "op": "store", "batch": 16, "q_len": 4096, "kv_heads": 8,
         "dim": 128, "page": 64, "fp8": True, "kind": "uniform", "lo": 0, "hi": 500, "layers": 1, "layer": 0},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["weights", "select", "compact", "attend", "store"])
    page = rng.choice([16, 32, 48, 64, 128])
    layers = rng.choice([1, 2])
    where = {"page": page, "layers": layers, "layer": rng.randrange(layers)}
    if op == "weights":
        batch, q_len = _log(rng, 1, 128), rng.choice([1, 1, 1, 2, 3])
        hi = _log(rng, 1, max(2, min(131072, 1000000 // (batch * q_len))))
        return {"op": op, "batch": batch, "q_len": q_len, "heads": rng.choice([1, 8, 16, 20, 64, 96, 128]), **where,
                "kind": "loguniform", "lo": 1, "hi": hi, "own_scale_pages": rng.random() < 0.5}
    if op in ("select", "compact"):
        batch = _log(rng, 1, 128)
        hi = _log(rng, 16, min(131072, 524288 // batch))
        lo = rng.randrange(1, hi + 1)
        keep = rng.randrange(8, hi + 1)
        sink = rng.choice([0, 1, 4])
        case = {"op": op, "batch": batch, "kind": "uniform", "lo": lo, "hi": hi, "keep": keep,
                "recent": rng.randrange(0, keep - sink + 1), "sink": sink}
        return case if op == "select" else {**case, **where, "own_scale_pages": rng.random() < 0.5}
    kv_heads, dim, fp8 = rng.choice([1, 2, 5, 8]), rng.choice([64, 128]), rng.random() < 0.5
    if op == "attend":
        batch, q_len, group = _log(rng, 1, 128), rng.choice([1, 1, 1, 2, 4]), rng.choice([1, 3, 4, 7, 8])
        hi = _log(rng, 1, max(2, min(131072, 4000000 // (batch * kv_heads))))
        return {"op": op, "batch": batch, "q_len": q_len, "heads": kv_heads * group, "kv_heads": kv_heads, "dim": dim,
                **where, "fp8": fp8, "kind": "loguniform", "lo": 1, "hi": hi}
    batch = _log(rng, 1, 128)
    return {"op": op, "batch": batch, "q_len": _log(rng, 1, 32768 // batch), "kv_heads": kv_heads, "dim": dim, **where,
            "fp8": fp8, "kind": "uniform", "lo": 0, "hi": 500}


# ---------------------------------------------------------------- inputs
def _lengths(case):
    """Cached tokens per request: part of the case (every seed has the same)."""
    b, lo, hi = case["batch"], case["lo"], case["hi"]
    rng = random.Random("%s %d %d %d" % (case["kind"], b, lo, hi))
    if case["kind"] == "fixed":
        return [hi] * b
    if case["kind"] == "uniform":
        return [rng.randint(lo, hi) for _ in range(b)]
    n = [min(hi, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))) for _ in range(b)]
    n[rng.randrange(b)] = hi
    return n


def _tables(case, stored, extra, gen):
    """Page table [batch, max_pages] over a permuted pool of the pages needed plus `extra`."""
    pages = [-(-n // case["page"]) for n in stored]
    pool = torch.randperm(sum(pages) + extra, generator=gen, device="cuda").to(torch.int32)
    table = torch.full((len(stored), max(max(pages), 1)), NO_PAGE, dtype=torch.int32, device="cuda")
    at = 0
    for b, k in enumerate(pages):
        table[b, :k] = pool[at:at + k]
        at += k
    return table, max(sum(pages) + extra, 1)


def _quantise(x):
    """Rows of the last dim to e4m3 codes with one fp32 scale each (amax / 448, 1 for a zero row)."""
    amax = x.float().abs().amax(-1, keepdim=True)
    scale = torch.where(amax > 0, amax / E4M3_MAX, torch.ones_like(amax))
    return (x.float() / scale).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn), scale


def _normal(shape, gen, outliers=0.0):
    x = torch.randn(shape, generator=gen, device="cuda", dtype=torch.bfloat16)
    if outliers:
        x *= 1 + 19 * (torch.rand(shape[:-1] + (1,), generator=gen, device="cuda") < outliers)
    return x


def _latent_cache(case, stored, gen):
    table, nb = _tables(case, stored, 5, gen)
    stable, nsb = _tables(case, stored, 37, gen) if case["own_scale_pages"] else (None, nb)
    blocks = torch.empty((nb, 1, case["layers"], case["page"], 1, LATENT), dtype=torch.uint8, device="cuda")
    own_scales = torch.empty((nb, 1, case["layers"], case["page"], 1, 1), device="cuda")
    for part, scale in zip(blocks.split(4096), own_scales.split(4096)):
        codes, s = _quantise(_normal(part.shape, gen, 0.01))
        part.copy_(codes.view(torch.uint8))
        scale.copy_(s)
    if stable is None:
        return {"blocks": blocks, "scales": own_scales, "table": table, "stable": None}
    # the scales in pages of their own: each request's go where its scale table says
    scales = torch.rand((nsb,) + own_scales.shape[1:], generator=gen, device="cuda") * 0.02
    used = table >= 0
    scales[stable[used].long()] = own_scales[table[used].long()]
    return {"blocks": blocks, "scales": scales, "table": table, "stable": stable}


def _mha_cache(case, stored, gen):
    table, nb = _tables(case, stored, 5, gen)
    shape = (nb, 2, case["layers"], case["page"], case["kv_heads"], case["dim"])
    if not case["fp8"]:
        return {"blocks": _normal(shape, gen), "scales": None, "table": table, "stable": None}
    blocks = torch.empty(shape, dtype=torch.uint8, device="cuda")
    scales = torch.empty(shape[:-1] + (1,), device="cuda")
    for part, scale in zip(blocks.split(2048), scales.split(2048)):
        codes, s = _quantise(_normal(part.shape, gen))
        part.copy_(codes.view(torch.uint8))
        scale.copy_(s)
    return {"blocks": blocks, "scales": scales, "table": table, "stable": None}


def _sums(shape, gen):
    """Accumulated weights as they come: a few heavy keys, a long tail, some keys never attended to, ties."""
    x = torch.exp(2 * torch.randn(shape, generator=gen, device="cuda")) * 0.05
    x = torch.where(torch.rand(shape, generator=gen, device="cuda") < 0.02, torch.zeros_like(x), x)
    return torch.where(torch.rand(shape, generator=gen, device="cuda") < 0.2, x.bfloat16().float(), x)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    op, n = case["op"], _lengths(case)
    s = {"case": case, "lengths": torch.tensor(n, dtype=torch.int32, device="cuda"), "max_length": max(n)}
    if op == "weights":
        t = case["q_len"]
        s |= _latent_cache(case, [x + t for x in n], gen)
        s["q"] = _normal((case["batch"], t, case["heads"], LATENT), gen)
        s["scores"] = _sums((case["batch"], max(n) + t), gen)
        s["out"] = torch.zeros_like(s["scores"])
        s["lse"] = torch.empty(s["q"].shape[:3], device="cuda")
        for b, length in enumerate(n):  # what the decode step before it returned
            k = _latent_rows(s, b, length + t).float()
            x = MLA_SCALE * torch.einsum("thd,kd->thk", s["q"][b].float(), k)
            late = torch.arange(length + t, device="cuda")[None] > length + torch.arange(t, device="cuda")[:, None]
            s["lse"][b] = x.masked_fill_(late[:, None], -math.inf).logsumexp(-1)
    elif op == "select":
        s["scores"] = _sums((case["batch"], max(n)), gen)
        s["kept"] = torch.full((case["batch"], case["keep"]), -1, dtype=torch.int32, device="cuda")
        s["kept_lengths"] = torch.empty(case["batch"], dtype=torch.int32, device="cuda")
    elif op == "compact":
        s |= _latent_cache(case, n, gen)
        s["scores"] = _sums((case["batch"], max(n)), gen)
        s["kept"] = torch.full((case["batch"], case["keep"]), -1, dtype=torch.int32, device="cuda")
        s["kept_lengths"] = torch.empty(case["batch"], dtype=torch.int32, device="cuda")
        _plain_select(s, case)
    elif op == "attend":
        t = case["q_len"]
        s |= _mha_cache(case, [x + t for x in n], gen)
        s["q"] = _normal((case["batch"], t, case["heads"], case["dim"]), gen)
        s["out"] = torch.empty_like(s["q"])
        s["lse"] = torch.empty(s["q"].shape[:3], device="cuda")
    else:
        s |= _mha_cache(case, [x + case["q_len"] for x in n], gen)
        s["k"] = _normal((case["batch"], case["q_len"], case["kv_heads"], case["dim"]), gen)
        s["v"] = _normal((case["batch"], case["q_len"], case["kv_heads"], case["dim"]), gen)
    return s


def _latent_rows(s, b, n):
    """Rows 0 .. n - 1 of request b, dequantised and rounded to bf16 as the decode reads them."""
    case = s["case"]
    t = torch.arange(n, device="cuda")
    page, slot = t // case["page"], t % case["page"]
    blk = s["table"][b, page].long()
    sblk = blk if s["stable"] is None else s["stable"][b, page].long()
    codes = s["blocks"].view(torch.float8_e4m3fn)[blk, 0, case["layer"], slot, 0]
    return (codes.float() * s["scales"][sblk, 0, case["layer"], slot, 0]).bfloat16()


# ---------------------------------------------------------------- plain forms
def _places(table, page, n):
    """(block, slot) of positions 0 .. n - 1 for every request; unused entries read block 0."""
    t = torch.arange(n, device=table.device)
    return table[:, t // page].long().clamp_(min=0), (t % page).expand(table.shape[0], n)


def _plain_weights(s, case):
    t, n = case["q_len"], s["scores"].shape[1]
    blk, slot = _places(s["table"], case["page"], n)
    sblk = blk if s["stable"] is None else _places(s["stable"], case["page"], n)[0]
    keys = s["blocks"].view(torch.float8_e4m3fn)[blk, 0, case["layer"], slot, 0].float()
    scale = s["scales"][sblk, 0, case["layer"], slot, 0, 0]
    x = torch.einsum("bthd,bkd->bthk", s["q"].float(), keys) * (MLA_SCALE * scale[:, None, None])
    at = torch.arange(n, device=x.device)
    last = s["lengths"][:, None] + torch.arange(t, device=x.device)
    seen = at <= last[..., None]
    p = torch.where(seen[:, :, None], torch.exp(x - s["lse"][..., None]), 0.0).sum((1, 2))
    old = torch.where(at < s["lengths"][:, None], s["scores"], 0.0)
    return torch.where(at < s["lengths"][:, None] + t, old + p, s["out"])


def _plain_select(s, case):
    scores, n, keep = s["scores"], s["lengths"][:, None], case["keep"]
    at = torch.arange(scores.shape[1], device=scores.device)
    rank = torch.where(at < n, scores.double(), -math.inf)
    rank = torch.where((at < n) & ((at < case["sink"]) | (at >= n - case["recent"])), math.inf, rank)
    order = torch.sort(rank, dim=1, descending=True, stable=True).indices[:, :keep]
    count = torch.clamp(n, max=keep)
    slot = torch.arange(order.shape[1], device=scores.device)
    order = torch.sort(torch.where(slot < count, order, scores.shape[1]), dim=1).values
    kept = s["kept"][:, :order.shape[1]]
    kept.copy_(torch.where(slot < count, order.to(torch.int32), kept))
    s["kept_lengths"].copy_(count[:, 0])
    return s["kept"], s["kept_lengths"]


def _plain_compact(s, case):
    page, layer = case["page"], case["layer"]
    b, j = torch.nonzero(torch.arange(case["keep"], device="cuda") < s["kept_lengths"][:, None], as_tuple=True)
    src = s["kept"][b, j].long()
    stable = s["table"] if s["stable"] is None else s["stable"]
    for store, table in ((s["blocks"], s["table"]), (s["scales"], stable)):
        rows = store[table[b, src // page].long(), :, layer, src % page]
        store[table[b, j // page].long(), :, layer, j % page] = rows
    s["scores"][b, j] = s["scores"][b, src]
    return s["blocks"], s["scales"], s["scores"]


def _plain_attend(s, case):
    t, n, kvh = case["q_len"], s["max_length"] + case["q_len"], case["kv_heads"]
    blk, slot = _places(s["table"], case["page"], n)
    kv = s["blocks"].view(torch.float8_e4m3fn) if case["fp8"] else s["blocks"]
    k, v = kv[blk, 0, case["layer"], slot].float(), kv[blk, 1, case["layer"], slot].float()
    if case["fp8"]:
        k, v = (x * s["scales"][blk, i, case["layer"], slot] for i, x in ((0, k), (1, v)))
    q = s["q"].float().unflatten(2, (kvh, -1))
    x = torch.einsum("btgrd,bkgd->btgrk", q, k) / math.sqrt(case["dim"])
    last = s["lengths"][:, None] + torch.arange(t, device=x.device)
    hidden = torch.arange(n, device=x.device) > last[..., None]
    x = x.masked_fill(hidden[:, :, None, None], -math.inf)
    # values behind a request's end may be anything, infinities among them
    v = v.masked_fill(hidden[:, -1, :, None, None], 0.0)
    m = x.amax(-1, keepdim=True)
    p = torch.exp(x - m)
    l = p.sum(-1, keepdim=True)
    out = torch.einsum("btgrk,bkgd->btgrd", p / l, v)
    return out.flatten(2, 3).bfloat16(), (m + torch.log(l)).flatten(2)


def _plain_store(s, case):
    t = case["q_len"]
    at = s["lengths"][:, None].long() + torch.arange(t, device="cuda")
    blk, slot = s["table"].gather(1, at // case["page"]).long(), at % case["page"]
    for i, x in ((0, s["k"]), (1, s["v"])):
        if case["fp8"]:
            codes, scale = _quantise(x)
            s["blocks"][blk, i, case["layer"], slot] = codes.view(torch.uint8)
            s["scales"][blk, i, case["layer"], slot] = scale
        else:
            s["blocks"][blk, i, case["layer"], slot] = x
    return (s["blocks"].view(torch.float8_e4m3fn), s["scales"]) if case["fp8"] else s["blocks"]


_PLAIN = {"weights": _plain_weights, "select": _plain_select, "compact": _plain_compact, "attend": _plain_attend,
          "store": _plain_store}


# ---------------------------------------------------------------- the framework's calls
def _own_run(s, case):
    import paged_fp8_kv_mla_b200 as M
    op = case["op"]
    if op == "weights":
        return M.accumulate_weights(s["q"], s["lse"], s["blocks"], s["scales"], s["lengths"], s["table"], s["stable"],
                                    case["q_len"], s["max_length"], case["layer"], MLA_SCALE, s["scores"],
                                    out=s["out"])
    if op == "select":
        return M.select_keys(s["scores"], s["lengths"], s["max_length"], case["keep"], case["recent"], case["sink"],
                             kept=s["kept"], kept_lengths=s["kept_lengths"])
    if op == "compact":
        return M.compact_cache(s["kept"], s["kept_lengths"], s["table"], s["stable"], case["layer"], s["blocks"],
                               s["scales"], s["scores"])
    if op == "attend":
        return M.mha_decode(s["q"], s["blocks"], s["scales"], s["lengths"], s["table"], s["stable"], case["q_len"],
                            s["max_length"], case["layer"], 1.0 / math.sqrt(case["dim"]), out=s["out"], lse=s["lse"])
    M.mha_kv_store(s["k"], s["v"], s["lengths"], s["table"], s["stable"], case["layer"], s["blocks"], s["scales"])
    return (s["blocks"].view(torch.float8_e4m3fn), s["scales"]) if case["fp8"] else s["blocks"]


def run(state):
    case = state["case"]
    return _own_run(state, case) if own else _PLAIN[case["op"]](state, case)


# ---------------------------------------------------------------- what a pass cannot do without
def work(case):
    op, n = case["op"], _lengths(case)
    b = case["batch"]
    if op == "weights":
        t, h = case["q_len"], case["heads"]
        keys = sum(n) + b * t
        pairs = sum(x + i + 1 for x in n for i in range(t))
        return {"bytes": keys * (LATENT + 4 + 4) + sum(n) * 4 + b * t * h * (LATENT * 2 + 4),
                "flops": 2 * LATENT * h * pairs}
    if op == "select":
        return {"bytes": 4 * sum(n) + 4 * sum(min(x, case["keep"]) for x in n) + 8 * b, "flops": sum(n)}
    if op == "compact":
        rows = sum(case["keep"] for x in n if x > case["keep"])
        return {"bytes": rows * (2 * (LATENT + 4 + 4) + 4) + 4 * b, "flops": 0}
    kvh, d = case["kv_heads"], case["dim"]
    row = kvh * (d + 4 if case["fp8"] else 2 * d)
    if op == "attend":
        t, h = case["q_len"], case["heads"]
        keys = sum(n) + b * t
        pairs = sum(x + i + 1 for x in n for i in range(t))
        return {"bytes": keys * 2 * row + b * t * h * (4 * d + 4), "flops": 4 * d * h * pairs}
    tokens = b * case["q_len"]
    return {"bytes": tokens * 2 * (2 * kvh * d + row), "flops": tokens * 2 * kvh * d * (2 if case["fp8"] else 0)}


# ---------------------------------------------------------------- 64-bit values
def exact(case, seed):
    op = case["op"]
    if op in ("select", "compact"):
        return None  # indices and moved rows: nothing is computed in floating point
    s = prepare(case, seed)
    page, layer, t = case["page"], case["layer"], case["q_len"]
    if op == "store":
        if not case["fp8"]:
            return None
        scales = s["scales"].double()
        for b, length in enumerate(_lengths(case)):
            pos = torch.arange(length, length + t, device="cuda")
            for i, x in ((0, s["k"][b]), (1, s["v"][b])):
                top = x.double().abs().max(-1, keepdim=True).values / 448
                top[top == 0] = 1
                scales[s["table"][b, pos // page].long(), i, layer, pos % page] = top
        return None, scales
    e4m3 = torch.arange(256, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn).double()
    outs, lses = [], []
    result = s["out"].double() if op == "weights" else None
    for b, length in enumerate(_lengths(case)):
        n = length + t
        pos = torch.arange(n, device="cuda")
        blk = s["table"][b, pos // page].long()
        late = pos[None] > length + torch.arange(t, device="cuda")[:, None]
        q = s["q"][b].double()
        if op == "weights":
            sblk = blk if s["stable"] is None else s["stable"][b, pos // page].long()
            rows = e4m3[s["blocks"][blk, 0, layer, pos % page, 0].int()] * s["scales"][sblk, 0, layer, pos % page, 0].double()
            x = (q.reshape(-1, LATENT) @ rows.T).reshape(t, -1, n) * MLA_SCALE
            weight = torch.exp(x - s["lse"][b].double()[..., None])
            weight[late[:, None].expand_as(weight)] = 0
            result[b, :n] = weight.sum((0, 1))
            result[b, :length] += s["scores"][b, :length].double()
            continue
        k, v = (s["blocks"][blk, i, layer, pos % page] for i in (0, 1))
        if case["fp8"]:
            k, v = (e4m3[y.int()] * s["scales"][blk, i, layer, pos % page].double() for i, y in ((0, k), (1, v)))
        group = case["heads"] // case["kv_heads"]
        k = k.double().permute(1, 2, 0)[None]                       # [1, kv heads, dim, n]
        v = v.double().permute(1, 0, 2)[None]                       # [1, kv heads, n, dim]
        x = (q.reshape(t, case["kv_heads"], group, -1) @ k) * case["dim"] ** -0.5
        x[late[:, None, None].expand_as(x)] = -math.inf
        lse = torch.logsumexp(x, -1, keepdim=True)
        outs.append((torch.exp(x - lse) @ v).reshape(t, case["heads"], -1))
        lses.append(lse.reshape(t, -1))
    return result if op == "weights" else (torch.stack(outs), torch.stack(lses))
