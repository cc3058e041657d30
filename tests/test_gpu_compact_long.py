"""Compaction in place over many chunks: every kernel's ring of chunks turns over several times, and the columns of
scales and sums take several chunks.  Every byte of the pool is compared with the definition.

Which kernel moves the rows follows from the number of 64-byte (32-byte) columns of all requests beside the 148
SMs: at least as many columns of 64 bytes: chunks of 256 rows, 3 deep; else more columns of 32 bytes than SMs:
chunks of 512 rows, 4 deep; else 1024 rows, 5 deep.  The scales and sums go in chunks of 8 words a thread."""
import pytest
import torch

from tests.cache_ref import LatentCache, MhaCache
from tests.test_gpu_select_compact import check_compact, pick

pytestmark = pytest.mark.gpu


def lists(kind, lengths, keep, seed=3):
    out = []
    for b, n in enumerate(lengths):
        k = min(n, keep)
        if kind == "random":
            out.append(pick(n, k, seed + b))
        elif kind == "dense":                                     # all but the first: each chunk's sources reach into the next
            out.append(list(range(1, n)))
        elif kind == "late":                                      # nothing moves until far in, then by one row
            out.append([j for j in range(n) if j != n // 2])
        else:                                                     # the tail alone: every row moves far
            out.append(list(range(n - k, n)))
    return out


@pytest.mark.parametrize("kind", ["random", "dense", "late", "tail"])
@pytest.mark.parametrize("lengths,keep,page,kw", [
    ([14000], 9500, 64, {}),                                      # 1024 rows a chunk, several of scales and of sums
    ([7000, 300, 6500], 6200, 48, dict(layers=2, layer=1, own_scale_pages=True)),
    ([4700] + [900] * 8 + [2600], 4200, 64, {}),                  # 512 rows a chunk
    ([4000] + [100] * 17 + [1300], 3500, 32, {}),                 # 256 rows a chunk
])
def test_latent_cache(lengths, keep, page, kw, kind):
    cache = LatentCache(lengths, page, seed=len(lengths), **kw)
    check_compact(cache, lists(kind, lengths, keep), torch.rand((len(lengths), max(lengths)), generator=torch.Generator().manual_seed(2)))


@pytest.mark.parametrize("kind", ["random", "dense"])
@pytest.mark.parametrize("fp8,heads,dim,lengths,keep", [
    (True, 8, 128, [4400, 3500, 700], 3200),                      # 512 rows a chunk, six chunks of scales
    (True, 1, 64, [9000], 7000),                                  # 1024 rows a chunk
    (True, 5, 64, [9900, 10], 7100),                              # rows of 320 bytes, scales that straddle chunks
    (False, 2, 64, [7000, 6000], 5500),
    (True, 8, 128, [1500] * 5, 1100),                             # 256 rows a chunk
])
def test_multi_head_cache(fp8, heads, dim, lengths, keep, kind):
    cache = MhaCache(lengths, 32, heads, dim, fp8, seed=6, own_scale_pages=True)
    check_compact(cache, lists(kind, lengths, keep), torch.rand((len(lengths), max(lengths)), generator=torch.Generator().manual_seed(2)))
