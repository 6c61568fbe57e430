"""Prefill over many key tiles (GPU): every loader form -- each cache type, head
size and block size -- passes enough tiles that its rings of pages, stages and
page infos come round several times, whole and split."""

import math

import pytest
import torch

import paged_kv_cache_471_b200 as pa
from kv_reference import FORMATS, Cache, attention

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.mark.parametrize("D,B", [(128, 16), (128, 32), (64, 16), (64, 32)])
@pytest.mark.parametrize("kv", FORMATS)
def test_many_tiles(kv, D, B):
    """31 and 9 tiles of 128 keys for each of two row tiles, in one partition, in
    the planner's and in forced ones; rows nobody owns in front and behind."""
    new, past = [40, 300, 1, 0], [3900, 900, 2000, 17]
    cache = Cache(kv, [n + p for n, p in zip(new, past)], 2, D, B, seed=23, pow2=D == 64)
    start = torch.tensor([2, 42, 342, 343, 343], dtype=torch.int32)
    g = torch.Generator().manual_seed(24)
    q = torch.randn((345, 8, D), generator=g).to(torch.bfloat16)
    scale = 1 / math.sqrt(D)
    ref, tol = attention(cache, q, start, scale)
    kc, vc = cache.packed(DEV)
    ks, vs = cache.scales(DEV)
    bt, sl, st, qd = (t.to(DEV) for t in (cache.tables, cache.lens, start, q))
    pa.read_status(device=DEV, clear=True)
    for pages in (4000 // B, 0, 128 // B, 640 // B):
        out = torch.full_like(qd, float("nan"))
        pa.prefill(out, qd, kc, vc, 2, scale, bt, sl, st, B, 3940, kv, ks, vs,
                   partition_pages=pages)
        torch.cuda.synchronize()
        got = out.cpu()
        assert torch.isnan(got[:2].float()).all() and torch.isnan(got[343:].float()).all()
        err = (got[2:343].double() - ref[2:343]).abs()
        assert (err <= tol[2:343]).all(), (pages, float((err / tol[2:343]).max()))
    assert pa.read_status(device=DEV) == 0
