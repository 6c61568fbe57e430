"""One workspace serves calls of every kind in turn (GPU): what a call leaves
behind in it means nothing to the next one."""

import pytest
import torch

import paged_kv_cache_471_b200 as pa
from kv_reference import Cache, attention

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def check(out, cache, query, start, scale, factor=1.0):
    ref, tol = attention(cache, query, start, scale)
    err = (out.cpu().double() - ref).abs()
    assert (err <= factor * tol).all(), float((err / tol.clamp(min=1e-300)).max())


def queries(T, Hq, D, seed=2):
    g = torch.Generator().manual_seed(seed)
    return torch.randn((T, Hq, D), generator=g).to(torch.bfloat16)


def test_a_prefill_s_partials_are_no_counts_of_the_dynamic_schedule():
    """Values of (-1, 0, -1, 0, ..) make a split prefill leave pairs of floats
    whose second is 0.0, where the dynamic schedule keeps its counters: in a
    fresh workspace, whose generation is 0 too, they must not read as counts."""
    Hk, G, D, B = 2, 4, 128, 16
    cache = Cache("bf16", [1500, 700], Hk, D, B, seed=21)
    bt, sl = cache.tables.to(DEV), cache.lens.to(DEV)
    kc, vc = cache.packed(DEV)
    flat = vc.clone()
    flat[:, :, 0::2] = -1.0
    flat[:, :, 1::2] = 0.0
    q = queries(2, Hk * G, D)
    few = queries(7, Hk * G, D).to(DEV)
    start = torch.tensor([0, 4, 7], dtype=torch.int32, device=DEV)
    need = max(pa.prefill_workspace_size(7, 2, Hk * G, Hk, D, B, 1500, "bf16", 8),
               pa.workspace_size(2, Hk * G, Hk, D, B, 1500, "bf16", schedule="dynamic"))
    ws = torch.zeros(need, dtype=torch.uint8, device=DEV)
    body = pa.WORKSPACE_HEADER_BYTES + pa.WORKSPACE_MERGE_COUNT_BYTES
    out = torch.empty_like(q, device=DEV)
    for _ in range(3):  # generations 0, 1, 2
        pa.prefill(torch.empty_like(few), few, kc, flat, Hk, 0.09, bt, sl, start, B, 1500,
                   workspace_tensor=ws, partition_pages=8)
        pair = ws[body:body + 8].view(torch.float32).cpu()
        assert float(pair[0]) < 0 and float(pair[1]) == 0
        pa.decode(out, q.to(DEV), kc, vc, Hk, 0.09, bt, sl, B, 1500, workspace_tensor=ws,
                  schedule="dynamic")
        torch.cuda.synchronize()
        # (Decode over bf16 pages also rounds the sum's weights: twice u A.)
        check(out, cache, q, torch.arange(3), 0.09, factor=2.0)
        out.fill_(float("nan"))
    assert pa.read_status(ws) == 0


def test_a_balanced_call_s_page_counts_are_no_counts_of_the_dynamic_schedule():
    """The balanced schedule leaves the running page counts of the sequences, small
    integers, where the dynamic schedule keeps its counters: at no generation may
    they read as pages that were handed out."""
    Hk, G, D, B = 1, 4, 64, 16
    lens = [16, 9, 16, 1, 13, 16]
    cache = Cache("bf16", lens, Hk, D, B, seed=22)
    bt, sl = cache.tables.to(DEV), cache.lens.to(DEV)
    kc, vc = cache.packed(DEV)
    q = queries(len(lens), Hk * G, D)
    q_dev = q.to(DEV)
    need = max(pa.workspace_size(len(lens), Hk * G, Hk, D, B, 16, "bf16", schedule=s)
               for s in ("dynamic", "balanced"))
    ws = torch.zeros(need, dtype=torch.uint8, device=DEV)
    for _ in range(9):
        for schedule in ("balanced", "dynamic"):
            out = torch.full_like(q_dev, float("nan"))
            pa.decode(out, q_dev, kc, vc, Hk, 0.125, bt, sl, B, 16, workspace_tensor=ws,
                      schedule=schedule)
            torch.cuda.synchronize()
            check(out, cache, q, torch.arange(len(lens) + 1), 0.125, factor=2.0)
    assert pa.read_status(ws) == 0
