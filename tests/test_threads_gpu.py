"""Calls of two host threads on one stream, without workspaces of their own
(GPU): the launches of one call stay together."""

import threading

import pytest
import torch

import paged_kv_cache_471_b200 as pa
from kv_reference import Cache, attention

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def queries(T, Hq, D, seed):
    g = torch.Generator().manual_seed(seed)
    return torch.randn((T, Hq, D), generator=g).to(torch.bfloat16)


@pytest.mark.parametrize("kind", ["decode", "dynamic", "prefill", "mixed"])
def test_two_threads_on_one_stream(kind):
    """Split calls: a kernel that leaves partials and one that merges them.  The
    stream is busy at first, so that launches wait for room in its queue."""
    Hk, Hq, D, B, calls = 2, 8, 128, 16, 1200
    cache = Cache("bf16", [3000], Hk, D, B, seed=41)
    kc, vc = cache.packed(DEV)
    bt, sl = cache.tables.to(DEV), cache.lens.to(DEV)
    assert pa.plan(1, Hq, Hk, D, B, 3000)["num_partitions"] > 1
    jobs = []
    for i in range(2):
        prefill = kind == "prefill" or (kind == "mixed" and i)
        n = 5 + i if prefill else 1
        q = queries(n, Hq, D, 42 + i)
        ref, tol = attention(cache, q, torch.tensor([0, n]), 0.09)
        outs = torch.full((calls, n, Hq, D), float("nan"), dtype=torch.bfloat16, device=DEV)
        jobs.append((prefill, q.to(DEV), torch.tensor([0, n], dtype=torch.int32, device=DEV),
                     outs, ref, 2 * tol))
    torch.cuda.synchronize()
    torch.cuda._sleep(200_000_000)  # about 0.1 s
    gate = threading.Barrier(2)
    failed = []

    def work(prefill, q, start, outs, *_):
        try:
            gate.wait()
            for out in outs:
                if prefill:
                    pa.prefill(out, q, kc, vc, Hk, 0.09, bt, sl, start, B, 3000,
                               partition_pages=64)
                else:
                    pa.decode(out, q, kc, vc, Hk, 0.09, bt, sl, B, 3000,
                              schedule="dynamic" if kind == "dynamic" else "auto")
        except Exception as e:
            failed.append(e)

    threads = [threading.Thread(target=work, args=j) for j in jobs]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not failed
    for *_, outs, ref, tol in jobs:
        err = (outs.cpu().double() - ref).abs()
        wrong = (~(err <= tol)).flatten(1).any(dim=1).nonzero().flatten()
        assert not len(wrong), wrong
