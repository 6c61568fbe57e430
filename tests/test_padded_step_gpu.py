"""A decode step over a padded batch (GPU): sequences of length 0 behind and
between the others, as a captured graph of a fixed batch size has them."""

import pytest
import torch

import paged_kv_cache_471_b200 as pa
from kv_reference import FORMATS, Cache, angle_table, attention, is_block

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.mark.parametrize("captured", [False, True])
@pytest.mark.parametrize("kv", FORMATS)
def test_rows_of_empty_sequences_are_padding(kv, captured):
    """They are not read or written, give a zero output row and set no status bit."""
    Hk, Hq, D, B = 2, 4, 64, 16
    lens = [17, 0, 1, 40, 0, 0]
    cache = Cache(kv, lens, Hk, D, B, seed=31)
    kc, vc = cache.packed(DEV)
    ks, vs = cache.scales(DEV)
    bt, sl = cache.tables.to(DEV), cache.lens.to(DEV)
    g = torch.Generator().manual_seed(32)
    host = {n: torch.randn((6, h, D), generator=g).to(torch.bfloat16)
            for n, h in (("query", Hq), ("key", Hk), ("value", Hk))}
    for t in host.values():
        t[1] = float("nan")
    rows = {n: t.to(DEV) for n, t in host.items()}
    angles = angle_table(40, D)
    table = angles.to(DEV)
    turned = torch.full_like(rows["query"], 5.0)
    out = torch.full_like(turned, float("nan"))

    def step():
        pa.append_kv(kc, vc, rows["key"], rows["value"], bt, sl, B, kv, ks, vs, cos_sin=table,
                     query=rows["query"], query_out=turned)
        pa.decode(out, turned, kc, vc, Hk, 0.125, bt, sl, B, 40, kv, ks, vs)

    pa.read_status(device=DEV, clear=True)
    if captured:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step()
        graph.replay()
    else:
        step()
    torch.cuda.synchronize()
    assert pa.read_status(device=DEV) == 0
    live = [s for s, t in enumerate(lens) if t]
    empty = [s for s, t in enumerate(lens) if not t]
    assert (turned[empty] == 5.0).all() and (out[empty] == 0).all()
    some = Cache(kv, [17], Hk, D, B)
    some.__dict__.update(cache.__dict__)
    some.tables, some.lens = cache.tables[live], cache.lens[live]
    start = torch.arange(len(live) + 1, dtype=torch.int32)
    q = some.append(host["key"][live], host["value"][live], start, angles,
                    query=host["query"][live], dtype=torch.float32).to(torch.bfloat16)
    assert torch.equal(turned[live].cpu(), q)
    k, v = cache.unpacked(kc, vc)
    for a, b in ((k, some.k), (v, some.v)):
        assert torch.equal(torch.nan_to_num(a.float(), 7.5), torch.nan_to_num(b.float(), 7.5))
    if is_block(kv):
        assert torch.equal(torch.nan_to_num(ks.cpu(), 7.5), torch.nan_to_num(some.ks, 7.5))
    ref, tol = attention(some, q, start, 0.125)
    # (Decode over bf16 pages also rounds the sum's weights: twice u A.)
    assert ((out[live].cpu().double() - ref).abs() <= 2 * tol).all()
