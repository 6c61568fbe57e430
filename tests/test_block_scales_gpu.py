"""Decode attention over 8-bit caches with a scale per block and kv head (GPU),
against the definition in fp64 within the rounding errors kv_reference counts."""

import math

import pytest
import torch

import paged_kv_cache_471_b200 as pa
from kv_reference import BLOCK_FORMATS, Cache, attention

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def decode(cache, query, scale, max_len=None, out=None, **kw):
    kc, vc = cache.packed(DEV)
    ks, vs = cache.scales(DEV)
    out = torch.full_like(query, float("nan"), device=DEV) if out is None else out
    max_len = int(cache.lens.max()) if max_len is None else max_len
    fn = kw.pop("fn", pa.decode)
    fn(out, query.to(DEV), kc, vc, cache.Hk, scale, cache.tables.to(DEV), cache.lens.to(DEV),
       cache.B, max_len, cache.kv, ks, vs, **kw)
    torch.cuda.synchronize()
    return out


def check(out, cache, query, scale, **kw):
    S = query.shape[0]
    ref, tol = attention(cache, query, torch.arange(S + 1), scale, **kw)
    err = (out.cpu().double() - ref).abs()
    assert (err <= tol).all(), float((err / tol.clamp(min=1e-300)).max())


def queries(S, Hq, D, seed=2, amp=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn((S, Hq, D), generator=g) * amp).to(torch.bfloat16)


@pytest.mark.parametrize("G", [1, 3, 8, 9, 16])
@pytest.mark.parametrize("D,B", [(128, 16), (128, 32), (64, 16), (64, 32)])
@pytest.mark.parametrize("kv", BLOCK_FORMATS)
def test_shapes_and_lengths(kv, D, B, G):
    lens = [1, 0, 17, 5 * B, 700, 33, 2]
    cache = Cache(kv, lens, 2, D, B, seed=G, pow2=G % 2 == 1)
    q = queries(len(lens), 2 * G, D)
    pa.read_status(device=DEV, clear=True)
    out = decode(cache, q, 1 / math.sqrt(D))
    check(out, cache, q, 1 / math.sqrt(D))
    assert (out[1] == 0).all()
    assert pa.read_status(device=DEV) == 0


@pytest.mark.parametrize("kw", [dict(partition_pages=3), dict(partition_pages=40),
                                dict(schedule="balanced"), dict(schedule="partitioned"),
                                dict(stages=5), dict(stages=6, num_sms=3),
                                dict(partition_pages=70), dict(mha_cuda_cores=True)])
@pytest.mark.parametrize("kv,B", [("fp8_e4m3_block", 16), ("int8_block", 32)])
def test_schedules(kv, B, kw):
    """Windows of more than 32 stages per warp, split and balanced plans."""
    lens = [9000, 3, 0, 4097, 8192 - 5]
    cache = Cache(kv, lens, 2, 128, B, seed=4)
    q = queries(len(lens), 8, 128)
    out = decode(cache, q, 0.09, **kw)
    check(out, cache, q, 0.09)
    assert pa.read_status(device=DEV) == 0


def test_split_tail_and_longest_first():
    """Whole units in two waves and a tail, mixed lengths: the plan of a batch of
    900 units on this GPU."""
    S, Hk = 100, 9
    lens = [(i * 37) % 500 + 16 for i in range(S)]
    p = pa.plan(S, Hk, Hk, 64, 16, 2048, "int8_block")
    assert p["tail_units"] > 0 and p["longest_first"]
    cache = Cache("int8_block", lens, Hk, 64, 16, seed=6)
    wide = torch.full((S, 128), -1, dtype=torch.int32)
    wide[:, :cache.tables.shape[1]] = cache.tables
    cache.tables = wide
    q = queries(S, Hk, 64)
    out = decode(cache, q, 0.125, max_len=2048)
    check(out, cache, q, 0.125)


@pytest.mark.parametrize("S,B,prefix", [(5, 16, 40), (5, 32, 3), (24, 16, 70), (40, 32, 5)])
@pytest.mark.parametrize("kv", BLOCK_FORMATS)
def test_shared_prefix(kv, S, B, prefix):
    """Few sequences (a CTA per row group) and many (the shared ring)."""
    lens = [prefix * B + (i * 29) % 200 for i in range(S)]
    cache = Cache(kv, lens, 2, 128, B, seed=8, shared_blocks=prefix)
    q = queries(S, 8, 128)
    out = decode(cache, q, 0.08, shared_prefix_blocks=prefix)
    check(out, cache, q, 0.08)
    assert pa.read_status(device=DEV) == 0


def test_alibi_and_noalloc():
    cache = Cache("fp8_e4m3_block", [300, 20], 2, 128, 16, seed=9)
    q = queries(2, 4, 128)
    slopes = torch.tensor([0.5, 0.25, 0.125, 0.0625])
    out = decode(cache, q, 0.09, alibi_slopes=slopes.to(DEV))
    check(out, cache, q, 0.09, alibi=slopes)
    out = decode(cache, q, 0.09, fn=pa.decode_noalloc)
    check(out, cache, q, 0.09)


@pytest.mark.parametrize("kv", BLOCK_FORMATS)
def test_scales_of_very_different_sizes(kv):
    """Blocks whose scales lie many binary orders apart, blocks of zeros with the
    smallest scale and with a scale of 0: the denominator counts every token
    whatever its value's size."""
    lens = [16 * 12] * 3
    cache = Cache(kv, lens, 2, 64, 16, seed=10)
    q = queries(3, 4, 64)
    for s in range(3):
        for j in range(12):
            blk = int(cache.tables[s, j])
            cache.vs[blk] *= 2.0 ** [0, -40, 13, -100, 5, 0, -20, 30, 0, -60, 1, -3][j]
            if s == 1:  # all small
                cache.vs[blk] *= 2.0 ** -30
            if s == 2:
                cache.vs[blk] = [1.0, 0.0, 2.0 ** -100][j % 3]
                if j % 3:
                    cache._raw(cache.v)[blk] = 0
    out = decode(cache, q, 0.125)
    check(out, cache, q, 0.125)
    out = decode(cache, q, 0.125, partition_pages=2)
    check(out, cache, q, 0.125)


def test_large_queries_and_keys():
    """Logits in the thousands: the running maximum keeps every weight finite."""
    cache = Cache("int8_block", [100, 50], 1, 64, 16, seed=11, amplitude=200.0)
    q = queries(2, 2, 64, amp=50.0)
    out = decode(cache, q, 1.0)
    assert torch.isfinite(out.float()).all()
    # the largest logit of each row is far ahead: the row is that token's value
    for s in range(2):
        k, v, _ = cache.values(s)
        for h in range(2):
            x = k[:, 0] @ q[s, h].double()
            top = torch.topk(x, 2)
            assert top.values[0] - top.values[1] > 40
            want = v[top.indices[0], 0]
            assert ((out[s, h].cpu().double() - want).abs() <= 2.0 ** -8 * want.abs()
                    + 2.0 ** -11 * want.abs()).all()


def test_bad_block_ids_are_skipped():
    cache = Cache("int8_block", [16 * 6], 2, 128, 16, seed=12)
    q = queries(1, 4, 128)
    good = cache.tables.clone()
    keep = [0, 2, 3, 5]
    cache.tables[0, 1], cache.tables[0, 4] = cache.num_blocks, -7
    pa.read_status(device=DEV, clear=True)
    out = decode(cache, q, 0.09)
    assert pa.read_status(device=DEV, clear=True) == pa.PA_DEV_BAD_BLOCK_ID
    cache.tables = good[:, keep].contiguous()
    cache.lens = torch.tensor([64], dtype=torch.int32)
    check(out, cache, q, 0.09)


def test_refusals():
    cache = Cache("fp8_e4m3_block", [40], 2, 128, 16)
    q = queries(1, 4, 128)
    for kw in (dict(schedule="dynamic"), dict(fp8_compute=True)):
        with pytest.raises(pa.PagedAttentionError):
            decode(cache, q, 0.1, **kw)
    cache.ks = cache.ks[:, :1].contiguous()
    with pytest.raises(ValueError):
        decode(cache, q, 0.1)


def test_two_graphs_and_an_eager_call_keep_their_workspaces():
    """Two captured calls with split plans, replayed on two streams at once, and
    an eager call between: each has a workspace of its own."""
    cache = Cache("int8_block", [6000], 2, 128, 16, seed=13)
    q = [queries(1, 8, 128, seed=s) for s in range(3)]
    kc, vc = cache.packed(DEV)
    ks, vs = cache.scales(DEV)
    bt, sl = cache.tables.to(DEV), cache.lens.to(DEV)
    assert pa.plan(1, 8, 2, 128, 16, 6000, "int8_block")["num_partitions"] > 1
    outs = [torch.empty_like(x, device=DEV) for x in q]
    qs = [x.to(DEV) for x in q]
    graphs, streams = [], [torch.cuda.Stream(), torch.cuda.Stream()]
    for i in range(2):
        g = torch.cuda.CUDAGraph()
        streams[i].wait_stream(torch.cuda.current_stream())
        with torch.cuda.graph(g, stream=streams[i]):
            for _ in range(20):
                pa.decode(outs[i], qs[i], kc, vc, 2, 0.09, bt, sl, 16, 6000, "int8_block", ks, vs)
        graphs.append(g)
    torch.cuda.synchronize()
    for i in range(2):
        with torch.cuda.stream(streams[i]):
            graphs[i].replay()
    pa.decode(outs[2], qs[2], kc, vc, 2, 0.09, bt, sl, 16, 6000, "int8_block", ks, vs)
    torch.cuda.synchronize()
    for i in range(3):
        check(outs[i], cache, q[i], 0.09)


@pytest.mark.parametrize("kv", BLOCK_FORMATS)
def test_copied_blocks_bring_their_scales(kv):
    cache = Cache(kv, [16 * 20], 3, 128, 16, seed=14, spare=30)
    kc, vc = cache.packed(DEV)
    ks, vs = cache.scales(DEV)
    src = cache.tables[0, :10].long()
    used = set(cache.tables[0].tolist())
    dst = torch.tensor([b for b in range(cache.num_blocks) if b not in used][:10])
    want = [t.clone() for t in (kc.view(torch.uint8), vc.view(torch.uint8), ks, vs)]
    for t in want:
        t[dst] = t[src]
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    bad = torch.tensor([cache.num_blocks])
    pa.copy_blocks(kc, vc, torch.cat([src, bad]).to(DEV), torch.cat([dst, bad]).to(DEV), kv,
                   status=status, k_scale=ks, v_scale=vs)
    torch.cuda.synchronize()
    assert int(status) == pa.PA_DEV_BAD_BLOCK_ID
    for t, w in zip((kc.view(torch.uint8), vc.view(torch.uint8), ks, vs), want):
        assert torch.equal(torch.nan_to_num(t.float(), 7.5), torch.nan_to_num(w.float(), 7.5))
    with pytest.raises(TypeError):
        pa.copy_blocks(kc, vc, src.to(DEV), dst.to(DEV), kv)
