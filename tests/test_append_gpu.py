"""Appending tokens to the paged cache (pa_append_kv, GPU).  What is written is
fixed to the bit by its description (fp32 products and sums, each rounded once,
then one rounding to the cache's type), so it is compared with the reference in
fp32 to the bit, and with the formula in fp64 within half a step."""

import math

import pytest
import torch

import paged_kv_cache_471_b200 as pa
from kv_reference import (BLOCK_FORMATS, FORMATS, Cache, angle_table, is_block, rotate)

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def same(a, b):
    """Equal to the bit, but for the sign and payload of NaNs."""
    a, b = a.cpu(), b.cpu()
    assert a.dtype == b.dtype and a.shape == b.shape
    if a.dtype in (torch.int8, torch.int32):
        return torch.equal(a, b)
    a, b = a.float(), b.float()
    return torch.equal(torch.nan_to_num(a, nan=777.0), torch.nan_to_num(b, nan=777.0)) \
        and torch.equal(torch.isnan(a), torch.isnan(b))


def make(kv, new, past, Hk, Hq, D, B, R, seed=1, pad=0, fused=True, **kw):
    """A cache that holds `past` tokens of each sequence, the tables for the new
    ones too, and the rows to append."""
    g = torch.Generator().manual_seed(seed)
    total = [n + p for n, p in zip(new, past)]
    # the new tokens taken out again: slots from past[s] on are as unused ones
    fresh = Cache(kv, total, Hk, D, B, seed=seed, **kw)
    for s, (p, t) in enumerate(zip(past, total)):
        for j in range(p // B, -(-t // B)):
            blk, off = int(fresh.tables[s, j]), max(0, p - j * B)
            for pages in (fresh.k, fresh.v):
                fresh._set(pages, blk, slice(off, B),
                           torch.full((Hk, B - off, D), float("nan") if kv != "int8_block"
                                      else -128.0).to(pages.dtype))
            if off == 0 and is_block(kv):
                fresh.ks[blk] = fresh.vs[blk] = float("nan")
    T = sum(new)
    ends = [0]
    for n in new:
        ends.append(ends[-1] + n)
    start = torch.tensor(ends, dtype=torch.int32)
    scale = torch.exp(torch.randn((T + pad, 1), generator=g))
    qkv = (torch.randn((T + pad, (Hq + 2 * Hk) * D), generator=g) * scale).to(torch.bfloat16)
    q, k, v = (qkv[:, :Hq * D], qkv[:, Hq * D:(Hq + Hk) * D], qkv[:, (Hq + Hk) * D:])
    on_gpu = qkv.to(DEV)
    parts = {}
    for name, lo, h in (("query", 0, Hq), ("key", Hq, Hk), ("value", Hq + Hk, Hk)):
        t = on_gpu[:, lo * D:(lo + h) * D]
        parts[name] = t.view(T + pad, h, D) if fused else t.reshape(T + pad, h, D).contiguous()
    host = {"query": q.reshape(-1, Hq, D), "key": k.reshape(-1, Hk, D),
            "value": v.reshape(-1, Hk, D)}
    angles = None if R is None else angle_table(max(1, max(total)), R)
    return fresh, start, host, parts, angles


def run(cache, start, parts, angles, **kw):
    kc, vc = cache.packed(DEV)
    ks, vs = cache.scales(DEV)
    qo = None
    if angles is not None and "query" in parts:
        qo = torch.full_like(parts["query"].contiguous(), float("nan"))
        kw.update(query=parts["query"], query_out=qo)
    pa.read_status(device=DEV, clear=True)
    pa.append_kv(kc, vc, parts["key"], parts["value"], cache.tables.to(DEV), cache.lens.to(DEV),
                 cache.B, cache.kv, ks, vs,
                 query_start=None if start is None else start.to(DEV),
                 cos_sin=None if angles is None else angles.to(DEV), **kw)
    torch.cuda.synchronize()
    return kc, vc, ks, vs, qo


def check(cache, got, start, host, angles, **kw):
    """cache: as before the call; got: run()'s answer."""
    kc, vc, ks, vs, qo = got
    k, v = cache.unpacked(kc, vc)
    q = cache.append(host["key"], host["value"], start, angles, query=host["query"],
                     dtype=torch.float32, **kw)
    assert same(k, cache.k) and same(v, cache.v)
    if is_block(cache.kv):
        assert same(ks, cache.ks) and same(vs, cache.vs)
    if qo is not None:
        T = int(start[-1])
        assert same(qo[:T], q[:T].to(torch.bfloat16))
        assert torch.isnan(qo[T:].float()).all()  # padding rows are left alone


SHAPES = [(128, 16), (128, 32), (64, 16), (64, 32)]


@pytest.mark.parametrize("D,B", SHAPES)
@pytest.mark.parametrize("kv", FORMATS)
def test_ragged_runs(kv, D, B):
    """Runs of no, one and many tokens that begin and end inside blocks."""
    new, past = [5, 0, 1, 3 * B, 2 * B + 3, B, 1], [3, 9, B - 1, 0, 5, B // 2, 0]
    for R, inter, Hk, Hq, fused in ((D, False, 2, 6, True), (D // 2, True, 1, 5, False),
                                    (16, False, 3, 3, True), (None, False, 2, 2, True)):
        args = make(kv, new, past, Hk, Hq, D, B, R, pad=4, fused=fused)
        cache, start, host, parts, angles = args
        got = run(cache, start, parts, angles, interleaved=inter)
        assert pa.read_status(device=DEV) == 0
        check(cache, got, start, host, angles, interleaved=inter)


@pytest.mark.parametrize("kv", FORMATS)
def test_within_half_a_step_of_the_formula(kv):
    """Against fp64: half a step of the cache's type (bf16 2^-8 relative, e4m3
    2^-4 relative or half its subnormal step 2^-10 of a scale, int8 half a
    scale), plus the rotation's fp32 roundings, each 2^-24 of a product of
    |x| <= amax and a cosine: 2^-22 amax.  A block's earlier tokens are rounded
    again when its scale grows: by half a step of the new scale, again."""
    new, past = [40, 3, 77], [5, 13, 0]
    cache, start, host, parts, angles = make(kv, new, past, 2, 4, 128, 16, 128)
    before = [cache.values(s)[:2] for s in range(3)]
    kc, vc, ks, vs, qo = run(cache, start, parts, angles)
    after = Cache(kv, [1], 2, 128, 16)
    after.__dict__.update(cache.__dict__)
    after.k, after.v = cache.unpacked(kc, vc)
    if is_block(kv):
        after.ks, after.vs = ks.cpu(), vs.cpu()
    for s in range(3):
        a, b, t = int(start[s]), int(start[s + 1]), int(cache.lens[s])
        pos = torch.arange(t - (b - a), t)
        want = (rotate(host["key"][a:b].double(), pos, angles, False), host["value"][a:b].double())
        gotk, gotv, _ = after.values(s)
        for got, new_x, old, scale in ((gotk, want[0], before[s][0], after.ks),
                                       (gotv, want[1], before[s][1], after.vs)):
            ids = after.tables[s, :-(-t // 16)].long()
            if is_block(kv):
                sc = scale[ids].double().repeat_interleave(16, 0)[:t, :, None]
            else:
                sc = torch.ones((t, 2, 1), dtype=torch.float64)
                sc = sc if scale is None else sc * float(scale)
            m = t - (b - a)
            for x, y, step in ((new_x, got[m:], sc[m:]), (old[:m], got[:m], sc[:m])):
                tol = {"bf16": 2.0 ** -8 * x.abs(), "int8_block": 0.5 * step}.get(
                    kv, 2.0 ** -4 * x.abs() + 2.0 ** -10 * step)
                tol = tol + 2.0 ** -22 * (x.abs().max() if x.numel() else 0.0)
                if kv == "fp8_e4m3":  # saturation of the fixed scale
                    x = x.clamp(-448 * float(scale), 448 * float(scale))
                assert ((y - x).abs() <= tol).all(), kv
        want_q = rotate(host["query"][a:b].double(), pos, angles, False)
        tol = 2.0 ** -8 * want_q.abs() + 2.0 ** -22 * want_q.abs().max()
        assert ((qo[a:b].cpu().double() - want_q).abs() <= tol).all()


@pytest.mark.parametrize("D,B", [(128, 16), (64, 32)])
@pytest.mark.parametrize("kv", FORMATS)
def test_one_token_at_a_time_fills_blocks(kv, D, B):
    """Decode steps (no query_start) from empty sequences over block ends, the
    tokens growing and shrinking so that block scales grow now and then."""
    S, Hk, Hq, steps = 3, 2, 4, B + 5
    empty, *_ = make(kv, [steps] * S, [0] * S, Hk, Hq, D, B, D, seed=3)
    kc, vc = empty.packed(DEV)
    ks, vs = empty.scales(DEV)
    angles = angle_table(steps, D)
    start = torch.arange(S + 1, dtype=torch.int32)
    g = torch.Generator().manual_seed(5)
    grown = 0
    for i in range(steps):
        amp = 2.0 ** (i % 7 - 3)
        rows = {n: (torch.randn((S, h, D), generator=g) * amp).to(torch.bfloat16)
                for n, h in (("query", Hq), ("key", Hk), ("value", Hk))}
        empty.lens = torch.full((S,), i + 1, dtype=torch.int32)
        old = None if not is_block(kv) else empty.ks.clone()
        q = rows["query"].to(DEV)
        out = pa.append_kv(kc, vc, rows["key"].to(DEV), rows["value"].to(DEV),
                           empty.tables.to(DEV), empty.lens.to(DEV), B, kv, ks, vs,
                           cos_sin=angles.to(DEV), query=q)
        assert out.data_ptr() == q.data_ptr()  # in place by default
        want = empty.append(rows["key"], rows["value"], start, angles, query=rows["query"],
                            dtype=torch.float32)
        assert same(out, want.to(torch.bfloat16))
        if old is not None and i % B:
            grown += int((empty.ks > old).sum())
    k, v = empty.unpacked(kc, vc)
    assert same(k, empty.k) and same(v, empty.v)
    if is_block(kv):
        assert same(ks, empty.ks) and same(vs, empty.vs) and grown > 0
    assert pa.read_status(device=DEV) == 0


@pytest.mark.parametrize("kv", BLOCK_FORMATS)
def test_scales_of_another_quantiser_are_kept(kv):
    """A partly filled block whose scale is no power of two keeps it while the
    new tokens fit, and its codes are x / scale, correctly rounded."""
    cache, start, host, parts, angles = make(kv, [3, 20], [5, 7], 2, 2, 128, 16, 64, pow2=False)
    got = run(cache, start, parts, angles)
    check(cache, got, start, host, angles)


@pytest.mark.parametrize("kv", FORMATS)
def test_extreme_values(kv):
    """Zeros, the smallest and largest numbers, infinities and NaNs in rows:
    neighbours keep their codes, a block of zeros has the smallest scale."""
    cache, start, host, parts, angles = make(kv, [16, 16, 20, 4], [0, 0, 4, 16], 2, 2, 64, 16, None)
    for name in ("key", "value"):
        x = host[name]
        x[0:16] = 0
        x[16:32] *= 1e-38
        x[33, 0, 5], x[34, 1, 6], x[35, 0, 7] = math.inf, -math.inf, math.nan
        x[40] *= 1e30
        x[52:, 1] = 3.0e38
    parts = {n: host[n].to(DEV) for n in ("key", "value")}
    got = run(cache, start, parts, None)
    check(cache, got, start, dict(host, query=None), None)
    if is_block(kv):
        blk = int(cache.tables[0, 0])
        assert (cache.ks[blk] == 2.0 ** -100).all()


def test_positions():
    """Given positions (the same one twice, far ones), and ones outside the
    table: clamped and flagged."""
    cache, start, host, parts, _ = make("bf16", [4, 3], [2, 15], 1, 2, 128, 16, 128)
    angles = angle_table(100000, 128)
    pos = torch.tensor([99999, 0, 7, 7, 54321, 3, 2], dtype=torch.int32)
    got = run(cache, start, parts, angles, positions=pos.to(DEV))
    assert pa.read_status(device=DEV) == 0
    check(cache, got, start, host, angles, positions=pos)
    cache, start, host, parts, _ = make("bf16", [4, 3], [2, 15], 1, 2, 128, 16, 128)
    out_of_range = torch.tensor([100000, -1, 7, 7, 2**31 - 1, -2**31, 2], dtype=torch.int32)
    got = run(cache, start, parts, angles, positions=out_of_range.to(DEV))
    assert pa.read_status(device=DEV, clear=True) == pa.PA_DEV_POSITION_OUT_OF_RANGE
    check(cache, got, start, host, angles, positions=out_of_range.long().clamp(0, 99999))


def test_many_sequences():
    """More sequences than one step of the search tells apart, most with no or
    one row, and rows before the first sequence's that nobody owns."""
    g = torch.Generator().manual_seed(9)
    S = 1500
    new = torch.randint(0, 3, (S,), generator=g)
    new[::97] = 40
    past = torch.randint(0, 20, (S,), generator=g)
    cache, start, host, parts, angles = make("int8_block", new.tolist(), past.tolist(), 1, 1, 64,
                                             16, 64)
    got = run(cache, start, parts, angles)
    check(cache, got, start, host, angles)
    # 37 rows in front
    cache, start, host, parts, angles = make("bf16", [3, 0, 20], [0, 4, 1], 1, 2, 64, 16, 64)
    front = {n: torch.cat([torch.zeros_like(parts[n])[:1].expand(37, -1, -1), parts[n]]).contiguous()
             for n in parts}
    kc, vc, ks, vs, qo = run(cache, start + 37, front, angles)
    assert torch.isnan(qo[:37].float()).all()
    check(cache, (kc, vc, ks, vs, qo[37:]), start, host, angles)


def test_bad_device_data_is_flagged_and_skipped():
    def once(change, bit):
        cache, start, host, parts, angles = make("fp8_e4m3_block", [5, 20, 3], [3, 0, 30], 2, 2,
                                                 64, 16, 64)
        start2 = start.clone()
        change(cache, start2)
        kc, vc, ks, vs, qo = run(cache, start2, parts, angles)
        assert pa.read_status(device=DEV, clear=True) == bit
        return cache, start, host, (kc, vc, ks, vs, qo), angles

    # a length that is shorter than the run, or longer than the table row (3
    # blocks of 16; up to 48 only the row's -1 entries are wrong)
    for bad_len, bit in ((2, pa.PA_DEV_SEQ_LEN_OUT_OF_RANGE), (-1, pa.PA_DEV_SEQ_LEN_OUT_OF_RANGE),
                         (49, pa.PA_DEV_SEQ_LEN_OUT_OF_RANGE),
                         (2**31 - 1, pa.PA_DEV_SEQ_LEN_OUT_OF_RANGE), (33, pa.PA_DEV_BAD_BLOCK_ID)):
        cache, start, host, got, angles = once(lambda c, s: c.lens.__setitem__(0, bad_len), bit)
        before = cache.unpacked(*cache.packed())
        k, v = cache.unpacked(got[0], got[1])
        blk = int(cache.tables[0, 0])
        assert same(k[blk], before[0][blk]) and same(v[blk], before[1][blk])
        assert bit == pa.PA_DEV_BAD_BLOCK_ID or torch.isnan(got[4][:5].float()).all()
        assert not torch.isnan(got[4][5:].float()).any()  # the other sequences' rows
    # block ids outside the pool: the block is skipped, queries are not
    for bad_id in (-1, 10**6, -2**31):
        cache, start, host, got, angles = once(
            lambda c, s: c.tables.__setitem__((1, 0), bad_id), pa.PA_DEV_BAD_BLOCK_ID)
        assert not torch.isnan(got[4].float()).any()
    # query_start out of range or decreasing
    for i, x in ((1, -3), (2, 2), (3, 29), (1, 2**31 - 1)):
        once(lambda c, s: s.__setitem__(i, x), pa.PA_DEV_BAD_QUERY_START)


# Prefix sums that decrease somewhere: the first has a unit whose search ends at
# sequence 1, which begins behind that unit.
DECREASING = [[0, 100, 120, 5, 200], [0, 190, 200, 3, 3], [150, 160, 20, 180, 190],
              [0, 64, 64, 32, 200], [0, 200, 0, 200, 0]]


@pytest.mark.parametrize("ends", DECREASING)
@pytest.mark.parametrize("kv", ["bf16", "int8_block"])
def test_a_decreasing_query_start_writes_nothing_out_of_place(kv, ends):
    S, B, D, raw = 4, 16, 64, Cache._raw
    cache, _, host, parts, angles = make(kv, [200] * S, [9] * S, 1, 1, D, B, D)
    kc, vc = cache.packed(DEV)
    ks, vs = cache.scales(DEV)
    rows = {n: t[:200].contiguous() for n, t in parts.items()}
    before = cache.unpacked(kc, vc)
    pa.read_status(device=DEV, clear=True)
    pa.append_kv(kc, vc, rows["key"], rows["value"], cache.tables.to(DEV), cache.lens.to(DEV), B,
                 kv, ks, vs, query_start=torch.tensor(ends, dtype=torch.int32, device=DEV),
                 cos_sin=angles.to(DEV), query=rows["query"])
    torch.cuda.synchronize()
    assert pa.read_status(device=DEV, clear=True) & pa.PA_DEV_BAD_QUERY_START
    for was, now in zip(before, cache.unpacked(kc, vc)):
        for blk in range(was.shape[0]):
            keep = slice(0, B)
            for s in range(S):
                at = (cache.tables[s] == blk).nonzero()
                n = ends[s + 1] - ends[s]
                if len(at) and 0 <= n <= 200:
                    # its last n tokens may have been written (and the tokens before
                    # them in a block, to the block's new scale)
                    first = max(0, min(B, int(cache.lens[s]) - n - int(at[0]) * B))
                    keep = slice(0, 0 if is_block(kv) and first < B else first)
            assert same(raw(was)[blk, :, keep], raw(now)[blk, :, keep]), (blk, keep)


@pytest.mark.parametrize("kv", ["bf16", "int8_block"])
def test_blocks_past_4_gib(kv):
    """Offsets past 32 bits."""
    Hk, D, B = 8, 128, 32
    page = Hk * D * B * (2 if kv == "bf16" else 1)
    nb = (1 << 32) // page + 40
    dt = torch.bfloat16 if kv == "bf16" else torch.int8
    x = 16 // dt.itemsize
    kc = torch.zeros((nb, Hk, D // x, B, x), dtype=dt, device=DEV)
    vc = torch.zeros((nb, Hk, D, B), dtype=dt, device=DEV)
    ks = torch.ones((nb, Hk), device=DEV)
    vs = torch.ones((nb, Hk), device=DEV)
    cache, start, host, parts, angles = make(kv, [33], [0], Hk, Hk, D, B, D)
    far = torch.tensor([[nb - 1, nb - 7]], dtype=torch.int32, device=DEV)
    pa.append_kv(kc, vc, parts["key"], parts["value"], far, cache.lens.to(DEV), B, kv, ks, vs,
                 query_start=start.to(DEV), cos_sin=angles.to(DEV))
    torch.cuda.synchronize()
    cache.append(host["key"], host["value"], start, angles, dtype=torch.float32)
    ids = far[0].long()
    k, v = cache.unpacked(kc[ids], vc[ids])
    want = cache.tables[0].long()
    assert same(k[0], cache.k[want[0]]) and same(v[0], cache.v[want[0]])
    assert same(k[1][:, :1], cache.k[want[1]][:, :1]) and same(v[1][:, :1], cache.v[want[1]][:, :1])
    others = torch.ones(nb, dtype=torch.bool, device=DEV)
    others[ids] = False
    for part in torch.arange(nb, device=DEV)[others].split(4096):
        assert not kc[part].view(torch.uint8).any() and not vc[part].view(torch.uint8).any()


@pytest.mark.parametrize("kv", FORMATS)
def test_caches_off_a_32_byte_boundary(kv):
    """The caches need 16 bytes only."""
    cache, start, host, parts, angles = make(kv, [40, 5], [0, 3], 2, 2, 128, 16, 128)
    kc, vc = cache.packed()
    odd = []
    for t in (kc, vc):
        raw = torch.zeros(t.numel() * t.element_size() + 48, dtype=torch.uint8, device=DEV)
        at = (16 - raw.data_ptr() % 32) % 32
        u = raw[at:at + t.numel() * t.element_size()].view(t.dtype).view(t.shape)
        u.view(torch.uint8).copy_(t.contiguous().view(torch.uint8))
        assert u.data_ptr() % 32 == 16
        odd.append(u)
    ks, vs = cache.scales(DEV)
    pa.append_kv(odd[0], odd[1], parts["key"], parts["value"], cache.tables.to(DEV),
                 cache.lens.to(DEV), 16, kv, ks, vs, query_start=start.to(DEV),
                 cos_sin=angles.to(DEV))
    check(cache, (odd[0], odd[1], ks, vs, None), start, host, angles)


def test_captured_and_on_another_stream():
    """A captured call replays on changed inputs, also on a side stream."""
    kv = "fp8_e4m3_block"
    cache, start, host, parts, angles = make(kv, [1] * 5, [0, 3, 15, 16, 40], 2, 4, 128, 16, 128)
    kc, vc = cache.packed(DEV)
    ks, vs = cache.scales(DEV)
    bt, sl, table = cache.tables.to(DEV), cache.lens.to(DEV), angles.to(DEV)
    k, v, q = (parts[n].contiguous() for n in ("key", "value", "query"))
    qo = torch.empty_like(q)
    first = [t.clone() for t in (kc.view(torch.uint8), vc.view(torch.uint8), ks, vs)]
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=st):
        pa.append_kv(kc, vc, k, v, bt, sl, 16, kv, ks, vs, cos_sin=table, query=q, query_out=qo)
    g = torch.Generator().manual_seed(77)
    for n, t in (("key", k), ("value", v), ("query", q)):
        host[n] = torch.randn(t.shape, generator=g).to(torch.bfloat16)
        t.copy_(host[n])
    for t, f in zip((kc.view(torch.uint8), vc.view(torch.uint8), ks, vs), first):
        t.copy_(f)
    graph.replay()
    torch.cuda.synchronize()
    check(cache, (kc, vc, ks, vs, qo), start, host, angles)


def test_binding_refusals():
    cache, start, host, parts, angles = make("bf16", [3, 4], [0, 0], 2, 4, 64, 16, 64)
    kc, vc = cache.packed(DEV)
    base = dict(key_cache=kc, value_cache=vc, key=parts["key"], value=parts["value"],
                block_tables=cache.tables.to(DEV), seq_lens=cache.lens.to(DEV), block_size=16,
                query_start=start.to(DEV))

    def refused(error, **over):
        with pytest.raises(error):
            pa.append_kv(**{**base, **over})

    refused(ValueError, query_start=None)  # 7 rows, 2 sequences
    refused(ValueError, key=parts["key"][:6])
    refused(ValueError, key=parts["key"].transpose(0, 1).contiguous().transpose(0, 1))
    refused(ValueError, key=parts["key"][:1].expand(7, -1, -1))  # rows that overlap
    refused(TypeError, key=parts["key"].float())
    refused(ValueError, key=parts["key"].cpu())
    refused(ValueError, block_size=32)
    refused(ValueError, query=parts["query"])  # no table
    refused(ValueError, positions=start.to(DEV))
    refused(TypeError, cos_sin=angles.to(DEV).double())
    refused(pa.PagedAttentionError, cos_sin=angles.to(DEV)[:, :40].contiguous())
    refused(TypeError, kv_dtype="fp8")  # a bf16 cache
    refused(ValueError, kv_dtype="fp4")
    refused(TypeError, kv_dtype="int8_block")
    refused(ValueError, query_start=start.to(DEV)[:-1])
    refused(ValueError, key_cache=kc[:2])
    refused(TypeError, status=torch.zeros(4, dtype=torch.uint8, device=DEV))
    refused(ValueError, status=torch.zeros(1, dtype=torch.int32))
    odd = torch.zeros(7 * 130, dtype=torch.bfloat16, device=DEV).as_strided((7, 2, 64), (130, 64, 1))
    refused(pa.PagedAttentionError, key=odd)  # a row stride that is no multiple of 8
    pa.append_kv(**base)


def test_no_tokens_is_a_no_op():
    cache, start, host, parts, angles = make("bf16", [0, 0], [3, 4], 2, 2, 64, 16, 64)
    got = run(cache, start, parts, angles)
    check(cache, got, start, host, angles)
