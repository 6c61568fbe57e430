"""V scales over the whole range that append writes, 2^-100 to 2^100, read by
decode and prefill (GPU), against the definition in fp64."""

import copy

import pytest
import torch

import paged_kv_cache_471_b200 as pa
from kv_reference import BLOCK_FORMATS, QMAX, Cache, attention

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def queries(T, Hq, D, seed=2):
    g = torch.Generator().manual_seed(seed)
    return torch.randn((T, Hq, D), generator=g).to(torch.bfloat16)


def attend(cache, q, n, scale, op="decode", alibi=None, **kw):
    """The last n tokens of each sequence."""
    kc, vc = cache.packed(DEV)
    ks, vs = cache.scales(DEV)
    out = torch.full_like(q, float("nan"), device=DEV)
    bt, sl = cache.tables.to(DEV), cache.lens.to(DEV)
    start = torch.arange(len(cache.lens) + 1, dtype=torch.int32) * n
    max_len = int(cache.lens.max())
    if op == "decode":
        pa.decode(out, q.to(DEV), kc, vc, cache.Hk, scale, bt, sl, cache.B, max_len, cache.kv, ks,
                  vs, alibi_slopes=None if alibi is None else alibi.to(DEV), **kw)
    else:
        pa.prefill(out, q.to(DEV), kc, vc, cache.Hk, scale, bt, sl, start.to(DEV), cache.B,
                   max_len, cache.kv, ks, vs, **kw)
    torch.cuda.synchronize()
    ref, tol = attention(cache, q, start, scale, alibi)
    # kv_reference's bound counts 2^-20 A for exponentials, A = sum_t p_t |v_t|.  A
    # logit's log2 here goes with a V scale's, up to 256 in all, which fp32 rounds
    # by 2^-17 a few times: 2^-15 of every weight, in the sum and in the denominator.
    size = copy.copy(cache)
    size.v = cache.v.float().abs().to(cache.v.dtype)
    return out.cpu().double(), ref, tol + 2.0 ** -14 * attention(size, q, start, scale, alibi)[0]


def check(out, ref, tol):
    err = (out - ref).abs()
    assert torch.isfinite(out).all()
    assert (err <= tol).all(), float((err / tol.clamp(min=1e-300)).max())


@pytest.mark.parametrize("op", ["decode", "prefill"])
@pytest.mark.parametrize("kv", BLOCK_FORMATS)
def test_what_append_writes_is_read(kv, op):
    """Sequences of one token, whose attention is its value: within half a step of
    its code (e4m3 2^-4 of it, int8 half a scale) and of bf16, whatever its size;
    above the largest code of 2^100 it saturates."""
    D, B, Hk = 64, 16, 2
    sizes = [1e-28, 1e-25, 1e-18, 1e-6, 1.0, 1e10, 2e14, 1e20, 1e27, 1e31, 3e38]
    S = len(sizes)
    cache = Cache(kv, [1] * S, Hk, D, B, seed=3)
    g = torch.Generator().manual_seed(4)
    v = torch.rand((S, Hk, D), generator=g) * 2 - 1
    v = (v * torch.tensor(sizes)[:, None, None]).to(torch.bfloat16)
    k = torch.randn((S, Hk, D), generator=g).to(torch.bfloat16)
    kc, vc = cache.packed(DEV)
    ks, vs = cache.scales(DEV)
    bt, sl = cache.tables.to(DEV), cache.lens.to(DEV)
    pa.append_kv(kc, vc, k.to(DEV), v.to(DEV), bt, sl, B, kv, ks, vs)
    q = queries(S, 2 * Hk, D).to(DEV)
    out = torch.empty_like(q)
    if op == "decode":
        pa.decode(out, q, kc, vc, Hk, 0.125, bt, sl, B, 1, kv, ks, vs)
    else:
        start = torch.arange(S + 1, dtype=torch.int32, device=DEV)
        pa.prefill(out, q, kc, vc, Hk, 0.125, bt, sl, start, B, 1, kv, ks, vs)
    torch.cuda.synchronize()
    want = v.double().repeat_interleave(2, dim=1)
    step = vs[bt[:, 0].long()].cpu().double().repeat_interleave(2, dim=1)[..., None]
    want = torch.maximum(torch.minimum(want, QMAX[kv] * step), -QMAX[kv] * step)
    assert float(step.max()) == 2.0 ** 100
    half = 0.5 * step if kv == "int8_block" else 2.0 ** -4 * want.abs() + 2.0 ** -10 * step
    tol = half + 2.0 ** -8 * (want.abs() + half)
    assert ((out.cpu().double() - want).abs() <= tol).all()


LOG2 = [0, 100, -100, 60, -60, 99, -99, 30, -30, 0, -100, 100]


def spread(cache, seed):
    g = torch.Generator().manual_seed(seed)
    e = torch.tensor(LOG2)[torch.randint(0, len(LOG2), (cache.num_blocks, 1), generator=g)]
    cache.vs[:] = torch.exp2(e.double()).float()


@pytest.mark.parametrize("kw", [dict(), dict(partition_pages=2), dict(schedule="balanced"),
                                dict(partition_pages=5), dict(op="prefill"),
                                dict(op="prefill", partition_pages=8)])
@pytest.mark.parametrize("kv", BLOCK_FORMATS)
def test_scales_over_the_whole_range_in_one_sequence(kv, kw):
    D, B, n = 128, 16, 9 if "op" in kw else 1
    lens = [16 * 40 - 3, 16 * 9, 16 * 23 + 1]
    cache = Cache(kv, lens, 2, D, B, seed=6)
    spread(cache, 7)
    q = queries(len(lens) * n, 8, D)
    check(*attend(cache, q, n, 0.125, **kw))


@pytest.mark.parametrize("kw", [dict(), dict(partition_pages=1), dict(partition_pages=40),
                                dict(shared=3), dict(op="prefill"),
                                dict(op="prefill", partition_pages=8)])
@pytest.mark.parametrize("order", ["small first", "large first", "among others"])
@pytest.mark.parametrize("kv", BLOCK_FORMATS)
def test_the_denominator_belongs_to_small_values(kv, order, kw):
    """Nearly all weight is on tokens whose values are as small as they get, while
    the largest values, of little weight, set the running maximum: the outputs
    are those few large values over the denominator of the small ones."""
    kw = dict(kw)
    D, B, n = 64, 16, 5 if "op" in kw else 1
    shared = kw.pop("shared", 0)
    blocks = 28
    cache = Cache(kv, [blocks * B] * 2, 1, D, B, seed=8, shared_blocks=shared)
    if shared:
        kw["shared_prefix_blocks"] = shared
    for s in range(2):
        for j in range(blocks):
            blk = int(cache.tables[s, j])
            large = {"small first": j >= blocks // 2, "large first": j < blocks // 2,
                     "among others": j % 9 == 4}[order]
            cache.vs[blk] = 2.0 ** (100 if large else -100)
            cache.ks[blk] = 2.0 ** -4
            # the first head dim decides: a logit of 0, or 46 (in log2) below
            cache._set(cache.k, blk, slice(0, B), torch.zeros((1, B, D)).to(cache.k.dtype))
            one = torch.zeros((1, B, D))
            one[..., 0] = -64.0 if large else 0.0
            cache._set(cache.k, blk, slice(0, B), one.to(cache.k.dtype))
    q = torch.zeros((2 * n, 4, D), dtype=torch.bfloat16)
    q[..., 0] = 8.0  # 8 * -64 * 2^-4 = -32 = -46.2 log2(e)
    out, ref, tol = attend(cache, q, n, 1.0, **kw)
    assert float(ref.abs().max()) > 2.0 ** 40
    check(out, ref, tol)


@pytest.mark.parametrize("op", ["decode", "prefill"])
def test_many_tokens_of_the_smallest_scale(op):
    """Thousands of cached zeros: sums near 2^100 times their number."""
    cache = Cache("int8_block", [9000], 1, 64, 32, seed=9)
    cache.vs[:] = 2.0 ** -100
    n = 5 if op == "prefill" else 1
    q = queries(n, 2, 64)
    for pages in (0, 64):
        out, ref, tol = attend(cache, q, n, 0.125, op=op, partition_pages=pages)
        check(out, ref, tol)


def test_a_scale_of_zero():
    cache = Cache("fp8_e4m3_block", [16 * 6], 1, 64, 16, seed=10)
    for j, e in enumerate([100, None, 0, None, -100, 40]):
        blk = int(cache.tables[0, j])
        cache.vs[blk] = 0.0 if e is None else 2.0 ** e
        if e is None:
            cache._raw(cache.v)[blk] = 0
    for op, n in (("decode", 1), ("prefill", 20)):
        check(*attend(cache, queries(n, 4, 64), n, 0.125, op=op))


@pytest.mark.parametrize("G", [1, 9])
@pytest.mark.parametrize("D,B", [(128, 16), (128, 32), (64, 16), (64, 32)])
@pytest.mark.parametrize("kv", BLOCK_FORMATS)
def test_every_form_over_long_sequences(kv, D, B, G):
    """More than 32 stages to a warp, one and two blocks of query rows, with and
    without ALiBi, whole and split; prefill over many tiles."""
    cache = Cache(kv, [9000, 33], 1, D, B, seed=11)
    spread(cache, 12)
    slopes = torch.linspace(0.001, 0.01, G)
    for kw in (dict(partition_pages=9000), dict(), dict(alibi=slopes, partition_pages=9000)):
        check(*attend(cache, queries(2, G, D), 1, 0.125, **kw))
    for kw in (dict(partition_pages=9000), dict()):
        check(*attend(cache, queries(6, G, D), 3, 0.125, op="prefill", **kw))


@pytest.mark.parametrize("S,B,prefix", [(5, 16, 40), (24, 16, 300), (40, 32, 150)])
@pytest.mark.parametrize("kv", BLOCK_FORMATS)
def test_shared_prefix_of_a_wide_range(kv, S, B, prefix):
    """Few sequences (a CTA per row group) and many (the shared ring)."""
    lens = [prefix * B + (i * 29) % 200 for i in range(S)]
    cache = Cache(kv, lens, 1, 64, B, seed=13, shared_blocks=prefix)
    spread(cache, 14)
    check(*attend(cache, queries(S, 4, 64), 1, 0.125, shared_prefix_blocks=prefix))
