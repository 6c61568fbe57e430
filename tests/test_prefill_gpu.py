"""Prefill attention over the paged cache (pa_prefill, GPU), against the
definition in fp64 within the rounding errors kv_reference counts."""

import math

import pytest
import torch

import paged_kv_cache_471_b200 as pa
from kv_reference import FORMATS, Cache, attention

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def ends(new):
    out = [0]
    for n in new:
        out.append(out[-1] + n)
    return torch.tensor(out, dtype=torch.int32)


def prefill(cache, query, start, scale, max_len=None, **kw):
    kc, vc = cache.packed(DEV)
    ks, vs = cache.scales(DEV)
    out = torch.full_like(query, float("nan"), device=DEV)
    max_len = int(cache.lens.max()) if max_len is None else max_len
    pa.prefill(out, query.to(DEV), kc, vc, cache.Hk, scale, cache.tables.to(DEV),
               cache.lens.to(DEV), start.to(DEV), cache.B, max_len, cache.kv, ks, vs, **kw)
    torch.cuda.synchronize()
    return out


def check(out, cache, query, start, scale):
    ref, tol = attention(cache, query, start, scale)
    n = int(start[-1])
    got = out[:n].cpu().double()
    assert torch.equal(torch.isfinite(got), torch.isfinite(ref[:n]))
    err = torch.nan_to_num(got - ref[:n]).abs()
    live = torch.isfinite(ref[:n])
    assert (err[live] <= tol[:n][live]).all(), \
        float((err[live] / tol[:n][live].clamp(min=1e-300)).max())
    assert torch.isnan(out[n:].float()).all()  # padding rows are left alone


def queries(T, Hq, D, seed=2, amp=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn((T, Hq, D), generator=g) * amp).to(torch.bfloat16)


@pytest.mark.parametrize("G", [1, 4, 5, 16])
@pytest.mark.parametrize("D,B", [(128, 16), (128, 32), (64, 16), (64, 32)])
@pytest.mark.parametrize("kv", FORMATS)
def test_ragged_prompts(kv, D, B, G):
    """Runs of no, one and many tokens, with and without cached ones before
    them, over tile ends (128 keys; 256 rows), and padding rows behind."""
    new = [1, 0, 128, 300, 3, 17]
    past = [0, 5, 0, 131, 255, 111]
    cache = Cache(kv, [n + p for n, p in zip(new, past)], 2, D, B, seed=G, pow2=G > 4)
    q = queries(sum(new) + 3, 2 * G, D)
    pa.read_status(device=DEV, clear=True)
    out = prefill(cache, q, ends(new), 1 / math.sqrt(D))
    check(out, cache, q, ends(new), 1 / math.sqrt(D))
    assert pa.read_status(device=DEV) == 0


@pytest.mark.parametrize("pages", [0, 8, 9, 40])
@pytest.mark.parametrize("kv,B", [("bf16", 32), ("fp8_e4m3", 16), ("int8_block", 16)])
def test_split_keys(kv, B, pages):
    """Few rows over many keys: partitions, some of them empty for the short
    sequences, merged; also past max_seq_len, which only plans the split."""
    new, past = [3, 40, 1, 0], [4000, 1000, 0, 17]
    cache = Cache(kv, [n + p for n, p in zip(new, past)], 1, 128, B, seed=3)
    q = queries(sum(new) + 2, 4, 128)
    out = prefill(cache, q, ends(new), 0.09, partition_pages=pages)
    check(out, cache, q, ends(new), 0.09)
    if pages:
        out = prefill(cache, q, ends(new), 0.09, partition_pages=pages, max_len=900)
        check(out, cache, q, ends(new), 0.09)


def test_the_decode_s_merge_counts_stay_zero():
    """A workspace serves prefill and decode in turn: a split call's partials
    stay off the counts that a split tail relies on."""
    cache = Cache("bf16", [2000], 2, 128, 16, seed=4)
    q = queries(5, 4, 128)
    n = pa.prefill_workspace_size(5, 1, 4, 2, 128, 16, 2000, "bf16")
    ws = torch.zeros(n, dtype=torch.uint8, device=DEV)
    out = prefill(cache, q, ends([5]), 0.09, workspace_tensor=ws)
    check(out, cache, q, ends([5]), 0.09)
    head = pa.WORKSPACE_HEADER_BYTES + pa.WORKSPACE_MERGE_COUNT_BYTES
    assert n > head and not ws[:head].any() and ws[head:].any()


@pytest.mark.parametrize("kv", ["bf16", "fp8_e4m3", "fp8_e4m3_block"])
def test_hidden_values_have_no_part(kv):
    """NaNs (and infinities) in values and keys that some rows do not see leave
    those rows alone, and make the rows that see them what they are."""
    new, past = [90, 150], [40, 100]
    cache = Cache(kv, [n + p for n, p in zip(new, past)], 2, 64, 16, seed=5)

    def spoil(pages, s, token, dims, x):
        blk, slot = int(cache.tables[s, token // 16]), token % 16
        page = pages[blk]
        page[1, slot, dims] = torch.tensor(x).to(pages.dtype)

    nan = float("nan")
    big = math.inf if kv == "bf16" else nan
    for s, token in ((0, 60), (0, 129), (1, 100), (1, 128), (1, 249), (1, 3)):
        spoil(cache.v, s, token, slice(3, 5), nan)
        spoil(cache.v, s, token, 7, big)
    spoil(cache.k, 0, 100, 9, nan)
    q = queries(sum(new), 4, 64)
    for pages in (0, 8):
        out = prefill(cache, q, ends(new), 0.125, partition_pages=pages)
        check(out, cache, q, ends(new), 0.125)


@pytest.mark.parametrize("scale", [-0.3, 0.0, 2.0])
def test_scales_of_any_sign(scale):
    for kv in ("bf16", "int8_block"):
        cache = Cache(kv, [200], 1, 128, 16, seed=6)
        q = queries(150, 2, 128)
        out = prefill(cache, q, ends([150]), scale)
        check(out, cache, q, ends([150]), scale)


def test_scales_of_any_sign_per_tensor():
    """Per-tensor scales below 0 work as they do in decode."""
    cache = Cache("fp8_e4m3", [200], 1, 64, 16, seed=6)
    cache.ks, cache.vs = -cache.ks, -cache.vs
    q = queries(150, 2, 64)
    out = prefill(cache, q, ends([150]), 0.2)
    check(out, cache, q, ends([150]), 0.2)


@pytest.mark.parametrize("kv", ["bf16", "int8_block"])
def test_rows_before_the_first_sequence(kv):
    """Rows below query_start[0] belong to nobody, with and without a split."""
    new = [3, 0, 300]
    cache = Cache(kv, [5, 9, 400], 2, 64, 16, seed=15)
    q = queries(sum(new) + 37, 4, 64)
    for pages in (0, 8):
        out = prefill(cache, q, ends(new) + 37, 0.125, partition_pages=pages)
        assert torch.isnan(out[:37].float()).all()
        check(out[37:], cache, q[37:], ends(new), 0.125)


def test_queries_beyond_f16():
    """8-bit caches meet the queries in f16: rows are scaled by a power of two."""
    cache = Cache("fp8_e4m3_block", [150], 1, 128, 16, seed=7)
    q = queries(150, 2, 128)
    q[::3] *= 1e30
    q[1::3] *= 1e-30
    q[5] = 0
    scale = 1e-30
    out = prefill(cache, q, ends([150]), scale)
    check(out, cache, q, ends([150]), scale)


def test_rising_logits_rescale_the_output():
    """Keys whose logits rise along the sequence move the maximum in every tile."""
    cache = Cache("bf16", [900], 1, 128, 16, seed=8)
    for j in range(57):
        blk = int(cache.tables[0, j])
        cache.k[blk, 0, :, 0] = 4.0 * (j % 29)
    q = queries(300, 1, 128)
    q[:, :, 0] = 3.0
    out = prefill(cache, q, ends([300]), 1.0)
    check(out, cache, q, ends([300]), 1.0)


def test_scales_of_very_different_sizes():
    cache = Cache("int8_block", [16 * 24], 2, 64, 16, seed=10)
    for j in range(24):
        blk = int(cache.tables[0, j])
        cache.vs[blk] *= 2.0 ** [0, -40, 13, -90, 5, 0, -20, 30][j % 8]
        if j % 5 == 0:
            cache.vs[blk] = 0.0
            cache.v[blk] = 0
        if j % 7 == 0:
            cache.ks[blk] = 0.0
    q = queries(300, 4, 64)
    out = prefill(cache, q, ends([300]), 0.125)
    check(out, cache, q, ends([300]), 0.125)


def test_bad_device_data_is_flagged_and_skipped():
    new, past = [20, 30, 5], [300, 0, 40]
    q = queries(55, 4, 64)

    def once(change, bit, rows, pages=0):
        cache = Cache("bf16", [n + p for n, p in zip(new, past)], 2, 64, 16, seed=11)
        start = ends(new)
        change(cache, start)
        pa.read_status(device=DEV, clear=True)
        out = prefill(cache, q, start, 0.125, max_len=320, partition_pages=pages)
        assert pa.read_status(device=DEV, clear=True) == bit
        assert torch.isnan(out[rows].float()).all()
        return cache, out

    for pages in (0, 8):
        for n in (19, -1, 321, 2**31 - 1):
            _, out = once(lambda c, s: c.lens.__setitem__(0, n), pa.PA_DEV_SEQ_LEN_OUT_OF_RANGE,
                          slice(0, 20), pages)
            assert torch.isfinite(out[20:].float()).all()
        once(lambda c, s: s.__setitem__(1, -3), pa.PA_DEV_BAD_QUERY_START, slice(0, 20), pages)
        # (sequence 1 decreases, and sequence 2 has more rows than its length)
        once(lambda c, s: s.__setitem__(2, 7),
             pa.PA_DEV_BAD_QUERY_START | pa.PA_DEV_SEQ_LEN_OUT_OF_RANGE, slice(20, 55), pages)
        once(lambda c, s: s.__setitem__(3, 56), pa.PA_DEV_BAD_QUERY_START, slice(50, 55), pages)
        # an illegal block: its keys are left out
        cache, out = once(lambda c, s: c.tables.__setitem__((0, 2), c.num_blocks),
                          pa.PA_DEV_BAD_BLOCK_ID, slice(0, 0), pages)
        cache.tables = torch.cat([cache.tables[:, :2], cache.tables[:, 3:]], dim=1)
        cache.lens[0] -= 16
        ref, tol = attention(cache, q, ends(new), 0.125)
        assert ((out[:20].cpu().double() - ref[:20]).abs() <= tol[:20]).all()


@pytest.mark.parametrize("pages", [0, 8])
@pytest.mark.parametrize("at", [[0, 100, 120, 5, 200], [0, 190, 200, 3, 3],
                                [150, 160, 20, 180, 190], [0, 64, 64, 32, 200],
                                [0, 200, 0, 200, 0], [0, 200, 199, 200, 1]])
def test_a_decreasing_query_start_stays_in_bounds(at, pages):
    """Flagged, and nothing is written but the rows of a sequence's legal range."""
    cache = Cache("fp8_e4m3", [230] * 4, 1, 64, 16, seed=12)
    room = torch.full((600, 1, 64), float("nan"), dtype=torch.bfloat16, device=DEV)
    kc, vc = cache.packed(DEV)
    ks, vs = cache.scales(DEV)
    pa.read_status(device=DEV, clear=True)
    pa.prefill(room[200:400], queries(200, 1, 64).to(DEV), kc, vc, 1, 0.125,
               cache.tables.to(DEV), cache.lens.to(DEV),
               torch.tensor(at, dtype=torch.int32, device=DEV), 16, 240, "fp8_e4m3", ks, vs,
               partition_pages=pages)
    torch.cuda.synchronize()
    assert pa.read_status(device=DEV, clear=True) == pa.PA_DEV_BAD_QUERY_START
    owned = torch.zeros(600, dtype=torch.bool)
    for a, b in zip(at, at[1:]):
        owned[200 + a:200 + max(a, b)] = True
    assert torch.isnan(room.float().cpu()[~owned]).all()


def test_many_sequences_and_blocks_past_4_gib():
    S = 700
    new = [(i * 7) % 4 for i in range(S)]
    past = [(i * 13) % 40 for i in range(S)]
    cache = Cache("bf16", [n + p for n, p in zip(new, past)], 1, 64, 16, seed=12)
    q = queries(sum(new), 2, 64)
    check(prefill(cache, q, ends(new), 0.125), cache, q, ends(new), 0.125)

    cache = Cache("bf16", [70], 8, 128, 32, seed=13)
    nb = (1 << 32) // (8 * 128 * 32 * 2) + 50
    kc = torch.zeros((nb, 8, 16, 32, 8), dtype=torch.bfloat16, device=DEV)
    vc = torch.zeros((nb, 8, 128, 32), dtype=torch.bfloat16, device=DEV)
    far = torch.tensor([[nb - 1, nb - 9, nb - 4]], device=DEV)
    k, v = cache.packed(DEV)
    kc[far[0]], vc[far[0]] = k[cache.tables[0].long().to(DEV)], v[cache.tables[0].long().to(DEV)]
    q = queries(70, 8, 128)
    out = torch.empty_like(q, device=DEV)
    pa.prefill(out, q.to(DEV), kc, vc, 8, 0.09, far.int(), cache.lens.to(DEV),
               ends([70]).to(DEV), 32, 96)
    check(out, cache, q, ends([70]), 0.09)


def test_captured_and_on_another_stream():
    """Two captured calls with a split and one without, replayed on two streams
    with other queries."""
    cache = Cache("int8_block", [3000, 700], 2, 128, 16, seed=14)
    kc, vc = cache.packed(DEV)
    ks, vs = cache.scales(DEV)
    bt, sl = cache.tables.to(DEV), cache.lens.to(DEV)
    runs = []
    for new in ([9, 4], [2, 300]):
        st = torch.cuda.Stream()
        st.wait_stream(torch.cuda.current_stream())
        q = torch.zeros((sum(new), 8, 128), dtype=torch.bfloat16, device=DEV)
        out, start = torch.empty_like(q), ends(new).to(DEV)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=st):
            for _ in range(5):
                pa.prefill(out, q, kc, vc, 2, 0.09, bt, sl, start, 16, 3000, "int8_block", ks, vs)
        runs.append((g, st, q, out, new))
    for i, (g, st, q, out, new) in enumerate(runs):
        q.copy_(queries(sum(new), 8, 128, seed=20 + i))
    torch.cuda.synchronize()
    for g, st, *_ in runs:
        with torch.cuda.stream(st):
            g.replay()
    torch.cuda.synchronize()
    for g, st, q, out, new in runs:
        check(out, cache, q.cpu(), ends(new), 0.09)


def test_binding_refusals():
    cache = Cache("bf16", [40, 3], 2, 64, 16)
    q = queries(10, 4, 64)
    with pytest.raises(ValueError):
        prefill(cache, q, ends([10]), 0.1)
    with pytest.raises(pa.PagedAttentionError):
        prefill(cache, q, ends([7, 3]), 0.1, max_len=49)
    with pytest.raises(pa.PagedAttentionError):
        prefill(cache, q, ends([7, 3]), float("inf"))
    with pytest.raises(pa.PagedAttentionError):
        prefill(cache, q, ends([7, 3]), 0.1, workspace_tensor=torch.zeros(
            64, dtype=torch.uint8, device=DEV))
    with pytest.raises(TypeError):
        prefill(cache, q.float(), ends([7, 3]), 0.1)
    with pytest.raises(ValueError):
        prefill(cache, q, torch.tensor([[0, 7, 10]], dtype=torch.int32), 0.1)
    out = prefill(cache, q[:0], ends([0, 0]), 0.1)
    assert out.numel() == 0
