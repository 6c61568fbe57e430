"""pa_append_kv, pa_prefill, pa_copy_blocks_ex and the block-scaled cache types
without a GPU: bad arguments are refused before any CUDA call."""

import ctypes
import shutil
import subprocess

import pytest

import paged_kv_cache_471_b200 as pa
from paged_kv_cache_471_b200 import build as pbuild


@pytest.fixture(scope="module")
def L():
    pbuild.build()
    return pa.lib()


APPEND_OPTS = dict(key_stride=0, value_stride=0, cos_sin=0x90000, max_position=100, rotary_dim=64,
                   interleaved=0, num_heads=8, positions=0xa0000, query=0xb0000,
                   query_out=0xc0000, query_stride=0, query_out_stride=0)


def _append(L, opts=None, **over):
    args = dict(key_cache=0x10000, value_cache=0x20000, key=0x30000, value=0x40000, num_tokens=5,
                num_seqs=2, num_kv_heads=2, head_size=128, block_tables=0x50000,
                max_blocks_per_seq=4, seq_lens=0x60000, query_start=0x70000, block_size=16,
                num_blocks=64, kv_dtype=0, k_scale=None, v_scale=None, status=0x80000,
                stream=None)
    args.update(over)
    o = pa.AppendOptions(**{**APPEND_OPTS, **(opts or {})})
    return L.pa_append_kv(*args.values(), ctypes.byref(o))


@pytest.mark.parametrize("over,opts,code", [
    (dict(num_tokens=-1), {}, pa.PA_ERR_INVALID_ARG),
    (dict(num_seqs=-1), {}, pa.PA_ERR_INVALID_ARG),
    (dict(num_kv_heads=0), {}, pa.PA_ERR_INVALID_ARG),
    (dict(head_size=96), {}, pa.PA_ERR_UNSUPPORTED),
    (dict(block_size=8), {}, pa.PA_ERR_UNSUPPORTED),
    (dict(kv_dtype=4), {}, pa.PA_ERR_UNSUPPORTED),
    (dict(max_blocks_per_seq=0), {}, pa.PA_ERR_INVALID_ARG),
    (dict(num_blocks=0), {}, pa.PA_ERR_INVALID_ARG),
    (dict(num_blocks=1 << 31), {}, pa.PA_ERR_INVALID_ARG),
    (dict(query_start=None), {}, pa.PA_ERR_INVALID_ARG),  # 5 rows, 2 sequences
    (dict(key=None), {}, pa.PA_ERR_INVALID_ARG),
    (dict(value=0x40008), {}, pa.PA_ERR_INVALID_ARG),
    (dict(key_cache=0x10008), {}, pa.PA_ERR_INVALID_ARG),
    (dict(value_cache=None), {}, pa.PA_ERR_INVALID_ARG),
    (dict(block_tables=0x50002), {}, pa.PA_ERR_INVALID_ARG),
    (dict(seq_lens=None), {}, pa.PA_ERR_INVALID_ARG),
    (dict(query_start=0x70002), {}, pa.PA_ERR_INVALID_ARG),
    (dict(status=0x80001), {}, pa.PA_ERR_INVALID_ARG),
    (dict(kv_dtype=1), {}, pa.PA_ERR_INVALID_ARG),  # no scales
    (dict(kv_dtype=2, k_scale=0x1000), {}, pa.PA_ERR_INVALID_ARG),
    (dict(kv_dtype=3, k_scale=0x1000, v_scale=0x1002), {}, pa.PA_ERR_INVALID_ARG),
    ({}, dict(key_stride=128), pa.PA_ERR_INVALID_ARG),   # rows overlap
    ({}, dict(value_stride=260), pa.PA_ERR_INVALID_ARG),  # not a multiple of 8
    ({}, dict(query_stride=1028), pa.PA_ERR_INVALID_ARG),
    ({}, dict(query_out_stride=8), pa.PA_ERR_INVALID_ARG),
    ({}, dict(rotary_dim=0), pa.PA_ERR_UNSUPPORTED),
    ({}, dict(rotary_dim=24), pa.PA_ERR_UNSUPPORTED),
    ({}, dict(rotary_dim=144), pa.PA_ERR_UNSUPPORTED),
    ({}, dict(max_position=0), pa.PA_ERR_INVALID_ARG),
    ({}, dict(cos_sin=0x90004), pa.PA_ERR_INVALID_ARG),
    ({}, dict(positions=0xa0002), pa.PA_ERR_INVALID_ARG),
    ({}, dict(cos_sin=None), pa.PA_ERR_INVALID_ARG),     # positions and query without it
    ({}, dict(query_out=None), pa.PA_ERR_INVALID_ARG),
    ({}, dict(query=0xb0008), pa.PA_ERR_INVALID_ARG),
    ({}, dict(num_heads=0), pa.PA_ERR_INVALID_ARG),
    (dict(num_tokens=2**31 - 1, num_kv_heads=1 << 20), dict(num_heads=65536),
     pa.PA_ERR_INVALID_ARG),  # more CTAs than a grid has
])
def test_append_refuses(L, over, opts, code):
    assert _append(L, opts, **over) == code
    assert L.pa_last_error_detail().decode() != ""


def test_append_of_nothing_is_a_no_op(L):
    assert _append(L, num_tokens=0, key=None) == pa.PA_OK
    assert _append(L, num_tokens=0, num_seqs=0, query_start=None, seq_lens=None) == pa.PA_OK


def _prefill(L, opts=None, **over):
    args = dict(out=0x10000, query=0x20000, key_cache=0x30000, value_cache=0x40000, num_tokens=5,
                num_seqs=2, num_heads=8, num_kv_heads=2, head_size=128, scale=0.1,
                block_tables=0x50000, max_blocks_per_seq=4, seq_lens=0x60000,
                query_start=0x70000, block_size=16, max_seq_len=64, num_blocks=64, kv_dtype=0,
                k_scale=None, v_scale=None, workspace=0x80000, workspace_bytes=1 << 20,
                stream=None)
    args.update(over)
    o = pa.Options(num_sms=148, **(opts or {}))
    return L.pa_prefill(*args.values(), ctypes.byref(o))


@pytest.mark.parametrize("over,opts,code", [
    (dict(num_tokens=-1), {}, pa.PA_ERR_INVALID_ARG),
    (dict(num_seqs=-1), {}, pa.PA_ERR_INVALID_ARG),
    (dict(num_heads=9), {}, pa.PA_ERR_INVALID_ARG),
    (dict(num_heads=34), {}, pa.PA_ERR_UNSUPPORTED),
    (dict(num_kv_heads=0), {}, pa.PA_ERR_INVALID_ARG),
    (dict(head_size=80), {}, pa.PA_ERR_UNSUPPORTED),
    (dict(block_size=64), {}, pa.PA_ERR_UNSUPPORTED),
    (dict(kv_dtype=-1), {}, pa.PA_ERR_UNSUPPORTED),
    (dict(scale=float("nan")), {}, pa.PA_ERR_INVALID_ARG),
    (dict(max_blocks_per_seq=0), {}, pa.PA_ERR_INVALID_ARG),
    (dict(max_seq_len=65), {}, pa.PA_ERR_INVALID_ARG),
    (dict(max_seq_len=-1), {}, pa.PA_ERR_INVALID_ARG),
    (dict(num_blocks=0), {}, pa.PA_ERR_INVALID_ARG),
    (dict(out=None), {}, pa.PA_ERR_INVALID_ARG),
    (dict(query=0x20008), {}, pa.PA_ERR_INVALID_ARG),
    (dict(key_cache=0x30004), {}, pa.PA_ERR_INVALID_ARG),
    (dict(query_start=None), {}, pa.PA_ERR_INVALID_ARG),
    (dict(seq_lens=0x60001), {}, pa.PA_ERR_INVALID_ARG),
    (dict(workspace=None), {}, pa.PA_ERR_INVALID_ARG),
    (dict(workspace_bytes=255), {}, pa.PA_ERR_WORKSPACE_TOO_SMALL),
    (dict(kv_dtype=1), {}, pa.PA_ERR_INVALID_ARG),
    (dict(kv_dtype=3, k_scale=0x1000), {}, pa.PA_ERR_INVALID_ARG),
    ({}, dict(schedule=1), pa.PA_ERR_UNSUPPORTED),
    ({}, dict(shared_prefix_blocks=1), pa.PA_ERR_UNSUPPORTED),
    ({}, dict(alibi_slopes=0x1000), pa.PA_ERR_UNSUPPORTED),
    ({}, dict(stages=2), pa.PA_ERR_UNSUPPORTED),
    ({}, dict(partition_pages=-1), pa.PA_ERR_INVALID_ARG),
    (dict(max_seq_len=16 * 1024, max_blocks_per_seq=1024), dict(partition_pages=8),
     pa.PA_ERR_INVALID_ARG),  # 128 partitions
    (dict(num_tokens=2**31 - 1), {}, pa.PA_ERR_INVALID_ARG),
])
def test_prefill_refuses(L, over, opts, code):
    assert _prefill(L, opts, **over) == code
    assert L.pa_last_error_detail().decode() != ""


def test_prefill_of_nothing_is_a_no_op(L):
    assert _prefill(L, num_tokens=0, out=None) == pa.PA_OK
    assert _prefill(L, num_tokens=0, num_seqs=0, query_start=None) == pa.PA_OK


def test_prefill_workspace():
    """Only calls with fewer CTAs (256 / G query tokens of a kv head each) than
    SMs split the keys; the workspace then holds (D + 2) floats per row and
    partition after the header and the decode's merge counts."""
    size = pa.prefill_workspace_size
    assert size(8192, 1, 32, 8, 128, 16, 8192, "bf16", num_sms=148) == pa.WORKSPACE_HEADER_BYTES
    assert size(0, 0, 32, 8, 128, 16, 0, "bf16", num_sms=148) == pa.WORKSPACE_HEADER_BYTES
    before = pa.WORKSPACE_HEADER_BYTES + pa.WORKSPACE_MERGE_COUNT_BYTES
    # 2 token groups x 8 kv heads on 148 SMs: 9 partitions of 235 key tiles
    n = size(14, 2, 32, 8, 128, 32, 30000, "int8_block", num_sms=148)
    body = 14 * 32 * 9 * (128 + 2) * 4
    assert n == -(-(before + body) // 256) * 256
    # partitions forced: 40 blocks of 16 tokens are 5 key tiles, so 1000 tokens make 2
    n = size(14, 2, 32, 8, 128, 16, 1000, "bf16", partition_pages=40, num_sms=148)
    body = 14 * 32 * 2 * (128 + 2) * 4
    assert n == -(-(before + body) // 256) * 256
    with pytest.raises(pa.PagedAttentionError):
        size(14, 2, 33, 8, 128, 16, 1000, "bf16", num_sms=148)


@pytest.mark.parametrize("over,code", [
    (dict(k_scale=None), pa.PA_ERR_INVALID_ARG),
    (dict(v_scale=0x4002), pa.PA_ERR_INVALID_ARG),
    (dict(kv_dtype=4), pa.PA_ERR_UNSUPPORTED),
    (dict(num_pairs=-1), pa.PA_ERR_INVALID_ARG),
    (dict(src=None), pa.PA_ERR_INVALID_ARG),
    (dict(key_cache=0x1008), pa.PA_ERR_INVALID_ARG),
])
def test_copy_blocks_refuses(L, over, code):
    args = dict(key_cache=0x1000, value_cache=0x2000, k_scale=0x3000, v_scale=0x4000,
                num_kv_heads=2, head_size=128, block_size=16, num_blocks=10, kv_dtype=2,
                src=0x5000, dst=0x6000, num_pairs=1, status=None, stream=None)
    args.update(over)
    assert L.pa_copy_blocks_ex(*args.values()) == code
    assert L.pa_bm_last_error_detail().decode() != ""


def test_copy_blocks_without_scales_refuses_block_scales(L):
    for code in (2, 3):
        assert L.pa_copy_blocks(0x1000, 0x2000, 2, 128, 16, 10, code, 0x5000, 0x6000, 1, None,
                                None) == pa.PA_ERR_INVALID_ARG


def test_plans_of_block_scaled_caches():
    """They plan like per-tensor codes; the dynamic schedule is refused."""
    for kv in ("fp8_e4m3_block", "int8_block"):
        for shape in ((64, 32, 8, 128, 16, 16384), (1, 32, 8, 128, 32, 131072)):
            assert pa.plan(*shape, kv, num_sms=148) == pa.plan(*shape, "fp8_e4m3", num_sms=148)
        with pytest.raises(pa.PagedAttentionError) as e:
            pa.plan(4, 8, 8, 64, 16, 256, kv, num_sms=148, schedule="dynamic")
        assert e.value.status == pa.PA_ERR_UNSUPPORTED


@pytest.mark.parametrize("over", [dict(kv_dtype=2), dict(kv_dtype=3, k_scale=0x1000)])
def test_decode_needs_both_scales(L, over):
    args = dict(out=0x10000, query=0x20000, key_cache=0x30000, value_cache=0x40000, num_seqs=2,
                num_heads=8, num_kv_heads=2, head_size=128, scale=0.088, block_tables=0x50000,
                max_blocks_per_seq=4, seq_lens=0x60000, block_size=16, max_seq_len=64,
                num_blocks=64, kv_dtype=0, k_scale=None, v_scale=None, workspace=0x70000,
                workspace_bytes=1 << 20, stream=None)
    args.update(over)
    assert L.pa_decode(*args.values()) == pa.PA_ERR_INVALID_ARG


@pytest.mark.skipif(shutil.which("nm") is None, reason="needs nm")
def test_two_copies_in_one_process_share_no_state(L):
    """A unique symbol is one for the process: a second copy of the library would believe that
    its kernels have the shared-memory limit which the first copy raised for its own."""
    out = subprocess.run(["nm", "-D", "--defined-only", pbuild.LIB], capture_output=True,
                         text=True, check=True).stdout
    names = [line.split() for line in out.splitlines()]
    assert any(n[-1] == "pa_append_kv" for n in names)
    assert not [n[-1] for n in names if n[-2] == "u"]
