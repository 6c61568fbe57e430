"""Python binding of libpagedattn (a paged KV cache and the attention over it,
B200 / sm_100a).

Argument marshalling only: every step of the computation runs in the CUDA
kernels of ``libpagedattn.so``; torch is used for device memory and streams.
If the library has not been built the calls raise -- there is no fallback.

``decode`` takes its arguments in the order of the call printed in the PR
#47361 benchmark snippet (out, query, key_cache, value_cache, num_kv_heads,
scale, block_tables, seq_lens, block_size, max_seq_len, kv dtype, k_scale,
v_scale), with the split-KV temporaries folded into one optional workspace.
``append_kv`` writes tokens into the cache, ``prefill`` is attention for many
query tokens of a sequence; both take the cache as ``decode`` does.
"""

from __future__ import annotations

import ctypes
import functools
import os
import threading

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libpagedattn.so")

PA_OK = 0
PA_ERR_INVALID_ARG = 1
PA_ERR_UNSUPPORTED = 2
PA_ERR_WORKSPACE_TOO_SMALL = 3
PA_ERR_CUDA = 4
PA_ERR_OUT_OF_BLOCKS = 5

PA_KV_BF16 = 0
PA_KV_FP8_E4M3 = 1
PA_KV_FP8_E4M3_BLOCK = 2
PA_KV_INT8_BLOCK = 3

PA_DEV_BAD_BLOCK_ID = 0x1
PA_DEV_SEQ_LEN_OUT_OF_RANGE = 0x2
PA_DEV_WAIT_TIMEOUT = 0x4
PA_DEV_PREFIX_MISMATCH = 0x8
PA_DEV_BAD_QUERY_START = 0x10
PA_DEV_POSITION_OUT_OF_RANGE = 0x20

WORKSPACE_HEADER_BYTES = 256
WORKSPACE_MERGE_COUNT_BYTES = 4096  # after the header when the plan needs more
NOALLOC_SCRATCH_BYTES = 16 << 20

_KV = {"bf16": PA_KV_BF16, "auto": PA_KV_BF16, "fp8": PA_KV_FP8_E4M3, "fp8_e4m3": PA_KV_FP8_E4M3,
       "fp8_e4m3_block": PA_KV_FP8_E4M3_BLOCK, "int8_block": PA_KV_INT8_BLOCK,
       PA_KV_BF16: PA_KV_BF16, PA_KV_FP8_E4M3: PA_KV_FP8_E4M3,
       PA_KV_FP8_E4M3_BLOCK: PA_KV_FP8_E4M3_BLOCK, PA_KV_INT8_BLOCK: PA_KV_INT8_BLOCK}


class PagedAttentionError(RuntimeError):
    def __init__(self, status: int, detail: str):
        self.status = status
        super().__init__(detail)


class Options(ctypes.Structure):
    _fields_ = [("partition_pages", ctypes.c_int), ("num_sms", ctypes.c_int),
                ("stages", ctypes.c_int), ("shared_prefix_blocks", ctypes.c_int),
                ("alibi_slopes", ctypes.c_void_p), ("fp8_compute", ctypes.c_int),
                ("test_stall_copies", ctypes.c_int), ("schedule", ctypes.c_int),
                ("mha_cuda_cores", ctypes.c_int)]


class AppendOptions(ctypes.Structure):
    _fields_ = [("key_stride", ctypes.c_int64), ("value_stride", ctypes.c_int64),
                ("cos_sin", ctypes.c_void_p), ("max_position", ctypes.c_int),
                ("rotary_dim", ctypes.c_int), ("interleaved", ctypes.c_int),
                ("num_heads", ctypes.c_int), ("positions", ctypes.c_void_p),
                ("query", ctypes.c_void_p), ("query_out", ctypes.c_void_p),
                ("query_stride", ctypes.c_int64), ("query_out_stride", ctypes.c_int64)]


class Plan(ctypes.Structure):
    _fields_ = [("num_partitions", ctypes.c_int), ("partition_pages", ctypes.c_int),
                ("stages", ctypes.c_int), ("warps_per_cta", ctypes.c_int),
                ("grid_ctas", ctypes.c_longlong), ("smem_bytes", ctypes.c_size_t),
                ("workspace_bytes", ctypes.c_size_t), ("prefix_partitions", ctypes.c_int),
                ("prefix_groups", ctypes.c_int), ("balanced", ctypes.c_int),
                ("dynamic", ctypes.c_int), ("tail_units", ctypes.c_longlong),
                ("tail_partitions", ctypes.c_int), ("tail_partition_pages", ctypes.c_int),
                ("combine", ctypes.c_int), ("longest_first", ctypes.c_int)]

    def as_dict(self):
        return {f: getattr(self, f) for f, _ in self._fields_}


_lib = None
_lock = threading.Lock()

_P = ctypes.c_void_p
_I = ctypes.c_int


def _bind(lib):
    decode_args = [_P, _P, _P, _P, _I, _I, _I, _I, ctypes.c_float, _P, _I, _P, _I, _I,
                   ctypes.c_int64, _I, _P, _P, _P, ctypes.c_size_t, _P]
    lib.pa_decode.argtypes = decode_args
    lib.pa_decode.restype = _I
    lib.pa_decode_ex.argtypes = decode_args + [ctypes.POINTER(Options)]
    lib.pa_decode_ex.restype = _I
    lib.pa_decode_noalloc.argtypes = decode_args[:18] + [_P]
    lib.pa_decode_noalloc.restype = _I
    lib.pa_plan_decode.argtypes = [ctypes.POINTER(Plan), _I, _I, _I, _I, _I, _I, _I,
                                   ctypes.POINTER(Options)]
    lib.pa_plan_decode.restype = _I
    lib.pa_decode_workspace_size.argtypes = [_I, _I, _I, _I, _I, _I, _I, ctypes.POINTER(Options)]
    lib.pa_decode_workspace_size.restype = ctypes.c_size_t
    lib.pa_read_device_status.argtypes = [_P, ctypes.POINTER(ctypes.c_uint32), _I, _P]
    lib.pa_read_device_status.restype = _I
    lib.pa_status_string.argtypes = [_I]
    lib.pa_status_string.restype = ctypes.c_char_p
    lib.pa_last_error_detail.argtypes = []
    lib.pa_last_error_detail.restype = ctypes.c_char_p
    lib.pa_version.argtypes = []
    lib.pa_version.restype = _I
    I64 = ctypes.c_int64
    lib.pa_bm_create.argtypes = [ctypes.POINTER(_P), I64, _I, _I]
    lib.pa_bm_create.restype = _I
    lib.pa_bm_destroy.argtypes = [_P]
    lib.pa_bm_destroy.restype = None
    lib.pa_bm_add_sequence.argtypes = [_P, ctypes.POINTER(_I)]
    lib.pa_bm_add_sequence.restype = _I
    lib.pa_bm_fork.argtypes = [_P, _I, ctypes.POINTER(_I)]
    lib.pa_bm_fork.restype = _I
    lib.pa_bm_free_sequence.argtypes = [_P, _I]
    lib.pa_bm_free_sequence.restype = _I
    lib.pa_bm_append_tokens.argtypes = [_P, _I, _I, ctypes.POINTER(I64), ctypes.POINTER(I64),
                                        ctypes.POINTER(_I)]
    lib.pa_bm_append_tokens.restype = _I
    lib.pa_bm_seq_len.argtypes = [_P, _I, ctypes.POINTER(I64)]
    lib.pa_bm_seq_len.restype = _I
    lib.pa_bm_export.argtypes = [_P, _P, _I, _P, _I, _P]
    lib.pa_bm_export.restype = _I
    lib.pa_bm_num_free_blocks.argtypes = [_P]
    lib.pa_bm_num_free_blocks.restype = I64
    lib.pa_bm_refcount.argtypes = [_P, I64]
    lib.pa_bm_refcount.restype = _I
    lib.pa_bm_last_error_detail.argtypes = []
    lib.pa_bm_last_error_detail.restype = ctypes.c_char_p
    lib.pa_copy_blocks.argtypes = [_P, _P, _I, _I, _I, I64, _I, _P, _P, _I, _P, _P]
    lib.pa_copy_blocks.restype = _I
    lib.pa_copy_blocks_ex.argtypes = [_P, _P, _P, _P, _I, _I, _I, I64, _I, _P, _P, _I, _P, _P]
    lib.pa_copy_blocks_ex.restype = _I
    lib.pa_append_kv.argtypes = [_P, _P, _P, _P, _I, _I, _I, _I, _P, _I, _P, _P, _I, I64, _I, _P,
                                 _P, _P, _P, ctypes.POINTER(AppendOptions)]
    lib.pa_append_kv.restype = _I
    lib.pa_prefill.argtypes = [_P, _P, _P, _P, _I, _I, _I, _I, _I, ctypes.c_float, _P, _I, _P, _P,
                               _I, _I, I64, _I, _P, _P, _P, ctypes.c_size_t, _P,
                               ctypes.POINTER(Options)]
    lib.pa_prefill.restype = _I
    lib.pa_prefill_workspace_size.argtypes = [_I] * 8 + [ctypes.POINTER(Options)]
    lib.pa_prefill_workspace_size.restype = ctypes.c_size_t
    lib.pa_capture_id.argtypes = [_P, ctypes.POINTER(ctypes.c_uint64)]
    lib.pa_capture_id.restype = _I
    lib.pa_capture_watch.argtypes = [_P, ctypes.POINTER(_P)]
    lib.pa_capture_watch.restype = _I
    lib.pa_capture_alive.argtypes = [_P]
    lib.pa_capture_alive.restype = _I
    lib.pa_capture_free.argtypes = [_P]
    lib.pa_capture_free.restype = None
    lib.pa_capture_mode.argtypes = [ctypes.POINTER(_I)]
    lib.pa_capture_mode.restype = _I
    return lib


def lib():
    """The loaded libpagedattn (raises if it was never built)."""
    global _lib
    if _lib is None:
        with _lock:
            if _lib is None:
                if not os.path.exists(LIB_PATH):
                    raise RuntimeError(
                        f"{LIB_PATH} is missing: build it with "
                        "`python -m paged_kv_cache_471_b200.build` (there is no fallback path)")
                _lib = _bind(ctypes.CDLL(LIB_PATH))
    return _lib


def _check(rc: int):
    if rc != PA_OK:
        L = lib()
        raise PagedAttentionError(rc, f"{L.pa_status_string(rc).decode()}: "
                                      f"{L.pa_last_error_detail().decode()}")


SCHEDULES = {"auto": 0, "balanced": 1, "partitioned": 2, "dynamic": 3}


def _opts(partition_pages=0, num_sms=0, stages=0, shared_prefix_blocks=0, alibi_ptr=None,
          fp8_compute=False, test_stall_copies=False, schedule="auto", mha_cuda_cores=False):
    if schedule not in SCHEDULES:
        raise ValueError(f"schedule must be one of {sorted(SCHEDULES)}")
    if not partition_pages and not num_sms and not stages and not shared_prefix_blocks \
            and not alibi_ptr and not fp8_compute and not test_stall_copies \
            and schedule == "auto" and not mha_cuda_cores:
        return None
    return ctypes.byref(Options(int(partition_pages), int(num_sms), int(stages),
                                int(shared_prefix_blocks), alibi_ptr, int(bool(fp8_compute)),
                                int(bool(test_stall_copies)), SCHEDULES[schedule],
                                int(bool(mha_cuda_cores))))


def kv_dtype_code(kv_dtype) -> int:
    try:
        return _KV[kv_dtype]
    except KeyError:
        raise ValueError(f"unsupported kv dtype {kv_dtype!r}") from None


def plan(num_seqs, num_heads, num_kv_heads, head_size, block_size, max_seq_len, kv_dtype="bf16",
         partition_pages=0, num_sms=0, stages=0, shared_prefix_blocks=0, fp8_compute=False,
         schedule="auto") -> dict:
    p = Plan()
    _check(lib().pa_plan_decode(ctypes.byref(p), num_seqs, num_heads, num_kv_heads, head_size,
                                block_size, max_seq_len, kv_dtype_code(kv_dtype),
                                _opts(partition_pages, num_sms, stages, shared_prefix_blocks,
                                      None, fp8_compute, False, schedule)))
    return p.as_dict()


def prefill_workspace_size(num_tokens, num_seqs, num_heads, num_kv_heads, head_size, block_size,
                           max_seq_len, kv_dtype="bf16", partition_pages=0, num_sms=0) -> int:
    n = lib().pa_prefill_workspace_size(num_tokens, num_seqs, num_heads, num_kv_heads, head_size,
                                        block_size, max_seq_len, kv_dtype_code(kv_dtype),
                                        _opts(partition_pages, num_sms))
    if n == 0:
        raise PagedAttentionError(PA_ERR_INVALID_ARG, lib().pa_last_error_detail().decode())
    return n


@functools.lru_cache(maxsize=4096)
def _prefill_workspace_size(device, *args):
    """prefill_workspace_size for the current device (number `device`)."""
    return prefill_workspace_size(*args)


@functools.lru_cache(maxsize=4096)
def _workspace_size(device, *args):
    """workspace_size for the current device (number `device`)."""
    return workspace_size(*args)


def workspace_size(num_seqs, num_heads, num_kv_heads, head_size, block_size, max_seq_len,
                   kv_dtype="bf16", partition_pages=0, num_sms=0, shared_prefix_blocks=0,
                   fp8_compute=False, schedule="auto", stages=0) -> int:
    n = lib().pa_decode_workspace_size(num_seqs, num_heads, num_kv_heads, head_size, block_size,
                                       max_seq_len, kv_dtype_code(kv_dtype),
                                       _opts(partition_pages, num_sms, stages, shared_prefix_blocks,
                                             None, fp8_compute, False, schedule))
    if n == 0:
        raise PagedAttentionError(PA_ERR_INVALID_ARG, lib().pa_last_error_detail().decode())
    return n


_ws_cache = {}     # (device number, stream) -> its calls' workspace (see _launching)
_captured = {}     # (device number, stream, capture id) -> the _Captured of its calls
_retired = {}      # device number -> status bits of graphs that are gone
_status_words = {}
_tables = threading.RLock()  # guards the three above
# (device number, stream) -> held while a call finds its workspace there and
# launches: a call may be two launches that hand partials on, and another
# thread's call on the same stream must not come between them.
_launching = {}


@functools.lru_cache(maxsize=None)
def _torch():
    """torch, which is imported by the first call, and the types that calls check."""
    import torch
    return torch, (torch.bfloat16,), (torch.float32,), (torch.int32,)


def _stream_ptr(stream, index):
    """The cudaStream_t of a call: the given stream's, or the current one's of
    device number `index`."""
    if stream is not None:
        return stream.cuda_stream
    return _torch()[0]._C._cuda_getCurrentRawStream(index)


def _capture_id(stream, index):
    """The id of the capture that a call's stream is in; 0 when it is in none."""
    if stream is None and not _torch()[0].cuda.is_current_stream_capturing():
        return 0
    n = ctypes.c_uint64(0)
    _check(lib().pa_capture_id(_stream_ptr(stream, index), ctypes.byref(n)))
    return n.value


class _outside:
    """``with _outside(index):`` -- torch work on device number `index` (the
    current one) that no capture takes in, whichever streams are being captured:
    on another stream, and complete at the end of the block."""

    def __init__(self, index):
        self.index = index

    def __enter__(self):
        torch = _torch()[0]
        self.mode = ctypes.c_int(2)
        _check(lib().pa_capture_mode(ctypes.byref(self.mode)))
        try:
            while True:  # (torch hands out a pool's streams in turn)
                side = torch.cuda.Stream(self.index)
                if not _capture_id(side, self.index):
                    break
            self.side = torch.cuda.stream(side)
            self.side.__enter__()
        except BaseException:
            _check(lib().pa_capture_mode(ctypes.byref(self.mode)))
            raise
        self.wait = side.synchronize

    def __exit__(self, *error):
        try:
            self.wait()
        finally:
            self.side.__exit__(*error)
            _check(lib().pa_capture_mode(ctypes.byref(self.mode)))


class _Captured:
    """The workspaces of the calls captured into one graph on one stream.  They
    run one after the other and share the largest; smaller ones that earlier
    calls of the capture took stay with them."""

    def __init__(self, index, stream):
        self.index, self.buffers, self.note = index, [], ctypes.c_void_p()
        _check(lib().pa_capture_watch(_stream_ptr(stream, index), ctypes.byref(self.note)))

    def __del__(self):
        if self.note and _lib is not None:  # (None at the end of the process)
            _lib.pa_capture_free(self.note)

    def alive(self):
        return lib().pa_capture_alive(self.note)

    def workspace(self, nbytes):
        if not self.buffers or self.buffers[-1].numel() < nbytes:
            torch = _torch()[0]
            with _outside(self.index):
                self.buffers.append(torch.zeros(nbytes, dtype=torch.uint8,
                                                device=torch.device("cuda", self.index)))
        return self.buffers[-1]


def _reap(index):
    """Let go of the workspaces of graphs of device number `index` (the current
    one) that are gone; their status bits are kept."""
    gone = [key for key, c in _captured.items() if c.index == index and not c.alive()]
    if not gone:
        return
    torch = _torch()[0]
    with _outside(index):
        if index not in _retired:
            _retired[index] = torch.zeros(4, dtype=torch.int32, device=torch.device("cuda", index))
        for key in gone:
            for ws in _captured.pop(key).buffers:
                _retired[index] |= ws[:16].view(torch.int32)


def workspace(nbytes: int, device, stream=None):
    """A zeroed workspace of at least nbytes on `device` for calls on `stream`
    (default: the current one), reused by the calls on that stream (its status
    word is sticky; see read_status).  Calls on different streams may overlap,
    so each stream has its own.  While the stream is being captured into a
    graph, the workspace belongs to that graph: the calls of the capture on that
    stream share it, nothing else does, and it is kept, status word and all,
    until the graph is gone."""
    torch = _torch()[0]
    dev = torch.device(device)
    index = torch.cuda.current_device() if dev.index is None else dev.index
    previous = _enter_device(index)
    try:
        key = (index, _stream_ptr(stream, index))
        with _launch_lock(key):
            return _workspace(max(nbytes, WORKSPACE_HEADER_BYTES), key, stream)
    finally:
        _leave_device(previous)


def _launch_lock(key):
    lock = _launching.get(key)
    return lock if lock is not None else _launching.setdefault(key, threading.Lock())


def _workspace(nbytes, key, stream):
    """workspace for the key (number of the current device, its stream's pointer),
    under the key's lock."""
    index = key[0]
    capture = _capture_id(stream, index)
    if capture:
        with _tables:
            _reap(index)
            held = _captured.get(key + (capture,))
            if held is None:
                held = _captured[key + (capture,)] = _Captured(index, stream)
            return held.workspace(nbytes)
    ws = _ws_cache.get(key)
    if ws is not None and ws.numel() >= nbytes:
        return ws
    torch = _torch()[0]
    with _tables:
        _reap(index)
    if stream is None:
        stream = torch.cuda.current_stream(index)
    with torch.cuda.stream(stream):  # zeroed, and later freed, in that stream's order
        new = torch.zeros(nbytes, dtype=torch.uint8, device=torch.device("cuda", index))
        if ws is not None:  # keep the status bits
            new[:4] = ws[:4]
    _ws_cache[key] = new
    return new


def _status_word(index):
    """The address of the device word that append_kv reports to by default;
    read_status reads it with the workspaces'.  Made, once, for device number
    `index` (the current one), where no capture and no stream's call sees it
    before it is zeroed."""
    word = _status_words.get(index)
    if word is None:
        torch = _torch()[0]
        with _tables:
            word = _status_words.get(index)
            if word is None:
                with _outside(index):
                    word = torch.zeros(4, dtype=torch.int32,
                                       device=torch.device("cuda", index))
                _status_words[index] = word
    return word.data_ptr()


def _enter_device(index):
    """Make device number `index` the current one, which the library plans for
    and launches on; returns the one to go back to, or None."""
    torch = _torch()[0]
    now = torch._C._cuda_getDevice()
    if now == index:
        return None
    torch.cuda.set_device(index)
    return now


def _leave_device(previous):
    if previous is not None:
        _torch()[0].cuda.set_device(previous)


def _refuse(t, name, dtypes, index):
    """Raise for what _ptr found wrong."""
    torch = _torch()[0]
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.get_device() != index:
        raise ValueError(f"{name} is on {t.device}, expected device {index}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    raise TypeError(f"{name} has dtype {t.dtype}, expected one of {dtypes}")


def _ptr(t, name, dtypes, index):
    """The address of a contiguous CUDA tensor on device number `index`."""
    try:
        if t.get_device() == index >= 0 and t.is_contiguous() \
                and (dtypes is None or t.dtype in dtypes):
            return t.data_ptr()
    except AttributeError:
        pass
    return _refuse(t, name, dtypes, index)


@functools.lru_cache(maxsize=None)
def _kv_types(code):
    import torch
    if code == PA_KV_BF16:
        return (torch.bfloat16,)
    if code == PA_KV_INT8_BLOCK:
        return (torch.int8, torch.uint8)
    return (torch.uint8, torch.float8_e4m3fn)


def _scale_ptrs(code, k_scale, v_scale, num_blocks, num_kv_heads, index):
    """Pointers to the scales of an 8-bit cache (None, None for bf16)."""
    if code == PA_KV_BF16:
        return None, None
    f32 = _torch()[2]
    ptrs = _ptr(k_scale, "k_scale", f32, index), _ptr(v_scale, "v_scale", f32, index)
    if code != PA_KV_FP8_E4M3:
        for t, name in ((k_scale, "k_scale"), (v_scale, "v_scale")):
            if t.shape != (num_blocks, num_kv_heads):
                raise ValueError(f"{name} must be [num_blocks, num_kv_heads] for block scales")
    return ptrs


def decode(out, query, key_cache, value_cache, num_kv_heads: int, scale: float, block_tables,
           seq_lens, block_size: int, max_seq_len: int, kv_dtype="bf16", k_scale=None,
           v_scale=None, workspace_tensor=None, partition_pages: int = 0, stream=None,
           stages: int = 0, shared_prefix_blocks: int = 0, alibi_slopes=None,
           fp8_compute: bool = False, test_stall_copies: bool = False, schedule: str = "auto",
           mha_cuda_cores: bool = False, num_sms: int = 0):
    """Paged decode attention into ``out`` (bf16 [num_seqs, num_heads, head_size]).

    key_cache: [num_blocks, num_kv_heads, head_size/x, block_size, x];
    value_cache: [num_blocks, num_kv_heads, head_size, block_size]; bf16, or
    uint8 / float8_e4m3fn holding e4m3 codes when kv_dtype is "fp8_e4m3"
    (then k_scale / v_scale are 1-element fp32 CUDA tensors), or e4m3 or int8
    codes when it is "fp8_e4m3_block" or "int8_block" (then k_scale / v_scale
    are fp32 [num_blocks, num_kv_heads], a scale for each block and kv head;
    no fp8_compute and no dynamic schedule).

    The keyword options are those of pa_options in include/pagedattn.h:
    partition_pages, stages, shared_prefix_blocks, alibi_slopes ([num_heads]
    fp32), fp8_compute, test_stall_copies, schedule ("auto",
    "partitioned", "balanced" or "dynamic"), mha_cuda_cores and num_sms (plan
    as if the GPU had that many SMs; 0 = the device's count).  workspace_tensor
    defaults to a cached zeroed buffer per device and stream; stream defaults
    to the current stream.
    """
    _, bf16, f32, i32 = _torch()
    code = kv_dtype_code(kv_dtype)
    index = query.get_device()
    S, Hq, D = query.shape
    kv_types = _kv_types(code)
    ptrs = (_ptr(out, "out", bf16, index), _ptr(query, "query", bf16, index),
            _ptr(key_cache, "key_cache", kv_types, index),
            _ptr(value_cache, "value_cache", kv_types, index))
    if out.shape != query.shape:
        raise ValueError("out must have the query's shape")
    if key_cache.dim() != 5 or value_cache.dim() != 4:
        raise ValueError("key_cache must be 5-D and value_cache 4-D")
    num_blocks, k_heads, groups, k_block, x = key_cache.shape
    if value_cache.shape != (num_blocks, num_kv_heads, D, block_size) \
            or k_heads != num_kv_heads or k_block != block_size or groups * x != D:
        raise ValueError("cache shapes do not match query / num_kv_heads / block_size")
    bt = _ptr(block_tables, "block_tables", i32, index)
    sl = _ptr(seq_lens, "seq_lens", i32, index)
    tables = block_tables.shape
    if len(tables) != 2 or tables[0] != S or seq_lens.shape != (S,):
        raise ValueError("block_tables must be [num_seqs, max_blocks] and seq_lens [num_seqs]")
    ks, vs = _scale_ptrs(code, k_scale, v_scale, num_blocks, num_kv_heads, index)
    alibi = None
    if alibi_slopes is not None:
        if alibi_slopes.shape != (Hq,):
            raise ValueError("alibi_slopes must be [num_heads]")
        alibi = _ptr(alibi_slopes, "alibi_slopes", f32, index)
    key = (index, _stream_ptr(stream, index))
    own = workspace_tensor is None  # (a given one is size-checked by the library)
    previous = _enter_device(index)
    if own:
        lock = _launch_lock(key)
        lock.acquire()
    try:
        if own:
            need = _workspace_size(index, S, Hq, num_kv_heads, D, block_size, max_seq_len, code,
                                   partition_pages, num_sms, shared_prefix_blocks,
                                   bool(fp8_compute) and code == PA_KV_FP8_E4M3, schedule, stages)
            workspace_tensor = _workspace(need, key, stream)
        ws = _ptr(workspace_tensor, "workspace", None, index)
        rc = lib().pa_decode_ex(*ptrs, S, Hq, int(num_kv_heads), D, float(scale), bt, tables[1],
                                sl, int(block_size), int(max_seq_len), num_blocks, code, ks, vs,
                                ws, workspace_tensor.numel() * workspace_tensor.element_size(),
                                key[1],
                                _opts(partition_pages, num_sms, stages, shared_prefix_blocks, alibi,
                                      fp8_compute, test_stall_copies, schedule, mha_cuda_cores))
    finally:
        if own:
            lock.release()
        _leave_device(previous)
    _check(rc)
    return out


def prefill(out, query, key_cache, value_cache, num_kv_heads: int, scale: float, block_tables,
            seq_lens, query_start, block_size: int, max_seq_len: int, kv_dtype="bf16",
            k_scale=None, v_scale=None, workspace_tensor=None, partition_pages: int = 0,
            stream=None, num_sms: int = 0):
    """Causal attention of each sequence's last tokens over its paged cache,
    into ``out`` (bf16 [num_tokens, num_heads, head_size], like query).

    Rows query_start[s] .. query_start[s + 1] - 1 (int32 [num_seqs + 1]) are
    the last tokens of sequence s, whose keys and values are in the cache
    already (append_kv) and counted in seq_lens[s]; a token sees the keys up to
    its own.  Rows that no sequence owns are left alone.  The cache, its types
    and scales, the workspace and the stream are those of decode;
    partition_pages > 0 forces a split of the keys into partitions of that many
    blocks (by default only batches with few rows are split).
    """
    _, bf16, _, i32 = _torch()
    code = kv_dtype_code(kv_dtype)
    index = query.get_device()
    kv_types = _kv_types(code)
    T, Hq, D = query.shape
    ptrs = (_ptr(out, "out", bf16, index), _ptr(query, "query", bf16, index),
            _ptr(key_cache, "key_cache", kv_types, index),
            _ptr(value_cache, "value_cache", kv_types, index))
    if out.shape != query.shape:
        raise ValueError("out must have the query's shape")
    num_blocks, x = key_cache.shape[0], 16 // key_cache.element_size()
    if key_cache.shape != (num_blocks, num_kv_heads, D // x, block_size, x) \
            or value_cache.shape != (num_blocks, num_kv_heads, D, block_size):
        raise ValueError("cache shapes do not match query / num_kv_heads / block_size")
    bt = _ptr(block_tables, "block_tables", i32, index)
    sl = _ptr(seq_lens, "seq_lens", i32, index)
    qs = _ptr(query_start, "query_start", i32, index)
    tables = block_tables.shape
    if seq_lens.dim() != 1 or len(tables) != 2 or tables[0] != seq_lens.shape[0] \
            or query_start.shape != (tables[0] + 1,):
        raise ValueError("block_tables must be [num_seqs, max_blocks], seq_lens [num_seqs] and "
                         "query_start [num_seqs + 1]")
    S = tables[0]
    ks, vs = _scale_ptrs(code, k_scale, v_scale, num_blocks, num_kv_heads, index)
    key = (index, _stream_ptr(stream, index))
    own = workspace_tensor is None  # (a given one is size-checked by the library)
    previous = _enter_device(index)
    if own:
        lock = _launch_lock(key)
        lock.acquire()
    try:
        if own:
            need = _prefill_workspace_size(index, T, S, Hq, num_kv_heads, D, block_size,
                                           max_seq_len, code, partition_pages, num_sms)
            workspace_tensor = _workspace(need, key, stream)
        ws = _ptr(workspace_tensor, "workspace", None, index)
        rc = lib().pa_prefill(*ptrs, T, S, Hq, int(num_kv_heads), D, float(scale), bt, tables[1],
                              sl, qs, int(block_size), int(max_seq_len), num_blocks, code, ks, vs,
                              ws, workspace_tensor.numel() * workspace_tensor.element_size(),
                              key[1], _opts(partition_pages, num_sms))
    finally:
        if own:
            lock.release()
        _leave_device(previous)
    _check(rc)
    return out


def decode_noalloc(out, query, key_cache, value_cache, num_kv_heads: int, scale: float,
                   block_tables, seq_lens, block_size: int, max_seq_len: int, kv_dtype="bf16",
                   k_scale=None, v_scale=None, stream=None):
    """``decode`` for callers that may not allocate device memory when they
    call: the split-KV scratch is the library's own fixed device array
    (NOALLOC_SCRATCH_BYTES per GPU), so nothing is allocated here.  Calls that
    overlap on the GPU share that array and must be serialised by the caller;
    the first call on a device should come before any stream capture."""
    torch, bf16, _, i32 = _torch()
    code = kv_dtype_code(kv_dtype)
    dev, index = query.device, query.get_device()
    S, Hq, D = query.shape
    kv_types = _kv_types(code)
    ks, vs = _scale_ptrs(code, k_scale, v_scale, key_cache.shape[0], num_kv_heads, index)
    st = stream if stream is not None else torch.cuda.current_stream(dev)
    ptrs = (_ptr(out, "out", bf16, index), _ptr(query, "query", bf16, index),
            _ptr(key_cache, "key_cache", kv_types, index),
            _ptr(value_cache, "value_cache", kv_types, index))
    bt = _ptr(block_tables, "block_tables", i32, index)
    sl = _ptr(seq_lens, "seq_lens", i32, index)
    with torch.cuda.device(dev):  # the scratch array of the tensors' device
        rc = lib().pa_decode_noalloc(*ptrs, S, Hq, int(num_kv_heads), D, float(scale), bt,
                                     block_tables.shape[1], sl, int(block_size), int(max_seq_len),
                                     int(key_cache.shape[0]), code, ks, vs, st.cuda_stream)
    _check(rc)
    return out


def read_status(workspace_tensor=None, device=None, clear=False, stream=None) -> int:
    """The sticky PA_DEV_* bits kernels set (synchronises): those of a
    workspace, or, without one, those of every call on the device that was
    given none, the replays of captured calls among them."""
    import torch
    if workspace_tensor is not None:
        dev, words = workspace_tensor.device, [workspace_tensor]
    else:
        dev = torch.device(device) if device is not None else torch.device("cuda")
        if dev.index is None:
            dev = torch.device("cuda", torch.cuda.current_device())
        previous = _enter_device(dev.index)
        try:
            with _tables:
                _reap(dev.index)
                words = [ws for key, ws in list(_ws_cache.items()) if key[0] == dev.index]
                words += [ws for c in _captured.values() if c.index == dev.index
                          for ws in c.buffers]
            words += [t[dev.index] for t in (_retired, _status_words) if dev.index in t]
        finally:
            _leave_device(previous)
        if words:  # calls of other streams may still be running
            torch.cuda.synchronize(dev)
    st = stream if stream is not None else torch.cuda.current_stream(dev)
    bits = 0
    with torch.cuda.device(dev):
        for w in words:
            flags = ctypes.c_uint32(0)
            _check(lib().pa_read_device_status(ctypes.c_void_p(w.data_ptr()), ctypes.byref(flags),
                                               int(bool(clear)), st.cuda_stream))
            bits |= int(flags.value)
        if clear and workspace_tensor is None and words:
            torch.cuda.synchronize(dev)  # cleared before calls on other streams follow
    return bits


def version() -> int:
    return int(lib().pa_version())


# --------------------------------------------------------------- block manager
def _bm_check(rc: int):
    if rc != PA_OK:
        L = lib()
        raise PagedAttentionError(rc, f"{L.pa_status_string(rc).decode()}: "
                                      f"{L.pa_bm_last_error_detail().decode()}")


class BlockManager:
    """Host block allocator of libpagedattn (``pa_bm_*``): blocks on demand,
    forked sequences sharing blocks, copy on write of a shared partial block."""

    def __init__(self, num_blocks: int, block_size: int, max_blocks_per_seq: int):
        self._h = ctypes.c_void_p()
        _bm_check(lib().pa_bm_create(ctypes.byref(self._h), int(num_blocks), int(block_size),
                                     int(max_blocks_per_seq)))
        self.num_blocks, self.block_size = int(num_blocks), int(block_size)
        self.max_blocks_per_seq = int(max_blocks_per_seq)

    def close(self):
        if self._h:
            lib().pa_bm_destroy(self._h)
            self._h = ctypes.c_void_p()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def add_sequence(self) -> int:
        i = ctypes.c_int()
        _bm_check(lib().pa_bm_add_sequence(self._h, ctypes.byref(i)))
        return i.value

    def fork(self, parent: int) -> int:
        i = ctypes.c_int()
        _bm_check(lib().pa_bm_fork(self._h, int(parent), ctypes.byref(i)))
        return i.value

    def free(self, seq: int):
        _bm_check(lib().pa_bm_free_sequence(self._h, int(seq)))

    def append(self, seq: int, num_tokens: int):
        """Grow a sequence; returns (src, dst) when a copy on write is needed."""
        a, b, n = ctypes.c_int64(), ctypes.c_int64(), ctypes.c_int()
        _bm_check(lib().pa_bm_append_tokens(self._h, int(seq), int(num_tokens), ctypes.byref(a),
                                            ctypes.byref(b), ctypes.byref(n)))
        return (a.value, b.value) if n.value else None

    def seq_len(self, seq: int) -> int:
        n = ctypes.c_int64()
        _bm_check(lib().pa_bm_seq_len(self._h, int(seq), ctypes.byref(n)))
        return n.value

    def export(self, seqs):
        """(block_tables int32 [n, max_blocks_per_seq], seq_lens int32 [n]) on the host."""
        import numpy as np
        ids = np.ascontiguousarray(np.asarray(seqs, dtype=np.int32))
        bt = np.empty((len(ids), self.max_blocks_per_seq), dtype=np.int32)
        sl = np.empty((len(ids),), dtype=np.int32)
        _bm_check(lib().pa_bm_export(self._h, ids.ctypes.data, len(ids), bt.ctypes.data,
                                     self.max_blocks_per_seq, sl.ctypes.data))
        return bt, sl

    def num_free_blocks(self) -> int:
        return int(lib().pa_bm_num_free_blocks(self._h))

    def refcount(self, block: int) -> int:
        return int(lib().pa_bm_refcount(self._h, int(block)))


def copy_blocks(key_cache, value_cache, src, dst, kv_dtype="bf16", status=None, stream=None,
                k_scale=None, v_scale=None):
    """Copy whole blocks (all kv heads, K and V): block dst[i] <- block src[i].
    src / dst: int64 CUDA tensors of block ids.  A cache with block scales
    needs k_scale and v_scale ([num_blocks, num_kv_heads]), whose rows are
    copied with the blocks."""
    import torch
    code = kv_dtype_code(kv_dtype)
    dev, index = key_cache.device, key_cache.get_device()
    kv_types = _kv_types(code)
    n = int(src.numel())
    if int(dst.numel()) != n:
        raise ValueError("src and dst must have the same length")
    Hk, D = value_cache.shape[1], value_cache.shape[2]
    st = stream if stream is not None else torch.cuda.current_stream(dev)
    ks = vs = None
    if code in (PA_KV_FP8_E4M3_BLOCK, PA_KV_INT8_BLOCK):
        ks, vs = _scale_ptrs(code, k_scale, v_scale, key_cache.shape[0], Hk, index)
    args = (_ptr(key_cache, "key_cache", kv_types, index),
            _ptr(value_cache, "value_cache", kv_types, index), ks, vs,
            int(Hk), int(D), int(value_cache.shape[3]), int(key_cache.shape[0]), code,
            _ptr(src, "src", (torch.int64,), index), _ptr(dst, "dst", (torch.int64,), index), n,
            None if status is None else _ptr(status, "status", None, index), st.cuda_stream)
    with torch.cuda.device(dev):
        rc = lib().pa_copy_blocks_ex(*args)
    _bm_check(rc)


# ------------------------------------------------------------- appending tokens
def _rows(t, name, tokens, heads, head_size, index):
    """Pointer and row stride of a bf16 [tokens, heads, head_size] tensor whose
    heads are dense (a view of a wider projection's output will do)."""
    try:
        if t.get_device() != index or t.dtype not in _torch()[1]:
            _refuse(t, name, _torch()[1], index)
    except AttributeError:
        _refuse(t, name, None, index)
    if t.shape != (tokens, heads, head_size):
        raise ValueError(f"{name} must be [{tokens}, {heads}, {head_size}]")
    if tokens == 0:
        return t.data_ptr(), 0
    row, head, element = t.stride()
    if element != 1 or (head != head_size and heads > 1):
        raise ValueError(f"{name}: a token's heads must be contiguous")
    if tokens == 1:
        return t.data_ptr(), 0
    if row < heads * head_size:
        raise ValueError(f"{name}: its rows overlap")
    return t.data_ptr(), row


def append_kv(key_cache, value_cache, key, value, block_tables, seq_lens, block_size: int,
              kv_dtype="bf16", k_scale=None, v_scale=None, *, query_start=None, cos_sin=None,
              interleaved: bool = False, positions=None, query=None, query_out=None, status=None,
              stream=None):
    """Write new tokens' keys and values into a paged cache, keys (and queries)
    rotated by their positions on the way.

    key, value: bf16 [num_tokens, num_kv_heads, head_size]; rows may be strided
    (views of one projection's output).  Rows query_start[s] ..
    query_start[s + 1] - 1 (int32 [num_seqs + 1]) are the last tokens of
    sequence s, whose length with them is seq_lens[s]; None: one row per
    sequence, as in a decode step (none for a length of 0).  Rows that no
    sequence owns (padding) are left alone.

    cos_sin: fp32 [max_position, rotary_dim], a row holding the cosines, then
    the sines of its position's rotary_dim / 2 angles; pairs are (d, d +
    rotary_dim / 2), or (2d, 2d + 1) with interleaved.  positions: int32
    [num_tokens] (default: a token's index in its sequence).  query is rotated
    into query_out (default: in place).

    kv_dtype and the scales are those of decode; with block scales, k_scale and
    v_scale are updated: see pa_append_kv in include/pagedattn.h.  status: an
    int32 / uint32 CUDA word for the PA_DEV_* bits (default: one that
    read_status reads).  Returns query_out (None without a query).
    """
    torch, _, f32, int32 = _torch()
    code = kv_dtype_code(kv_dtype)
    index = key_cache.get_device()
    kv_types = _kv_types(code)
    kc = _ptr(key_cache, "key_cache", kv_types, index)
    vc = _ptr(value_cache, "value_cache", kv_types, index)
    if key_cache.dim() != 5 or value_cache.dim() != 4:
        raise ValueError("key_cache must be 5-D and value_cache 4-D")
    num_blocks, Hk, D, B = value_cache.shape
    x = 8 if code == PA_KV_BF16 else 16
    if B != block_size or key_cache.shape != (num_blocks, Hk, D // x, B, x):
        raise ValueError("cache shapes do not match each other / block_size")
    bt = _ptr(block_tables, "block_tables", int32, index)
    sl = _ptr(seq_lens, "seq_lens", int32, index)
    T, S, tables = key.shape[0], seq_lens.shape[0], block_tables.shape
    if len(tables) != 2 or tables[0] != S or seq_lens.dim() != 1:
        raise ValueError("block_tables must be [num_seqs, max_blocks] and seq_lens [num_seqs]")
    qs = None
    if query_start is not None:
        qs = _ptr(query_start, "query_start", int32, index)
        if query_start.shape != (S + 1,):
            raise ValueError("query_start must be [num_seqs + 1]")
    elif T != S:
        raise ValueError("without query_start, key and value need a row per sequence")
    k, k_stride = _rows(key, "key", T, Hk, D, index)
    v, v_stride = _rows(value, "value", T, Hk, D, index)
    ks, vs = _scale_ptrs(code, k_scale, v_scale, num_blocks, Hk, index)
    table = pos = q = qo = None
    max_position = rotary_dim = Hq = q_stride = qo_stride = 0
    if cos_sin is not None:
        table = _ptr(cos_sin, "cos_sin", f32, index)
        if cos_sin.dim() != 2:
            raise ValueError("cos_sin must be [max_position, rotary_dim]")
        max_position, rotary_dim = cos_sin.shape
        if positions is not None:
            pos = _ptr(positions, "positions", int32, index)
            if positions.shape != (T,):
                raise ValueError("positions must be [num_tokens]")
        if query is not None:
            if query_out is None:
                query_out = query
            if query.dim() != 3:
                raise ValueError("query must be [num_tokens, num_heads, head_size]")
            Hq = query.shape[1]
            q, q_stride = _rows(query, "query", T, Hq, D, index)
            qo, qo_stride = _rows(query_out, "query_out", T, Hq, D, index)
        elif query_out is not None:
            raise ValueError("query_out needs query")
    elif positions is not None or query is not None or query_out is not None or interleaved:
        raise ValueError("positions, query, query_out and interleaved need cos_sin")
    o = AppendOptions(k_stride, v_stride, table, max_position, rotary_dim, bool(interleaved), Hq,
                      pos, q, qo, q_stride, qo_stride)
    previous = _enter_device(index)
    try:
        if status is None:
            word = _status_word(index)
        else:
            word = _ptr(status, "status", (torch.int32, torch.uint32), index)
        rc = lib().pa_append_kv(kc, vc, k, v, T, S, Hk, D, bt, tables[1], sl, qs, B, num_blocks,
                                code, ks, vs, word, _stream_ptr(stream, index), ctypes.byref(o))
    finally:
        _leave_device(previous)
    _check(rc)
    return query_out
