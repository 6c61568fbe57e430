"""pa_capture_*: argument checks, without a GPU."""

import ctypes

import pytest

import paged_kv_cache_471_b200 as pa
from paged_kv_cache_471_b200 import build as pbuild


@pytest.fixture(scope="module")
def L():
    pbuild.build()
    return pa.lib()


def test_refusals(L):
    assert L.pa_capture_id(None, None) == pa.PA_ERR_INVALID_ARG
    assert L.pa_capture_watch(None, None) == pa.PA_ERR_INVALID_ARG
    assert L.pa_capture_mode(None) == pa.PA_ERR_INVALID_ARG
    for mode in (-1, 3):
        assert L.pa_capture_mode(ctypes.byref(ctypes.c_int(mode))) == pa.PA_ERR_INVALID_ARG
        assert L.pa_last_error_detail().decode() != ""


def test_no_note_is_not_alive(L):
    assert L.pa_capture_alive(None) == 0
    L.pa_capture_free(None)
