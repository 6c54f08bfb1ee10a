"""Refusals of the calls that take new tokens and of the microscaled transitions that need
no GPU: a missing context or a negative count, before anything else is looked at."""

import ctypes

import pytest


def test_a_null_context_is_refused(ekv_lib):
    L, inv = ekv_lib._lib, ekv_lib.EKV_ERR_INVALID_ARG
    n = None
    assert L.ekv_append_kv_rope(n, n, n, n, 0, 0, 0, n, 0, 0, 0, n, n, n, 0, 0, n, 0, n, 0, n, 0, n, n, 1, 1, n) == inv
    assert L.ekv_extend_attention(n, n, n, n, 0, 0, n, 0, n, 0, n, 0, n, n, 1, 1, 1, 0, ctypes.c_float(0), n, n, n) == inv
    assert L.ekv_demote_pages_micro(n, n, 0, 0, n, 1, n, n) == inv
    assert L.ekv_expand_pages_micro(n, n, 0, 0, n, 1, n, n) == inv


@pytest.mark.parametrize("name", ["ekv_append_kv_rope", "ekv_extend_attention", "ekv_demote_pages_micro", "ekv_expand_pages_micro"])
def test_the_binding_raises(ekv_lib, name):
    import inspect
    f = getattr(ekv_lib, name)
    args = [None if p == "ctx" else 0 for p in inspect.signature(f).parameters]
    with pytest.raises(ekv_lib.EkvError) as e:
        f(*args)
    assert e.value.status == ekv_lib.EKV_ERR_INVALID_ARG
