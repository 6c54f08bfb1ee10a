"""Refusals of the rotary table, the normalising writer and the attention of packed prompts that need no GPU: a missing
context, before anything else is looked at."""

import ctypes
import inspect

import pytest


def test_a_null_context_is_refused(ekv_lib):
    L, inv, n = ekv_lib._lib, ekv_lib.EKV_ERR_INVALID_ARG, None
    cfg = ekv_lib.ekv_rope_config(1e4, 0, 1.0, 1.0, 1.0, 2.0, 1.0)
    assert L.ekv_rope_table(n, ctypes.byref(cfg), n, 0, 1, 64, n) == inv
    assert L.ekv_append_kv_norm_rope(n, n, n, n, 0, 0, 0, n, n, ctypes.c_float(0), n, 0, 0, 0, n, n, n, n, 0, 0, n, 0, 0, n, 0,
                                     n, 0, n, n, 1, 1, n) == inv
    assert L.ekv_prompt_attention(n, n, n, n, 0, 0, 0, n, 1, 1, 0, ctypes.c_float(0), n, n, n) == inv


@pytest.mark.parametrize("name", ["ekv_rope_table", "ekv_append_kv_norm_rope", "ekv_prompt_attention"])
def test_the_binding_raises(ekv_lib, name):
    f = getattr(ekv_lib, name)
    args = [None if p in ("ctx", "cfg") else 0 for p in inspect.signature(f).parameters]
    with pytest.raises(ekv_lib.EkvError) as e:
        f(*args)
    assert e.value.status == ekv_lib.EKV_ERR_INVALID_ARG
