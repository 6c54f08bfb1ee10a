"""The bounded waits of ekv_prompt_attention, made to run out one after the other in the test library: a barrier of
CTA 0 expects 16 bytes that no copy delivers, so that the role that waits for it gives up and all others wind down. The
call returns and reports the timeout; the next calls on the context are right."""

import ctypes
import os
import time

import numpy as np
import pytest

from _extend import cu_of
from test_prompt_gpu import check, rows_of

pytestmark = pytest.mark.gpu

# (kv_empty and q_empty are waited for when a stage or tile is used again, o_free when a second item ends its first block)
WAITS = ("q_full", "kv_full of keys", "kv_full of values", "v_raw", "s_full", "p_full", "pv_done", "kv_empty", "q_empty", "o_free")


@pytest.fixture(scope="module")
def waitlib(ekv_lib):
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    lib = ctypes.CDLL(os.path.join(os.path.dirname(ekv_lib.LIB_PATH), "libekv_waittest.so"))
    vp, i = ctypes.c_void_p, ctypes.c_int
    lib.ekv_create.argtypes = [ctypes.POINTER(vp), ctypes.POINTER(ekv_lib.ekv_config)]
    lib.ekv_destroy.argtypes = [vp]
    lib.ekv_prompt_attention.argtypes = ekv_lib._lib.ekv_prompt_attention.argtypes
    lib.ekv_get_error.argtypes = [vp, ctypes.POINTER(i), ctypes.POINTER(i)]
    lib.ekv_test_inject_prompt_timeout.argtypes = [i]
    return lib, torch


@pytest.mark.parametrize("d", [128, 64])
def test_each_wait_runs_out_and_the_context_recovers(ekv_lib, waitlib, d):
    lib, torch = waitlib
    lens = [100] * 600                                   # one block an item, its values past the prompt's end
    cu, T = cu_of(lens), sum(lens)
    x = rows_of(np.random.default_rng(240), T, 8, 2, d)
    q, k, v = torch.from_numpy(x).cuda().split((8, 2, 2), 1)
    dcu = torch.from_numpy(cu).cuda()
    out, lse = torch.empty((T, 8, d), device="cuda", dtype=torch.float16), torch.empty((T, 8), device="cuda")
    ctx, cfg = ctypes.c_void_p(), ekv_lib.ekv_config(8, 2, d, 600)
    assert lib.ekv_create(ctypes.byref(ctx), ctypes.byref(cfg)) == 0

    def call():
        st = torch.cuda.current_stream().cuda_stream
        assert lib.ekv_prompt_attention(ctx, q.data_ptr(), k.data_ptr(), v.data_ptr(), q.stride(0), k.stride(0), v.stride(0), dcu.data_ptr(),
                                        600, T, 0, 0.0, out.data_ptr(), lse.data_ptr(), st) == 0
        code, detail = ctypes.c_int(-1), ctypes.c_int(-1)
        assert lib.ekv_get_error(ctx, ctypes.byref(code), ctypes.byref(detail)) == 0
        return code.value, detail.value

    try:
        assert call() == (0, 0)
        some = cu_of(lens[:5])
        check(x[:500, :8], x[:500, 8:10], x[:500, 10:], some, out[:500], lse[:500])
        good = out.clone(), lse.clone()
        for wait in range(1, len(WAITS) + 1):
            assert lib.ekv_test_inject_prompt_timeout(wait) == 0
            t0 = time.perf_counter()
            err = call()
            assert time.perf_counter() - t0 < 5.0
            assert err == (ekv_lib.EKV_ERR_DEVICE_CHECK, ekv_lib.EKV_DETAIL_TIMEOUT), WAITS[wait - 1]
            out.fill_(float("nan"))
            lse.fill_(float("nan"))
            assert call() == (0, 0), WAITS[wait - 1]
            assert torch.equal(out, good[0]) and torch.equal(lse, good[1]), WAITS[wait - 1]
    finally:
        lib.ekv_destroy(ctx)
