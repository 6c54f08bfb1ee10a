"""The bounded waits of ekv_extend_attention, made to run out one after the other in the test library:
a barrier of CTA 0 expects 16 bytes that no copy delivers, so that the role that waits for it gives up and
all others wind down. The call returns and reports the timeout; the next calls on the context are right."""

import ctypes
import os
import time

import numpy as np
import pytest

from _extend import check, cu_of, make_case, to_device

pytestmark = pytest.mark.gpu

WAITS = ("q_full", "k_full", "v_full", "raw_full", "s_full", "p_full", "pv_done", "seg_full", "meta_full")


@pytest.fixture(scope="module")
def waitlib(ekv_lib):
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    lib = ctypes.CDLL(os.path.join(os.path.dirname(ekv_lib.LIB_PATH), "libekv_waittest.so"))
    vp, i = ctypes.c_void_p, ctypes.c_int
    lib.ekv_create.argtypes = [ctypes.POINTER(vp), ctypes.POINTER(ekv_lib.ekv_config)]
    lib.ekv_destroy.argtypes = [vp]
    lib.ekv_extend_attention.argtypes = ekv_lib._lib.ekv_extend_attention.argtypes
    lib.ekv_get_error.argtypes = [vp, ctypes.POINTER(i), ctypes.POINTER(i)]
    lib.ekv_test_inject_extend_timeout.argtypes = [i]
    return lib, torch


@pytest.mark.parametrize("fmt,sm,d", [("fp16", 0, 128), ("e4m3", 1, 128), ("micro", 0, 64), ("all", 1, 128), ("all", 1, 64)])
@pytest.mark.parametrize("new", [[2, 1], [200, 30]])
def test_each_wait_runs_out_and_the_context_recovers(ekv_lib, waitlib, fmt, sm, d, new):
    lib, torch = waitlib
    lens = [100000, 500]                                 # (CTA 0 has blocks enough to reach every wait)
    case = make_case(lens, 8, 2, d, fmt, sm, 120)
    cu = cu_of(new)
    q = np.random.default_rng(121).standard_normal((int(cu[-1]), 8, d)).astype(np.float16)
    dv, dq, dcu = to_device(case), torch.from_numpy(q).cuda(), torch.from_numpy(cu).cuda()
    out, lse = torch.empty_like(dq), torch.empty(dq.shape[:2], device="cuda")
    ctx, cfg = ctypes.c_void_p(), ekv_lib.ekv_config(8, 2, d, 2)
    assert lib.ekv_create(ctypes.byref(ctx), ctypes.byref(cfg)) == 0

    def ptr(x):
        return None if x is None else x.data_ptr()

    def call():
        st = torch.cuda.current_stream().cuda_stream
        assert lib.ekv_extend_attention(ctx, ptr(dq), ptr(dv.k_pages), ptr(dv.v_pages), dv.v_page_stride, dv.num_pages,
                                        ptr(dv.v_scales), dv.scale_mode, ptr(dv.page_mode), dv.uniform_mode,
                                        ptr(dv.block_table), int(dv.block_table.shape[1]), ptr(dv.seq_lens), ptr(dcu), 2,
                                        int(cu[-1]), max(new), 0, 0.0, ptr(out), ptr(lse), st) == 0
        code, detail = ctypes.c_int(-1), ctypes.c_int(-1)
        assert lib.ekv_get_error(ctx, ctypes.byref(code), ctypes.byref(detail)) == 0
        return code.value, detail.value

    try:
        assert call() == (0, 0)
        check(case, cu, q, out, lse, rows={0, int(cu[-1]) - 1})
        good = out.clone(), lse.clone()
        for wait in range(1, len(WAITS) + 1):
            assert lib.ekv_test_inject_extend_timeout(wait) == 0
            t0 = time.perf_counter()
            err = call()
            assert time.perf_counter() - t0 < 5.0
            if WAITS[wait - 1] == "raw_full" and fmt == "fp16":
                assert err == (0, 0)                         # (no raw pages)
            else:
                assert err == (ekv_lib.EKV_ERR_DEVICE_CHECK, ekv_lib.EKV_DETAIL_TIMEOUT), WAITS[wait - 1]
            out.fill_(float("nan"))
            lse.fill_(float("nan"))
            assert call() == (0, 0), WAITS[wait - 1]
            assert torch.equal(out, good[0]) and torch.equal(lse, good[1]), WAITS[wait - 1]
    finally:
        lib.ekv_destroy(ctx)
