"""A bounded wait of the page transitions, made to run out in the test library: a wait of CTA 0 for its
third page (its first, where the ring has one slot) expects 16 bytes more than its copy delivers (the copy itself lands). The call returns and
reports the timeout; CTA 0's pages from there on stay as they were, all others are done, and the next
call does the rest."""

import ctypes
import os

import numpy as np
import pytest

from oracle import micro as om

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def waitlib(ekv_lib):
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    lib = ctypes.CDLL(os.path.join(os.path.dirname(ekv_lib.LIB_PATH), "libekv_waittest.so"))
    vp, i = ctypes.c_void_p, ctypes.c_int
    lib.ekv_create.argtypes = [ctypes.POINTER(vp), ctypes.POINTER(ekv_lib.ekv_config)]
    lib.ekv_destroy.argtypes = [vp]
    for f in (lib.ekv_demote_pages_micro, lib.ekv_expand_pages_micro):
        f.argtypes = [vp, vp, ctypes.c_longlong, i, vp, i, vp, vp]
    lib.ekv_get_error.argtypes = [vp, ctypes.POINTER(i), ctypes.POINTER(i)]
    lib.ekv_test_inject_wait_timeout.argtypes = [i]
    return lib, torch


def error(lib, ctx):
    code, detail = ctypes.c_int(-1), ctypes.c_int(-1)
    assert lib.ekv_get_error(ctx, ctypes.byref(code), ctypes.byref(detail)) == 0
    return code.value, detail.value


@pytest.mark.parametrize("hkv,d,slot", [(1, 64, 2), (2, 64, 2), (8, 128, 0)])
def test_a_wait_runs_out_between_stored_pages(ekv_lib, waitlib, hkv, d, slot):
    lib, torch = waitlib
    grid = 4 * torch.cuda.get_device_properties(0).multi_processor_count
    P, n, micro = 6 * grid + 3, 16 * hkv * d, om.page_bytes(hkv, d)
    rng = np.random.default_rng(110)
    x = rng.standard_normal((32, 16, hkv, d)).astype(np.float16)
    kind = torch.from_numpy(rng.integers(0, 32, P)).cuda()

    def rows(a):
        return torch.from_numpy(np.ascontiguousarray(a).reshape(32, -1).view(np.uint8).copy()).cuda()[kind]

    coded = np.stack([om.encode_page(p) for p in x])
    back = np.stack([om.decode_page(c, hkv, d) for c in coded]).astype(np.float16)
    v = rows(x)
    m, ids = torch.zeros(P, dtype=torch.uint8, device="cuda"), torch.arange(P, dtype=torch.int32, device="cuda")
    first = ids % grid == 0                                 # CTA 0's; demoting, it ends before the page of number `slot`
    left = first & (ids // grid >= slot)
    ctx, cfg = ctypes.c_void_p(), ekv_lib.ekv_config(hkv, hkv, d, 1)
    assert lib.ekv_create(ctypes.byref(ctx), ctypes.byref(cfg)) == 0

    def call(f, inject):
        assert lib.ekv_test_inject_wait_timeout(inject) == 0
        st = torch.cuda.current_stream().cuda_stream
        assert f(ctx, v.data_ptr(), 2 * n, P, ids.data_ptr(), P, m.data_ptr(), st) == 0
        want = (ekv_lib.EKV_ERR_DEVICE_CHECK, ekv_lib.EKV_DETAIL_TIMEOUT) if inject else (0, 0)
        assert error(lib, ctx) == want                       # (synchronises)

    try:
        before, after = v.clone(), v.clone()
        after[:, :micro] = rows(coded)
        call(lib.ekv_demote_pages_micro, 1)
        assert torch.equal(m, torch.where(left, 0, 3).to(torch.uint8))
        assert torch.equal(v, torch.where(left[:, None], before, after))
        call(lib.ekv_demote_pages_micro, 0)
        assert bool((m == 3).all()) and torch.equal(v, after)
        call(lib.ekv_expand_pages_micro, 1)
        left = first & (ids // grid >= 2)                    # (a ring of five pages at least)
        assert torch.equal(m, torch.where(left, 3, 0).to(torch.uint8))
        assert torch.equal(v, torch.where(left[:, None], after, rows(back)))
        call(lib.ekv_expand_pages_micro, 0)
        assert not m.any() and torch.equal(v, rows(back))
    finally:
        lib.ekv_destroy(ctx)
