"""ekv_append_kv_norm_rope on many tokens: blocks in rounds, tokens in parts, the ring run through many times. Rows do not depend on
one another, so a call of thousands of tokens gives bit for bit what calls of a few give, which the oracle checks elsewhere; and
the wait for a ring's copies, run out once in the test library."""

import ctypes
import os
import time

import numpy as np
import pytest

from _extend import cu_of, make_case, to_device
from _prompt import rope_table, write

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch_cuda():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return torch


@pytest.mark.parametrize("grow", [0, 1])
@pytest.mark.parametrize("fmt", ["e4m3", "all"])
@pytest.mark.parametrize("hq,hkv,d,queries", [(32, 8, 128, True), (64, 8, 128, True), (3, 1, 64, True), (16, 8, 64, True), (8, 2, 128, False)])
def test_one_call_is_many_small_ones(ekv_lib, torch_cuda, grow, fmt, hq, hkv, d, queries):
    torch = torch_cuda
    rng = np.random.default_rng(300)
    new = [int(n) for n in rng.integers(1, 400, 40)] + [9000, 0, 3000, 1]
    ctx_len = [int(n) for n in rng.integers(0, 40, len(new))]
    lens = np.array([n + c for n, c in zip(new, ctx_len)], np.int32)
    case = make_case(lens, hq, hkv, d, fmt, 1, 301, stride_pad=16)
    T, cu = sum(new), cu_of(new)
    rows = torch.randn((T, hq + 2 * hkv, d), device="cuda", dtype=torch.float16)
    q, k, v = rows.split((hq, hkv, hkv), 1)
    q = q if queries else None
    w = torch.from_numpy((1 + 0.5 * rng.standard_normal((2, d))).astype(np.float16)).cuda()
    rope = torch.from_numpy(rope_table(int(lens.max()), d // 2)).cuda()
    ctx = ekv_lib.Context(hq, hkv, d, 1)

    def run(pieces):
        dev = to_device(case)
        qo, ko = (torch.full((T, h, d), float("nan"), device="cuda", dtype=torch.float16) for h in (hq, hkv))
        for b0, b1 in pieces:
            a, z = int(cu[b0]), int(cu[b1])
            if a == z:
                continue
            part = torch.from_numpy(cu[b0:b1 + 1] - cu[b0]).cuda()
            write(ekv_lib, ctx, dev, None if q is None else q[a:z], k[a:z], v[a:z], rope, d // 2, 1, qo[a:z], dev.seq_lens[b0:b1].contiguous(), part,
                  b1 - b0, z - a, q_weight=w[0], k_weight=w[1], k_out=ko[a:z], grow_scales=grow,
                  block_table=dev.block_table[b0:b1].contiguous())
        assert ctx.error() == (0, 0)
        return dev, qo, ko

    one, q1, k1 = run([(0, len(new))])
    dev, q2, k2 = run([(b, b + 1) for b in range(len(new))])
    assert not torch.isnan(k1).any() and (q is None or not torch.isnan(q1).any())
    for x, y in ((q1, q2), (k1, k2), (one.k_pages, dev.k_pages)):
        assert torch.equal(x.view(torch.int16), y.view(torch.int16))
    assert torch.equal(one.v_pages, dev.v_pages)
    assert torch.equal(one.v_scales.view(torch.int32), dev.v_scales.view(torch.int32))


def test_the_wait_for_a_ring_runs_out_and_the_context_recovers(ekv_lib, torch_cuda):
    torch = torch_cuda
    lib = ctypes.CDLL(os.path.join(os.path.dirname(ekv_lib.LIB_PATH), "libekv_waittest.so"))
    vp, i = ctypes.c_void_p, ctypes.c_int
    lib.ekv_create.argtypes = [ctypes.POINTER(vp), ctypes.POINTER(ekv_lib.ekv_config)]
    lib.ekv_destroy.argtypes = [vp]
    lib.ekv_append_kv_norm_rope.argtypes = ekv_lib._lib.ekv_append_kv_norm_rope.argtypes
    lib.ekv_get_error.argtypes = [vp, ctypes.POINTER(i), ctypes.POINTER(i)]
    lib.ekv_test_inject_wait_timeout.argtypes = [i]
    hq, hkv, d, n = 8, 2, 128, 5000
    case = make_case([n], hq, hkv, d, "e4m3", 1, 302)
    q, k, v = torch.randn((n, hq + 2 * hkv, d), device="cuda", dtype=torch.float16).split((hq, hkv, hkv), 1)
    w = torch.ones(d, device="cuda", dtype=torch.float16)
    rope = torch.from_numpy(rope_table(n, d)).cuda()
    cu = torch.tensor([0, n], device="cuda", dtype=torch.int32)
    ctx, cfg = ctypes.c_void_p(), ekv_lib.ekv_config(hq, hkv, d, 1)
    assert lib.ekv_create(ctypes.byref(ctx), ctypes.byref(cfg)) == 0

    def call(grow):
        dev, qo, ko = to_device(case), torch.empty((n, hq, d), device="cuda", dtype=torch.float16), torch.empty((n, hkv, d), device="cuda", dtype=torch.float16)
        p = lambda x: x.data_ptr()
        assert lib.ekv_append_kv_norm_rope(ctx, p(q), p(k), p(v), q.stride(0), k.stride(0), v.stride(0), p(w), p(w), 1e-6, p(rope), n, d, 0, p(qo),
                                           p(ko), p(dev.k_pages), p(dev.v_pages), dev.v_page_stride, dev.num_pages, p(dev.v_scales), 1, grow, None, 1,
                                           p(dev.block_table), int(dev.block_table.shape[1]), p(dev.seq_lens), p(cu), 1, n,
                                           torch.cuda.current_stream().cuda_stream) == 0
        code, detail = ctypes.c_int(-1), ctypes.c_int(-1)
        assert lib.ekv_get_error(ctx, ctypes.byref(code), ctypes.byref(detail)) == 0
        return (code.value, detail.value), (qo, ko, dev.k_pages, dev.v_pages.view(torch.int8), dev.v_scales)

    try:
        for grow in (0, 1):
            err, good = call(grow)
            assert err == (0, 0)
            assert lib.ekv_test_inject_wait_timeout(1) == 0
            t0 = time.perf_counter()
            assert call(grow)[0] == (ekv_lib.EKV_ERR_DEVICE_CHECK, ekv_lib.EKV_DETAIL_TIMEOUT)
            assert time.perf_counter() - t0 < 5.0
            err, again = call(grow)
            assert err == (0, 0) and all(torch.equal(torch.nan_to_num(x), torch.nan_to_num(y)) for x, y in zip(good, again))
    finally:
        lib.ekv_destroy(ctx)
