"""ekv_demote_pages_micro and ekv_expand_pages_micro, byte for byte against the oracle."""

import numpy as np
import pytest

from oracle import micro as om

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch_cuda():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return torch


def pool(P, hkv, d, seed, pad=0):
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((P, 16, hkv, d)) * np.exp(rng.uniform(-18, 9, (P, 16, hkv, 1)))
    x = x.clip(-65504, 65504).astype(np.float16)
    x[0, :4] = 0
    x[1 % P, 2, 0, :32] = -0.0
    x[2 % P, 3, 0, :32] = np.float16(65504)
    return np.concatenate([x.reshape(P, -1).view(np.uint8), np.full((P, pad), 0xCD, np.uint8)], 1)


@pytest.mark.parametrize("hkv,d,P,pad", [(8, 128, 40, 0), (1, 64, 7, 16), (2, 64, 700, 0), (4, 128, 33, 48), (1, 128, 1, 0)])
def test_round_trip_matches_the_oracle(ekv_lib, torch_cuda, hkv, d, P, pad):
    torch = torch_cuda
    vb = pool(P, hkv, d, 40 + P, pad)
    rng = np.random.default_rng(P)
    mode = np.where(rng.random(P) < 0.2, rng.integers(1, 4, P), 0).astype(np.uint8)
    # pages already in the microscaled form hold such bytes
    for p in np.flatnonzero(mode == 3):
        vb[p][: om.page_bytes(hkv, d)] = om.encode_page(rng.standard_normal((16, hkv, d)))
    ids = rng.permutation(P)[: max(1, P * 3 // 4)].astype(np.int32)
    v, m, di = (torch.from_numpy(x.copy()).cuda() for x in (vb, mode, ids))
    ctx = ekv_lib.Context(hkv, hkv, d, 1)
    ekv_lib.ekv_demote_pages_micro(ctx.handle, v, vb.shape[1], P, di, len(ids), m)
    torch.cuda.synchronize()
    assert ctx.error() == (0, 0)
    rv, rm, _ = om.demote_pages(vb, ids, mode, hkv, d)
    assert np.array_equal(m.cpu().numpy(), rm) and np.array_equal(v.cpu().numpy(), rv)
    ekv_lib.ekv_expand_pages_micro(ctx.handle, v, vb.shape[1], P, di, len(ids), m)
    torch.cuda.synchronize()
    assert ctx.error() == (0, 0)
    rv, rm = om.expand_pages(rv, ids, rm, hkv, d)
    assert np.array_equal(m.cpu().numpy(), rm) and np.array_equal(v.cpu().numpy(), rv)


def test_every_fp16_magnitude_as_a_block_maximum(ekv_lib, torch_cuda):
    """Each finite fp16 value heads a block of its own, under multiples that meet every tie."""
    torch = torch_cuda
    bits = np.arange(0x7c00, dtype=np.uint16)
    a = bits.view(np.float16).astype(np.float64)
    frac = np.linspace(-1, 1, 32)
    frac[5:12] = [1, 1 / 12, 1 / 8, 5 / 24, 7 / 24, 5 / 12, 5 / 6]
    x = (a[:, None] * frac).astype(np.float16)
    x[:, 5] = a.astype(np.float16)
    x = np.concatenate([x.reshape(-1), np.zeros(-x.size % (16 * 128), np.float16)]).reshape(-1, 16, 1, 128)
    vb = x.reshape(x.shape[0], -1).view(np.uint8)
    P = vb.shape[0]
    v, m, ids = torch.from_numpy(vb.copy()).cuda(), torch.zeros(P, dtype=torch.uint8, device="cuda"), torch.arange(P, dtype=torch.int32, device="cuda")
    ctx = ekv_lib.Context(1, 1, 128, 1)
    ekv_lib.ekv_demote_pages_micro(ctx.handle, v, vb.shape[1], P, ids, P, m)
    torch.cuda.synchronize()
    assert ctx.error() == (0, 0)
    rv, _, _ = om.demote_pages(vb, range(P), np.zeros(P, np.uint8), 1, 128)
    assert np.array_equal(v.cpu().numpy(), rv)


def test_nonfinite_bad_ids_and_bad_scales(ekv_lib, torch_cuda):
    torch = torch_cuda
    vb = pool(4, 2, 64, 50)
    vb.view(np.float16).reshape(4, 16, 2, 64)[1, 15, 1, 63] = np.inf
    v, m = torch.from_numpy(vb.copy()).cuda(), torch.zeros(4, dtype=torch.uint8, device="cuda")
    ctx = ekv_lib.Context(2, 2, 64, 1)
    ids = torch.tensor([0, 1, 3], dtype=torch.int32, device="cuda")
    ekv_lib.ekv_demote_pages_micro(ctx.handle, v, vb.shape[1], 4, ids, 3, m)
    assert ctx.error() == (ekv_lib.EKV_ERR_DEVICE_CHECK, ekv_lib.EKV_DETAIL_NONFINITE_PAGE)
    rv, rm, bad = om.demote_pages(vb, [0, 1, 3], np.zeros(4, np.uint8), 2, 64)
    assert bad == [1] and np.array_equal(v.cpu().numpy(), rv) and np.array_equal(m.cpu().numpy(), rm)
    v[0, 16 * 32] = 141                                   # a scale above the range
    v[3, 16 * 32 + 1] = 102                               # and one below
    raw = v.cpu().numpy()
    ekv_lib.ekv_expand_pages_micro(ctx.handle, v, vb.shape[1], 4, ids, 3, m)
    assert ctx.error() == (ekv_lib.EKV_ERR_DEVICE_CHECK, ekv_lib.EKV_DETAIL_SCALE)
    assert np.array_equal(v.cpu().numpy(), om.expand_pages(raw, [0, 1, 3], rm, 2, 64)[0])
    for bad_id in (-1, 4):
        ids[0] = bad_id
        ekv_lib.ekv_demote_pages_micro(ctx.handle, v, vb.shape[1], 4, ids, 1, m)
        assert ctx.error() == (ekv_lib.EKV_ERR_DEVICE_CHECK, ekv_lib.EKV_DETAIL_PAGE_ID)
    for f in (ekv_lib.ekv_demote_pages_micro, ekv_lib.ekv_expand_pages_micro):
        for a in ((None, v, vb.shape[1], 4, ids, 1, m), (ctx.handle, None, vb.shape[1], 4, ids, 1, m),
                  (ctx.handle, v, vb.shape[1] - 16, 4, ids, 1, m), (ctx.handle, v, vb.shape[1], 4, None, 1, m),
                  (ctx.handle, v, vb.shape[1], 4, ids, 1, None), (ctx.handle, v, vb.shape[1], 4, ids, -1, m)):
            with pytest.raises(ekv_lib.EkvError) as e:
                f(*a)
            assert e.value.status == ekv_lib.EKV_ERR_INVALID_ARG
        f(ctx.handle, None, 0, 0, None, 0, None)          # no pages: nothing to do
    with pytest.raises(ekv_lib.EkvError):                 # no located form
        ekv_lib.ekv_transition_pages(ctx.handle, 3, v, vb.shape[1], 4, 4, ids, None, None, 1, m)


def test_a_step_over_moving_pages(ekv_lib, torch_cuda):
    """Demote, write, attend, expand, attend: the run of the calls together."""
    torch = torch_cuda
    from _extend import check, cu_of, make_case, run_extend, to_device
    from test_append_rope_gpu import call, rope_table
    lens = np.array([130, 300], np.int32)
    case = make_case(lens, 8, 2, 128, "fp16", 0, 51)
    case.page_mode, P = np.zeros(case.num_pages, np.uint8), case.num_pages
    d = to_device(case)
    ctx = ekv_lib.Context(8, 2, 128, 2)
    ids = torch.from_numpy(case.block_table[1, :18].copy()).cuda()      # the full pages of sequence 1
    ekv_lib.ekv_demote_pages_micro(ctx.handle, d.v_pages, d.v_page_stride, P, ids, 18, d.page_mode)
    cu = cu_of([1, 20])                                   # sequence 1's chunk reaches into two of them
    dcu, rope = torch.from_numpy(cu).cuda(), torch.from_numpy(rope_table(300, 128)).cuda()
    q, k, v = (torch.randn((21, h, 128), dtype=torch.float16, device="cuda") for h in (8, 2, 2))
    call(ekv_lib, ctx, d, q, k, v, rope, 128, 0, q, d.seq_lens, dcu, 2, 21)
    out, lse = run_extend(ekv_lib, ctx, d, q, dcu, 20)
    ekv_lib.ekv_expand_pages_micro(ctx.handle, d.v_pages, d.v_page_stride, P, ids, 18, d.page_mode)
    out2, lse2 = run_extend(ekv_lib, ctx, d, q, dcu, 20)
    assert ctx.error() == (0, 0)
    assert not d.page_mode.any()
    case.k_pages, case.v_pages, case.page_mode = d.k_pages.cpu().numpy(), d.v_pages.cpu().numpy(), d.page_mode.cpu().numpy()
    check(case, cu, q.cpu().numpy(), out, lse)            # the values are the same in either form
    check(case, cu, q.cpu().numpy(), out2, lse2)
