"""ekv_extend_attention over E4M3 pages whose scales lie far apart: the smallest fp32 values, the
largest that the call takes, and those beyond, which are reported."""

import numpy as np
import pytest

from oracle import extend as oe

from _extend import bounds, check, cu_of, make_case, run_extend, to_device

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch_cuda():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return torch


def run(ekv, torch, case, new, seed, window=0):
    cu = cu_of(new)
    q = np.random.default_rng(seed).standard_normal((int(cu[-1]), 8, 128)).astype(np.float16)
    ctx = ekv.Context(8, 2, 128, len(new))
    out, lse = run_extend(ekv, ctx, to_device(case), torch.from_numpy(q).cuda(), torch.from_numpy(cu).cuda(), max(new), window)
    err = ctx.error()
    ctx.close()
    return cu, q, out, lse, err


FORMS = [("e4m3", [200, 160, 90], [1, 1, 1]), ("e4m3", [200, 160, 90], [50, 60, 70]), ("all", [200, 160, 90], [16, 2, 9]),
         ("all", [200, 160, 90], [50, 60, 70]), ("e4m3", [6000, 90, 1], [3, 1, 1]), ("e4m3", [2500, 90, 1], [40, 1, 1])]


@pytest.mark.parametrize("fmt,lens,new", FORMS)
@pytest.mark.parametrize("small", [1e-45, 1e-40, 1e-38, 2.0 ** -100, 2.0 ** -60, 2.0 ** -44, 2.0 ** -43])
def test_small_scales_beside_ordinary_ones(ekv_lib, torch_cuda, fmt, lens, new, small):
    """The keys of such pages count in the sum as all others do; their values add next to nothing."""
    case = make_case(lens, 8, 2, 128, fmt, 1, 70)
    rng = np.random.default_rng(71)
    case.v_scales = np.where(rng.random(case.v_scales.shape) < 0.5, np.float32(small), case.v_scales).astype(np.float32)
    cu, q, out, lse, err = run(ekv_lib, torch_cuda, case, new, 72)
    assert err == (0, 0)
    check(case, cu, q, out, lse)


@pytest.mark.parametrize("fmt,lens,new", FORMS)
def test_the_whole_range_in_one_call(ekv_lib, torch_cuda, fmt, lens, new):
    """Scales from the smallest to 2^40; pages of the large ones hold zeros, so that every output is an fp16 value. The
    outputs themselves are not compared: a weight is rounded to fp16 relative to the row's largest weight times scale, which
    a page of zeros under 2^40 sets 2^40 above the others, so that all of them may be lost."""
    case = make_case(lens, 8, 2, 128, fmt, 1, 73)
    rng = np.random.default_rng(74)
    pick = rng.integers(0, 6, case.v_scales.shape)
    case.v_scales = np.choose(pick, [case.v_scales, np.float32(1e-45), np.float32(1e-30), np.float32(2.0 ** -50),
                                     np.float32(2.0 ** 40), np.float32(2.0 ** 30)]).astype(np.float32)
    mode = np.full(case.num_pages, 1) if case.page_mode is None else case.page_mode
    codes = case.v_pages[:, : 16 * 2 * 128].reshape(-1, 16, 2, 128)
    for h in range(2):
        codes[(pick[:, h] >= 4) & (mode == 1), :, h] = 0
    case.v_pages = np.concatenate([codes.reshape(len(codes), -1), case.v_pages[:, 16 * 2 * 128:]], 1)
    cu, q, out, lse, err = run(ekv_lib, torch_cuda, case, new, 75)
    assert err == (0, 0) and torch_cuda.isfinite(out).all()
    ref = oe.attention(q, case, cu)
    _, tol = bounds(case, cu, ref, max(lens))
    assert np.all(np.abs(lse.cpu().numpy() - ref[1]) <= tol)


@pytest.mark.parametrize("new", [[1, 1], [50, 60]])
@pytest.mark.parametrize("scale", [2.0 ** 41, 3e38])
def test_scales_beyond_the_range_are_reported(ekv_lib, torch_cuda, new, scale):
    torch = torch_cuda
    case = make_case([200, 160], 8, 2, 128, "e4m3", 1, 76)
    case.v_scales[case.block_table[1, 1], 1] = np.float32(scale)
    cu, q, out, lse, err = run(ekv_lib, torch, case, new, 77)
    assert err == (ekv_lib.EKV_ERR_DEVICE_CHECK, ekv_lib.EKV_DETAIL_SCALE)
    hit = torch.zeros_like(lse, dtype=torch.bool)
    hit[new[0]:, 4:] = True
    assert torch.all(out[hit] == 0) and torch.all(lse[hit] == -float("inf"))
    case.v_scales[case.block_table[1, 1], 1] = np.float32(0.01)
    _, _, good, good_lse, err = run(ekv_lib, torch, case, new, 77)
    assert err == (0, 0) and torch.equal(out[~hit], good[~hit]) and torch.equal(lse[~hit], good_lse[~hit])


@pytest.mark.parametrize("new", [[1, 1], [50, 60]])
@pytest.mark.parametrize("scale", [1e-45, 1e-38, 2.0 ** -30, 2.0 ** 41, 3e38])
def test_one_scale_for_all_codes_may_be_any(ekv_lib, torch_cuda, new, scale):
    torch = torch_cuda
    case = make_case([200, 160], 8, 2, 128, "e4m3", 0, 78)
    unit = run(ekv_lib, torch, case, new, 79)
    case.v_scales[:] = np.float32(scale)
    cu, q, out, lse, err = run(ekv_lib, torch, case, new, 79)
    assert err == (0, 0) and torch.equal(lse, unit[3])
    if scale <= 1:
        check(case, cu, q, out, lse)
    else:                                                # sums of the codes times the scale: infinite, or zero
        assert not torch.isnan(out).any()
        assert torch.equal(torch.sign(out), torch.sign(unit[2])) and torch.isinf(out[unit[2] != 0]).all()
