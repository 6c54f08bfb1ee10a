"""ekv_extend_attention over E4M3 pages of small values beside a page of zeros, to which the demotion
gives the scale 1: the zeros take their share of the weights and no precision from the others."""

import numpy as np
import pytest

from oracle import extend as oe

from _extend import cu_of, make_case, run_extend, to_device

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch_cuda():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return torch


def weight_rounding(case, q, cu, scales):
    """What the rounding of small weights can cost, [T][H_q]: a weight is held as w s / max(w s), times 2^7, in fp16, so
    below 2^-14 it is off by up to half of fp16's least step, 2^-25: 2^-32 of the largest. With codes up to
    448 that is 448 n 2^-32 max(w s) / sum(w) of n keys (1 / sum(w / max(w s)) is the result's divisor)."""
    T, Hq, D = q.shape
    G = Hq // case.k_pages.shape[2]
    out = np.zeros((T, Hq))
    for i, b, t in oe.places(case.seq_lens, cu):
        K, _ = oe.sequence_kv(b, case, t + 1)
        pages = case.block_table[b, np.arange(t + 1) // 16]
        for h in range(Hq):
            z = K[:, h // G] @ q[i, h].astype(np.float64) / np.sqrt(D)
            w = np.exp(z - z.max())
            out[i, h] = 448 * (t + 1) * 2.0 ** -32 * (w * scales[pages, h // G]).max() / w.sum()
    return out


@pytest.mark.parametrize("lens,new", [([200, 90], [1, 2]), ([200, 90], [50, 60]), ([3000, 90], [2, 1]), ([1500, 90], [40, 1])])
@pytest.mark.parametrize("power", [-16, -20, -22])
def test_a_page_of_zeros_beside_small_values(ekv_lib, torch_cuda, lens, new, power):
    torch = torch_cuda
    case = make_case(lens, 8, 2, 128, "e4m3", 1, 95)
    case.v_scales = (case.v_scales * 0 + np.float32(1.03 * 2.0 ** power)).astype(np.float32)
    for b in range(2):                                   # a page in the middle of each sequence
        page = case.block_table[b, 2]
        case.v_pages[page] = 0
        case.v_scales[page] = 1.0
    cu = cu_of(new)
    q = (0.05 * np.random.default_rng(96).standard_normal((int(cu[-1]), 8, 128))).astype(np.float16)
    ctx = ekv_lib.Context(8, 2, 128, 2)
    out, lse = run_extend(ekv_lib, ctx, to_device(case), torch.from_numpy(q).cuda(), torch.from_numpy(cu).cuda(), max(new))
    assert ctx.error() == (0, 0)
    ref, ref_lse, wabs, qk = oe.attention(q, case, cu)
    w = (128 + 4) * 2.0 ** -24 * qk + 2.0 ** -19 + max(lens) * 2.0 ** -24      # relative error of a weight before its rounding
    # the result's rounding, the weights' (2^-11, and w twice: product and divisor), and the small weights'
    tol = 2.0 ** -11 * np.abs(ref) + 2.0 ** -25 + (2.0 ** -11 + 2 * w[..., None]) * wabs * 1.01
    tol += weight_rounding(case, q, cu, case.v_scales)[..., None]
    err = np.abs(out.float().cpu().numpy() - ref)
    assert np.all(err <= tol), f"{err.max():.3e}, {(err / tol).max():.2f} of the bound"
    ctx.close()
