"""ekv_extend_attention with a failing page that only some queries of a sequence see: those get zeros
and lse -inf, the others keep the bits that they have over a good page."""

import numpy as np
import pytest

from _extend import check, cu_of, make_case, run_extend, to_device

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch_cuda():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return torch


# length and new tokens of the sequence, failing page, window: queries before it, on it and past it
PLACES = [(90, 16, 5, 0), (90, 16, 4, 5), (90, 50, 3, 0), (90, 50, 3, 20), (300, 16, 18, 40), (700, 300, 30, 100),
          (9000, 16, 562, 0), (9000, 16, 561, 4), (9000, 300, 550, 0), (9000, 300, 550, 64), (9000, 300, 556, 5000)]


@pytest.mark.parametrize("fmt", ["e4m3", "all"])
@pytest.mark.parametrize("what", ["id", "mode", "scale"])
@pytest.mark.parametrize("length,n,page,window", PLACES)
def test_only_the_queries_that_see_it(ekv_lib, torch_cuda, fmt, what, length, n, page, window):
    torch = torch_cuda
    if what == "mode" and fmt == "e4m3":
        pytest.skip("a uniform pool has no mode bytes")
    lens, new = [100, length, 33], [3, n, 1]
    base = make_case(lens, 8, 2, 64, fmt, 1, 80)
    at = int(base.block_table[1, page])
    if base.page_mode is not None:                       # an E4M3 page: its scale can fail
        base.page_mode[at] = 1
        base.v_pages[at][: 16 * 2 * 64] = 0x38
        base.v_scales[at] = 0.01
    cu = cu_of(new)
    q = np.random.default_rng(81).standard_normal((int(cu[-1]), 8, 64)).astype(np.float16)
    ctx = ekv_lib.Context(8, 2, 64, 3)
    dq, dcu = torch.from_numpy(q).cuda(), torch.from_numpy(cu).cuda()
    good, good_lse = run_extend(ekv_lib, ctx, to_device(base), dq, dcu, n, window=window)
    assert ctx.error() == (0, 0)
    check(base, cu, q, good, good_lse, window, rows={0, 2, 3, 3 + n // 3, 2 + n, 3 + n})

    d, heads = to_device(base), slice(0, 8)
    if what == "id":
        d.block_table[1, page] = -7
    elif what == "mode":
        d.page_mode[at] = 77
    else:
        d.v_scales[at, 1] = float("inf")
        heads = slice(4, 8)
    out, lse = run_extend(ekv_lib, ctx, d, dq, dcu, n, window=window)
    detail = {"id": ekv_lib.EKV_DETAIL_PAGE_ID, "mode": ekv_lib.EKV_DETAIL_PAGE_MODE, "scale": ekv_lib.EKV_DETAIL_SCALE}[what]
    assert ctx.error() == (ekv_lib.EKV_ERR_DEVICE_CHECK, detail)
    pos = length - n + np.arange(n)
    sees = (pos >= 16 * page) & ((pos - window + 1 <= 16 * page + 15) | (window == 0))
    assert sees.any() and not sees.all()
    hit = torch.zeros((int(cu[-1]), 8), dtype=torch.bool, device="cuda")
    hit[3:3 + n, heads] = torch.from_numpy(sees).cuda()[:, None]
    assert torch.all(out[hit] == 0) and torch.all(lse[hit] == -float("inf"))
    assert torch.equal(out[~hit], good[~hit]) and torch.equal(lse[~hit], good_lse[~hit])
    ctx.close()
