"""ekv_extend_attention over pools whose pages lie past 2^31 and 2^32 bytes, in slots of an odd stride."""

import numpy as np
import pytest

from _extend import check, cu_of, make_case, run_extend, to_device

pytestmark = pytest.mark.gpu

STRIDE = 32768 + 16                                    # in 16-byte units, 2049 a page: past 2^31 of them in a pool of 35 GB


@pytest.fixture(scope="module")
def torch_cuda():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return torch


@pytest.fixture(scope="module")
def pools(torch_cuda):
    """K and V pools (not filled) of so many pages that the units of the last one's values pass 2^31."""
    torch = torch_cuda
    pages = 2 ** 31 // (STRIDE // 16) + 40
    if torch.cuda.mem_get_info()[0] < 60 << 30:
        pytest.skip("needs 60 GB")
    k = torch.empty((pages, 16, 1, 64), dtype=torch.float16, device="cuda")
    v = torch.empty((pages, STRIDE), dtype=torch.uint8, device="cuda")
    yield k, v
    del k, v
    torch.cuda.empty_cache()


def place(torch, case, pools, first):
    """The case with its pages at `first` and on."""
    k, v = pools
    d = to_device(case)
    n = case.num_pages
    k[first:first + n] = d.k_pages
    v[first:first + n, :case.v_pages.shape[1]] = d.v_pages
    scales = torch.ones((len(k), 1), dtype=torch.float32, device="cuda")
    if case.v_scales is not None and case.scale_mode == 1:
        scales[first:first + n] = d.v_scales
    d.v_scales = scales if case.scale_mode == 1 else d.v_scales
    d.k_pages, d.v_pages = k, v
    d.block_table = d.block_table + first
    if case.page_mode is not None:
        modes = torch.full((len(k),), 255, dtype=torch.uint8, device="cuda")
        modes[first:first + n] = d.page_mode
        d.page_mode = modes
    return d


@pytest.mark.parametrize("new", [[1, 1], [50, 60]])
@pytest.mark.parametrize("fmt,sm", [("e4m3", 0), ("e4m3", 1), ("micro", 0), ("fp16", 0), ("all", 1)])
def test_pages_at_the_end_of_a_large_pool(ekv_lib, torch_cuda, pools, fmt, sm, new):
    """E4M3 and microscaled pools are taken whole; FP16 pages up to the 2^31 units that a coordinate names."""
    torch = torch_cuda
    case = make_case([200, 160], 2, 1, 64, fmt, sm, 98)
    cu = cu_of(new)
    q = np.random.default_rng(99).standard_normal((int(cu[-1]), 2, 64)).astype(np.float16)
    dq, dcu = torch.from_numpy(q).cuda(), torch.from_numpy(cu).cuda()
    ctx = ekv_lib.Context(2, 1, 64, 2)
    fp16_pages = fmt in ("fp16", "all")
    pages = len(pools[0]) if not fp16_pages else (2 ** 31 - 1) // (STRIDE // 16)
    d = place(torch, case, pools, pages - case.num_pages)
    if fp16_pages:
        with pytest.raises(ekv_lib.EkvError) as e:
            run_extend(ekv_lib, ctx, d, dq, dcu, max(new))
        assert e.value.status == ekv_lib.EKV_ERR_UNSUPPORTED
        d.k_pages, d.v_pages = d.k_pages[:pages], d.v_pages[:pages]
    out, lse = run_extend(ekv_lib, ctx, d, dq, dcu, max(new))
    assert ctx.error() == (0, 0)
    check(case, cu, q, out, lse)
    ctx.close()
