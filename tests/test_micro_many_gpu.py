"""Microscaled transitions of many pages a CTA: refills of the ring, further chunks of ids, and stored
pages with skipped and non-finite ones between them, byte for byte against the oracle."""

import numpy as np
import pytest

from oracle import micro as om

pytestmark = pytest.mark.gpu

KINDS = 48                                            # different pages; the pool repeats them


@pytest.fixture(scope="module")
def torch_cuda():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return torch


# items a CTA (4 an SM): 263 reach into a second chunk of 256 ids
@pytest.mark.parametrize("hkv,d,per_cta,pad", [(1, 64, 263, 0), (2, 64, 40, 16), (4, 128, 7, 0), (8, 128, 7, 32)])
@pytest.mark.parametrize("skipped,nonfinite", [(0.0, 0.0), (0.4, 0.0), (0.0, 0.4), (0.3, 0.2)])
def test_many_pages_a_cta(ekv_lib, torch_cuda, hkv, d, per_cta, pad, skipped, nonfinite):
    torch = torch_cuda
    rng = np.random.default_rng(60 + hkv)
    n = 16 * hkv * d
    size, micro = 2 * n + pad, om.page_bytes(hkv, d)
    x = (rng.standard_normal((KINDS, 16, hkv, d)) * np.exp(rng.uniform(-9, 9, (KINDS, 16, hkv, 1)))).clip(-65504, 65504)
    x = x.astype(np.float16)
    wrong = x.copy()
    wrong[np.arange(KINDS), rng.integers(0, 16, KINDS), rng.integers(0, hkv, KINDS), rng.integers(0, d, KINDS)] = np.inf
    coded = np.stack([om.encode_page(p) for p in x])
    back = np.stack([om.decode_page(c, hkv, d) for c in coded]).astype(np.float16)

    P = per_cta * 4 * torch.cuda.get_device_properties(0).multi_processor_count + 5
    kind = torch.from_numpy(rng.integers(0, KINDS, P)).cuda()
    mode = torch.from_numpy(np.where(rng.random(P) < skipped, rng.integers(1, 4, P), 0).astype(np.uint8)).cuda()
    bad = torch.from_numpy(rng.random(P) < nonfinite).cuda() & (mode == 0)

    def bytes_of(a):
        return torch.from_numpy(np.ascontiguousarray(a).reshape(KINDS, -1).view(np.uint8).copy()).cuda()[kind]

    def with_codes(v, which):
        out = v.clone()
        out[which, :micro] = bytes_of(coded)[which]
        return out

    v = torch.full((P, size), 0xCD, dtype=torch.uint8, device="cuda")
    v[:, :2 * n] = torch.where(bad[:, None], bytes_of(wrong), bytes_of(x))
    v = with_codes(v, mode == 3)                         # pages that are microscaled already
    demoted = (mode == 0) & ~bad
    want_v, want_m = with_codes(v, demoted), torch.where(demoted, 3, mode).to(torch.uint8)
    ids = torch.randperm(P, generator=torch.Generator().manual_seed(hkv)).to(torch.int32).cuda()
    m = mode.clone()
    ctx = ekv_lib.Context(hkv, hkv, d, 1)
    ekv_lib.ekv_demote_pages_micro(ctx.handle, v, size, P, ids, P, m)
    torch.cuda.synchronize()
    found = ctx.error()
    assert found == ((ekv_lib.EKV_ERR_DEVICE_CHECK, ekv_lib.EKV_DETAIL_NONFINITE_PAGE) if bool(bad.any()) else (0, 0))
    assert torch.equal(m, want_m) and torch.equal(v, want_v)

    ekv_lib.ekv_expand_pages_micro(ctx.handle, v, size, P, ids, P, m)
    torch.cuda.synchronize()
    assert ctx.error() == (0, 0)
    want_v[:, :2 * n] = torch.where((want_m == 3)[:, None], bytes_of(back), want_v[:, :2 * n])
    assert torch.equal(m, torch.where(want_m == 3, 0, want_m).to(torch.uint8)) and torch.equal(v, want_v)
    ctx.close()
