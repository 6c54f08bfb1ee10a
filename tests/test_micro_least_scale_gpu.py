"""The microscaled form at its least scale, 2^-24: codes .5 and 1.5, which the library's own writers never
make there, are rounded to fp16; and the form's largest relative errors."""

import numpy as np
import pytest

from oracle import micro as om


def test_the_largest_errors_of_a_block():
    """A fifth of the block's maximum (5 becomes 4), and a quarter where the block saturates."""
    for a, share in ((5.0, 0.2), (5.0 * 2.0 ** -24, 0.2), (65504.0, 1 - 49152 / 65504)):
        x = np.zeros((1, 32))
        x[0, 3] = a
        c, k = om.encode_rows(x)
        got = om.VALUES[c[0, 3] & 7] * 2.0 ** float(k[0, 0])
        assert abs(got - a) / a == pytest.approx(share, abs=1e-12)
    x = np.random.default_rng(130).standard_normal((4000, 32)).astype(np.float16).astype(np.float64)
    c, k = om.encode_rows(x)
    got = np.where(c & 8, -1, 1) * om.VALUES[c & 7] * 2.0 ** k.astype(np.float64)
    assert (np.abs(got - x).max(1) <= np.abs(x).max(1) / 5).all()


def test_fp16_values_need_no_half_codes_at_the_least_scale():
    x = np.arange(0, 7)[:, None] * 2.0 ** -24 * np.ones((1, 32))
    c, k = om.encode_rows(x)
    assert (k == -24).all() and not np.isin(c & 7, (1, 3)).any()


@pytest.mark.gpu
def test_half_codes_at_the_least_scale_round(ekv_lib):
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from _extend import make_case, run_extend, to_device
    v = torch.zeros((1, 2 * 16 * 64), dtype=torch.uint8, device="cuda")
    v[0, :16 * 32] = 0x31 | 0x80                         # codes .5 (low) and -1.5
    v[0, 16 * 32:16 * 34] = 103
    case = make_case([16], 1, 1, 64, "micro", 0, 131)
    d = to_device(case)
    d.v_pages[int(case.block_table[0, 0]), :16 * 34] = v[0, :16 * 34]
    m, ids = torch.full((1,), 3, dtype=torch.uint8, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    ctx = ekv_lib.Context(1, 1, 64, 1)
    ekv_lib.ekv_expand_pages_micro(ctx.handle, v, v.shape[1], 1, ids, 1, m)
    got = v.view(torch.float16).view(16, 64)
    assert torch.all(got[:, 0::2] == 0) and torch.all(got[:, 1::2] == -2.0 ** -23)
    q = torch.zeros((1, 1, 64), dtype=torch.float16, device="cuda")
    out, _ = run_extend(ekv_lib, ctx, d, q, torch.tensor([0, 1], dtype=torch.int32, device="cuda"), 1)
    assert torch.all(out[0, 0, 0::2] == 0) and torch.all(out[0, 0, 1::2] == -2.0 ** -23)
    assert ctx.error() == (0, 0)
