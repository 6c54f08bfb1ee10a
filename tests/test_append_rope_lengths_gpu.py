"""ekv_append_kv_rope with cu_q arrays that are not what the call asks for: reported, nothing written
for the sequences that fail, nothing touched outside the tensors."""

import numpy as np
import pytest

from _extend import make_case, to_device
from test_append_rope_gpu import call, rope_table

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch_cuda():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return torch


def run(ekv, torch, cu, lens, total, table_rows):
    """Error word, and which rows of q_out and pages of K were written."""
    case = make_case([40] * table_rows, 4, 2, 64, "e4m3", 0, 97)
    d = to_device(case)
    q, k, v = (torch.ones((total, h, 64), dtype=torch.float16, device="cuda") for h in (4, 2, 2))
    qo = torch.full_like(q, 7.0)
    before = d.k_pages.view(torch.int16).clone()
    ctx = ekv.Context(4, 2, 64, table_rows)
    call(ekv, ctx, d, q, k, v, torch.from_numpy(rope_table(64, 64)).cuda(), 64, 0, qo,
         torch.tensor(lens, dtype=torch.int32, device="cuda"), torch.tensor(cu, dtype=torch.int32, device="cuda"), len(lens), total)
    torch.cuda.synchronize()
    err = ctx.error()
    pages = (d.k_pages.view(torch.int16) != before).flatten(1).any(1).nonzero().flatten().tolist()
    ctx.close()
    return err, (qo != 7).flatten(1).any(1).cpu().numpy(), {int(p) for p in pages}, case.block_table


def test_a_first_row_below_zero(ekv_lib, torch_cuda):
    """cu_q[b] far below 0: the number of new tokens passes 32 bits, and the first would stand before position 0."""
    for low in (-2 ** 31 + 8, -2 ** 31, -5):
        err, rows, pages, _ = run(ekv_lib, torch_cuda, [0, low, 8], [40, 40 if low == -5 else 3], 8, 2)
        assert err == (ekv_lib.EKV_ERR_DEVICE_CHECK, ekv_lib.EKV_DETAIL_SEQ_LEN)
        assert not rows.any() and not pages


@pytest.mark.parametrize("batch,at", [(3, 1), (3, 2), (300, 277), (2000, 1999)])
def test_fewer_than_no_new_tokens(ekv_lib, torch_cuda, batch, at):
    """No row belongs to such a sequence; the others are written."""
    new = [1] * batch
    new[at] = -1
    cu = np.cumsum([0] + new).tolist()
    err, rows, pages, table = run(ekv_lib, torch_cuda, cu, [40] * batch, batch, batch)
    assert err == (ekv_lib.EKV_ERR_DEVICE_CHECK, ekv_lib.EKV_DETAIL_SEQ_LEN)
    assert rows[:at - 1].all() and not rows[cu[-1]:].any()
    assert int(table[at, 2]) not in pages and {int(p) for p in table[:at - 1, 2]} <= pages
    new[at] = 0                                          # none at all is no error
    err, rows, pages, _ = run(ekv_lib, torch_cuda, np.cumsum([0] + new).tolist(), [40] * batch, batch, batch)
    assert err == (0, 0) and rows[:batch - 1].all() and len(pages) == batch - 1
