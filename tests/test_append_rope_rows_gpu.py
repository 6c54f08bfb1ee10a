"""ekv_append_kv_rope with more rows announced than the sequences have, as a captured step of a
padded batch has: k_new, v_new and q end with the last sequence."""

import numpy as np
import pytest

from _extend import cu_of, make_case, to_device
from test_append_rope_gpu import call, check, rope_table

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch_cuda():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return torch


@pytest.mark.parametrize("total", [0, 1, 7, 4096, 1 << 20])
@pytest.mark.parametrize("new", [[1, 1, 1], [3, 0, 20], [0, 0, 0], [300, 2, 1]])
def test_tensors_that_end_with_the_last_sequence(ekv_lib, torch_cuda, new, total):
    """`total` rows more are announced than there are; only q_out's rows up to cu_q[batch] are written."""
    torch = torch_cuda
    lens = np.array([400, 2, 30], np.int32)
    case = make_case(lens, 8, 2, 128, "all", 1, 90)
    cu, T = cu_of(new), sum(new)
    rng = np.random.default_rng(91)
    q, k, v = (rng.standard_normal((T, h, 128)).astype(np.float16) for h in (8, 2, 2))
    rope = rope_table(400, 128)
    dev = to_device(case)
    dq, dk, dv = (torch.zeros((max(1, T), h, 128), dtype=torch.float16, device="cuda") for h in (8, 2, 2))
    for x, y in ((dq, q), (dk, k), (dv, v)):
        x[:T] = torch.from_numpy(y).cuda()
    qo = torch.full((T + 3, 8, 128), 5.0, dtype=torch.float16, device="cuda")
    ctx = ekv_lib.Context(8, 2, 128, 3)
    call(ekv_lib, ctx, dev, dq, dk, dv, torch.from_numpy(rope).cuda(), 128, 0, qo, dev.seq_lens, torch.from_numpy(cu).cuda(), 3,
         T + total)
    torch.cuda.synchronize()
    assert ctx.error() == (0, 0)
    assert torch.all(qo[T:] == 5.0)
    if T:
        check(case, rope, 0, 128, q, k, v, lens, cu, qo.cpu().numpy(), dev.k_pages.cpu().numpy(), dev.v_pages.cpu().numpy())
    else:
        assert np.array_equal(dev.k_pages.cpu().numpy().view(np.uint16), case.k_pages.view(np.uint16))
        assert np.array_equal(dev.v_pages.cpu().numpy(), case.v_pages)
    ctx.close()
