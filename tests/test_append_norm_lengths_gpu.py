"""ekv_append_kv_norm_rope with cu_q arrays that are not what the call asks for: reported, nothing written for the sequences
that fail, in any of the call's outputs; the others are written as the oracle has them."""

import numpy as np
import pytest

from _extend import make_case, to_device
from _prompt import check_write, rope_table, write

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch_cuda():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return torch


def bits(x):
    return x.cpu().numpy().view(np.uint16)


def run(ekv, torch, case, rope, hq, hkv, d, lens, cu, total, rows, grow, **kw):
    dev, x = to_device(case), torch.from_numpy(rows).cuda()
    qo, ko = (torch.full((total, h, d), 7.0, dtype=torch.float16, device="cuda") for h in (hq, hkv))
    w = torch.ones(d, dtype=torch.float16, device="cuda")
    q, k, v = x.split((hq, hkv, hkv), 1)
    ctx = ekv.Context(hq, hkv, d, len(lens))
    write(ekv, ctx, dev, q, k, v, torch.from_numpy(rope).cuda(), rope.shape[1], 0, qo,
          torch.tensor(lens, dtype=torch.int32, device="cuda"), torch.tensor(cu, dtype=torch.int32, device="cuda"), len(lens), total,
          q_weight=w, k_weight=w, k_out=ko, grow_scales=grow, **kw)
    torch.cuda.synchronize()
    return ctx.error(), dev, qo, ko, w.cpu().numpy()


@pytest.mark.parametrize("grow", [0, 1])
@pytest.mark.parametrize("low", [-1, -5, -2 ** 31 + 4, -2 ** 31 + 100, -2 ** 31])
@pytest.mark.parametrize("batch", [1, 4, 40])
def test_a_first_row_below_zero(ekv_lib, torch_cuda, grow, low, batch):
    """The first sequence fails; the others are written as a call writes them that does not have it."""
    torch = torch_cuda
    hq, hkv, d, n = 4, 2, 64, 3
    lens = [20] * batch
    case = make_case(np.array(lens), hq, hkv, d, "e4m3", 1, 310)
    rows = np.random.default_rng(311).standard_normal((n * batch, hq + 2 * hkv, d)).astype(np.float16)
    rope = rope_table(20, d)
    cu = np.arange(0, n * batch + 1, n, dtype=np.int32)
    bad = cu.copy()
    bad[0] = low
    err, dev, qo, ko, w = run(ekv_lib, torch, case, rope, hq, hkv, d, lens, bad, n * batch, rows, grow)
    assert err == (ekv_lib.EKV_ERR_DEVICE_CHECK, ekv_lib.EKV_DETAIL_SEQ_LEN)
    assert torch.all(qo[:n] == 7) and torch.all(ko[:n] == 7)
    if batch == 1:
        assert np.array_equal(bits(dev.k_pages), case.k_pages.view(np.uint16))
        assert np.array_equal(dev.v_pages.cpu().numpy(), case.v_pages) and np.array_equal(dev.v_scales.cpu().numpy(), case.v_scales)
        return
    case.block_table = case.block_table[1:]
    r = rows[n:]
    check_write(case, rope, 0, r[:, :hq], r[:, hq:hq + hkv], r[:, hq + hkv:], w, w, 1e-6, lens[1:], cu[1:] - n, grow,
                qo[n:].cpu().numpy(), ko[n:].cpu().numpy(), dev)


@pytest.mark.parametrize("grow", [0, 1])
def test_arrays_of_anything_are_reported(ekv_lib, torch_cuda, grow):
    """Ends of 32 bits, falling and random arrays: an error, or rows inside the call's outputs alone."""
    torch = torch_cuda
    hq, hkv, d, total = 4, 2, 64, 12
    rng = np.random.default_rng(312)
    case = make_case(np.full(6, 40), hq, hkv, d, "e4m3", 1, 313)
    rows = rng.standard_normal((total, hq + 2 * hkv, d)).astype(np.float16)
    rope = rope_table(64, d)
    ends = np.array([-2 ** 31, -2 ** 31 + 9, -9, 0, 9, 2 ** 31 - 9, 2 ** 31 - 1])
    used = {int(p) for p in case.block_table.flatten()}
    for turn in range(40):
        cu = (rng.choice(ends, 7) if turn % 2 else rng.integers(-2 ** 31, 2 ** 31, 7)).astype(np.int32)
        cu[-1] = abs(int(cu[-1])) if cu[-1] > -2 ** 31 else 5
        lens = rng.choice([-2 ** 31, -1, 0, 3, 40, 2 ** 31 - 1], 6)
        err, dev, qo, ko, _ = run(ekv_lib, torch, case, rope, hq, hkv, d, lens, cu, total, rows, grow)
        if np.any(np.diff(cu.astype(np.int64)) < 0):
            assert err == (ekv_lib.EKV_ERR_DEVICE_CHECK, ekv_lib.EKV_DETAIL_SEQ_LEN), (cu, lens)
        changed = np.any(bits(dev.k_pages) != case.k_pages.view(np.uint16), (1, 2, 3)).nonzero()[0]
        assert {int(p) for p in changed} <= used


@pytest.mark.parametrize("grow", [0, 1])
@pytest.mark.parametrize("rope_len", [1, 16, 33, 39, 40, 47])
@pytest.mark.parametrize("hkv,d", [(2, 64), (8, 128)])
def test_positions_behind_the_table(ekv_lib, torch_cuda, grow, rope_len, hkv, d):
    """Tokens at such positions are reported and leave everything as it was; what stands before them is written as a call writes it
    that does not have them. Their values are large: counted in, they would grow every scale."""
    torch = torch_cuda
    hq, lens, new = 2 * hkv, [40, 48, 3, 40, 64], [2, 48, 3, 25, 30]
    cu = np.cumsum([0] + new)
    case = make_case(np.array(lens), hq, hkv, d, "all", 1, 314, pool_pages=30)
    at = np.concatenate([np.arange(n - m, n) for n, m in zip(lens, new)])
    rows = np.random.default_rng(315).standard_normal((sum(new), hq + 2 * hkv, d)).astype(np.float16)
    rows[at >= rope_len] *= 200
    rope = rope_table(64, d)
    err, dev, qo, ko, w = run(ekv_lib, torch, case, rope, hq, hkv, d, lens, cu.tolist(), len(rows), rows, grow, rope_len=rope_len)
    assert err == (ekv_lib.EKV_ERR_DEVICE_CHECK, ekv_lib.EKV_DETAIL_SEQ_LEN)
    good = torch.from_numpy(at < rope_len).cuda()
    assert torch.all(qo[~good] == 7) and torch.all(ko[~good] == 7)
    kept = [int(np.sum(at[a:b] < rope_len)) for a, b in zip(cu, cu[1:])]
    r = rows[at < rope_len]
    check_write(case, rope, 0, r[:, :hq], r[:, hq:hq + hkv], r[:, hq + hkv:], w, w, 1e-6,
                np.array([n - m + k for n, m, k in zip(lens, new, kept)]), np.cumsum([0] + kept), grow, qo[good].cpu().numpy(), ko[good].cpu().numpy(), dev)
