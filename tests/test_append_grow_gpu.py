"""ekv_append_kv_norm_rope with grow_scales: E4M3 codes and scales bit for bit against the oracle, over pages begun, continued
and whole, every page form beside them, odd values and scales; and the cache read back."""

import numpy as np
import pytest

from mixed_precision_paged_gb300 import workloads as wl
from oracle import decode as od
from oracle import demote

from _extend import cu_of, make_case, to_device
from _prompt import check_write, rope_table, write

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch_cuda():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return torch


def gpu(torch, x):
    return None if x is None else torch.from_numpy(np.ascontiguousarray(x)).cuda()


def run(ekv, torch, case, ctx, rows, hq, hkv, lens, new, rope_dim=64):
    """One call on slices of `rows`; checked against the oracle."""
    cu, T = cu_of(new), int(sum(new))
    rope = rope_table(int(max(lens)), rope_dim)
    dev, x = to_device(case), gpu(torch, rows)
    q, k, v = x.split((hq, hkv, hkv), 1)
    qo, ko = (torch.full(y.shape, float("nan"), dtype=torch.float16, device="cuda") for y in (q, k))
    w = torch.ones(rows.shape[2], dtype=torch.float16, device="cuda")
    write(ekv, ctx, dev, q, k, v, gpu(torch, rope) if rope_dim else None, rope_dim, 0, qo, gpu(torch, np.asarray(lens, np.int32)),
          gpu(torch, cu), len(lens), rows.shape[0], q_weight=w, k_weight=w, k_out=ko, grow_scales=1)
    torch.cuda.synchronize()
    assert ctx.error() == (0, 0)
    one = w.cpu().numpy()
    check_write(case, rope, 0, rows[:, :hq], rows[:, hq:hq + hkv], rows[:, hq + hkv:], one, one, 1e-6, lens, cu, 1,
                qo.cpu().numpy(), ko.cpu().numpy(), dev)
    assert torch.isnan(qo[T:]).all() and torch.isnan(ko[T:]).all()
    return dev


@pytest.mark.parametrize("fmt", ["e4m3", "all"])
@pytest.mark.parametrize("hq,hkv,d", [(8, 2, 128), (4, 4, 64), (5, 1, 64), (8, 8, 128)])
@pytest.mark.parametrize("size", [1.0, 40.0])
def test_ragged_batches(ekv_lib, torch_cuda, fmt, hq, hkv, d, size):
    """New rows that begin in the middle of a page, end in one, fill whole ones; `size` 40: every scale grows."""
    lens, new = np.array([40, 17, 1, 200, 33, 16, 48], np.int32), [7, 1, 1, 150, 0, 16, 31]
    case = make_case(lens, hq, hkv, d, fmt, 1, 130, pool_pages=40, stride_pad=16)
    rng = np.random.default_rng(131)
    rows = (rng.standard_normal((sum(new) + 3, hq + 2 * hkv, d)) * size).astype(np.float16)
    run(ekv_lib, torch_cuda, case, ekv_lib.Context(hq, hkv, d, 7), rows, hq, hkv, lens, new)


@pytest.mark.parametrize("batch,n,ctx_len", [(1, 1, 0), (1, 1, 15), (1, 1, 16), (40, 1, 21), (700, 3, 14), (2, 900, 7), (1, 5000, 0)])
def test_sizes(ekv_lib, torch_cuda, batch, n, ctx_len):
    """From one row an item to chunks of rows; more sequences than the context was made for."""
    lens, new = np.full(batch, n + ctx_len, np.int32), [n] * batch
    case = make_case(lens, 8, 8, 64, "e4m3", 1, 132)
    rng = np.random.default_rng(133)
    rows = (rng.standard_normal((n * batch, 24, 64)) * np.exp2(rng.integers(-3, 4, (n * batch, 1, 1)))).astype(np.float16)
    run(ekv_lib, torch_cuda, case, ekv_lib.Context(8, 8, 64, 1), rows, 8, 8, lens, new)


def test_many_empty_sequences(ekv_lib, torch_cuda):
    new = [0] * 37 + [1] + [0] * 70 + [18, 0, 2]
    lens = np.array([n + 9 for n in new], np.int32)
    case = make_case(lens, 4, 2, 64, "e4m3", 1, 134)
    rows = np.random.default_rng(135).standard_normal((sum(new), 8, 64)).astype(np.float16)
    run(ekv_lib, torch_cuda, case, ekv_lib.Context(4, 2, 64, 1), rows, 4, 2, lens, new)


@pytest.mark.parametrize("value", [0.0, -0.0, np.inf, -np.inf, np.nan, 65504.0, 6e-8])
@pytest.mark.parametrize("begun", [False, True])
def test_odd_values(ekv_lib, torch_cuda, value, begun):
    """One such value among ones, a row of it, and a page of nothing else."""
    lens = np.array([16, 16, 16], np.int32) + (3 if begun else 0)
    case = make_case(lens + 16, 2, 1, 64, "e4m3", 1, 136)
    rows = np.ones((48, 4, 64), np.float16)
    rows[3, 3, 5], rows[17, 3], rows[32:, 3] = value, value, value
    run(ekv_lib, torch_cuda, case, ekv_lib.Context(2, 1, 64, 3), rows, 2, 1, lens, [16, 16, 16], rope_dim=0)


@pytest.mark.parametrize("scale", [1.0, 2.0 ** -40, 1e-38, 1e-44, 2.9e38, 1e30, 2.0 ** 90, 1 / 448])
def test_odd_scales(ekv_lib, torch_cuda, scale):
    """Scales at the ends of fp32's range, under which the quotient takes the slow way."""
    lens = np.array([20, 9], np.int32)
    case = make_case(lens, 2, 1, 128, "e4m3", 1, 137)
    case.v_scales[:] = np.float32(scale)
    rows = np.random.default_rng(138).standard_normal((8, 4, 128)).astype(np.float16)
    run(ekv_lib, torch_cuda, case, ekv_lib.Context(2, 1, 128, 2), rows, 2, 1, lens, [4, 4], rope_dim=0)


def test_growth_of_every_code(ekv_lib, torch_cuda):
    """All 256 codes in the earlier rows, under growth by one power of two and by many."""
    lens = np.array([5], np.int32)
    for top in (900.0, 65504.0):
        case = make_case(lens, 1, 1, 64, "e4m3", 1, 139)
        p = int(case.block_table[0, 0])
        case.v_pages[p, :256] = np.arange(256)
        case.v_scales[p] = 1.0
        rows = np.zeros((1, 3, 64), np.float16)
        rows[0, 2] = np.linspace(-top, top, 64)
        run(ekv_lib, torch_cuda, case, ekv_lib.Context(1, 1, 64, 1), rows, 1, 1, lens, [1], rope_dim=0)


def test_whole_pages_are_as_demoted(ekv_lib, torch_cuda):
    torch = torch_cuda
    lens = np.array([64], np.int32)
    case = make_case(lens, 8, 2, 128, "e4m3", 1, 140)
    rows = (np.random.default_rng(141).standard_normal((64, 12, 128)) * 3).astype(np.float16)
    dev = run(ekv_lib, torch, case, ekv_lib.Context(8, 2, 128, 1), rows, 8, 2, lens, [64])
    for j in range(4):
        p, x = int(case.block_table[0, j]), rows[16 * j:16 * j + 16, 10:]
        s = demote.page_scales(x)
        assert np.array_equal(dev.v_scales[p].cpu().numpy(), s)
        assert np.array_equal(dev.v_pages[p].cpu().numpy()[: 16 * 2 * 128], demote.quantise_page(x, s).reshape(-1))


def test_a_cache_grown_token_by_token_is_read_by_decode(ekv_lib, torch_cuda):
    """40 decode steps from an empty cache whose scales were never set, under the programmatic launch, each followed
    by a decode that sees the page just written."""
    torch = torch_cuda
    hq, hkv, d, B = 8, 2, 128, 3
    case = make_case(np.full(B, 40, np.int32), hq, hkv, d, "e4m3", 1, 142)
    case.v_scales[:] = np.nan
    dev = to_device(case)
    ctx = ekv_lib.Context(hq, hkv, d, B, pdl=True)
    rng = np.random.default_rng(143)
    cu = torch.arange(B + 1, dtype=torch.int32, device="cuda")
    rope = gpu(torch, rope_table(40, d))
    w = torch.ones(d, dtype=torch.float16, device="cuda")
    for t in range(40):
        size = 2.0 ** rng.integers(-2, 3)
        x = [gpu(torch, (rng.standard_normal((B, h, d)) * size).astype(np.float16)) for h in (hq, hkv, hkv)]
        lens = torch.full((B,), t + 1, dtype=torch.int32, device="cuda")
        q = torch.empty_like(x[0])
        out, again = torch.empty_like(q), torch.empty_like(q)
        write(ekv_lib, ctx, dev, *x, rope, d, 0, q, lens, cu, B, B, q_weight=w, k_weight=w, grow_scales=1)
        step = wl.DecodeCase(**{**dev.__dict__, "q": q, "seq_lens": lens})
        ctx.decode(step, out)
        torch.cuda.synchronize()
        ctx.decode(step, again)
        assert ctx.error() == (0, 0) and torch.equal(out, again), t
    ref, _ = od.paged_decode(q.cpu().numpy(), dev.k_pages.cpu().numpy(), dev.v_pages.cpu().numpy(), dev.v_scales.cpu().numpy(), 1, None,
                             1, case.block_table, lens.cpu().numpy())
    # the result's rounding and the weights', 2^-11 of values up to four times the largest result each, and the decode's fp32 steps
    assert np.abs(out.float().cpu().numpy() - ref).max() <= 2.0 ** -8 * np.abs(ref).max()
