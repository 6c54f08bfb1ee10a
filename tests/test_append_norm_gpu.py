"""ekv_append_kv_norm_rope with given scales: normalised and rotated queries and keys within their rounding, value bytes bit for
bit, over page forms, pair styles, strides, weights and ragged batches; refusals and device checks."""

import numpy as np
import pytest

from _extend import cu_of, make_case, to_device
from _prompt import check_write, rope_table, write

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch_cuda():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return torch


def weights(rng, d, which):
    return [(1 + 0.5 * rng.standard_normal(d)).astype(np.float16) if x in which else None for x in "qk"]


def gpu(torch, x):
    return None if x is None else torch.from_numpy(np.ascontiguousarray(x)).cuda()


@pytest.mark.parametrize("fmt,sm", [("fp16", 0), ("e4m3", 0), ("e4m3", 1), ("all", 1)])
@pytest.mark.parametrize("hq,hkv,d,dim,style,which", [(8, 2, 128, 128, 0, "qk"), (4, 4, 64, 32, 0, "qk"), (32, 8, 128, 64, 1, "qk"),
                                                      (5, 1, 64, 64, 1, "k"), (7, 1, 128, 16, 0, "q"), (6, 2, 64, 0, 0, "qk"),
                                                      (8, 8, 128, 128, 0, "")])
def test_ragged_batches(ekv_lib, torch_cuda, fmt, sm, hq, hkv, d, dim, style, which):
    torch = torch_cuda
    lens, new = np.array([40, 17, 1, 200, 33], np.int32), [7, 1, 1, 70, 0]
    case = make_case(lens, hq, hkv, d, fmt, sm, 30, pool_pages=30, stride_pad=16)
    cu, T = cu_of(new), sum(new)
    rng = np.random.default_rng(31)
    rows = (rng.standard_normal((T + 3, hq + 2 * hkv, d)) * np.exp2(rng.integers(-6, 7, (T + 3, 1, 1)))).astype(np.float16)
    qw, kw = weights(rng, d, which)
    rope = rope_table(200, dim)
    dev, x = to_device(case), torch.from_numpy(rows).cuda()
    q, k, v = x.split((hq, hkv, hkv), 1)                 # slices of one projection's rows
    qo = torch.full((T + 3, hq, d), float("nan"), dtype=torch.float16, device="cuda")
    ko = torch.full((T + 3, hkv, d), float("nan"), dtype=torch.float16, device="cuda")
    ctx = ekv_lib.Context(hq, hkv, d, 5)
    write(ekv_lib, ctx, dev, q, k, v, gpu(torch, rope) if dim else None, dim, style, qo, dev.seq_lens, gpu(torch, cu), 5, T + 3,
          q_weight=gpu(torch, qw), k_weight=gpu(torch, kw), norm_eps=1e-3, k_out=ko)
    torch.cuda.synchronize()
    assert ctx.error() == (0, 0)
    assert torch.isnan(qo[T:]).all() and torch.isnan(ko[T:]).all()   # rows behind the last sequence
    check_write(case, rope, style, rows[:, :hq], rows[:, hq:hq + hkv], rows[:, hq + hkv:], qw, kw, 1e-3, lens, cu, 0,
                qo.cpu().numpy(), ko.cpu().numpy(), dev)


@pytest.mark.parametrize("batch,n", [(1, 1), (33, 1), (300, 2), (2, 700), (1, 3000)])
def test_sizes_and_in_place(ekv_lib, torch_cuda, batch, n):
    """q_out is q and k_out is k itself; the batch is larger than the context's; from one token to thousands."""
    torch = torch_cuda
    lens, new = np.full(batch, n + 5, np.int32), [n] * batch
    case = make_case(lens, 8, 2, 64, "e4m3", 1, 32)
    cu, T = cu_of(new), n * batch
    rng = np.random.default_rng(33)
    q, k, v = (rng.standard_normal((T, h, 64)).astype(np.float16) for h in (8, 2, 2))
    qw, kw = weights(rng, 64, "qk")
    rope = rope_table(n + 5, 64)
    dev, dq, dk = to_device(case), gpu(torch, q), gpu(torch, k)
    ctx = ekv_lib.Context(8, 2, 64, 1)
    write(ekv_lib, ctx, dev, dq, dk, gpu(torch, v), gpu(torch, rope), 64, 0, dq, dev.seq_lens, gpu(torch, cu), batch, T,
          q_weight=gpu(torch, qw), k_weight=gpu(torch, kw), k_out=dk)
    torch.cuda.synchronize()
    assert ctx.error() == (0, 0)
    check_write(case, rope, 0, q, k, v, qw, kw, 1e-6, lens, cu, 0, dq.cpu().numpy(), dk.cpu().numpy(), dev)


@pytest.mark.parametrize("value", [0.0, 65504.0, 6e-8, np.inf, np.nan])
def test_odd_values(ekv_lib, torch_cuda, value):
    """Rows of zeros, of the largest and least values; one that is not finite makes its row NaN and no other."""
    torch = torch_cuda
    lens = np.array([3], np.int32)
    case = make_case(lens, 2, 1, 128, "fp16", 0, 34)
    x = np.ones((3, 2, 128), np.float16)
    if np.isfinite(value):
        x[1] = value
    else:
        x[1, 0, 7] = value
    k = x[:, :1]
    w = np.full(128, 2, np.float16)
    dev = to_device(case)
    qo = torch.empty((3, 2, 128), dtype=torch.float16, device="cuda")
    ctx = ekv_lib.Context(2, 1, 128, 1)
    write(ekv_lib, ctx, dev, gpu(torch, x), gpu(torch, k), gpu(torch, k), None, 0, 0, qo, dev.seq_lens,
          torch.tensor([0, 3], dtype=torch.int32, device="cuda"), 1, 3, q_weight=gpu(torch, w), k_weight=gpu(torch, w), norm_eps=1e-12)
    assert ctx.error() == (0, 0)
    got = qo.cpu().numpy().astype(np.float64)
    if np.isfinite(value):
        ref = x.astype(np.float64) / np.sqrt(x.astype(np.float64) ** 2 + 1e-12) * 2
        assert np.all(np.abs(got - ref) <= 2.0 ** -10 * np.abs(ref) + 2.0 ** -24)
    else:
        assert np.isnan(got[1, 0]).any() and np.all(got[[0, 2]] == 2) and np.all(got[1, 1] == 2)


def test_device_checks_write_nothing(ekv_lib, torch_cuda):
    torch = torch_cuda
    lens = np.array([40, 40, 40], np.int32)
    case = make_case(lens, 4, 2, 64, "all", 1, 35)
    case.page_mode[case.block_table[1]] = 1
    case.v_scales[:] = 0.02
    ctx = ekv_lib.Context(4, 2, 64, 3)
    cu = torch.tensor([0, 2, 4, 6], dtype=torch.int32, device="cuda")
    q, k, v = (torch.randn((6, h, 64), dtype=torch.float16, device="cuda") for h in (4, 2, 2))
    rope = gpu(torch, rope_table(64, 64))
    w = torch.ones(64, dtype=torch.float16, device="cuda")
    page = int(case.block_table[1, 2])

    def run(change, **kw):
        d = to_device(case)
        change(d)
        before = d.k_pages.clone(), d.v_pages.clone()
        qo, ko = torch.full_like(q, 7.0), torch.full_like(k, 7.0)
        write(ekv_lib, ctx, d, q, k, v, rope, 64, 0, qo, d.seq_lens, kw.pop("cu_q", cu), 3, 6, q_weight=w, k_weight=w, k_out=ko, **kw)
        err = ctx.error()
        changed = (d.k_pages.view(torch.int16) != before[0].view(torch.int16)).flatten(1).any(1), (d.v_pages != before[1]).any(1)
        return err, bool(changed[0][page]), bool(changed[1][page]), qo, ko

    check_ = ekv_lib.EKV_ERR_DEVICE_CHECK
    for grow in (0, 1):
        assert run(lambda d: None, grow_scales=grow)[:3] == ((0, 0), True, True)
        for bad in (1, 49):
            err, kc, vc, qo, ko = run(lambda d: d.seq_lens.__setitem__(1, bad), grow_scales=grow)
            assert err == (check_, ekv_lib.EKV_DETAIL_SEQ_LEN) and not kc and not vc and torch.all(qo[2:4] == 7) and torch.all(ko[2:4] == 7)
        err, kc, vc, qo, ko = run(lambda d: None, rope_len=39, grow_scales=grow)   # the last token stands behind the table
        assert err == (check_, ekv_lib.EKV_DETAIL_SEQ_LEN) and torch.all(qo[1] == 7) and not torch.any(qo[0] == 7)
        for bad in (-3, case.num_pages):
            err, kc, vc, qo, ko = run(lambda d: d.block_table.__setitem__((1, 2), bad), grow_scales=grow)
            assert err == (check_, ekv_lib.EKV_DETAIL_PAGE_ID) and not kc and not vc and not torch.any(qo == 7) and not torch.any(ko == 7)
        err, kc, vc, _, ko = run(lambda d: d.page_mode.__setitem__(page, 200), grow_scales=grow)
        assert err == (check_, ekv_lib.EKV_DETAIL_PAGE_MODE) and not kc and not vc and not torch.any(ko == 7)
        for bad in (0.0, float("nan"), float("inf"), -1.0):
            err, kc, vc, _, _ = run(lambda d: d.v_scales.__setitem__(page, bad), grow_scales=grow)
            assert err == (check_, ekv_lib.EKV_DETAIL_SCALE) and kc and not vc
        err = run(lambda d: None, grow_scales=grow, cu_q=torch.tensor([0, 4, 2, 6], dtype=torch.int32, device="cuda"))[0]
        assert err == (check_, ekv_lib.EKV_DETAIL_SEQ_LEN)


def test_refusals(ekv_lib, torch_cuda):
    torch = torch_cuda
    case = make_case(np.array([40], np.int32), 4, 2, 64, "e4m3", 1, 36)
    d = to_device(case)
    ctx = ekv_lib.Context(4, 2, 64, 1)
    q, k, v = (torch.zeros((2, h, 64), dtype=torch.float16, device="cuda") for h in (4, 2, 2))
    cu = torch.tensor([0, 2], dtype=torch.int32, device="cuda")
    rope = gpu(torch, rope_table(64, 64))
    w = torch.ones(72, dtype=torch.float16, device="cuda")
    for kw in (dict(ctx=None), dict(k_new=None), dict(v_new=None), dict(q_out=None), dict(rope_table=None), dict(rope_len=0),
               dict(rope_dim=8), dict(rope_dim=80), dict(rope_style=2), dict(q_stride=248), dict(k_stride=124), dict(v_stride=129),
               dict(k_pages=None), dict(cu_q=None), dict(seq_lens=None), dict(batch=-1), dict(total_q=-1), dict(uniform_mode=0),
               dict(v_scales=None), dict(v_page_stride_bytes=2052), dict(q=q.data_ptr() + 2), dict(q_weight=w.data_ptr() + 2),
               dict(k_weight=w.data_ptr() + 8), dict(k_out=k.data_ptr() + 2), dict(norm_eps=0.0), dict(norm_eps=-1.0),
               dict(norm_eps=float("nan")), dict(norm_eps=float("inf")), dict(grow_scales=2), dict(grow_scales=1, scale_mode=0),
               dict(grow_scales=1, v_scales=None)):
        a = dict(ctx=ctx.handle, q=q, k_new=k, v_new=v, q_stride=256, k_stride=128, v_stride=128, q_weight=w, k_weight=None, norm_eps=1e-6,
                 rope_table=rope, rope_len=64, rope_dim=64, rope_style=0, q_out=q, k_out=None, k_pages=d.k_pages, v_pages=d.v_pages,
                 v_page_stride_bytes=d.v_page_stride, num_pages=d.num_pages, v_scales=d.v_scales, scale_mode=1, grow_scales=0,
                 page_mode=None, uniform_mode=1, block_table=d.block_table, block_table_stride=int(d.block_table.shape[1]),
                 seq_lens=d.seq_lens, cu_q=cu, batch=1, total_q=2)
        with pytest.raises(ekv_lib.EkvError) as e:
            ekv_lib.ekv_append_kv_norm_rope(**{**a, **kw})
        assert e.value.status == ekv_lib.EKV_ERR_INVALID_ARG, kw
    write(ekv_lib, ctx, d, q, k, v, rope, 64, 0, q, d.seq_lens, cu, 0, 2)
    write(ekv_lib, ctx, d, q, k, v, rope, 64, 0, q, d.seq_lens, cu, 1, 0)
    write(ekv_lib, ctx, d, q, k, v, rope, 64, 0, q, d.seq_lens, cu, 1, 2, norm_eps=0.0)   # (no weights)
    assert ctx.error() == (0, 0)
