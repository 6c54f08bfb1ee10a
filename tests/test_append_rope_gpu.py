"""ekv_append_kv_rope against the oracle: rotated queries and keys within their rounding, value
bytes bit for bit, over page forms, pair styles, strides and ragged batches; refusals."""

import numpy as np
import pytest

from oracle import extend as oe

from _extend import cu_of, make_case, to_device

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch_cuda():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return torch


def rope_table(n, dim, seed=0):
    pos = np.arange(n)[:, None] * 10000.0 ** (-np.arange(dim // 2) / max(1, dim // 2))
    return np.concatenate([np.cos(pos), np.sin(pos)], 1).astype(np.float32)


def call(ekv, owner, d, queries, k, v, rope, dim, style, qo, lens, cu, nseq, total, **kw):
    a = dict(ctx=owner.handle, q=queries, k_new=k, v_new=v, q_stride=queries.stride(0) if queries is not None else 0, k_stride=k.stride(0),
             v_stride=v.stride(0), rope_table=rope, rope_len=rope.shape[0] if rope is not None else 0, rope_dim=dim,
             rope_style=style, q_out=qo, k_pages=d.k_pages, v_pages=d.v_pages, v_page_stride_bytes=d.v_page_stride,
             num_pages=d.num_pages, v_scales=d.v_scales, scale_mode=d.scale_mode, page_mode=d.page_mode,
             uniform_mode=d.uniform_mode, block_table=d.block_table, block_table_stride=int(d.block_table.shape[1]),
             seq_lens=lens, cu_q=cu, batch=nseq, total_q=total)
    a.update(kw)
    ekv.ekv_append_kv_rope(**a)


def check(case, rope, style, dim, q, k, v, lens, cu, qo, kp, vp):
    """Rotated values: half an fp16 step (2^-11 relative, 2^-25 where subnormal) and three fp32
    roundings of the products and their sum; bytes of V and untouched rows exactly."""
    T = int(cu[-1])
    rq, rk, rv = oe.append(q, k, v, rope, style, case.k_pages, case.v_pages, case.v_scales, case.scale_mode, case.page_mode,
                           case.uniform_mode, case.block_table, lens, cu)
    def near(got, ref, size):
        return np.all(np.abs(got.astype(np.float64) - ref) <= 2.0 ** -11 * np.abs(ref) + 2.0 ** -25 + 3 * 2.0 ** -24 * size)
    assert near(qo[:T], rq[:T], 2 * np.abs(q[:T].astype(np.float64)).max())
    assert np.array_equal(qo[:T, :, dim:], q[:T, :, dim:])
    written = np.zeros(kp.shape[:2], bool)
    for i, b, t in oe.places(lens, cu):
        written[case.block_table[b][t // 16], t % 16] = True
    assert near(kp[written], rk[written], 2 * np.abs(k.astype(np.float64)).max())
    assert np.array_equal(kp[~written].view(np.uint16), case.k_pages[~written].view(np.uint16))
    assert np.array_equal(vp, rv)


@pytest.mark.parametrize("fmt,sm", [("fp16", 0), ("e4m3", 0), ("e4m3", 1), ("base", 0), ("micro", 0), ("all", 1)])
@pytest.mark.parametrize("hq,hkv,d,dim,style", [(8, 2, 128, 128, 0), (4, 4, 64, 32, 0), (32, 8, 128, 64, 1), (5, 1, 64, 64, 1),
                                                (7, 1, 128, 16, 0), (6, 2, 64, 0, 0)])
def test_ragged_batches(ekv_lib, torch_cuda, fmt, sm, hq, hkv, d, dim, style):
    torch = torch_cuda
    lens, new = np.array([40, 17, 1, 200, 33], np.int32), [7, 1, 1, 70, 0]
    case = make_case(lens, hq, hkv, d, fmt, sm, 30, pool_pages=30, stride_pad=16)
    cu, T = cu_of(new), sum(new)
    rng = np.random.default_rng(31)
    rows = (rng.standard_normal((T + 3, hq + 2 * hkv, d)) * 2).astype(np.float16)
    rope = rope_table(200, dim) if dim else np.zeros((200, 0), np.float32)
    dev, x = to_device(case), torch.from_numpy(rows).cuda()
    q, k, v = x.split((hq, hkv, hkv), 1)                 # slices of one projection's rows
    qo = torch.full((T + 3, hq, d), float("nan"), dtype=torch.float16, device="cuda")
    ctx = ekv_lib.Context(hq, hkv, d, 5)
    call(ekv_lib, ctx, dev, q, k, v, torch.from_numpy(rope).cuda() if dim else None, dim, style, qo, dev.seq_lens,
         torch.from_numpy(cu).cuda(), 5, T + 3)
    torch.cuda.synchronize()
    assert ctx.error() == (0, 0)
    assert torch.isnan(qo[T:]).all()                     # rows behind the last sequence
    check(case, rope, style, dim, rows[:, :hq], rows[:, hq:hq + hkv], rows[:, hq + hkv:], lens, cu, qo.cpu().numpy(),
          dev.k_pages.cpu().numpy(), dev.v_pages.cpu().numpy())


@pytest.mark.parametrize("batch,n", [(1, 1), (33, 1), (300, 2), (2, 700), (1, 3000)])
def test_sizes_and_in_place(ekv_lib, torch_cuda, batch, n):
    """q_out is q itself; the batch is larger than the context's; from one token to thousands."""
    torch = torch_cuda
    lens, new = np.full(batch, n + 5, np.int32), [n] * batch
    case = make_case(lens, 8, 2, 64, "e4m3", 1, 32)
    cu, T = cu_of(new), n * batch
    rng = np.random.default_rng(33)
    q, k, v = (rng.standard_normal((T, h, 64)).astype(np.float16) for h in (8, 2, 2))
    rope = rope_table(n + 5, 64)
    dev, dq = to_device(case), torch.from_numpy(q).cuda()
    ctx = ekv_lib.Context(8, 2, 64, 1)
    call(ekv_lib, ctx, dev, dq, torch.from_numpy(k).cuda(), torch.from_numpy(v).cuda(), torch.from_numpy(rope).cuda(), 64, 0,
         dq, dev.seq_lens, torch.from_numpy(cu).cuda(), batch, T)
    torch.cuda.synchronize()
    assert ctx.error() == (0, 0)
    check(case, rope, 0, 64, q, k, v, lens, cu, dq.cpu().numpy(), dev.k_pages.cpu().numpy(), dev.v_pages.cpu().numpy())


@pytest.mark.parametrize("value", [np.inf, -np.inf, np.nan, 65504.0, -0.0, 6e-8])
def test_odd_values(ekv_lib, torch_cuda, value):
    torch = torch_cuda
    lens = np.array([3], np.int32)
    for fmt in ("fp16", "micro", "base", "e4m3"):
        case = make_case(lens, 2, 1, 64, fmt, 0, 34)
        v = np.ones((3, 1, 64), np.float16)
        v[1, 0, 5], v[2, 0, 40:] = value, value
        k = np.zeros((3, 1, 64), np.float16)
        dev = to_device(case)
        ctx = ekv_lib.Context(2, 1, 64, 1)
        call(ekv_lib, ctx, dev, None, torch.from_numpy(k).cuda(), torch.from_numpy(v).cuda(), None, 0, 0, None, dev.seq_lens,
             torch.tensor([0, 3], dtype=torch.int32, device="cuda"), 1, 3)
        assert ctx.error() == (0, 0)
        _, _, rv = oe.append(np.zeros((3, 2, 64), np.float16), k, v, np.zeros((3, 0), np.float32), 0, case.k_pages,
                             case.v_pages, case.v_scales, 0, case.page_mode, case.uniform_mode, case.block_table, lens,
                             np.array([0, 3]))
        assert np.array_equal(dev.v_pages.cpu().numpy(), rv), fmt


def test_device_checks_write_nothing(ekv_lib, torch_cuda):
    torch = torch_cuda
    lens = np.array([40, 40, 40], np.int32)
    case = make_case(lens, 4, 2, 64, "all", 1, 35)
    case.page_mode[case.block_table[1]] = 1
    case.v_scales[:] = 0.02
    ctx = ekv_lib.Context(4, 2, 64, 3)
    cu = torch.tensor([0, 2, 4, 6], dtype=torch.int32, device="cuda")
    q, k, v = (torch.randn((6, h, 64), dtype=torch.float16, device="cuda") for h in (4, 2, 2))
    rope = torch.from_numpy(rope_table(64, 64)).cuda()

    def run(change, **kw):
        d = to_device(case)
        change(d)
        before = d.k_pages.clone(), d.v_pages.clone()
        qo = torch.full_like(q, 7.0)
        call(ekv_lib, ctx, d, q, k, v, rope, 64, 0, qo, d.seq_lens, cu, 3, 6, **kw)
        err = ctx.error()
        page = int(case.block_table[1, 2])
        changed = (d.k_pages.view(torch.int16) != before[0].view(torch.int16)).flatten(1).any(1), (d.v_pages != before[1]).any(1)
        return err, bool(changed[0][page]), bool(changed[1][page]), qo

    check_ = ekv_lib.EKV_ERR_DEVICE_CHECK
    assert run(lambda d: None)[:3] == ((0, 0), True, True)
    err, kc, vc, qo = run(lambda d: d.seq_lens.__setitem__(1, 1))
    assert err == (check_, ekv_lib.EKV_DETAIL_SEQ_LEN) and not kc and not vc and torch.all(qo[2:4] == 7)
    err, kc, vc, qo = run(lambda d: d.seq_lens.__setitem__(1, 49))
    assert err == (check_, ekv_lib.EKV_DETAIL_SEQ_LEN) and not kc and not vc and torch.all(qo[2:4] == 7)
    err, kc, vc, qo = run(lambda d: None, rope_len=39)   # the last token stands behind the table
    assert err == (check_, ekv_lib.EKV_DETAIL_SEQ_LEN) and torch.all(qo[1] == 7) and not torch.any(qo[0] == 7)
    err, kc, vc, qo = run(lambda d: d.block_table.__setitem__((1, 2), -3))
    assert err == (check_, ekv_lib.EKV_DETAIL_PAGE_ID) and not kc and not vc and not torch.any(qo == 7)
    err, kc, vc, _ = run(lambda d: d.page_mode.__setitem__(int(case.block_table[1, 2]), 200))
    assert err == (check_, ekv_lib.EKV_DETAIL_PAGE_MODE) and not kc and not vc
    err, kc, vc, _ = run(lambda d: d.v_scales.__setitem__(int(case.block_table[1, 2]), 0.0))
    assert err == (check_, ekv_lib.EKV_DETAIL_SCALE) and kc and not vc


def test_refusals(ekv_lib, torch_cuda):
    torch = torch_cuda
    case = make_case(np.array([40], np.int32), 4, 2, 64, "e4m3", 0, 36)
    d = to_device(case)
    ctx = ekv_lib.Context(4, 2, 64, 1)
    q, k, v = (torch.zeros((2, h, 64), dtype=torch.float16, device="cuda") for h in (4, 2, 2))
    cu = torch.tensor([0, 2], dtype=torch.int32, device="cuda")
    rope = torch.from_numpy(rope_table(64, 64)).cuda()
    for kw in (dict(ctx=None), dict(k_new=None), dict(v_new=None), dict(q_out=None), dict(rope_table=None), dict(rope_len=0),
               dict(rope_dim=8), dict(rope_dim=80), dict(rope_dim=-16), dict(rope_style=2), dict(q_stride=248),
               dict(k_stride=124), dict(v_stride=129), dict(k_stride=64), dict(k_pages=None), dict(cu_q=None),
               dict(seq_lens=None), dict(batch=-1), dict(total_q=-1), dict(uniform_mode=0), dict(v_scales=None),
               dict(v_page_stride_bytes=2052), dict(q=q.data_ptr() + 2), dict(k_new=k.data_ptr() + 8),
               dict(rope_table=rope.data_ptr() + 4)):
        with pytest.raises(ekv_lib.EkvError) as e:
            call(ekv_lib, ctx, d, q, k, v, rope, 64, 0, q, d.seq_lens, cu, 1, 2, **kw)
        assert e.value.status == ekv_lib.EKV_ERR_INVALID_ARG, kw
    call(ekv_lib, ctx, d, q, k, v, rope, 64, 0, q, d.seq_lens, cu, 0, 2)
    call(ekv_lib, ctx, d, q, k, v, rope, 64, 0, q, d.seq_lens, cu, 1, 0)
    assert ctx.error() == (0, 0)


def test_a_programmatic_decode_after_a_chunk_reads_it(ekv_lib, torch_cuda):
    """The writer may fill any page of a sequence: a decode launched right behind it under
    ekv_set_pdl sees every row."""
    torch = torch_cuda
    lens = np.array([2000, 1500], np.int32)
    case = make_case(lens, 8, 2, 128, "mixed", 1, 37)
    ctx = ekv_lib.Context(8, 2, 128, 2, pdl=True)
    cu = torch.tensor([0, 1000, 1900], dtype=torch.int32, device="cuda")
    d = to_device(case)
    rope = torch.from_numpy(rope_table(2000, 128)).cuda()
    for _ in range(20):
        k, v = (torch.randn((1900, 2, 128), dtype=torch.float16, device="cuda") for _ in range(2))
        out, out2 = torch.empty_like(d.q), torch.empty_like(d.q)
        ctx.decode(d, out)
        call(ekv_lib, ctx, d, None, k, v, rope, 128, 0, None, d.seq_lens, cu, 2, 1900)
        ctx.decode(d, out)
        torch.cuda.synchronize()
        ctx.decode(d, out2)
        assert ctx.error() == (0, 0) and torch.equal(out, out2)
