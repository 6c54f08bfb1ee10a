"""ekv_extend_attention against the float64 oracle: one token to long chunks, page forms, head
layouts, windows, lengths at tile borders, refusals, streams and captured graphs."""

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


def run_and_check(ekv, torch, lens, new, hq, hkv, d, fmt="all", scale_mode=1, window=0, seed=0, rows=None, q_gain=1.0,
                  sm_scale=0.0, stride_pad=0, max_q=None):
    case = make_case(lens, hq, hkv, d, fmt, scale_mode, seed, stride_pad=stride_pad)
    cu = cu_of(new)
    q = (np.random.default_rng(seed + 9).standard_normal((int(cu[-1]), hq, d)) * q_gain).astype(np.float16)
    ctx = ekv.Context(hq, hkv, d, len(lens))
    out, lse = run_extend(ekv, ctx, to_device(case), torch.from_numpy(q).cuda(), torch.from_numpy(cu).cuda(),
                          max(new) if max_q is None else max_q, window, sm_scale)
    torch.cuda.synchronize()
    assert ctx.error() == (0, 0)
    check(case, cu, q, out, lse, window, sm_scale if sm_scale > 0 else None, rows)
    ctx.close()


FORMS = [("fp16", 0), ("e4m3", 0), ("e4m3", 1), ("base", 0), ("micro", 0), ("all", 1), ("all", 0)]


@pytest.mark.parametrize("fmt,sm", FORMS)
@pytest.mark.parametrize("new", [[1, 1, 1, 1, 1], [5, 1, 3, 4, 2], [40, 1, 130, 17, 0]])
def test_forms_of_pages(ekv_lib, torch_cuda, fmt, sm, new):
    run_and_check(ekv_lib, torch_cuda, [300, 1, 131, 17, 64], new, 8, 2, 128, fmt, sm, seed=1)


@pytest.mark.parametrize("hq,hkv,d", [(4, 2, 64), (8, 1, 128), (8, 8, 64), (24, 4, 128), (5, 1, 64), (14, 2, 128),
                                      (32, 8, 128), (16, 2, 64), (3, 1, 128)])
@pytest.mark.parametrize("new", [[1, 2], [9, 3], [70, 33]])
def test_head_layouts(ekv_lib, torch_cuda, hq, hkv, d, new):
    run_and_check(ekv_lib, torch_cuda, [200, 77], new, hq, hkv, d, "all", 1, seed=2)


@pytest.mark.parametrize("n", [1, 2, 4, 5, 8, 9, 16, 31, 32, 33, 63, 64, 65, 127, 128, 129, 200, 257])
def test_numbers_of_new_tokens(ekv_lib, torch_cuda, n):
    run_and_check(ekv_lib, torch_cuda, [n + 100, n, max(n, 16)], [n, n, max(1, n // 2)], 8, 2, 64, "e4m3", 0, seed=n)


@pytest.mark.parametrize("length", [1, 2, 15, 16, 17, 127, 128, 129, 255, 256, 257, 1000])
@pytest.mark.parametrize("n", [1, 12])
def test_lengths_at_borders(ekv_lib, torch_cuda, length, n):
    n = min(n, length)
    run_and_check(ekv_lib, torch_cuda, [length], [n], 8, 2, 128, "all", 1, seed=length)


@pytest.mark.parametrize("window", [1, 2, 15, 16, 17, 100, 128, 129, 300, 5000])
@pytest.mark.parametrize("new", [[1, 1], [6, 3], [90, 300]])
def test_windows(ekv_lib, torch_cuda, window, new):
    run_and_check(ekv_lib, torch_cuda, [700, 333], new, 8, 2, 128, "all", 1, window=window, seed=window)


def test_a_long_sequence_is_split_and_joined(ekv_lib, torch_cuda):
    run_and_check(ekv_lib, torch_cuda, [20011], [1], 8, 2, 128, "e4m3", 1, seed=4, q_gain=2.0)
    run_and_check(ekv_lib, torch_cuda, [20011], [3], 8, 2, 128, "micro", 0, seed=5)
    run_and_check(ekv_lib, torch_cuda, [9000], [40], 8, 2, 128, "all", 1, seed=6, rows={0, 13, 39})
    run_and_check(ekv_lib, torch_cuda, [9000], [300], 8, 2, 64, "fp16", 0, seed=7, rows={0, 1, 128, 255, 256, 299})


def test_many_sequences_of_odd_lengths(ekv_lib, torch_cuda):
    rng = np.random.default_rng(8)
    lens = rng.integers(1, 500, 150)
    run_and_check(ekv_lib, torch_cuda, lens, [1] * 150, 8, 4, 64, "all", 1, seed=9)
    new = [int(min(n, rng.integers(0, 30))) for n in lens]
    run_and_check(ekv_lib, torch_cuda, lens, new, 8, 4, 64, "all", 1, seed=10, rows=set(rng.integers(0, sum(new), 200).tolist()))


@pytest.mark.parametrize("new", [[1, 1], [40, 60]])
def test_sharp_scores_strides_and_scale(ekv_lib, torch_cuda, new):
    run_and_check(ekv_lib, torch_cuda, [150, 333], new, 8, 2, 128, "all", 1, seed=11, q_gain=8.0)
    run_and_check(ekv_lib, torch_cuda, [150, 333], new, 8, 2, 128, "all", 1, seed=12, stride_pad=16)
    run_and_check(ekv_lib, torch_cuda, [150, 333], new, 8, 2, 64, "e4m3", 1, seed=13, stride_pad=48, sm_scale=0.31)
    run_and_check(ekv_lib, torch_cuda, [150, 333], new, 8, 2, 64, "micro", 1, seed=14, stride_pad=80, max_q=500)


@pytest.mark.parametrize("new", [[1, 1, 1], [50, 60, 70]])
def test_scales_of_very_different_size(ekv_lib, torch_cuda, new):
    """E4M3 pages whose scales differ by 2^30: the small ones still count where they are alone."""
    torch = torch_cuda
    case = make_case([200, 160, 90], 8, 2, 128, "e4m3", 1, 15)
    rng = np.random.default_rng(15)
    case.v_scales = (case.v_scales * 2.0 ** rng.integers(-24, 7, case.v_scales.shape)).astype(np.float32)
    case.v_scales[case.block_table[1, :10]] *= np.float32(2.0 ** -10)
    cu = cu_of(new)
    q = rng.standard_normal((int(cu[-1]), 8, 128)).astype(np.float16)
    ctx = ekv_lib.Context(8, 2, 128, 3)
    out, lse = run_extend(ekv_lib, ctx, to_device(case), torch.from_numpy(q).cuda(), torch.from_numpy(cu).cuda(), max(new))
    assert ctx.error() == (0, 0)
    check(case, cu, q, out, lse)


@pytest.mark.parametrize("new", [[1, 0, 2, 0], [0, 0, 0, 1], [40, 0, 80, 0]])
def test_rows_behind_the_last_sequence_stay(ekv_lib, torch_cuda, new):
    torch = torch_cuda
    case = make_case([60, 20, 100, 1], 8, 2, 64, "all", 1, 16)
    case.seq_lens = np.array([60, 20, 100, new[3]], np.int32)
    cu = cu_of(new)
    T = int(cu[-1])
    q = np.random.default_rng(3).standard_normal((T + 5, 8, 64)).astype(np.float16)
    ctx = ekv_lib.Context(8, 2, 64, 4)
    out, lse = run_extend(ekv_lib, ctx, to_device(case), torch.from_numpy(q).cuda(), torch.from_numpy(cu).cuda(), max(new))
    assert ctx.error() == (0, 0)
    assert torch.isnan(out[T:]).all() and torch.isnan(lse[T:]).all()
    check(case, cu, q[:T], out[:T], lse[:T])


@pytest.mark.parametrize("n", [1, 50])
def test_no_lse_and_masked_infinities(ekv_lib, torch_cuda, n):
    """Keys outside a query's range hold infinities and NaN; lse is not asked for."""
    torch = torch_cuda
    case = make_case([300], 8, 2, 128, "fp16", 0, 17)
    rows = np.arange(16 * 19)
    page, row = case.block_table[0, rows // 16], rows % 16
    v = case.v_pages.view("<f2").reshape(-1, 16, 2, 128)
    old = rows < 300 - n - 60                            # behind every query's window
    case.k_pages[page[old], row[old]] = np.inf
    v[page[old], row[old]] = np.nan
    q = np.random.default_rng(4).standard_normal((n, 8, 128)).astype(np.float16)
    ctx = ekv_lib.Context(8, 2, 128, 1)
    d, cu = to_device(case), torch.tensor([0, n], dtype=torch.int32, device="cuda")
    qd = torch.from_numpy(q).cuda()
    out, lse = run_extend(ekv_lib, ctx, d, qd, cu, n, window=60)
    out2 = torch.empty_like(qd)
    ekv_lib.ekv_extend_attention(ctx.handle, qd, d.k_pages, d.v_pages, d.v_page_stride, d.num_pages, None, 0, None, 0,
                                 d.block_table, int(d.block_table.shape[1]), d.seq_lens, cu, 1, n, n, 60, 0.0, out2)
    assert ctx.error() == (0, 0)
    assert torch.equal(out, out2)
    case.k_pages[page[old], row[old]] = 0
    v[page[old], row[old]] = 0
    check(case, [0, n], q, out, lse, window=60)


@pytest.mark.parametrize("new", [[2, 1, 3], [40, 33, 50]])
def test_failing_pages_zero_the_queries_that_see_them(ekv_lib, torch_cuda, new):
    torch = torch_cuda
    lens = [200, 90, 150]
    base = make_case(lens, 8, 2, 64, "all", 1, 18)
    base.page_mode[base.block_table[1, 2]] = 1           # an E4M3 page: its scale can fail
    base.v_pages[base.block_table[1, 2]][: 16 * 2 * 64] = 0x38
    base.v_scales[base.block_table[1, 2]] = 0.01
    cu = cu_of(new)
    q = np.random.default_rng(5).standard_normal((int(cu[-1]), 8, 64)).astype(np.float16)
    ctx = ekv_lib.Context(8, 2, 64, 3)
    dq, dcu = torch.from_numpy(q).cuda(), torch.from_numpy(cu).cuda()
    good, _ = run_extend(ekv_lib, ctx, to_device(base), dq, dcu, max(new))
    assert ctx.error() == (0, 0)
    seq1 = slice(int(cu[1]), int(cu[2]))
    for what, detail in (("id", ekv_lib.EKV_DETAIL_PAGE_ID), ("mode", ekv_lib.EKV_DETAIL_PAGE_MODE),
                         ("scale", ekv_lib.EKV_DETAIL_SCALE), ("scales", ekv_lib.EKV_DETAIL_SCALE)):
        d = to_device(base)
        heads = slice(0, 8)
        if what == "id":
            d.block_table[1, 2] = d.num_pages
        elif what == "mode":
            d.page_mode[int(base.block_table[1, 2])] = 4
        elif what == "scale":
            d.v_scales[int(base.block_table[1, 2]), 1] = float("nan")
            heads = slice(4, 8)
        else:
            d.v_scales = None
        out, lse = run_extend(ekv_lib, ctx, d, dq, dcu, max(new))
        assert ctx.error() == (ekv_lib.EKV_ERR_DEVICE_CHECK, detail), what
        assert torch.all(out[seq1, heads] == 0) and torch.all(lse[seq1, heads] == -float("inf")), what
        if what != "scales":
            keep = torch.ones_like(out, dtype=torch.bool)
            keep[seq1, heads] = False
            assert torch.equal(out[keep], good[keep]), what
    # a window that leaves the failing page behind some queries: those are as before
    d = to_device(base)
    d.block_table[1, 2] = -1                             # keys 32 .. 47 of 90
    n, w = new[1], 60
    out, lse = run_extend(ekv_lib, ctx, d, dq, dcu, max(new), window=w)
    assert ctx.error()[0] in (0, ekv_lib.EKV_ERR_DEVICE_CHECK)
    pos = 90 - n + np.arange(n)
    sees = (pos - w + 1 <= 47) & (pos >= 32)
    got = out[seq1].float().cpu().numpy()
    assert np.all(got[sees] == 0) and np.all(np.abs(got[~sees]).max(axis=(1, 2)) > 0)


@pytest.mark.parametrize("n", [1, 50])
def test_bad_micro_scale_reads_as_zero(ekv_lib, torch_cuda, n):
    torch = torch_cuda
    case = make_case([64], 2, 1, 64, "micro", 0, 19)
    d = to_device(case)
    d.v_pages[:, 16 * 32:16 * 34] = 255                  # every scale byte
    q = torch.randn((n, 2, 64), dtype=torch.float16, device="cuda")
    ctx = ekv_lib.Context(2, 1, 64, 1)
    out, _ = run_extend(ekv_lib, ctx, d, q, torch.tensor([0, n], dtype=torch.int32, device="cuda"), n)
    assert ctx.error() == (ekv_lib.EKV_ERR_DEVICE_CHECK, ekv_lib.EKV_DETAIL_SCALE)
    assert torch.all(out == 0)


@pytest.mark.parametrize("n", [2, 40])
def test_lengths_that_fail(ekv_lib, torch_cuda, n):
    torch = torch_cuda
    case = make_case([100, 100, 100], 8, 2, 64, "e4m3", 0, 20)
    ctx = ekv_lib.Context(8, 2, 64, 3)
    cu = torch.tensor(cu_of([n, n, n]), device="cuda")
    q = torch.randn((3 * n, 8, 64), dtype=torch.float16, device="cuda")
    good, _ = run_extend(ekv_lib, ctx, to_device(case), q, cu, n)
    for bad in (-1, 1, 16 * 7 + 1, 1 << 30):             # below its new tokens, above the table
        d = to_device(case)
        d.seq_lens[1] = bad
        out, lse = run_extend(ekv_lib, ctx, d, q, cu, n)
        assert ctx.error() == (ekv_lib.EKV_ERR_DEVICE_CHECK, ekv_lib.EKV_DETAIL_SEQ_LEN), bad
        assert torch.all(out[n:2 * n] == 0) and torch.all(lse[n:2 * n] == -float("inf"))
        assert torch.equal(out[:n], good[:n]) and torch.equal(out[2 * n:], good[2 * n:])
    out, lse = run_extend(ekv_lib, ctx, to_device(case), q, cu, n - 1)      # max_q below the truth
    assert ctx.error() == (ekv_lib.EKV_ERR_DEVICE_CHECK, ekv_lib.EKV_DETAIL_SEQ_LEN)
    assert torch.all(out == 0)


def test_refusals(ekv_lib, torch_cuda):
    torch = torch_cuda
    case = make_case([40], 8, 2, 64, "e4m3", 0, 21)
    d = to_device(case)
    ctx = ekv_lib.Context(8, 2, 64, 1)
    q = torch.zeros((2, 8, 64), dtype=torch.float16, device="cuda")
    cu = torch.tensor([0, 2], dtype=torch.int32, device="cuda")
    out, lse = torch.empty_like(q), torch.empty((2, 8), device="cuda")

    def call(**kw):
        a = dict(ctx=ctx.handle, q=q, k_pages=d.k_pages, v_pages=d.v_pages, v_page_stride_bytes=d.v_page_stride,
                 num_pages=d.num_pages, v_scales=d.v_scales, scale_mode=0, page_mode=None, uniform_mode=1,
                 block_table=d.block_table, block_table_stride=3, seq_lens=d.seq_lens, cu_q=cu, batch=1, total_q=2,
                 max_q=2, window=0, sm_scale=0.0, out=out, lse=lse)
        a.update(kw)
        ekv_lib.ekv_extend_attention(**a)

    call()
    inv = ekv_lib.EKV_ERR_INVALID_ARG
    for kw, status in ((dict(ctx=None), inv), (dict(q=None), inv), (dict(out=None), inv), (dict(k_pages=None), inv),
                       (dict(v_pages=None), inv), (dict(seq_lens=None), inv), (dict(cu_q=None), inv),
                       (dict(block_table=None), inv), (dict(window=-1), inv), (dict(max_q=-1), inv), (dict(batch=-1), inv),
                       (dict(total_q=-1), inv), (dict(batch=2), ekv_lib.EKV_ERR_CAPACITY), (dict(uniform_mode=4), inv),
                       (dict(uniform_mode=-1), inv), (dict(scale_mode=2), inv), (dict(v_scales=None), inv),
                       (dict(uniform_mode=0), inv), (dict(uniform_mode=2), inv), (dict(q=q.data_ptr() + 2), inv),
                       (dict(out=out.data_ptr() + 8), inv), (dict(lse=lse.data_ptr() + 2), inv),
                       (dict(v_page_stride_bytes=d.v_page_stride + 8), inv), (dict(v_page_stride_bytes=1024), inv),
                       (dict(num_pages=0), inv), (dict(block_table_stride=0), inv)):
        with pytest.raises(ekv_lib.EkvError) as e:
            call(**kw)
        assert e.value.status == status, kw
    call(batch=0)
    call(total_q=0)
    assert ctx.error() == (0, 0)


@pytest.mark.parametrize("new", [[3, 1, 2], [60, 2, 90]])
def test_captured_and_replayed_on_another_stream(ekv_lib, torch_cuda, new):
    """A graph of writer and attention, replayed over new tokens and lengths that its buffers
    receive, beside eager calls between the replays; twice the same result."""
    torch = torch_cuda
    lens = np.array([200, 30, 150], np.int32)
    case = make_case(lens + 20, 8, 2, 128, "all", 1, 22)
    case.seq_lens = lens
    cu = cu_of(new)
    T = int(cu[-1])
    rng = np.random.default_rng(6)
    ang = rng.standard_normal((256, 64))
    rope = torch.from_numpy(np.concatenate([np.cos(ang), np.sin(ang)], 1).astype(np.float32)).cuda()
    d, dcu = to_device(case), torch.from_numpy(cu).cuda()
    ctx = ekv_lib.Context(8, 2, 128, 3)
    q, k, v = (torch.randn((T, h, 128), dtype=torch.float16, device="cuda") for h in (8, 2, 2))
    qr, out, lse = torch.empty_like(q), torch.empty_like(q), torch.empty((T, 8), device="cuda")

    def step(stream=None):
        ekv_lib.ekv_append_kv_rope(ctx.handle, q, k, v, 8 * 128, 256, 256, rope, 256, 128, 0, qr, d.k_pages, d.v_pages,
                                   d.v_page_stride, d.num_pages, d.v_scales, 1, d.page_mode, 0, d.block_table,
                                   int(d.block_table.shape[1]), d.seq_lens, dcu, 3, T, stream)
        run_extend(ekv_lib, ctx, d, qr, dcu, max(new), out=out, lse=lse, stream=stream)

    step()
    torch.cuda.synchronize()
    g, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(g, stream=s):
        step()
    for grow in (1, 7, 20):
        for x in (q, k, v):
            x.copy_(torch.randn_like(x))
        d.seq_lens.copy_(torch.from_numpy(lens + grow))
        torch.cuda.synchronize()
        with torch.cuda.stream(s):
            g.replay()
        s.synchronize()
        first = out.clone(), lse.clone()
        out.zero_()
        step()
        torch.cuda.synchronize()
        assert torch.equal(out, first[0]) and torch.equal(lse, first[1])
        assert ctx.error() == (0, 0)
        host = make_case(lens + 20, 8, 2, 128, "all", 1, 22)
        host.k_pages, host.v_pages = d.k_pages.cpu().numpy(), d.v_pages.cpu().numpy()
        host.seq_lens = lens + grow
        check(host, cu, qr.cpu().numpy(), out, lse)


def test_one_token_agrees_with_the_decode(ekv_lib, torch_cuda):
    torch = torch_cuda
    lens = [1000, 17, 300, 4097]
    case = make_case(lens, 32, 8, 128, "mixed", 1, 23)
    d = to_device(case)
    ctx = ekv_lib.Context(32, 8, 128, 4)
    out, lse = torch.empty_like(d.q), torch.empty((4, 32), device="cuda")
    ctx.decode(d, out, lse)
    cu = torch.arange(5, dtype=torch.int32, device="cuda")
    out2, lse2 = run_extend(ekv_lib, ctx, d, d.q, cu, 1)
    assert ctx.error() == (0, 0)
    check(case, cu_of([1] * 4), case.q, out, lse)
    check(case, cu_of([1] * 4), case.q, out2, lse2)
    # the elder decode reports microscaled pages and zeroes their sequence; this one reads them
    case = make_case(lens, 32, 8, 128, "all", 1, 24)
    d = to_device(case)
    ctx.decode(d, out, lse)
    assert ctx.error() == (ekv_lib.EKV_ERR_DEVICE_CHECK, ekv_lib.EKV_DETAIL_PAGE_MODE)
    out2, lse2 = run_extend(ekv_lib, ctx, d, d.q, cu, 1)
    assert ctx.error() == (0, 0)
    check(case, cu_of([1] * 4), case.q, out2, lse2)


@pytest.mark.parametrize("most", [1, 30])
def test_batches_of_more_sequences_than_threads(ekv_lib, torch_cuda, most):
    """The plan reads sequences in passes of one per thread; empty ones among them."""
    rng = np.random.default_rng(30 + most)
    lens = rng.integers(1, 200, 1300)
    new = [int(min(n, rng.integers(0, most + 1))) for n in lens]
    run_and_check(ekv_lib, torch_cuda, lens, new, 4, 2, 64, "e4m3", 0, seed=31, max_q=most,
                  rows=set(rng.integers(0, sum(new), 300).tolist()) | {0, sum(new) - 1})


@pytest.mark.parametrize("length,n", [(300, 1), (300, 50), (9000, 2), (9000, 40)])
def test_nan_goes_to_the_queries_that_meet_it(ekv_lib, torch_cuda, length, n):
    """A NaN query or visible NaN key gives NaN, as the formula does; the other queries keep their bits."""
    torch = torch_cuda
    case = make_case([length], 8, 2, 128, "e4m3", 0, 32)
    d, cu = to_device(case), torch.tensor([0, n], dtype=torch.int32, device="cuda")
    q = torch.randn((n, 8, 128), dtype=torch.float16, device="cuda")
    ctx = ekv_lib.Context(8, 2, 128, 1)
    out, lse = run_extend(ekv_lib, ctx, d, q, cu, n)
    q2 = q.clone()
    q2[n // 2, 5, 77] = float("nan")
    out2, lse2 = run_extend(ekv_lib, ctx, d, q2, cu, n)
    hit = torch.zeros((n, 8), dtype=torch.bool, device="cuda")
    hit[n // 2, 5] = True
    assert torch.isnan(out2[hit]).all() and torch.isnan(lse2[hit]).all()
    assert torch.equal(out2[~hit], out[~hit]) and torch.equal(lse2[~hit], lse[~hit])
    t = length - 1 - n // 3                              # a key that the last third of the queries see
    d.k_pages[int(case.block_table[0, t // 16]), t % 16, 1, 3] = float("nan")
    out3, lse3 = run_extend(ekv_lib, ctx, d, q, cu, n)
    hit[:] = False
    hit[n - 1 - n // 3:, 4:] = True
    assert torch.isnan(out3[hit]).all() and torch.isnan(lse3[hit]).all()
    assert torch.equal(out3[~hit], out[~hit]) and torch.equal(lse3[~hit], lse[~hit])
    assert ctx.error() == (0, 0)


@pytest.mark.parametrize("n", [1, 70])
def test_stale_table_entries_outside_the_window(ekv_lib, torch_cuda, n):
    torch = torch_cuda
    case = make_case([900, 33], 8, 2, 64, "all", 1, 33)
    cu = cu_of([n, min(n, 33)])
    q = np.random.default_rng(34).standard_normal((int(cu[-1]), 8, 64)).astype(np.float16)
    d = to_device(case)
    seen = 900 - n - 100 + 1                             # first key that a query of sequence 0 sees
    d.block_table[0, :seen // 16] = torch.tensor(2 ** 31 - 1, dtype=torch.int32)
    d.block_table[1, 3:] = -5
    ctx = ekv_lib.Context(8, 2, 64, 2)
    out, lse = run_extend(ekv_lib, ctx, d, torch.from_numpy(q).cuda(), torch.from_numpy(cu).cuda(), n, window=100)
    assert ctx.error() == (0, 0)
    check(case, cu, q, out, lse, window=100)


def test_two_contexts_at_once_and_again(ekv_lib, torch_cuda):
    """Calls of two contexts that overlap on two streams, repeated: each keeps its bits."""
    torch = torch_cuda
    runs = []
    for i, (lens, new) in enumerate((([5000, 300, 2000], [1, 2, 3]), ([3000, 700], [200, 90]))):
        case = make_case(lens, 8, 2, 128, "all", 1, 40 + i)
        cu = cu_of(new)
        q = torch.randn((int(cu[-1]), 8, 128), dtype=torch.float16, device="cuda")
        ctx, d, dcu = ekv_lib.Context(8, 2, 128, 3), to_device(case), torch.from_numpy(cu).cuda()
        runs.append((ctx, d, q, dcu, max(new), torch.cuda.Stream(), run_extend(ekv_lib, ctx, d, q, dcu, max(new))))
    torch.cuda.synchronize()
    got = []
    for _ in range(8):
        for ctx, d, q, dcu, mq, s, _ref in runs:
            with torch.cuda.stream(s):
                got.append((run_extend(ekv_lib, ctx, d, q, dcu, mq, stream=s.cuda_stream), _ref))
    torch.cuda.synchronize()
    for (out, lse), ref in got:
        assert torch.equal(out, ref[0]) and torch.equal(lse, ref[1])
    for r in runs:
        assert r[0].error() == (0, 0)
