"""ekv_prompt_attention against the oracle: lengths from none to thousands around the tile and block borders, every group size,
windows, strides, dead rows; replays, streams; refusals and device checks."""

import numpy as np
import pytest

from oracle import prompt as op

from _extend import bounds, cu_of

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch_cuda():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return torch


def attend(ekv, ctx, q, k, v, cu, n, total, window=0, sm_scale=0.0, stream=None):
    import torch
    out = torch.full(q.shape, float("nan"), dtype=torch.float16, device="cuda")
    lse = torch.full(q.shape[:2], float("nan"), dtype=torch.float32, device="cuda")
    ekv.ekv_prompt_attention(ctx.handle, q, k, v, q.stride(0), k.stride(0), v.stride(0), cu, n, total, window, sm_scale, out, lse, stream)
    return out, lse


def check(q, k, v, cu, out, lse, window=0, sm_scale=None):
    ref = op.attention(q, k, v, cu, window, sm_scale)
    T, longest = int(cu[-1]), int(np.diff(cu).max())
    tol, ltol = bounds(None, None, ref, min(window, longest) if window else longest)
    o, l = out.float().cpu().numpy().astype(np.float64)[:T], lse.cpu().numpy().astype(np.float64)[:T]
    assert np.all(np.isfinite(o)) and np.all(np.isfinite(l))
    err, lerr = np.abs(o - ref[0][:T]), np.abs(l - ref[1][:T])
    assert np.all(err <= tol[:T]), f"out off by {err.max():.3e}, {(err / tol[:T]).max():.2f} of the bound"
    assert np.all(lerr <= ltol[:T]), f"lse off by {lerr.max():.3e}, {(lerr / ltol[:T]).max():.2f} of the bound"


def rows_of(rng, total, hq, hkv, d):
    x = rng.standard_normal((total, hq + 2 * hkv, d)).astype(np.float16)
    x[:, :hq] *= np.float16(1.5)
    return x


BORDERS = [1, 2, 15, 16, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 256, 257, 300, 0, 5]


@pytest.mark.parametrize("hq,hkv,d", [(8, 2, 128), (4, 4, 64), (8, 1, 64), (3, 1, 128), (10, 2, 64), (6, 1, 128), (14, 2, 64),
                                      (16, 8, 128), (1, 1, 128)])
@pytest.mark.parametrize("window", [0, 1, 33, 128, 200])
def test_lengths_and_groups(ekv_lib, torch_cuda, hq, hkv, d, window):
    torch = torch_cuda
    rng = np.random.default_rng(200 + hq)
    lens = list(rng.permutation(BORDERS))
    cu, T = cu_of(lens), sum(lens)
    x = rows_of(rng, T + 9, hq, hkv, d)
    x[T:] = np.nan                                       # rows behind the last prompt
    q, k, v = torch.from_numpy(x).cuda().split((hq, hkv, hkv), 1)
    ctx = ekv_lib.Context(hq, hkv, d, len(lens))
    out, lse = attend(ekv_lib, ctx, q, k, v, torch.from_numpy(cu).cuda(), len(lens), T + 9, window)
    assert ctx.error() == (0, 0)
    check(x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:], cu, out, lse, window)
    assert torch.isnan(out[T:]).all() and torch.isnan(lse[T:]).all()


@pytest.mark.parametrize("lens", [[1], [7], [0], [0, 0, 3, 0], [2000, 1, 700], [1024] * 3, [1] * 300, [100] * 40])
@pytest.mark.parametrize("hq,hkv,d", [(8, 2, 128), (4, 2, 64)])
def test_batches(ekv_lib, torch_cuda, lens, hq, hkv, d):
    torch = torch_cuda
    rng = np.random.default_rng(210)
    cu, T = cu_of(lens), sum(lens)
    x = rows_of(rng, max(T, 1), hq, hkv, d)
    q, k, v = (torch.from_numpy(np.ascontiguousarray(y)).cuda() for y in np.split(x, [hq, hq + hkv], 1))
    ctx = ekv_lib.Context(hq, hkv, d, 300)
    out, lse = attend(ekv_lib, ctx, q, k, v, torch.from_numpy(cu).cuda(), len(lens), max(T, 1))
    assert ctx.error() == (0, 0)
    if T:
        check(x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:], cu, out, lse)


@pytest.mark.parametrize("n", [31, 32, 33, 1000, 4096])
def test_many_prompts_are_sorted_and_found(ekv_lib, torch_cuda, n):
    """Prompts of every number of query blocks in no order; all rows against torch in 64 bits."""
    torch = torch_cuda
    rng = np.random.default_rng(220 + n)
    lens = rng.integers(0, 12, n) if n > 2000 else np.where(rng.random(n) < 0.1, rng.integers(0, 700, n), rng.integers(0, 90, n))
    cu, T = cu_of(lens), int(lens.sum())
    q, k, v = torch.randn((T, 8, 64), device="cuda", dtype=torch.float16).split((4, 2, 2), 1)
    ctx = ekv_lib.Context(4, 2, 64, 4096)
    out, lse = attend(ekv_lib, ctx, q, k, v, torch.from_numpy(cu).cuda(), n, T)
    assert ctx.error() == (0, 0)
    top = int(lens.max())
    live = torch.arange(top, device="cuda") < torch.from_numpy(lens).cuda()[:, None]
    at = (torch.from_numpy(cu[:-1]).cuda().long()[:, None] + torch.arange(top, device="cuda")).clamp(max=T - 1)
    seen = torch.arange(top, device="cuda") <= torch.arange(top, device="cuda")[:, None]
    for b0 in range(0, n, 256):
        b = slice(b0, b0 + 256)
        for h in range(4):
            x, y, z = q[:, h][at[b]].double(), k[:, h // 2][at[b]].double(), v[:, h // 2][at[b]].double()
            s = (x @ y.transpose(1, 2) / 8).masked_fill_(~seen, -np.inf)
            ref, ref_l = torch.softmax(s, -1) @ z, torch.logsumexp(s, -1)
            # |v| < 6: half a step of the result and of the weights, 2^-11 each, and the scores' rounding (see _extend.bounds)
            assert ((out[:, h][at[b]].double() - ref).abs()[live[b]] <= 2.0 ** -11 * 12 + 2.0 ** -12).all()
            assert ((lse[:, h][at[b]].double() - ref_l).abs()[live[b]] <= 1e-4).all()


@pytest.mark.parametrize("kind", ["nan", "inf"])
def test_what_other_prompts_hold_does_not_matter(ekv_lib, torch_cuda, kind):
    torch = torch_cuda
    lens = [70, 130, 1, 260]
    cu, T = cu_of(lens), sum(lens)
    rng = np.random.default_rng(230)
    x = rows_of(rng, T, 8, 2, 128)
    ctx = ekv_lib.Context(8, 2, 128, 4)
    dcu = torch.from_numpy(cu).cuda()

    def run(y):
        q, k, v = torch.from_numpy(y).cuda().split((8, 2, 2), 1)
        return attend(ekv_lib, ctx, q, k, v, dcu, 4, T)

    out, lse = run(x)
    for i in range(4):
        y = x.copy()
        y[:cu[i]], y[cu[i + 1]:] = np.float16(kind), np.float16(kind)
        o, l = run(y)
        assert torch.equal(o[cu[i]:cu[i + 1]], out[cu[i]:cu[i + 1]]) and torch.equal(l[cu[i]:cu[i + 1]], lse[cu[i]:cu[i + 1]])
    assert ctx.error() == (0, 0)


def test_a_nan_key_reaches_the_queries_that_meet_it(ekv_lib, torch_cuda):
    torch = torch_cuda
    x = rows_of(np.random.default_rng(231), 300, 4, 2, 64)
    x[140, 4, 3] = np.nan                                # a key of KV head 0
    q, k, v = torch.from_numpy(x).cuda().split((4, 2, 2), 1)
    ctx = ekv_lib.Context(4, 2, 64, 1)
    for window in (0, 50):
        out, lse = attend(ekv_lib, ctx, q, k, v, torch.tensor([0, 300], dtype=torch.int32, device="cuda"), 1, 300, window)
        hit = torch.isnan(out).any(-1).cpu().numpy()
        meets = np.zeros((300, 4), bool)
        meets[140:190 if window else 300, :2] = True
        assert np.array_equal(hit, meets) and np.array_equal(torch.isnan(lse).cpu().numpy(), meets)
    assert ctx.error() == (0, 0)


def test_scores_that_grow_and_fall(ekv_lib, torch_cuda):
    """Maxima that move block after block, up and down, and scores far apart (weights that all but vanish)."""
    torch = torch_cuda
    rng = np.random.default_rng(232)
    x = rows_of(rng, 1500, 4, 2, 64)
    for size in (np.linspace(0.1, 12, 1500), np.linspace(12, 0.1, 1500), 8 * np.abs(np.sin(np.arange(1500) / 150))):
        y = x.copy()
        y[:, 4:6] = (y[:, 4:6] * size[:, None, None]).astype(np.float16)
        q, k, v = torch.from_numpy(y).cuda().split((4, 2, 2), 1)
        ctx = ekv_lib.Context(4, 2, 64, 2)
        cu = cu_of([1000, 500])
        out, lse = attend(ekv_lib, ctx, q, k, v, torch.from_numpy(cu).cuda(), 2, 1500, sm_scale=0.25)
        assert ctx.error() == (0, 0)
        check(y[:, :4], y[:, 4:6], y[:, 6:], cu, out, lse, sm_scale=0.25)


def test_scores_of_minus_infinity(ekv_lib, torch_cuda):
    """A query that only meets scores of -inf gets zeros and lse -inf; a prompt beside it its own."""
    torch = torch_cuda
    x = rows_of(np.random.default_rng(233), 40, 1, 1, 64)
    x[:20, 1], x[:20, 0] = 0, np.float16(1)
    x[:20, 1, 0] = -np.inf
    q, k, v = torch.from_numpy(x).cuda().split((1, 1, 1), 1)
    ctx = ekv_lib.Context(1, 1, 64, 2)
    out, lse = attend(ekv_lib, ctx, q, k, v, torch.tensor([0, 20, 40], dtype=torch.int32, device="cuda"), 2, 40)
    assert ctx.error() == (0, 0) and torch.all(out[:20] == 0) and torch.all(torch.isneginf(lse[:20]))
    check(x[20:, :1], x[20:, 1:2], x[20:, 2:], np.array([0, 20]), out[20:], lse[20:])


def test_packed_prompts_equal_the_prefill_over_their_pages(ekv_lib, torch_cuda):
    torch = torch_cuda
    lens = [512, 1000, 96]                               # (whole pages but the middle one's last)
    cu, T = cu_of(lens), sum(lens)
    q, k, v = torch.randn((T, 48, 128), device="cuda", dtype=torch.float16).split((32, 8, 8), 1)
    ctx = ekv_lib.Context(32, 8, 128, 3)
    out, lse = attend(ekv_lib, ctx, q, k, v, torch.from_numpy(cu).cuda(), 3, T)
    off = np.cumsum([0] + [-(-n // 16) for n in lens]).astype(np.int32)
    ws = [torch.zeros((int(off[-1]) * 16, 8, 128), device="cuda", dtype=torch.float16) for _ in range(2)]
    for i in range(3):
        for w, y in zip(ws, (k, v)):
            w[16 * off[i]:16 * off[i] + lens[i]] = y[cu[i]:cu[i + 1]]
    o, l = torch.empty_like(out), torch.empty_like(lse)
    ekv_lib.ekv_prefill_attention(ctx.handle, q.contiguous(), *ws, int(off[-1]), torch.from_numpy(cu).cuda(), torch.from_numpy(off).cuda(), 3,
                                  1000, 0.0, o, l)
    assert ctx.error() == (0, 0)
    # both round weights and results to half a step each: |out| < 5 at the first rows, whose keys are few
    assert (out - o).abs().max().item() <= 4 * 2.0 ** -11 * 5 and (lse - l).abs().max().item() <= 1e-4


def test_replayed_on_another_stream_with_other_lengths(ekv_lib, torch_cuda):
    torch = torch_cuda
    rng = np.random.default_rng(234)
    x = rows_of(rng, 900, 8, 2, 64)
    dx = torch.from_numpy(x).cuda()
    q, k, v = dx.split((8, 2, 2), 1)
    ctx = ekv_lib.Context(8, 2, 64, 4)
    cu = torch.tensor([0, 10, 300, 300, 900], dtype=torch.int32, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        attend(ekv_lib, ctx, q, k, v, cu, 4, 900, 100)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, lse = attend(ekv_lib, ctx, q, k, v, cu, 4, 900, 100)
    for lens in ([10, 290, 0, 600], [900, 0, 0, 0], [1, 2, 3, 4]):
        dx.copy_(torch.from_numpy(rows_of(rng, 900, 8, 2, 64)))
        cu.copy_(torch.from_numpy(cu_of(lens)))
        graph.replay()
        torch.cuda.synchronize()
        y = dx.cpu().numpy()
        check(y[:, :8], y[:, 8:10], y[:, 10:], cu_of(lens), out, lse, 100)
        assert torch.isnan(out[sum(lens):]).all()
    assert ctx.error() == (0, 0)


def test_results_do_not_depend_on_the_batch(ekv_lib, torch_cuda):
    """The same prompt twice among others: bit for bit."""
    torch = torch_cuda
    x = torch.randn((1500, 12, 128), device="cuda", dtype=torch.float16)
    q, k, v = x.split((8, 2, 2), 1)
    ctx = ekv_lib.Context(8, 2, 128, 6)
    many = torch.tensor([0, 100, 101, 101, 700, 1400, 1500], dtype=torch.int32, device="cuda")
    out, lse = attend(ekv_lib, ctx, q, k, v, many, 6, 1500)
    again, l2 = attend(ekv_lib, ctx, q, k, v, many, 6, 1500)
    assert torch.equal(out, again) and torch.equal(lse, l2)
    x[701:] = 3                                          # the others change
    o, l = attend(ekv_lib, ctx, q, k, v, many, 6, 1500)
    assert torch.equal(o[:700], out[:700]) and torch.equal(l[:700], lse[:700])


def test_alignment_of_results_and_wide_strides(ekv_lib, torch_cuda):
    """out on a 16-byte border that is none of 32; rows further apart than their heads, by different amounts."""
    torch = torch_cuda
    rng = np.random.default_rng(235)
    lens = [130, 40]
    cu, T = cu_of(lens), 170
    x = rows_of(rng, T, 8, 2, 64)
    wide = [torch.zeros((T, h * 64 + pad), device="cuda", dtype=torch.float16) for h, pad in ((8, 8), (2, 24), (2, 200))]
    for y, z in zip(wide, np.split(x, [8, 10], 1)):
        y[:, : z.shape[1] * 64] = torch.from_numpy(z.reshape(T, -1).copy()).cuda()
    ctx = ekv_lib.Context(8, 2, 64, 2)
    room = torch.full((T * 512 + 16,), float("nan"), device="cuda", dtype=torch.float16)
    lse = torch.empty((T, 8), device="cuda")
    for shift in (0, 8):
        out = room[shift:shift + T * 512]
        ekv_lib.ekv_prompt_attention(ctx.handle, *wide, *(y.stride(0) for y in wide), torch.from_numpy(cu).cuda(), 2, T, 0, 0.0, out, lse)
        assert ctx.error() == (0, 0)
        check(x[:, :8], x[:, 8:10], x[:, 10:], cu, out.view(T, 8, 64), lse)
    ekv_lib.ekv_prompt_attention(ctx.handle, *wide, *(y.stride(0) for y in wide), torch.from_numpy(cu).cuda(), 2, T, 0, 0.0, out, None)
    assert ctx.error() == (0, 0)


@pytest.mark.parametrize("lens", [[5000, 4100], [8192]])
def test_long_prompts(ekv_lib, torch_cuda, lens):
    """Lengths from which on a tile takes one head: sampled rows against 64 bits."""
    torch = torch_cuda
    cu, T = cu_of(lens), sum(lens)
    q, k, v = torch.randn((T, 12, 128), device="cuda", dtype=torch.float16).split((8, 2, 2), 1)
    ctx = ekv_lib.Context(8, 2, 128, 2)
    out, lse = attend(ekv_lib, ctx, q, k, v, torch.from_numpy(cu).cuda(), len(lens), T)
    assert ctx.error() == (0, 0)
    rng = np.random.default_rng(236)
    for a, b in zip(cu, cu[1:]):
        for r in sorted({0, 1, 127, 128, 255, 256, 4095, int(b - a) - 1} | {int(x) for x in rng.integers(0, b - a, 40)}):
            for h in range(8):
                s = (k[a:a + r + 1, h // 4].double() @ q[a + r, h].double()) / 128 ** 0.5
                p = torch.softmax(s, 0)
                ref, big = p @ v[a:a + r + 1, h // 4].double(), p @ v[a:a + r + 1, h // 4].double().abs()
                # the result's rounding and the weights', and the scores' (see _extend.bounds)
                assert ((out[a + r, h].double() - ref).abs() <= 2.0 ** -11 * ref.abs() + 2.0 ** -10.5 * big + 2.0 ** -24).all()
                assert abs(lse[a + r, h].double() - torch.logsumexp(s, 0)) <= 1e-4


def test_lengths_that_claim_rows_many_times_over_are_refused(ekv_lib, torch_cuda):
    torch = torch_cuda
    q, k, v = torch.randn((500, 8, 64), device="cuda", dtype=torch.float16).split((4, 2, 2), 1)
    ctx = ekv_lib.Context(4, 2, 64, 400)
    out, _ = attend(ekv_lib, ctx, q, k, v, torch.tensor([0, 500] * 200 + [0], dtype=torch.int32, device="cuda"), 400, 500)
    assert ctx.error() == (ekv_lib.EKV_ERR_DEVICE_CHECK, ekv_lib.EKV_DETAIL_SEQ_LEN) and torch.isnan(out).all()


def test_calls_on_two_streams_at_once(ekv_lib, torch_cuda):
    """The call keeps nothing in its context but the error word."""
    torch = torch_cuda
    q, k, v = torch.randn((4000, 12, 128), device="cuda", dtype=torch.float16).split((8, 2, 2), 1)
    ctx = ekv_lib.Context(8, 2, 128, 40)
    cus = [torch.arange(0, 4001, 4000 // n, dtype=torch.int32, device="cuda") for n in (40, 5)]
    alone = [attend(ekv_lib, ctx, q, k, v, c, len(c) - 1, 4000) for c in cus]
    streams = [torch.cuda.Stream() for _ in cus]
    torch.cuda.synchronize()
    for _ in range(5):
        got = []
        for s, c in zip(streams, cus):
            with torch.cuda.stream(s):
                got.append(attend(ekv_lib, ctx, q, k, v, c, len(c) - 1, 4000))
        torch.cuda.synchronize()
        assert all(torch.equal(a[0], g[0]) and torch.equal(a[1], g[1]) for a, g in zip(alone, got))
    assert ctx.error() == (0, 0)


def test_bad_lengths_are_reported(ekv_lib, torch_cuda):
    torch = torch_cuda
    q, k, v = torch.randn((200, 8, 64), device="cuda", dtype=torch.float16).split((4, 2, 2), 1)
    ctx = ekv_lib.Context(4, 2, 64, 3)
    whole = attend(ekv_lib, ctx, q, k, v, torch.tensor([0, 50, 100, 150], dtype=torch.int32, device="cuda"), 3, 200)
    assert ctx.error() == (0, 0)
    for cu, good in (([-5, 50, 100, 150], [(50, 100), (100, 150)]), ([0, 50, 100, 201], [(0, 50), (50, 100)]),
                     ([0, 2000000000, 100, 150], [(100, 150)]), ([0, 50, -50, 201], [(0, 50)])):
        out, lse = attend(ekv_lib, ctx, q, k, v, torch.tensor(cu, dtype=torch.int32, device="cuda"), 3, 200)
        assert ctx.error() == (ekv_lib.EKV_ERR_DEVICE_CHECK, ekv_lib.EKV_DETAIL_SEQ_LEN)
        rows = torch.ones(200, dtype=torch.bool, device="cuda")
        for a, b in good:
            assert torch.equal(out[a:b], whole[0][a:b]) and torch.equal(lse[a:b], whole[1][a:b])
            rows[a:b] = False
        assert torch.isnan(out[rows]).all() and torch.isnan(lse[rows]).all()
    assert ctx.error() == (0, 0)


def test_refusals(ekv_lib, torch_cuda):
    torch = torch_cuda
    q, k, v = (torch.zeros((20, h, 64), dtype=torch.float16, device="cuda") for h in (4, 2, 2))
    cu = torch.tensor([0, 20], dtype=torch.int32, device="cuda")
    ctx = ekv_lib.Context(4, 2, 64, 2)
    inv, cap, uns = ekv_lib.EKV_ERR_INVALID_ARG, ekv_lib.EKV_ERR_CAPACITY, ekv_lib.EKV_ERR_UNSUPPORTED
    args = dict(ctx=ctx.handle, q=q, k=k, v=v, q_stride=256, k_stride=128, v_stride=128, cu_seqlens=cu, n=1, total=20, window=0,
                sm_scale=0.0, out=torch.empty_like(q))
    for status, kw in ((inv, dict(ctx=None)), (inv, dict(q=None)), (inv, dict(k=None)), (inv, dict(v=None)), (inv, dict(cu_seqlens=None)),
                       (inv, dict(out=None)), (inv, dict(n=-1)), (inv, dict(total=-1)), (inv, dict(window=-1)), (cap, dict(n=3)),
                       (inv, dict(q=q.data_ptr() + 2)), (inv, dict(k=k.data_ptr() + 8)), (inv, dict(v=v.data_ptr() + 2)),
                       (inv, dict(out=q.data_ptr() + 8)), (inv, dict(lse=q.data_ptr() + 2)), (inv, dict(q_stride=248)),
                       (inv, dict(q_stride=260)), (inv, dict(k_stride=120)), (inv, dict(v_stride=132)), (uns, dict(total=(1 << 24) + 1))):
        with pytest.raises(ekv_lib.EkvError) as e:
            ekv_lib.ekv_prompt_attention(**{**args, **kw})
        assert e.value.status == status, kw
    ekv_lib.ekv_prompt_attention(**{**args, "n": 0})
    ekv_lib.ekv_prompt_attention(**{**args, "total": 0})
    assert ctx.error() == (0, 0)
