"""A prompt's whole way, as a program runs it: the rotary table is made, the prompts are normalised, rotated and written into E4M3
pages whose scales the writer makes, and attend to themselves from the packed rows; then the same program decodes
over the pages, token after token. Against the oracle, and captured into one graph."""

import numpy as np
import pytest

from mixed_precision_paged_gb300 import workloads as wl
from oracle import decode as od
from oracle import prompt as op

from _extend import bounds, cu_of, make_case, run_extend, to_device
from _prompt import write

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch_cuda():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return torch


@pytest.mark.parametrize("graphed", [False, True])
@pytest.mark.parametrize("hq,hkv,d,dim,style,window", [(8, 2, 128, 128, 0, 0), (4, 4, 64, 32, 1, 40)])
def test_prompts_then_decode(ekv_lib, torch_cuda, graphed, hq, hkv, d, dim, style, window):
    torch = torch_cuda
    rng = np.random.default_rng(250)
    lens, steps = [130, 1, 47, 16], 3
    B, T, cu = len(lens), sum(lens), cu_of(lens)
    case = make_case(np.array(lens) + steps, hq, hkv, d, "e4m3", 1, 251)
    case.v_scales[:] = np.nan                            # (never set)
    dev = to_device(case)
    ctx = ekv_lib.Context(hq, hkv, d, B)
    cfg = dict(theta=1e4, scaling=2, factor=4.0, original_len=64.0, slow=1.0, fast=4.0, magnitude=1.1)
    table = torch.empty((256, dim), device="cuda")
    qw, kw = ((1 + 0.2 * rng.standard_normal(d)).astype(np.float16) for _ in range(2))
    dqw, dkw = torch.from_numpy(qw).cuda(), torch.from_numpy(kw).cuda()
    x = rng.standard_normal((T, hq + 2 * hkv, d)).astype(np.float16)
    rows = torch.from_numpy(x).cuda()
    q, k, v = rows.split((hq, hkv, hkv), 1)
    dcu, dlens = torch.from_numpy(cu).cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda")
    qo, ko = torch.empty((T, hq, d), device="cuda", dtype=torch.float16), torch.empty((T, hkv, d), device="cuda", dtype=torch.float16)
    out, lse = torch.empty_like(qo), torch.empty((T, hq), device="cuda")

    def prompts():
        ekv_lib.ekv_rope_table(ctx.handle, ekv_lib.ekv_rope_config(**cfg), table, 0, 256, dim)
        write(ekv_lib, ctx, dev, q, k, v, table, dim, style, qo, dlens, dcu, B, T, q_weight=dqw, k_weight=dkw, k_out=ko, grow_scales=1)
        ekv_lib.ekv_prompt_attention(ctx.handle, qo, ko, v, hq * d, hkv * d, v.stride(0), dcu, B, T, window, 0.0, out, lse)

    prompts()
    if graphed:
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            prompts()
        x = x[::-1].copy()
        rows.copy_(torch.from_numpy(x))
        graph.replay()
    torch.cuda.synchronize()
    assert ctx.error() == (0, 0)
    # the attention against the oracle over the rows that the writer made
    got_q, got_k = qo.cpu().numpy(), ko.cpu().numpy()
    ref = op.attention(got_q, got_k, x[:, hq + hkv:], cu, window)
    tol, ltol = bounds(None, None, ref, max(lens))
    assert np.all(np.abs(out.float().cpu().numpy() - ref[0]) <= tol) and np.all(np.abs(lse.cpu().numpy() - ref[1]) <= ltol)
    # those rows against the formula: half an fp16 step, and the table's, the norm's and the rotation's fp32 steps
    rope = op.rope_table(0, 256, dim, **cfg)
    rq = op.append(x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:], qw, kw, 1e-6, rope, style, case.k_pages, case.v_pages, case.v_scales,
                   1, 1, None, 1, case.block_table, np.array(lens), cu)[0]
    assert np.all(np.abs(got_q - rq) <= 2.0 ** -11 * np.abs(rq) + 2.0 ** -25 + 32 * 2.0 ** -24 * 2 * np.abs(rq).max())
    # decode steps over the pages
    for step in range(1, steps + 1):
        y = torch.from_numpy(rng.standard_normal((B, hq + 2 * hkv, d)).astype(np.float16)).cuda()
        q1, k1, v1 = y.split((hq, hkv, hkv), 1)
        now = dlens + step
        one = torch.arange(B + 1, dtype=torch.int32, device="cuda")
        qd = torch.empty((B, hq, d), device="cuda", dtype=torch.float16)
        write(ekv_lib, ctx, dev, q1, k1, v1, table, dim, style, qd, now, one, B, B, q_weight=dqw, k_weight=dkw, grow_scales=1)
        d1 = wl.DecodeCase(**{**dev.__dict__, "q": qd, "seq_lens": now})
        dec = torch.empty_like(qd)
        ctx.decode(d1, dec)
        ext, _ = run_extend(ekv_lib, ctx, d1, qd, one, 1)
        assert ctx.error() == (0, 0)
        refd, _ = od.paged_decode(qd.cpu().numpy(), dev.k_pages.cpu().numpy(), dev.v_pages.cpu().numpy(), dev.v_scales.cpu().numpy(), 1,
                                  None, 1, case.block_table, now.cpu().numpy())
        for o in (dec, ext):                             # (the decode's tolerance, see tests/_helpers.py)
            assert np.abs(o.float().cpu().numpy() - refd).max() <= 2e-3
