"""Shared pieces of the tests of a prompt's way into the cache."""

import numpy as np

from oracle import extend as oe
from oracle import prompt as op


def rope_table(n, dim):
    return op.rope_table(0, n, dim, theta=1e4).astype(np.float32) if dim else np.zeros((n, 0), np.float32)


def write(ekv, owner, d, q, k, v, rope, dim, style, qo, lens, cu, nseq, total, **kw):
    """ekv_append_kv_norm_rope with a case's pages; kw: what differs."""
    a = dict(ctx=owner.handle, q=q, k_new=k, v_new=v, q_stride=q.stride(0) if q is not None else 0, k_stride=k.stride(0),
             v_stride=v.stride(0), q_weight=None, k_weight=None, norm_eps=1e-6, rope_table=rope,
             rope_len=rope.shape[0] if rope is not None else 0, rope_dim=dim, rope_style=style, q_out=qo, k_out=None,
             k_pages=d.k_pages, v_pages=d.v_pages, v_page_stride_bytes=d.v_page_stride, num_pages=d.num_pages,
             v_scales=d.v_scales, scale_mode=d.scale_mode, grow_scales=0, page_mode=d.page_mode, uniform_mode=d.uniform_mode,
             block_table=d.block_table, block_table_stride=int(d.block_table.shape[1]), seq_lens=lens, cu_q=cu, batch=nseq,
             total_q=total)
    a.update(kw)
    ekv.ekv_append_kv_norm_rope(**a)


def check_write(case, rope, style, q, k, v, qw, kw, eps, lens, cu, grow, qo, ko, dev):
    """Against the oracle. Queries and keys: the sum of squares of 16 products a lane and 3 additions (19 roundings,
    halved by the root), the root (2 units, 2^-22), two products: 16 units of 2^-24 of each value; the rotation three
    more of the pair's size; the result half an fp16 step (2^-11 relative, 2^-25 where subnormal). Value bytes and scales
    exactly, and every other row of the pages as it was."""
    T = int(cu[-1])
    rq, rk, rv, rs = op.append(q, k, v, qw, kw, eps, rope, style, case.k_pages, case.v_pages, case.v_scales, case.scale_mode, grow,
                               case.page_mode, case.uniform_mode, case.block_table, lens, cu)

    def near(got, ref, rows, w):
        size = 2 * np.abs(op.normed(rows, w, eps)).max(-1, keepdims=True)
        return np.all(np.abs(got.astype(np.float64) - ref) <= 2.0 ** -11 * np.abs(ref) + 2.0 ** -25 + 20 * 2.0 ** -24 * size)
    if qo is not None:
        assert near(qo[:T], rq[:T], q[:T], qw)
    kp = dev.k_pages.cpu().numpy()
    written = np.zeros(kp.shape[:2], bool)
    for i, b, t in oe.places(lens, cu):
        page, row = case.block_table[b][t // 16], t % 16
        written[page, row] = True
        assert near(kp[page, row], rk[page, row], k[i], kw)
        if ko is not None:
            assert np.array_equal(ko[i].view(np.uint16), kp[page, row].view(np.uint16))
    assert np.array_equal(kp[~written].view(np.uint16), case.k_pages[~written].view(np.uint16))
    if rs is not None:
        assert np.array_equal(dev.v_scales.cpu().numpy(), rs)
    assert np.array_equal(dev.v_pages.cpu().numpy(), rv)
