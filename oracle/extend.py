"""New tokens of a ragged batch: the rotary cache writer and their attention over the
paged cache, in float64. Oracle only.

Sequence b has n_b = cu_q[b+1] - cu_q[b] new tokens, the last of its seq_lens[b]; its r-th is row
i = cu_q[b] + r at position t = seq_lens[b] - n_b + r.

* writer: q and k rotated, (x_i, x_j) -> (x_i cos - x_j sin, x_j cos + x_i sin) over the pairs of
  the first rope_dim values, by the table row of t (its first half cosines, its second sines); the K
  row and the V row go to row t % 16 of page block_table[b][t // 16], V in the page's form.
* attention: query row i, head h_q over keys max(0, t - window + 1) .. t of sequence b
  (window 0: from key 0), KV head h_q // G.
"""

import math

import numpy as np

from . import decode, micro, writer

PAGE_SIZE = 16


def rotate(x, cos, sin, style):
    """x float64 [..., D] turned by the angles of one position (cos, sin [rope_dim / 2])."""
    y = np.array(x, dtype=np.float64)
    half = cos.size
    for j in range(half):
        a, b = (j, j + half) if style == 0 else (2 * j, 2 * j + 1)
        y[..., a] = x[..., a] * cos[j] - x[..., b] * sin[j]
        y[..., b] = x[..., b] * cos[j] + x[..., a] * sin[j]
    return y


def places(seq_lens, cu_q):
    """(row i, sequence b, position t) of every new token."""
    for b in range(len(seq_lens)):
        n = int(cu_q[b + 1]) - int(cu_q[b])
        for r in range(n):
            yield int(cu_q[b]) + r, b, int(seq_lens[b]) - n + r


def append(q, k_new, v_new, rope, rope_style, k_pages, v_pages, v_scales, scale_mode, page_mode, uniform_mode,
           block_table, seq_lens, cu_q):
    """q' float64 [T][H_q][D], K pool float64, V pool bytes. V bytes are exact; q' and K are
    not rounded."""
    kp, vp = k_pages.astype(np.float64), np.array(v_pages, copy=True)
    qo = q.astype(np.float64)
    H, D = k_new.shape[1:]
    half = rope.shape[1] // 2
    for i, b, t in places(seq_lens, cu_q):
        cos, sin = rope[t, :half].astype(np.float64), rope[t, half:].astype(np.float64)
        qo[i] = rotate(q[i].astype(np.float64), cos, sin, rope_style)
        page, row = int(block_table[b][t // PAGE_SIZE]), t % PAGE_SIZE
        kp[page, row] = rotate(k_new[i].astype(np.float64), cos, sin, rope_style)
        mode = uniform_mode if page_mode is None else int(page_mode[page])
        if mode == micro.MODE_MICRO_FP4:
            n, cb = micro.page_bytes(1, D), PAGE_SIZE * D // 2
            for h in range(H):
                for j in range(D // 32):
                    c, k = micro.encode_block(v_new[i, h, 32 * j:32 * j + 32])
                    at = h * n + row * D // 2 + 16 * j
                    vp[page, at:at + 16] = c[0::2] | (c[1::2] << 4)
                    vp[page, h * n + cb + row * (D // 32) + j] = k + 127
        else:
            one = np.array([[page]])
            _, v2 = writer.append_token(np.zeros((1,) + k_pages.shape[1:], np.float16), vp[page:page + 1],
                                        v_scales if scale_mode == 0 or v_scales is None else v_scales[page:page + 1],
                                        scale_mode, None, mode, np.zeros_like(one), [row],
                                        np.zeros((1, H, D), np.float16), v_new[i:i + 1])
            vp[page] = v2[0]
    return qo, kp, vp


def sequence_kv(b, case, L):
    """float64 K, V [L][H_kv][D] of sequence b of a case with the fields of workloads.DecodeCase."""
    H, D = case.k_pages.shape[2:]
    ks, vs = [], []
    for j in range(-(-L // PAGE_SIZE)):
        p = int(case.block_table[b][j])
        mode = case.uniform_mode if case.page_mode is None else int(case.page_mode[p])
        ks.append(case.k_pages[p].astype(np.float64))
        if mode == micro.MODE_MICRO_FP4:
            vs.append(micro.decode_page(case.v_pages[p], H, D))
        else:
            srow = decode._scale_row(case.v_scales, case.scale_mode, p, H) if mode == 1 else None
            vs.append(decode.dequant_value_page(case.v_pages[p], mode, srow, H, D, PAGE_SIZE))
    return np.concatenate(ks)[:L], np.concatenate(vs)[:L]


def attention(q, case, cu_q, window=0, sm_scale=None, rows=None):
    """out [T][H_q][D], lse [T][H_q], and for error bounds: wabs = sum_k p_k |v_k| [T][H_q][D]
    and qk = max_k sm_scale * sum_d |q_d k_d| [T][H_q]. `rows`: only these rows (the rest stay 0 / -inf)."""
    T, H_q, D = q.shape
    H = case.k_pages.shape[2]
    G = H_q // H
    sm = 1.0 / math.sqrt(D) if sm_scale is None or sm_scale <= 0 else sm_scale
    out, wabs = np.zeros((T, H_q, D)), np.zeros((T, H_q, D))
    lse, qk = np.full((T, H_q), -np.inf), np.zeros((T, H_q))
    kv = {}
    for i, b, t in places(case.seq_lens, cu_q):
        if rows is not None and i not in rows:
            continue
        if b not in kv:
            kv = {b: sequence_kv(b, case, int(case.seq_lens[b]))}
        K, V = kv[b]
        lo = max(0, t - window + 1) if window else 0
        for hq in range(H_q):
            h = hq // G
            k, v, x = K[lo:t + 1, h], V[lo:t + 1, h], q[i, hq].astype(np.float64)
            z = (k @ x) * sm
            m = z.max()
            w = np.exp(z - m)
            out[i, hq] = (w @ v) / w.sum()
            wabs[i, hq] = (w @ np.abs(v)) / w.sum()
            lse[i, hq] = m + math.log(w.sum())
            qk[i, hq] = (np.abs(k) @ np.abs(x)).max() * sm
    return out, lse, wabs, qk
