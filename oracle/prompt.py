"""A prompt's way into the cache, in float64: rotary angles under a stretched context, the writer
that normalises heads and lets E4M3 scales grow, and causal attention of packed prompts.
Oracle only.

* angles: pair i of rope_dim / 2 makes w_i = theta^(-2 i / rope_dim) / (2 pi) turns a position; scaling divides w_i by
  `factor` wholly (linear), by the turns r = original_len * w_i over the original context (kept from `fast` turns on,
  divided up to `slow`, a straight line between), or with the line drawn over i instead (B. Peng et al., "YaRN:
  Efficient Context Window Extension of Large Language Models", 2023, for the idea of dividing by parts).
* writer: x_d / sqrt(mean x^2 + eps) * w_d per head row of q and k, then oracle.extend's rotation and pages. Growing scales: per
  (page, KV head) with a the largest finite magnitude written (infinities: 65504), row 0 written: s = fp32(max(a, 2^-24) / 448);
  else s 2^k, k >= 0 least with fp32(448 s) 2^k >= a, the earlier rows' codes re-encoded from value 2^-k.
* attention: query s of a prompt over its keys max(0, s - window + 1) .. s, KV head h_q // G.
"""

import math

import numpy as np

from . import e4m3, extend

PAGE_SIZE = 16
PLAIN, LINEAR, BY_TURNS, BY_DIMS = 0, 1, 2, 3


def turns(rope_dim, theta, scaling=PLAIN, factor=1.0, original_len=1.0, slow=1.0, fast=2.0):
    """float64 [rope_dim / 2]: whole turns of each pair from a position to the next."""
    out = []
    for i in range(rope_dim // 2):
        w = theta ** (-2.0 * i / rope_dim) / (2 * math.pi)
        g = 1.0
        if scaling == LINEAR:
            g = 0.0
        elif scaling == BY_TURNS:
            r = original_len * w
            g = 1.0 if r >= fast else 0.0 if r <= slow else (r - slow) / (fast - slow)
        elif scaling == BY_DIMS:
            def dim_of(r):
                return rope_dim * math.log(original_len / (2 * math.pi * r)) / (2 * math.log(theta))
            lo, hi = max(0, math.floor(dim_of(fast))), min(rope_dim - 1, math.ceil(dim_of(slow)))
            g = 1.0 if i <= lo else 0.0 if i >= hi else (hi - i) / (hi - lo)
        out.append(w * g + w / factor * (1 - g))
    return np.array(out)


def rope_table(first, n, rope_dim, magnitude=1.0, **cfg):
    """float64 [n][rope_dim]: cosines, then sines."""
    x = np.arange(first, first + n, dtype=np.float64)[:, None] * turns(rope_dim, **cfg)
    a = 2 * math.pi * (x - np.floor(x))
    return magnitude * np.concatenate([np.cos(a), np.sin(a)], 1)


def normed(x, weight, eps):
    """Head rows [..., D] normalised; unchanged without a weight."""
    x = x.astype(np.float64)
    if weight is None:
        return x
    return x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * weight.astype(np.float64)


def grow(v_new, v_pages, v_scales, page_mode, uniform_mode, block_table, seq_lens, cu_q, D):
    """(V pool bytes, scales) before the new rows are encoded: scales made or grown, earlier codes brought under them."""
    vp, sc = np.array(v_pages, copy=True), np.array(v_scales, dtype=np.float32, copy=True)
    H = v_new.shape[1]
    rows = {}
    for i, b, t in extend.places(seq_lens, cu_q):
        rows.setdefault(int(block_table[b][t // PAGE_SIZE]), []).append((t % PAGE_SIZE, i))
    for page, at in rows.items():
        if (uniform_mode if page_mode is None else int(page_mode[page])) != 1:
            continue
        r0 = min(r for r, _ in at)
        for h in range(H):
            x = np.abs(v_new[[i for _, i in at], h].astype(np.float64))
            a = np.minimum(np.where(np.isnan(x), 0.0, x), 65504.0).max()
            if r0 == 0:
                sc[page, h] = np.float32(max(a, 2.0 ** -24) / 448)
                continue
            with np.errstate(over="ignore"):
                top = float(np.float32(448.0 * float(sc[page, h])))
            k = 0
            while top * 2.0 ** k < a:
                k += 1
            if k:
                codes = vp[page, : PAGE_SIZE * H * D].reshape(PAGE_SIZE, H, D)
                y = e4m3.decode(codes[:r0, h]) * 2.0 ** -k
                nan = np.isnan(y)
                codes[:r0, h] = np.where(nan, 0x7F, e4m3.encode_rne_satfinite(np.where(nan, 0.0, y)))
                sc[page, h] = np.float32(float(sc[page, h]) * 2.0 ** k)
    return vp, sc


def append(q, k_new, v_new, q_weight, k_weight, eps, rope, style, k_pages, v_pages, v_scales, scale_mode, grow_scales,
           page_mode, uniform_mode, block_table, seq_lens, cu_q):
    """q' and K pool float64 (not rounded), V pool bytes and scales (exact)."""
    sc = v_scales
    if grow_scales:
        v_pages, sc = grow(v_new, v_pages, v_scales, page_mode, uniform_mode, block_table, seq_lens, cu_q, k_new.shape[2])
    qo, kp, vp = extend.append(normed(q, q_weight, eps), normed(k_new, k_weight, eps), v_new, rope, style, k_pages, v_pages, sc,
                               scale_mode, page_mode, uniform_mode, block_table, seq_lens, cu_q)
    return qo, kp, vp, sc


def attention(q, k, v, cu, window=0, sm_scale=None):
    """out, lse, and for error bounds wabs and qk as in oracle.extend.attention, of packed rows
    q [T][H_q][D], k and v [T][H_kv][D]; rows of no prompt stay 0 / -inf."""
    T, H_q, D = q.shape
    G = H_q // k.shape[1]
    sm = 1.0 / math.sqrt(D) if sm_scale is None or sm_scale <= 0 else sm_scale
    out, wabs = np.zeros((T, H_q, D)), np.zeros((T, H_q, D))
    lse, qk = np.full((T, H_q), -np.inf), np.zeros((T, H_q))
    for a, b in zip(cu, cu[1:]):
        a, b = int(a), int(b)
        i = np.arange(b - a)
        seen = i[None, :] <= i[:, None]
        if window:
            seen &= i[None, :] > i[:, None] - window
        for hq in range(H_q if b > a else 0):
            x, K, V = (y[a:b, h].astype(np.float64) for y, h in ((q, hq), (k, hq // G), (v, hq // G)))
            z = np.where(seen, x @ K.T * sm, -np.inf)
            m = z.max(1, keepdims=True)
            w = np.exp(z - m)
            s = w.sum(1, keepdims=True)
            out[a:b, hq], wabs[a:b, hq] = (w / s) @ V, (w / s) @ np.abs(V)
            lse[a:b, hq] = (m + np.log(s))[:, 0]
            qk[a:b, hq] = np.where(seen, np.abs(x) @ np.abs(K).T, 0.0).max(1) * sm
    return out, lse, wabs, qk
