"""Microscaled FP4 value pages. Oracle only, exact.

Definition (the element and scale formats are the OCP Microscaling Formats v1.0 E2M1 and
E8M0; the choice of the scale is this library's):

* a block is 32 consecutive values of one token's row of one KV head;
* its scale is 2^k, k the least integer in [-24, 13] with absmax <= 6 * 2^k (13 when none);
* a code is the E2M1 value (0, .5, 1, 1.5, 2, 3, 4, 6 and a sign) nearest to x / 2^k, ties to
  the even code, saturating at 6, the sign of x kept (-0.0 -> 8);
* a page's bytes: for each KV head the 16 rows of D / 2 code bytes (element 2i in the low half of
  byte i), then the 16 rows of D / 32 scale bytes, k + 127.
"""

import numpy as np

PAGE_SIZE = 16
MODE_TARGET_FP16 = 0
MODE_MICRO_FP4 = 3
BLOCK = 32
K_MIN, K_MAX = -24, 13
VALUES = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def page_bytes(H_kv, D):
    return PAGE_SIZE * H_kv * (D // 2 + D // BLOCK)


def encode_block(x):
    """(codes uint8 [32], k) of 32 finite values; infinite values saturate, a NaN becomes +6."""
    x = np.asarray(x, dtype=np.float64)
    finite_max = np.inf if not np.all(np.isfinite(x)) else np.abs(x).max()
    k = next((k for k in range(K_MIN, K_MAX + 1) if finite_max <= 6.0 * 2.0 ** k), K_MAX)
    codes = np.zeros(x.size, dtype=np.uint8)
    for i, v in enumerate(x):
        if np.isnan(v):
            codes[i] = 7
            continue
        y = min(abs(v) / 2.0 ** k, 6.0)
        d = np.abs(VALUES - y)
        best = np.flatnonzero(d == d.min())
        c = int(best[0]) if best.size == 1 else int(best[best % 2 == 0][0])
        codes[i] = c | (8 if np.signbit(v) else 0)
    return codes, k


def encode_rows(x):
    """Vectorised ``encode_block`` over the last axis of finite float64 x [..., D]:
    codes uint8 [..., D], k int [..., D / 32]."""
    b = np.asarray(x, dtype=np.float64).reshape(*x.shape[:-1], -1, BLOCK)
    a = np.abs(b).max(-1)
    k = np.full(a.shape, K_MIN)
    for e in range(K_MIN, K_MAX):
        k = np.where(a > 6.0 * 2.0 ** e, e + 1, k)
    y = np.minimum(np.abs(b) / (2.0 ** k.astype(np.float64))[..., None], 6.0)
    hi = np.clip(np.searchsorted(VALUES, y), 1, 7)
    lo = hi - 1
    d_hi, d_lo = VALUES[hi] - y, y - VALUES[lo]
    c = np.where((d_hi < d_lo) | ((d_hi == d_lo) & (hi % 2 == 0)), hi, lo).astype(np.uint8)
    c |= np.where(np.signbit(b), 8, 0).astype(np.uint8)
    return c.reshape(x.shape), k


def encode_page(x):
    """Bytes [page_bytes] of the values x [16][H_kv][D]."""
    S, H, D = x.shape
    out = []
    for h in range(H):
        c, k = encode_rows(x[:, h].astype(np.float64))
        out.append((c[:, 0::2] | (c[:, 1::2] << 4)).reshape(-1))
        out.append((k + 127).astype(np.uint8).reshape(-1))
    return np.concatenate(out)


def decode_page(raw, H_kv, D):
    """float64 [16][H_kv][D] of a page's bytes; a scale byte outside the range gives zeros."""
    n = page_bytes(1, D)
    out = np.zeros((PAGE_SIZE, H_kv, D))
    for h in range(H_kv):
        s = np.asarray(raw[h * n:(h + 1) * n])
        codes = s[: PAGE_SIZE * D // 2].reshape(PAGE_SIZE, D // 2)
        k = s[PAGE_SIZE * D // 2:].reshape(PAGE_SIZE, D // BLOCK).astype(np.int64) - 127
        v = np.empty((PAGE_SIZE, D))
        for at, c in ((0, codes & 15), (1, codes >> 4)):
            v[:, at::2] = np.where(c & 8, -1.0, 1.0) * VALUES[c & 7]
        good = np.repeat((k >= K_MIN) & (k <= K_MAX), BLOCK, axis=1)
        out[:, h] = np.where(good, v * np.repeat(2.0 ** k.astype(np.float64), BLOCK, axis=1), 0.0)
    return out


def demote_pages(v_pages, page_ids, page_mode, H_kv, D):
    """Oracle of ``ekv_demote_pages_micro``: (v_pages', page_mode', skipped non-finite pages)."""
    v, mode, bad = np.array(v_pages, copy=True), np.array(page_mode, copy=True), []
    n = PAGE_SIZE * H_kv * D
    for p in page_ids:
        if mode[p] != MODE_TARGET_FP16:
            continue
        x = np.ascontiguousarray(v[p][: 2 * n]).view("<f2").reshape(PAGE_SIZE, H_kv, D)
        if not np.all(np.isfinite(x)):
            bad.append(int(p))
            continue
        v[p][: page_bytes(H_kv, D)] = encode_page(x)
        mode[p] = MODE_MICRO_FP4
    return v, mode, bad


def expand_pages(v_pages, page_ids, page_mode, H_kv, D):
    """Oracle of ``ekv_expand_pages_micro``: (v_pages', page_mode')."""
    v, mode = np.array(v_pages, copy=True), np.array(page_mode, copy=True)
    n = PAGE_SIZE * H_kv * D
    for p in page_ids:
        if mode[p] != MODE_MICRO_FP4:
            continue
        x = decode_page(v[p], H_kv, D).astype(np.float16)
        v[p][: 2 * n] = x.reshape(-1).view(np.uint8)
        mode[p] = MODE_TARGET_FP16
    return v, mode
