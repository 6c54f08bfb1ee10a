"""Shared pieces of the tests of new tokens over the paged cache: cases with pages of all
four forms, device copies, and the error bounds of the attention."""

import dataclasses

import numpy as np

from mixed_precision_paged_gb300 import workloads as wl
from oracle import extend as oe
from oracle import micro as om

MICRO = 3


def make_case(lens, hq, hkv, d, fmt="mixed", scale_mode=1, seed=0, pool_pages=None, stride_pad=0):
    """A host DecodeCase (its q unused). fmt 'all': TARGET, E4M3, BASE and microscaled pages
    mixed; 'micro': a uniform microscaled pool in slots of its own size; else as
    workloads.make_decode_case. Rows behind a sequence and unused pages hold NaN."""
    if fmt not in ("all", "micro"):
        c = wl.make_decode_case(lens, hq, hkv, d, v_format=fmt, scale_mode=scale_mode, seed=seed, pool_pages=pool_pages)
    else:
        c = wl.make_decode_case(lens, hq, hkv, d, v_format="mixed", scale_mode=scale_mode, seed=seed,
                                pool_pages=pool_pages, p_compact=0.25 if fmt == "all" else 0.0,
                                p_base=0.25 if fmt == "all" else 0.0)
        rng = np.random.default_rng(seed + 1)
        n, mb = 16 * hkv * d, om.page_bytes(hkv, d)
        for p in range(c.num_pages):
            if c.page_mode[p] == 0 and (fmt == "micro" or rng.random() < 0.5):
                x = np.ascontiguousarray(c.v_pages[p][: 2 * n]).view("<f2").reshape(16, hkv, d)
                raw = om.encode_page(np.where(np.isfinite(x), x, 0))
                # rows behind the sequence: values of their own, far larger than the others
                dead = ~np.isfinite(x).all(axis=(1, 2))
                for h in range(hkv):
                    s = raw[h * (mb // hkv):(h + 1) * (mb // hkv)]
                    s[: 8 * d].reshape(16, -1)[dead] = 0x77
                    s[8 * d:].reshape(16, -1)[dead] = 127 + 13
                c.v_pages[p][:mb] = raw
                c.page_mode[p] = MICRO
        if fmt == "micro":
            c.v_pages = np.ascontiguousarray(c.v_pages[:, :mb])
            c.page_mode, c.uniform_mode, c.v_scales = None, MICRO, None
    if stride_pad:
        c.v_pages = np.concatenate([c.v_pages, np.full((c.num_pages, stride_pad), 0x7E, np.uint8)], 1)
    return c


def to_device(case):
    import torch

    def t(x):
        return torch.from_numpy(np.ascontiguousarray(x)).cuda() if isinstance(x, np.ndarray) else x
    return dataclasses.replace(case, **{f.name: t(getattr(case, f.name)) for f in dataclasses.fields(case) if f.name != "extra"})


def cu_of(new):
    return np.cumsum([0] + list(new)).astype(np.int32)


def run_extend(ekv, ctx, d, q, cu, max_q, window=0, sm_scale=0.0, total=None, stream=None, out=None, lse=None):
    import torch
    out = torch.full(q.shape, float("nan"), dtype=torch.float16, device="cuda") if out is None else out
    lse = torch.full(q.shape[:2], float("nan"), dtype=torch.float32, device="cuda") if lse is None else lse
    ekv.ekv_extend_attention(ctx.handle, q, d.k_pages, d.v_pages, d.v_page_stride, d.num_pages, d.v_scales,
                             d.scale_mode, d.page_mode, d.uniform_mode, d.block_table, int(d.block_table.shape[1]),
                             d.seq_lens, cu, d.batch, q.shape[0] if total is None else total, max_q, window, sm_scale,
                             out, lse, stream)
    return out, lse


def bounds(case, cu, ref, n_keys):
    """Bounds of |out| and |lse| errors. Steps that round: the fp32 scores (D products and sums:
    an absolute error of at most (D + 4) 2^-24 sm sum|q k|, which is a relative error of each weight; the
    exponent's argument and 2^x add 2^-20), the weights to fp16 (2^-11 relative, 2^-25 of the
    largest weight where subnormal), fp32 sums (n 2^-24) and the result to fp16 (2^-11, 2^-25)."""
    out, lse, wabs, qk = ref
    D = out.shape[-1]
    w = (D + 4) * 2.0 ** -24 * qk + 2.0 ** -20 + n_keys * 2.0 ** -24
    vmax = wabs.max(initial=1.0) * 8
    tol = 2.0 ** -11 * np.abs(out) + (2.0 ** -11 + 2 * w[..., None]) * wabs * 1.01 + n_keys * 2.0 ** -25 * vmax + 2.0 ** -24
    return tol, 2 * w + 2.0 ** -22 * np.abs(np.where(np.isfinite(lse), lse, 0))


def check(case, cu, q, out, lse, window=0, sm_scale=None, rows=None):
    """Compare with the oracle (all rows, or some)."""
    ref = oe.attention(q, case, cu, window=window, sm_scale=sm_scale, rows=rows)
    sel = np.array(sorted(rows)) if rows is not None else np.arange(int(cu[-1]))
    tol, ltol = bounds(case, cu, ref, min(window, int(case.seq_lens.max())) if window else int(case.seq_lens.max()))
    o, l = out.float().cpu().numpy().astype(np.float64)[sel], lse.cpu().numpy().astype(np.float64)[sel]
    assert np.all(np.isfinite(o)) and np.all(np.isfinite(l))
    err, lerr = np.abs(o - ref[0][sel]), np.abs(l - ref[1][sel])
    assert np.all(err <= tol[sel]), f"out off by {err.max():.3e}, {(err / tol[sel]).max():.2f} of the bound"
    assert np.all(lerr <= ltol[sel]), f"lse off by {lerr.max():.3e}, {(lerr / ltol[sel]).max():.2f} of the bound"
