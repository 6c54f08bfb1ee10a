"""Cases of the paged-cache operators that take new tokens: what they compute in plain
form, and the calls of the ekv library that compute the same.

Three operators, over one page layout (include/ekv.h: 16-token pages, FP16 keys, value
pages in FP16, E4M3, BASE or microscaled FP4 form):

* append   the new tokens of every sequence (one or many each): their queries and keys are
           rotated by the position (rotary embedding from a cos / sin table), keys and
           values written into the pages of the cache;
* extend   attention of those new tokens over the paged cache: causal among themselves,
           over everything cached before them, or over a sliding window of it;
* micro    value pages quantised in place to microscaled FP4 (blocks of 32 values with a
           power-of-two scale) and expanded again into the FP16 values that they stand for.
"""

import functools
import math
import random

import numpy as np
import torch

own = False

PAGE = 16
TARGET, E4M3, BASE, MICRO = 0, 1, 2, 3
PER_TENSOR, PER_PAGE_HEAD = 0, 1
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ------------------------------------------------------------------------------- cases
def _append(name, batch, new, ctx, hq, hkv, d, rope_dim, style, fmt, lens, fused):
    return dict(name=name, op="append", batch=batch, new_lo=new[0], new_hi=new[1], ctx_lo=ctx[0], ctx_hi=ctx[1],
                hq=hq, hkv=hkv, d=d, rope_dim=rope_dim, style=style, fmt=fmt, lens=lens, fused=fused)


def _extend(name, batch, new, ctx, hq, hkv, d, window, fmt, scale, lens):
    return dict(name=name, op="extend", batch=batch, new_lo=new[0], new_hi=new[1], ctx_lo=ctx[0], ctx_hi=ctx[1],
                hq=hq, hkv=hkv, d=d, window=window, fmt=fmt, scale=scale, lens=lens)


def _micro(name, pool, pages, hkv, d):
    return dict(name=name, op="micro", pool=pool, pages=pages, hkv=hkv, d=d)


def listed():
    """`new` and `ctx`: the range of each sequence's new and earlier tokens; `lens`: which
    draw of the lengths; `scale`: one value scale per tensor (0) or per page and head (1)."""
    return [
        # one decode step of a batch of 32: the latency of the writer
        _append("append step 32", 32, (1, 1), (512, 1024), 32, 8, 128, 128, 0, "e4m3", 1, True),
        # draft tokens and short chunks of many users, half of each head rotated in
        # interleaved pairs, four key heads
        _append("append ragged 96", 96, (1, 333), (0, 700), 32, 4, 128, 64, 1, "e4m3", 2, False),
        # the prompts of a whole admission
        _append("append prompts 8x8192", 8, (8192, 8192), (0, 0), 32, 8, 128, 128, 0, "fp16", 3, True),
        # the smallest decode: two short contexts
        _extend("extend tiny", 2, (1, 1), (36, 99), 4, 2, 64, 0, "e4m3", 0, 4),
        # one decode step at a batch of 32 and 8K of context
        _extend("extend decode 32x8k", 32, (1, 1), (8192, 8319), 32, 8, 128, 0, "e4m3", 0, 5),
        # verification of four draft tokens and the last accepted one, pages of every form
        _extend("extend verify 48", 48, (5, 5), (512, 8192), 32, 8, 128, 0, "mixed", 1, 6),
        # many users, most of them short, eight query heads a key head, values in 4 bits
        _extend("extend micro 200", 200, (1, 4), (1, 4096), 32, 4, 128, 0, "micro", 0, 7),
        # chunks of four prompts behind 8K of cached prefix
        _extend("extend chunks 4x512", 4, (512, 512), (7900, 8192), 32, 8, 128, 0, "fp16", 0, 8),
        # ragged chunks under a sliding window, pages of every form
        _extend("extend window 1024", 12, (1, 700), (2000, 6000), 32, 8, 128, 1024, "mixed", 1, 9),
        # a long chunk of one long prompt, values in 8 bits
        _extend("extend chunk 4096 of 20k", 1, (4096, 4096), (16384, 16384), 32, 8, 128, 0, "e4m3", 1, 10),
        # a few pages that an eviction policy moves down
        _micro("micro 48 pages", 256, 48, 8, 128),
        # half of a pool of 16,384 pages
        _micro("micro 8192 pages", 16384, 8192, 8, 128),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    op = rng.choice(("append", "append", "extend", "extend", "extend", "extend", "micro"))
    hq, hkv, d = rng.choice(((32, 8, 128), (32, 8, 128), (32, 4, 128), (16, 8, 64), (4, 2, 64), (8, 1, 128), (24, 4, 128),
                             (8, 8, 64)))
    lens = rng.randrange(1, 1 << 20)
    if op == "micro":
        pages = _log_int(rng, 1, 8192)
        return dict(_micro("", pages + _log_int(rng, 1, 8192), pages, hkv, d))
    batch = _log_int(rng, 1, 200)
    if op == "append":
        hi = _log_int(rng, 1, max(1, 65536 // batch))
        lo = rng.choice((1, hi, rng.randint(1, hi)))
        c = _append("", batch, (lo, hi), (0, _log_int(rng, 1, 2048)), hq, hkv, d, rng.choice((d, d, d // 2, 16)),
                    rng.randrange(2), rng.choice(("fp16", "e4m3")), lens, rng.random() < 0.5)
    else:
        fmt = rng.choice(("fp16", "e4m3", "mixed", "mixed", "micro"))
        while True:
            batch = _log_int(rng, 1, 200)
            hi = rng.choice((1, rng.randint(2, 8), _log_int(rng, 9, 4096)))
            ctx = _log_int(rng, 16, 20480)
            if batch * hq * hi * (ctx + hi) <= 32 * 4096 * 20480 and batch * (ctx + hi) * hkv <= 32 * 8320 * 8:
                break
        window = rng.choice((0, 0, 0, _log_int(rng, 1, 4096)))
        c = _extend("", batch, (rng.choice((1, hi)), hi), (rng.choice((0, ctx // 2, ctx)), ctx), hq, hkv, d, window, fmt,
                    rng.randrange(2), lens)
    del c["name"]
    return c


def _lengths(case):
    """(new tokens, total tokens) of every sequence: they go by the case alone."""
    r = random.Random(case["lens"])
    new = [r.randint(case["new_lo"], case["new_hi"]) for _ in range(case["batch"])]
    return new, [r.randint(case["ctx_lo"], case["ctx_hi"]) + n for n in new]


# ----------------------------------------------------------------------------- formats
def _micro_stride(hkv, d):
    return PAGE * hkv * (d // 2 + d // 32)


def _micro_codes(x):
    """Sign and E2M1 code (4 bits) and biased scale exponent of blocks of 32 float32 values."""
    b = x.unflatten(-1, (-1, 32))
    m, e = torch.frexp(b.abs().amax(-1))
    k = (e - 3 + (m > 0.75).to(e.dtype)).clamp(-24, 13)     # the least k with absmax <= 6 * 2^k
    y = torch.ldexp(b.abs(), -k.unsqueeze(-1))
    code = sum(c.to(torch.uint8) for c in (y > 0.25, y >= 0.75, y > 1.25, y >= 1.75, y > 2.5, y >= 3.5, y > 5.0))
    code = code | (torch.signbit(b).to(torch.uint8) << 3)
    return code.flatten(-2), (k + 127).to(torch.uint8)


def _micro_values(code, scale):
    """float32 values of 4-bit codes [..., n] under biased scale exponents [..., n / 32]."""
    lut = torch.tensor(E2M1, device=code.device)
    v = lut[(code & 7).long()]
    v = torch.where((code & 8) != 0, -v, v).unflatten(-1, (-1, 32))
    return torch.ldexp(v, (scale.to(torch.int32) - 127).unsqueeze(-1)).flatten(-2)


def _micro_pack(x):
    """[P][16][H][D] float32 -> [P][H * 16 * (D / 2 + D / 32)] bytes: per KV head the 16 rows
    of codes (two to a byte, the first in the low half), then the 16 rows of scales."""
    code, scale = _micro_codes(x.transpose(1, 2))
    two = code.unflatten(-1, (-1, 2))
    packed = (two[..., 0] | (two[..., 1] << 4)).flatten(-2)
    return torch.cat((packed, scale.flatten(-2)), -1).flatten(1)


def _micro_unpack(raw, hkv, d):
    """The float32 values [..., 16, H, D] of page bytes [..., >= micro page]."""
    raw = raw[..., :_micro_stride(hkv, d)].unflatten(-1, (hkv, -1))
    packed = raw[..., :PAGE * d // 2].unflatten(-1, (PAGE, d // 2))
    scale = raw[..., PAGE * d // 2:].unflatten(-1, (PAGE, d // 32))
    code = torch.stack((packed & 15, packed >> 4), -1).flatten(-2)
    return _micro_values(code, scale).transpose(-3, -2)


def _pool(case, pages, gen):
    """K pool, V pool bytes, modes and scales of `pages` pages in the case's format."""
    hkv, d, n = case["hkv"], case["d"], PAGE * case["hkv"] * case["d"]
    k = torch.randn((pages, PAGE, hkv, d), generator=gen, device="cuda", dtype=torch.float16)
    # values with an offset of their own in every channel, as projections have them
    offset = 0.5 * torch.randn((hkv, d), generator=gen, device="cuda")
    fmt, scale_mode = case["fmt"], case.get("scale", PER_PAGE_HEAD)
    stride = {"e4m3": n, "micro": _micro_stride(hkv, d)}.get(fmt, 2 * n)
    v = torch.empty((pages, stride), dtype=torch.uint8, device="cuda")
    modes = None
    if fmt == "mixed":
        modes = torch.randint(0, 4, (pages,), generator=gen, device="cuda", dtype=torch.uint8)
    scales = None
    if fmt in ("e4m3", "mixed"):
        if scale_mode == PER_TENSOR:
            scales = torch.full((1,), 6.0 / 448, device="cuda")
        else:
            scales = torch.empty((pages, hkv), device="cuda")
    for p0 in range(0, pages, 4096):
        x = torch.randn((min(4096, pages - p0), PAGE, hkv, d), generator=gen, device="cuda") + offset
        m = slice(p0, p0 + x.shape[0])
        if scales is not None and scale_mode == PER_PAGE_HEAD:
            scales[m] = x.abs().amax((1, 3)) / 448
        forms = []
        if fmt in ("fp16", "mixed"):
            forms.append((TARGET, x.half().flatten(1).view(torch.uint8)))
        if fmt in ("e4m3", "mixed"):
            s = scales if scale_mode == PER_TENSOR else scales[m].view(-1, 1, hkv, 1)
            forms.append((E4M3, (x / s).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8).flatten(1)))
        if fmt in ("base", "mixed"):
            forms.append((BASE, (x.half().view(torch.int16) >> 8).to(torch.uint8).flatten(1)))
        if fmt in ("micro", "mixed"):
            forms.append((MICRO, _micro_pack(x)))
        for mode, raw in forms:
            if modes is None:
                v[m, :raw.shape[1]] = raw
            else:
                v[m, :raw.shape[1]] = torch.where((modes[m] == mode)[:, None], raw, v[m, :raw.shape[1]])
    uniform = {"fp16": TARGET, "e4m3": E4M3, "base": BASE, "micro": MICRO, "mixed": TARGET}[fmt]
    return dict(k_pages=k, v_pages=v, modes=modes, scales=scales, uniform=uniform,
                scale_mode=scale_mode if scales is not None else PER_TENSOR)


def _tables(case, gen, lens):
    """Block table over a random permutation of the pool; entries past a sequence's pages repeat its last."""
    need = [max(1, -(-n // PAGE)) for n in lens]
    perm = torch.randperm(sum(need), generator=gen, device="cuda").to(torch.int32)
    first = torch.tensor(np.cumsum([0] + need[:-1]), device="cuda")
    last = torch.tensor(need, device="cuda") - 1
    j = torch.arange(max(need), device="cuda")
    return perm[first[:, None] + torch.minimum(j[None, :], last[:, None])].contiguous(), sum(need)


# ----------------------------------------------------------------------------- prepare
def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    hkv, d = case["hkv"], case["d"]
    if case["op"] == "micro":
        v = torch.empty((case["pool"], PAGE, hkv, d), dtype=torch.float16, device="cuda")
        offset = 0.5 * torch.randn((hkv, d), generator=gen, device="cuda")
        for p0 in range(0, case["pool"], 4096):
            v[p0:p0 + 4096] = torch.randn(v[p0:p0 + 4096].shape, generator=gen, device="cuda") + offset
        ids = torch.randperm(case["pool"], generator=gen, device="cuda")[:case["pages"]].to(torch.int32)
        return dict(case=case, v=v, ids=ids, modes=torch.zeros(case["pool"], dtype=torch.uint8, device="cuda"))
    hq = case["hq"]
    new, lens = _lengths(case)
    total = sum(new)
    st = dict(case=case, total=total, max_new=max(new),
              cu=torch.tensor(np.cumsum([0] + new), dtype=torch.int32, device="cuda"),
              lens=torch.tensor(lens, dtype=torch.int32, device="cuda"))
    st["table"], pages = _tables(case, gen, lens)
    st.update(_pool(case, pages, gen))
    if case["op"] == "extend":
        # queries sharp enough that attention prefers some keys
        st["q"] = 1.5 * torch.randn((total, hq, d), generator=gen, device="cuda", dtype=torch.float16)
        return st
    if case["fused"]:                                       # one projection's rows: q, k and v side by side
        rows = torch.randn((total, hq + 2 * hkv, d), generator=gen, device="cuda", dtype=torch.float16)
        st["q"], st["k"], st["v"] = rows.split((hq, hkv, hkv), 1)
    else:
        st["q"] = torch.randn((total, hq, d), generator=gen, device="cuda", dtype=torch.float16)
        st["k"] = torch.randn((total, hkv, d), generator=gen, device="cuda", dtype=torch.float16)
        st["v"] = torch.randn((total, hkv, d), generator=gen, device="cuda", dtype=torch.float16)
    half = case["rope_dim"] // 2
    freq = 10000.0 ** (-torch.arange(half, dtype=torch.float64, device="cuda") / half)
    angle = torch.arange(max(lens), dtype=torch.float64, device="cuda")[:, None] * freq
    st["rope"] = torch.cat((angle.cos(), angle.sin()), 1).float().contiguous()
    st["q_out"] = torch.empty((total, hq, d), dtype=torch.float16, device="cuda")
    return st


# ------------------------------------------------------------------------- plain forms
def _places(s):
    """Sequence, index among the new tokens, and position of every new token."""
    i = torch.arange(s["total"], device="cuda")
    b = torch.searchsorted(s["cu"][1:].contiguous(), i.to(torch.int32), right=True)
    r = i - s["cu"][b].long()
    return b, r, r + s["lens"][b].long() - (s["cu"][b + 1] - s["cu"][b]).long()


def _rotate(x, cos, sin, style, dim):
    a, rest = x[..., :dim].float(), x[..., dim:].float()
    if style == 0:
        u, w = a[..., :dim // 2], a[..., dim // 2:]
        a = torch.cat((u * cos - w * sin, w * cos + u * sin), -1)
    else:
        u, w = a[..., 0::2], a[..., 1::2]
        a = torch.stack((u * cos - w * sin, w * cos + u * sin), -1).flatten(-2)
    return torch.cat((a, rest), -1).half()


def _plain_append(s):
    c = s["case"]
    hkv, d, dim = c["hkv"], c["d"], c["rope_dim"]
    b, r, t = _places(s)
    cos, sin = s["rope"][t][:, None].split(dim // 2, -1)
    s["q_out"].copy_(_rotate(s["q"], cos, sin, c["style"], dim))
    page, row = s["table"][b, t // PAGE].long(), t % PAGE
    s["k_pages"][page, row] = _rotate(s["k"], cos, sin, c["style"], dim)
    if c["fmt"] == "fp16":
        s["v_pages"].view(torch.float16).view(-1, PAGE, hkv, d)[page, row] = s["v"]
    else:
        y = (s["v"].float() / s["scales"][page][:, :, None]).clamp(-448, 448)
        s["v_pages"].view(-1, PAGE, hkv, d)[page, row] = y.to(torch.float8_e4m3fn).view(torch.uint8)


def _plain_values(s, page):
    """float32 values [..., 16, H, D] of the pages."""
    c = s["case"]
    hkv, d, n = c["hkv"], c["d"], PAGE * c["hkv"] * c["d"]
    raw, fmt, shape = s["v_pages"][page], c["fmt"], (PAGE, hkv, d)
    if fmt == "fp16":
        return raw.view(torch.float16).float().unflatten(-1, shape)
    if fmt == "micro":
        return _micro_unpack(raw, hkv, d)
    scale = s["scales"] if s["scale_mode"] == PER_TENSOR else s["scales"][page][..., None, :, None]
    e4m3 = raw[..., :n].view(torch.float8_e4m3fn).float().unflatten(-1, shape) * scale
    if fmt == "e4m3":
        return e4m3
    mode = s["modes"][page][..., None, None, None]
    v = torch.where(mode == E4M3, e4m3, raw.view(torch.float16).float().unflatten(-1, shape))
    base = (raw[..., :n].to(torch.int16) << 8).view(torch.float16).float().unflatten(-1, shape)
    v = torch.where(mode == BASE, base, v)
    return torch.where(mode == MICRO, _micro_unpack(raw, hkv, d), v)


def _plain_extend(s):
    c = s["case"]
    hq, hkv, d, g = c["hq"], c["hkv"], c["d"], c["hq"] // c["hkv"]
    b, r, _ = _places(s)
    page = s["table"].long()
    k = s["k_pages"][page].float().flatten(1, 2)            # [B][keys][H][D]
    v = _plain_values(s, page).flatten(1, 2)
    n = (s["cu"][1:] - s["cu"][:-1]).long()
    q = torch.zeros((c["batch"], s["max_new"], hkv, g, d), device="cuda")
    q[b, r] = s["q"].float().view(-1, hkv, g, d)
    score = torch.einsum("bqhgd,bkhd->bhgqk", q, k) / math.sqrt(d)
    pos = torch.arange(s["max_new"], device="cuda")[None, :] + (s["lens"].long() - n)[:, None]
    key = torch.arange(k.shape[1], device="cuda")
    seen = key <= pos[..., None]
    if c["window"]:
        seen &= key > pos[..., None] - c["window"]
    score.masked_fill_(~seen[:, None, None], -math.inf)
    top = score.amax(-1, keepdim=True)
    score.sub_(top).exp_()
    total = score.sum(-1, keepdim=True)
    out = (torch.einsum("bhgqk,bkhd->bhgqd", score, v) / total).permute(0, 3, 1, 2, 4)[b, r].reshape(-1, hq, d).half()
    lse = (top + total.log())[..., 0].permute(0, 3, 1, 2)[b, r].reshape(-1, hq)
    return out, lse


def _plain_micro(s):
    ids = s["ids"].long()
    x = s["v"][ids].float().transpose(1, 2)
    s["v"][ids] = _micro_values(*_micro_codes(x)).transpose(1, 2).half()


# --------------------------------------------------------------------------------- run
@functools.lru_cache(maxsize=None)
def _context(hq, hkv, d):
    """The handle that a program keeps for a model's head layout."""
    from mixed_precision_paged_gb300 import ekv
    return ekv, ekv.Context(hq, hkv, d, 256)


def run(state):
    s, c = state, state["case"]
    if c["op"] == "micro":
        if own:
            ekv, ctx = _context(c["hkv"], c["hkv"], c["d"])
            stride = 2 * PAGE * c["hkv"] * c["d"]
            args = (ctx.handle, s["v"], stride, c["pool"], s["ids"], c["pages"], s["modes"])
            ekv.ekv_demote_pages_micro(*args)
            ekv.ekv_expand_pages_micro(*args)
        else:
            _plain_micro(s)
        return {"values": s["v"], "modes": s["modes"]}
    if c["op"] == "append":
        if own:
            ekv, ctx = _context(c["hq"], c["hkv"], c["d"])
            ekv.ekv_append_kv_rope(ctx.handle, s["q"], s["k"], s["v"], s["q"].stride(0), s["k"].stride(0), s["v"].stride(0),
                                   s["rope"], s["rope"].shape[0], c["rope_dim"], c["style"], s["q_out"], s["k_pages"],
                                   s["v_pages"], s["v_pages"].shape[1], s["k_pages"].shape[0], s["scales"],
                                   s["scale_mode"], s["modes"], s["uniform"], s["table"], s["table"].shape[1],
                                   s["lens"], s["cu"], c["batch"], s["total"])
        else:
            _plain_append(s)
        kind = torch.float16 if c["fmt"] == "fp16" else torch.float8_e4m3fn
        return {"q": s["q_out"], "k_pages": s["k_pages"], "v_pages": s["v_pages"].view(kind)}
    if own:
        ekv, ctx = _context(c["hq"], c["hkv"], c["d"])
        out = torch.empty_like(s["q"])
        lse = torch.empty(s["q"].shape[:2], dtype=torch.float32, device="cuda")
        ekv.ekv_extend_attention(ctx.handle, s["q"], s["k_pages"], s["v_pages"], s["v_pages"].shape[1],
                                 s["k_pages"].shape[0], s["scales"], s["scale_mode"], s["modes"], s["uniform"],
                                 s["table"], s["table"].shape[1], s["lens"], s["cu"], c["batch"], s["total"],
                                 s["max_new"], c["window"], 0.0, out, lse)
    else:
        out, lse = _plain_extend(s)
    return {"out": out, "lse": lse}


# -------------------------------------------------------------------------------- work
def work(case):
    hkv, d = case["hkv"], case["d"]
    if case["op"] == "micro":                               # FP16 to 17/32 of a byte a value, and back
        n = case["pages"] * PAGE * hkv * d
        return {"bytes": 2 * n * (2 + 17 / 32), "flops": 0}
    hq = case["hq"]
    new, lens = _lengths(case)
    value = {"fp16": 2, "e4m3": 1, "base": 1, "micro": 17 / 32, "mixed": (2 + 1 + 1 + 17 / 32) / 4}[case["fmt"]]
    if case["op"] == "append":
        spans = sorted((l - n, l) for n, l in zip(new, lens))
        rows, end = 0, 0                                    # rows of the table that any token reads
        for lo, hi in spans:
            rows += max(0, hi - max(lo, end))
            end = max(end, hi)
        return {"bytes": sum(new) * d * (2 * 2 * hq + 2 * 2 * hkv + (2 + value) * hkv) + rows * 4 * case["rope_dim"], "flops": 0}
    w = case["window"] or (1 << 30)
    keys = sum(l - max(0, l - n - w + 1) for n, l in zip(new, lens))
    pairs = sum(sum(min(l - n + r + 1, w) for r in range(n)) for n, l in zip(new, lens))
    return {"bytes": keys * hkv * d * (2 + value) + sum(new) * hq * (4 * d + 4), "flops": 4 * d * hq * pairs}


# ------------------------------------------------------------------------------- exact
def _byte_table(mode):
    """The 256 values of a byte as an E4M3 code, or as the high byte of an FP16 word."""
    out = []
    for b in range(256):
        sign, bits = (-1.0 if b & 128 else 1.0), b & 127
        if mode == E4M3:
            e, m = bits >> 3, bits & 7
            val = math.nan if bits == 127 else (8 + m) * 2.0 ** (e - 10) if e else m * 2.0 ** -9
        else:
            e, m = bits >> 2, bits & 3
            val = (math.nan if m else math.inf) if e == 31 else (4 + m) * 2.0 ** (e - 17) if e else m * 2.0 ** -16
        out.append(sign * val)
    return torch.tensor(out, dtype=torch.float64, device="cuda")


def _nearest(y, grid):
    """The nearest of an ascending grid of magnitudes, the even index at a tie, beyond its end its end; y >= 0 in float64."""
    hi = torch.searchsorted(grid, y).clamp(1, len(grid) - 1)
    lo = hi - 1
    up = (y - grid[lo] > grid[hi] - y) | ((y - grid[lo] == grid[hi] - y) & (hi % 2 == 0))
    return torch.where(up, grid[hi], grid[lo])


def _exact_micro(x):
    """What blocks of 32 values (the last axis, in float64) stand for after their quantisation."""
    y = x.reshape(*x.shape[:-1], -1, 32)
    a = y.abs().amax(-1, keepdim=True)
    step = torch.full_like(a, 2.0 ** -24)
    for k in range(-23, 14):
        step = torch.where(a > 6 * 2.0 ** (k - 1), torch.full_like(a, 2.0 ** k), step)
    grid = torch.tensor(E2M1, dtype=torch.float64, device=x.device)
    return (torch.copysign(_nearest(y.abs() / step, grid), y) * step).reshape(x.shape)


def _exact_values(s, pages, h):
    """float64 values [keys][D] of one sequence's pages for KV head h."""
    c = s["case"]
    hkv, d = c["hkv"], c["d"]
    raw, got = s["v_pages"][pages], []
    modes = [s["uniform"]] * len(pages) if s["modes"] is None else s["modes"][pages].tolist()
    v = torch.empty((len(pages), PAGE, d), dtype=torch.float64, device="cuda")
    for mode in set(modes):
        at = torch.tensor([i for i, m in enumerate(modes) if m == mode], device="cuda")
        r = raw[at]
        if mode == TARGET:
            got = r.view(torch.float16).view(-1, PAGE, hkv, d)[:, :, h].double()
        elif mode == MICRO:
            each = PAGE * d // 2 + PAGE * d // 32
            slab = r[:, h * each:(h + 1) * each]
            codes = slab[:, :PAGE * d // 2].reshape(-1, PAGE, d // 2).long()
            power = 2.0 ** (slab[:, PAGE * d // 2:].reshape(-1, PAGE, d // 32).double() - 127)
            lut = torch.tensor(list(E2M1) + [-x for x in E2M1], dtype=torch.float64, device="cuda")
            got = torch.empty((len(at), PAGE, d), dtype=torch.float64, device="cuda")
            got[..., 0::2], got[..., 1::2] = lut[codes % 16], lut[codes // 16]
            got *= power.repeat_interleave(32, -1)
        else:
            got = _byte_table(mode)[r[:, :PAGE * hkv * d].view(-1, PAGE, hkv, d)[:, :, h].long()]
            if mode == E4M3:
                got = got * (s["scales"].double() if s["scale_mode"] == PER_TENSOR else s["scales"].double()[pages[at], h].view(-1, 1, 1))
        v[at] = got
    return v.view(-1, d)


def _exact_extend(s):
    c = s["case"]
    hq, hkv, d, g = c["hq"], c["hkv"], c["d"], c["hq"] // c["hkv"]
    out = torch.empty((s["total"], hq, d), dtype=torch.float64, device="cuda")
    lse = torch.empty((s["total"], hq), dtype=torch.float64, device="cuda")
    cu, lens = s["cu"].tolist(), s["lens"].tolist()
    for b, n in enumerate(lens):
        pages = s["table"][b, :-(-n // PAGE)].long()
        first = n - (cu[b + 1] - cu[b])
        for h in range(hkv):
            k = s["k_pages"][pages, :, h].double().view(-1, d)[:n]
            v = _exact_values(s, pages, h)[:n]
            for r0 in range(cu[b], cu[b + 1], 512):
                r1 = min(r0 + 512, cu[b + 1])
                q = s["q"][r0:r1, h * g:(h + 1) * g].double()
                z = torch.tensordot(q, k, ([2], [1])) * d ** -0.5
                at = first - cu[b] + torch.arange(r0, r1, device="cuda")[:, None, None]
                j = torch.arange(n, device="cuda")
                z = z.where((j <= at) & (j > at - (c["window"] or n + 1)), torch.tensor(-math.inf, dtype=z.dtype, device="cuda"))
                norm = torch.logsumexp(z, -1)
                lse[r0:r1, h * g:(h + 1) * g] = norm
                out[r0:r1, h * g:(h + 1) * g] = torch.tensordot(torch.exp(z - norm[..., None]), v, ([2], [0]))
    return {"out": out, "lse": lse}


def _exact_append(s):
    c = s["case"]
    hkv, d, dim = c["hkv"], c["d"], c["rope_dim"]
    fp16 = c["fmt"] == "fp16"
    cu, lens = s["cu"].tolist(), s["lens"].tolist()
    at = torch.cat([torch.arange(n - (cu[b + 1] - cu[b]), n) for b, n in enumerate(lens)]).cuda()
    seq = torch.repeat_interleave(torch.arange(len(lens)), torch.tensor(cu).diff()).cuda()
    page, row = s["table"].long()[seq, at // PAGE], at % PAGE
    first, second = (torch.arange(dim // 2), torch.arange(dim // 2) + dim // 2) if c["style"] == 0 else \
        (2 * torch.arange(dim // 2), 2 * torch.arange(dim // 2) + 1)

    def turned(x):                                          # each pair as a complex number times cos + i sin
        x = x.double()
        t = s["rope"][at].double()
        z = torch.complex(x[..., first], x[..., second]) * torch.complex(t[:, None, :dim // 2], t[:, None, dim // 2:])
        x[..., first], x[..., second] = z.real, z.imag
        return x

    k = s["k_pages"].double()
    k[page, row] = turned(s["k"])
    if fp16:
        v = s["v_pages"].view(torch.float16).view(-1, PAGE, hkv, d).double()
        v[page, row] = s["v"].double()
    else:
        grid = _byte_table(E4M3)
        v = grid[s["v_pages"].view(-1, PAGE, hkv, d).long()]
        # the quotient is rounded to 32 bits before its code is chosen: part of the definition
        y = (s["v"].double() / s["scales"].double()[page][:, :, None]).float().double()
        v[page, row] = torch.copysign(_nearest(y.abs(), grid[:127]), y)
    return {"q": turned(s["q"]), "k_pages": k, "v_pages": v.view(s["v_pages"].shape[0], -1)}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "extend":
        return _exact_extend(s)
    if case["op"] == "append":
        return _exact_append(s)
    ids = s["ids"].long()
    v = s["v"].double()
    v[ids] = _exact_micro(v[ids].flatten(0, 1)).view(len(ids), PAGE, case["hkv"], case["d"])
    return {"values": v, "modes": None}
