"""Cases of the operators that bring a fresh prompt from its projection into the paged cache:
what they compute in plain form, and the calls of the ekv library that compute the same.

* angles   the table of cosines and sines that the rotary writers read, with the frequencies of a
           model whose context was stretched (all divided, or only the slow ones);
* write    the new tokens of every sequence (one or many each): queries and keys are normalised per
           head, rotated by the position, keys and values written into the pages of the cache, and the
           rotated keys also packed for the attention of the prompt. Values go to FP16 pages, to E4M3 pages
           whose scales are there, or to E4M3 pages whose scales the writer makes and lets grow;
* prompt   causal attention of whole prompts of different lengths, packed behind one another, straight
           from the rows of the projection, over all earlier tokens or a sliding window of them.
"""

import functools
import math
import random

import numpy as np
import torch

own = False

PAGE = 16
TARGET, E4M3 = 0, 1
PER_PAGE_HEAD = 1
TINY = 2.0 ** -24                                           # the least FP16 magnitude


# ------------------------------------------------------------------------------- cases
def _angles(name, first, rows, dim, scaling, factor, original, slow, fast):
    return dict(name=name, op="angles", first=first, rows=rows, dim=dim, scaling=scaling, factor=factor, original=original,
                slow=slow, fast=fast)


def _write(name, batch, new, ctx, hq, hkv, d, rope_dim, style, fmt, lens, fused, packed):
    return dict(name=name, op="write", batch=batch, new_lo=new[0], new_hi=new[1], ctx_lo=ctx[0], ctx_hi=ctx[1], hq=hq,
                hkv=hkv, d=d, rope_dim=rope_dim, style=style, fmt=fmt, lens=lens, fused=fused, packed=packed)


def _prompt(name, batch, new, hq, hkv, d, window, lens, fused):
    return dict(name=name, op="prompt", batch=batch, new_lo=new[0], new_hi=new[1], ctx_lo=0, ctx_hi=0, hq=hq, hkv=hkv, d=d,
                window=window, lens=lens, fused=fused)


def listed():
    """`new` and `ctx`: the range of each sequence's new and earlier tokens; `lens`: which draw of
    the lengths; `fmt` "grow": E4M3 pages whose scales the writer makes."""
    return [
        # a small model's positions, as a program starts
        _angles("angles 4096x64", 0, 4096, 64, "plain", 1.0, 4096, 1.0, 4.0),
        # a context stretched eightfold, the slow frequencies alone
        _angles("angles 131072x128", 0, 131072, 128, "turns", 8.0, 8192, 1.0, 4.0),
        # one decode step of a batch of 32
        _write("write step 32", 32, (1, 1), (512, 1024), 32, 8, 128, 128, 0, "e4m3", 1, True, False),
        # draft tokens and short chunks of many users, half of each head rotated in interleaved pairs
        _write("write ragged 96", 96, (1, 333), (0, 700), 32, 4, 128, 64, 1, "e4m3", 2, False, True),
        # the prompts of a whole admission
        _write("write prompts 8x8192", 8, (8192, 8192), (0, 0), 32, 8, 128, 128, 0, "fp16", 3, True, True),
        # one decode step of 256 users, each with a page begun, or beginning one, in 8 bits
        _write("grow step 256", 256, (1, 1), (100, 600), 32, 8, 128, 128, 0, "grow", 4, True, False),
        # ragged prompts straight into 8-bit pages
        _write("grow prompts 24", 24, (700, 4000), (0, 0), 32, 8, 128, 128, 0, "grow", 5, True, True),
        # two short prompts of a small model
        _prompt("prompt tiny", 2, (37, 100), 4, 2, 64, 0, 6, False),
        # an admission of many short prompts, eight query heads a key head
        _prompt("prompt short 200", 200, (1, 300), 32, 4, 128, 0, 7, True),
        # prompts of very different lengths, together
        _prompt("prompt ragged 16", 16, (100, 4096), 32, 8, 128, 0, 8, True),
        # long prompts under a sliding window
        _prompt("prompt window 1024", 4, (6000, 8192), 32, 8, 128, 1024, 9, False),
        # the prompts of a whole admission
        _prompt("prompt 8x8192", 8, (8192, 8192), 32, 8, 128, 0, 10, True),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    op = rng.choice(("angles", "write", "write", "write", "prompt", "prompt", "prompt"))
    lens = rng.randrange(1, 1 << 20)
    if op == "angles":
        dim = 16 * rng.randint(1, 8)
        slow = rng.choice((1.0, 0.5, 2.0))
        c = _angles("", _log_int(rng, 1, 1 << 20) - 1, _log_int(rng, 1, 131072 * 128 // dim), dim,
                    rng.choice(("plain", "linear", "turns", "dims")), rng.choice((1.0, 2.0, 4.0, 8.0, 32.0)),
                    rng.choice((2048, 4096, 8192, 32768)), slow, slow * rng.choice((4.0, 32.0)))
        del c["name"]
        return c
    hq, hkv, d = rng.choice(((32, 8, 128), (32, 8, 128), (32, 4, 128), (16, 8, 64), (4, 2, 64), (8, 1, 128), (24, 4, 128),
                             (8, 8, 64)))
    if op == "write":
        batch = _log_int(rng, 1, 256)
        hi = _log_int(rng, 1, max(1, 65536 // batch))
        lo = rng.choice((1, hi, rng.randint(1, hi)))
        c = _write("", batch, (lo, hi), (0, _log_int(rng, 1, 1024)), hq, hkv, d, rng.choice((d, d, d // 2, 16)),
                   rng.randrange(2), rng.choice(("fp16", "e4m3", "grow", "grow")), lens, rng.random() < 0.5,
                   rng.random() < 0.5)
    else:
        while True:
            batch, hi = _log_int(rng, 1, 256), _log_int(rng, 1, 16384)
            if batch * hi <= 65536 and batch * hq * hi * hi <= 32 * 8 * 8192 * 8192:
                break
        c = _prompt("", batch, (rng.choice((1, hi, rng.randint(1, hi))), hi), hq, hkv, d,
                    rng.choice((0, 0, 0, _log_int(rng, 1, 4096))), lens, rng.random() < 0.5)
    del c["name"]
    return c


def _lengths(case):
    """(new tokens, total tokens) of every sequence: they go by the case alone."""
    r = random.Random(case["lens"])
    new = [r.randint(case["new_lo"], case["new_hi"]) for _ in range(case["batch"])]
    return new, [r.randint(case["ctx_lo"], case["ctx_hi"]) + n for n in new]


def _magnitude(case):
    """What stretched models multiply cosines and sines by: it keeps the scores' spread."""
    return 0.1 * math.log(case["factor"]) + 1.0 if case["scaling"] in ("turns", "dims") else 1.0


# ----------------------------------------------------------------------------- prepare
def _rows(case, total, gen):
    """q, k and v rows: slices of one projection's output, or tensors of their own."""
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    if case["fused"]:
        rows = torch.randn((total, hq + 2 * hkv, d), generator=gen, device="cuda", dtype=torch.float16)
        return rows.split((hq, hkv, hkv), 1)
    return [torch.randn((total, h, d), generator=gen, device="cuda", dtype=torch.float16) for h in (hq, hkv, hkv)]


def prepare(case, seed):
    if case["op"] == "angles":                              # from a position on: a table may be made, or added to, in pieces
        return dict(case=case, first=case["first"] + random.Random(seed).randrange(4096),
                    table=torch.empty((case["rows"], case["dim"]), dtype=torch.float32, device="cuda"))
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    new, lens = _lengths(case)
    total = sum(new)
    st = dict(case=case, total=total, new=new, cu=torch.tensor(np.cumsum([0] + new), dtype=torch.int32, device="cuda"))
    st["q"], st["k"], st["v"] = _rows(case, total, gen)
    if case["op"] == "prompt":
        st["q"].mul_(1.5)                                   # sharp enough that attention prefers some keys
        return st
    st["lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
    # block table over a random permutation of the pool; entries past a sequence's pages repeat its last
    need = [max(1, -(-n // PAGE)) for n in lens]
    pages = sum(need)
    perm = torch.randperm(pages, generator=gen, device="cuda").to(torch.int32)
    first = torch.tensor(np.cumsum([0] + need[:-1]), device="cuda")
    j = torch.arange(max(need), device="cuda")
    st["table"] = perm[first[:, None] + torch.minimum(j[None, :], torch.tensor(need, device="cuda")[:, None] - 1)].contiguous()
    st["k_pages"] = torch.randn((pages, PAGE, hkv, d), generator=gen, device="cuda", dtype=torch.float16)
    st["scales"] = None
    if case["fmt"] == "fp16":
        st["v_pages"] = torch.randn((pages, PAGE * hkv * d), generator=gen, device="cuda", dtype=torch.float16).view(torch.uint8)
    else:
        # pages as earlier calls left them: their scale is some row's largest magnitude, so later rows may need more
        x = torch.randn((pages, PAGE, hkv, d), generator=gen, device="cuda")
        st["scales"] = x.abs().amax((1, 3)) / 448 * (0.4 + 0.6 * torch.rand((pages, hkv), generator=gen, device="cuda"))
        y = (x / st["scales"][:, None, :, None]).clamp(-448, 448)
        st["v_pages"] = y.to(torch.float8_e4m3fn).view(torch.uint8).flatten(1)
    # values with channels of their own size, weights of a trained norm
    st["v"].mul_(torch.rand((hkv, d), generator=gen, device="cuda").half() + 0.5)
    st["q_weight"] = (1 + 0.3 * torch.randn(d, generator=gen, device="cuda")).half()
    st["k_weight"] = (1 + 0.3 * torch.randn(d, generator=gen, device="cuda")).half()
    half = case["rope_dim"] // 2
    freq = 10000.0 ** (-torch.arange(half, dtype=torch.float64, device="cuda") / half)
    angle = torch.arange(max(lens), dtype=torch.float64, device="cuda")[:, None] * freq
    st["rope"] = torch.cat((angle.cos(), angle.sin()), 1).float().contiguous()
    st["q_out"] = torch.empty((total, hq, d), dtype=torch.float16, device="cuda")
    st["k_out"] = torch.empty((total, hkv, d), dtype=torch.float16, device="cuda") if case["packed"] else None
    return st


EPS = 1e-6
THETA = 10000.0


# ------------------------------------------------------------------------- plain forms
def _plain_angles(s):
    """In 64 bits: the angle of a far position has few bits behind its whole turns."""
    c = s["case"]
    dim, half = c["dim"], c["dim"] // 2
    i = torch.arange(half, dtype=torch.float64, device="cuda")
    f = THETA ** (-2 * i / dim)
    if c["scaling"] == "linear":
        f = f / c["factor"]
    elif c["scaling"] == "turns":                           # ramp over the turns within the original context
        g = ((c["original"] * f / (2 * math.pi) - c["slow"]) / (c["fast"] - c["slow"])).clamp(0, 1)
        f = f * (g + (1 - g) / c["factor"])
    elif c["scaling"] == "dims":                            # ramp over the pairs, between those of so many turns
        at = [dim * math.log(c["original"] / (2 * math.pi * r)) / (2 * math.log(THETA)) for r in (c["fast"], c["slow"])]
        lo, hi = max(math.floor(at[0]), 0), min(math.ceil(at[1]), dim - 1)
        g = 1 - ((i - lo) / max(hi - lo, 0.001)).clamp(0, 1)
        f = f * (g + (1 - g) / c["factor"])
    angle = torch.arange(s["first"], s["first"] + c["rows"], dtype=torch.float64, device="cuda")[:, None] * f
    s["table"][:, :half] = angle.cos() * _magnitude(c)
    s["table"][:, half:] = angle.sin() * _magnitude(c)


def _places(s):
    """Sequence and position of every new token."""
    i = torch.arange(s["total"], device="cuda")
    b = torch.searchsorted(s["cu"][1:].contiguous(), i.to(torch.int32), right=True)
    return b, i - s["cu"][b + 1].long() + s["lens"][b].long()


def _normed(x, w):
    x = x.float()
    return x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * w.float()


def _rotate(x, cos, sin, style, dim):
    a, rest = x[..., :dim], x[..., dim:]
    if style == 0:
        u, w = a[..., :dim // 2], a[..., dim // 2:]
        a = torch.cat((u * cos - w * sin, w * cos + u * sin), -1)
    else:
        u, w = a[..., 0::2], a[..., 1::2]
        a = torch.stack((u * cos - w * sin, w * cos + u * sin), -1).flatten(-2)
    return torch.cat((a, rest), -1).half()


def _plain_grow(s, page, row):
    """The scales of the pages that the call writes, and the codes that were there under them."""
    c = s["case"]
    pages, hkv = s["scales"].shape
    big = torch.zeros((pages, hkv), device="cuda")
    big.scatter_reduce_(0, page[:, None].expand(-1, hkv), s["v"].float().abs().amax(-1), "amax")
    first = torch.full((pages,), PAGE, device="cuda").scatter_reduce_(0, page, row, "amin")
    (m, e), (n, f) = torch.frexp(big), torch.frexp(s["scales"] * 448)
    k = (e - f + (m > n)).clamp_(min=0) * (big > 0) * ((first > 0) & (first < PAGE))[:, None]
    at = (k > 0).any(-1).nonzero()[:, 0]                    # pages whose codes are brought under a larger scale
    codes = s["v_pages"].view(torch.float8_e4m3fn).view(pages, PAGE, hkv, c["d"])
    old = codes[at].float()
    old = torch.where((torch.arange(PAGE, device="cuda") < first[at, None])[..., None, None],
                      torch.ldexp(old, -k[at][:, None, :, None]), old)
    codes[at] = old.to(torch.float8_e4m3fn)
    fresh = big.clamp(min=TINY) / torch.full_like(big, 448)   # (a number would be multiplied by its reciprocal)
    grown = torch.where((first == 0)[:, None], fresh, torch.ldexp(s["scales"], k))
    s["scales"].copy_(grown)


def _plain_write(s):
    c = s["case"]
    hkv, d, dim = c["hkv"], c["d"], c["rope_dim"]
    b, t = _places(s)
    cos, sin = s["rope"][t][:, None].split(dim // 2, -1)
    s["q_out"].copy_(_rotate(_normed(s["q"], s["q_weight"]), cos, sin, c["style"], dim))
    k = _rotate(_normed(s["k"], s["k_weight"]), cos, sin, c["style"], dim)
    page, row = s["table"][b, t // PAGE].long(), t % PAGE
    s["k_pages"][page, row] = k
    if s["k_out"] is not None:
        s["k_out"].copy_(k)
    if c["fmt"] == "fp16":
        s["v_pages"].view(torch.float16).view(-1, PAGE, hkv, d)[page, row] = s["v"]
        return
    if c["fmt"] == "grow":
        _plain_grow(s, page, row)
    y = (s["v"].float() / s["scales"][page][:, :, None]).clamp(-448, 448)
    s["v_pages"].view(-1, PAGE, hkv, d)[page, row] = y.to(torch.float8_e4m3fn).view(torch.uint8)


def _plain_prompt(s):
    """Prompts that fit together are padded to one length; KV heads of long ones go in turns."""
    c = s["case"]
    hq, hkv, d, g, n = c["hq"], c["hkv"], c["d"], c["hq"] // c["hkv"], c["batch"]
    out = torch.empty((s["total"], hq, d), dtype=torch.float16, device="cuda")
    lse = torch.empty((s["total"], hq), dtype=torch.float32, device="cuda")
    most = 1 << 30
    b0 = 0
    while b0 < n:
        b1, top = b0 + 1, s["new"][b0]
        while b1 < n and (b1 + 1 - b0) * hq * max(top, s["new"][b1]) ** 2 <= most:
            top = max(top, s["new"][b1])
            b1 += 1
        cu = s["cu"][b0:b1 + 1].long()
        pos = torch.arange(top, device="cuda")
        at = (cu[:-1, None] + pos).clamp(max=s["total"] - 1)
        real = pos < (cu[1:] - cu[:-1])[:, None]
        rows = at[real]
        seen = pos <= pos[:, None]
        if c["window"]:
            seen &= pos > pos[:, None] - c["window"]
        step = max(1, min(hkv, most // ((b1 - b0) * g * top * top)))
        for h in range(0, hkv, step):
            q = s["q"][:, h * g:(h + step) * g][at].float().unflatten(2, (-1, g))
            k, v = s["k"][:, h:h + step][at].float(), s["v"][:, h:h + step][at].float()
            score = torch.einsum("bqhgd,bkhd->bhgqk", q, k).div_(math.sqrt(d))
            score.masked_fill_(~seen, -math.inf)
            peak = score.amax(-1, keepdim=True)
            score.sub_(peak).exp_()
            total = score.sum(-1, keepdim=True)
            o = (torch.einsum("bhgqk,bkhd->bhgqd", score, v) / total).permute(0, 3, 1, 2, 4).flatten(2, 3)
            out[rows, h * g:(h + step) * g] = o[real].half()
            lse[rows, h * g:(h + step) * g] = (peak + total.log())[..., 0].permute(0, 3, 1, 2).flatten(2, 3)[real]
        b0 = b1
    return out, lse


# --------------------------------------------------------------------------------- run
@functools.lru_cache(maxsize=None)
def _context(hq, hkv, d):
    """The handle that a program keeps for a model's head layout."""
    from mixed_precision_paged_gb300 import ekv
    return ekv, ekv.Context(hq, hkv, d, 256)


def run(state):
    s, c = state, state["case"]
    if c["op"] == "angles":
        if own:
            ekv, ctx = _context(32, 8, 128)
            kind = {"plain": ekv.EKV_ROPE_PLAIN, "linear": ekv.EKV_ROPE_LINEAR, "turns": ekv.EKV_ROPE_BY_TURNS,
                    "dims": ekv.EKV_ROPE_BY_DIMS}[c["scaling"]]
            cfg = ekv.ekv_rope_config(THETA, kind, c["factor"], c["original"], c["slow"], c["fast"], _magnitude(c))
            ekv.ekv_rope_table(ctx.handle, cfg, s["table"], s["first"], c["rows"], c["dim"])
        else:
            _plain_angles(s)
        return s["table"]
    if c["op"] == "write":
        if own:
            ekv, ctx = _context(c["hq"], c["hkv"], c["d"])
            ekv.ekv_append_kv_norm_rope(ctx.handle, s["q"], s["k"], s["v"], s["q"].stride(0), s["k"].stride(0),
                                        s["v"].stride(0), s["q_weight"], s["k_weight"], EPS, s["rope"], s["rope"].shape[0],
                                        c["rope_dim"], c["style"], s["q_out"], s["k_out"], s["k_pages"], s["v_pages"],
                                        s["v_pages"].shape[1], s["k_pages"].shape[0], s["scales"], PER_PAGE_HEAD,
                                        c["fmt"] == "grow", None, TARGET if c["fmt"] == "fp16" else E4M3, s["table"],
                                        s["table"].shape[1], s["lens"], s["cu"], c["batch"], s["total"])
        else:
            _plain_write(s)
        kind = torch.float16 if c["fmt"] == "fp16" else torch.float8_e4m3fn
        return {"q": s["q_out"], "k": s["k_out"], "k_pages": s["k_pages"], "v_pages": s["v_pages"].view(kind),
                "scales": s["scales"]}
    if own:
        ekv, ctx = _context(c["hq"], c["hkv"], c["d"])
        out = torch.empty((s["total"], c["hq"], c["d"]), dtype=torch.float16, device="cuda")
        lse = torch.empty((s["total"], c["hq"]), dtype=torch.float32, device="cuda")
        ekv.ekv_prompt_attention(ctx.handle, s["q"], s["k"], s["v"], s["q"].stride(0), s["k"].stride(0), s["v"].stride(0),
                                 s["cu"], c["batch"], s["total"], c["window"], 0.0, out, lse)
    else:
        out, lse = _plain_prompt(s)
    return {"out": out, "lse": lse}


# -------------------------------------------------------------------------------- work
def work(case):
    if case["op"] == "angles":
        return {"bytes": 4 * case["rows"] * case["dim"], "flops": 0}
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    new, lens = _lengths(case)
    total = sum(new)
    if case["op"] == "prompt":
        w = case["window"] or (1 << 30)
        pairs = sum(n * (n + 1) // 2 - max(0, n - w) * (max(0, n - w) + 1) // 2 for n in new)
        return {"bytes": total * ((2 * hq + 2 * hkv) * 2 * d + 4 * hq), "flops": 4 * d * hq * pairs}
    rows, end = 0, 0                                        # rows of the table that any token reads
    for lo, hi in sorted((l - n, l) for n, l in zip(new, lens)):
        rows += max(0, hi - max(lo, end))
        end = max(end, hi)
    value = 2 if case["fmt"] == "fp16" else 1
    each = 2 * 2 * hq + (4 + 2 * case["packed"]) * hkv + (2 + value) * hkv
    return {"bytes": total * d * each + rows * 4 * case["rope_dim"], "flops": 0}


# ------------------------------------------------------------------------------- exact
def _exact_angles(case, at):
    half = case["dim"] // 2
    turns = []                                              # of each pair, a position
    pair_of = lambda r: half * math.log(case["original"] / (2 * math.pi * r), THETA)
    lo = max(0, math.floor(pair_of(case["fast"]))) if case["scaling"] == "dims" else 0
    hi = min(case["dim"] - 1, math.ceil(pair_of(case["slow"]))) if case["scaling"] == "dims" else 0
    for i in range(half):
        f = math.exp(-i / half * math.log(THETA)) / (2 * math.pi)
        kept = {"plain": 1.0, "linear": 0.0}.get(case["scaling"])
        if case["scaling"] == "turns":
            kept = min(1.0, max(0.0, (case["original"] * f - case["slow"]) / (case["fast"] - case["slow"])))
        elif case["scaling"] == "dims":
            kept = min(1.0, max(0.0, (hi - i) / (hi - lo))) if hi > lo else float(i <= lo)
        turns.append(f * kept + f / case["factor"] * (1 - kept))
    turns = torch.tensor(turns, dtype=torch.float64, device="cuda")
    x = torch.arange(case["rows"], dtype=torch.float64, device="cuda").add_(at)[:, None] * turns
    z = torch.polar(torch.full_like(x, _magnitude(case)), (x - x.round()) * (2 * math.pi))
    return torch.cat((z.real, z.imag), 1)


def _code_values():
    """The values of the E4M3 codes 0 .. 126, ascending."""
    return torch.tensor([(8 + c % 8) * 2.0 ** (c // 8 - 10) if c > 7 else c * 2.0 ** -9 for c in range(127)],
                        dtype=torch.float64, device="cuda")


def _nearest(y, grid):
    """The nearest of an ascending grid of magnitudes, the even index at a tie, beyond its end its end; y >= 0 in float64."""
    hi = torch.searchsorted(grid, y).clamp(1, len(grid) - 1)
    lo = hi - 1
    up = (y - grid[lo] > grid[hi] - y) | ((y - grid[lo] == grid[hi] - y) & (hi % 2 == 0))
    return torch.where(up, grid[hi], grid[lo])


def _exact_write(s):
    c = s["case"]
    hkv, d, dim = c["hkv"], c["d"], c["rope_dim"]
    cu, lens = s["cu"].tolist(), s["lens"].tolist()
    at = torch.cat([torch.arange(n - (cu[b + 1] - cu[b]), n) for b, n in enumerate(lens)]).cuda()
    seq = torch.repeat_interleave(torch.arange(len(lens)), torch.tensor(cu).diff()).cuda()
    page, row = s["table"].long()[seq, at // PAGE], at % PAGE
    j = torch.arange(dim // 2)
    first, second = (j, j + dim // 2) if c["style"] == 0 else (2 * j, 2 * j + 1)

    def turned(x, w):                                       # each pair as a complex number times cos + i sin
        x = x.double()
        x = x / (x.square().sum(-1, keepdim=True) / d + EPS).sqrt() * w.double()
        t = s["rope"][at].double()
        z = torch.complex(x[..., first], x[..., second]) * torch.complex(t[:, None, :dim // 2], t[:, None, dim // 2:])
        x[..., first], x[..., second] = z.real, z.imag
        return x

    new_k = turned(s["k"], s["k_weight"])
    k = s["k_pages"].double()
    k[page, row] = new_k
    scales = None
    if c["fmt"] == "fp16":
        v = s["v_pages"].view(torch.float16).view(-1, PAGE, hkv, d).double()
        v[page, row] = s["v"].double()
    else:
        grid = _code_values()
        raw = s["v_pages"].view(-1, PAGE, hkv, d).long()
        v = torch.where(raw > 127, -1.0, 1.0).double() * grid[raw & 127]
        scales = s["scales"].double()
        if c["fmt"] == "grow":
            # page after page, as it stands after the call; 32 bits where a scale is stored
            begun = torch.zeros(len(scales), dtype=torch.bool, device="cuda")
            begun[page[row == 0]] = True
            wide = torch.zeros((len(scales), hkv), dtype=torch.float64, device="cuda")
            wide.index_reduce_(0, page, s["v"].double().abs().amax(-1), "amax")
            room = (scales * 448).float().double()
            more = torch.zeros_like(scales)
            for k2 in range(1, 60):
                more[(room * 2.0 ** (k2 - 1) < wide) & ~begun[:, None]] = k2
            lowest = torch.full((len(scales),), PAGE, device="cuda").index_reduce_(0, page, row, "amin")
            kept = torch.arange(PAGE, device="cuda") < lowest[:, None]
            shrunk = v / 2.0 ** more[:, None, :, None]
            for p0 in range(0, len(v), 1024):
                p = slice(p0, p0 + 1024)
                moved = kept[p][:, :, None, None] & (more[p] > 0)[:, None, :, None] & (lowest[p] < PAGE)[:, None, None, None]
                v[p] = torch.where(moved, torch.copysign(_nearest(shrunk[p].abs(), grid), v[p]), v[p])
            scales = torch.where(begun[:, None], (wide.clamp(min=TINY) / 448).float().double(), scales * 2.0 ** more)
        # the quotient is rounded to 32 bits before its code is chosen: part of the definition
        y = (s["v"].double() / scales[page][:, :, None]).float().double()
        v[page, row] = torch.copysign(_nearest(y.abs(), grid), y)
    return {"q": turned(s["q"], s["q_weight"]), "k": new_k if c["packed"] else None, "k_pages": k,
            "v_pages": v.view(s["v_pages"].shape[0], -1), "scales": scales}


def _exact_prompt(s):
    c = s["case"]
    hq, hkv, d, g = c["hq"], c["hkv"], c["d"], c["hq"] // c["hkv"]
    out = torch.empty((s["total"], hq, d), dtype=torch.float64, device="cuda")
    lse = torch.empty((s["total"], hq), dtype=torch.float64, device="cuda")
    cu = s["cu"].tolist()
    for a, z in zip(cu, cu[1:]):
        for r0 in range(a, z, 1024):
            r1 = min(r0 + 1024, z)
            low = max(a, r0 - c["window"] + 1) if c["window"] else a
            i, j = torch.arange(r0, r1, device="cuda")[:, None], torch.arange(low, r1, device="cuda")
            hidden = (j > i) | (j <= i - c["window"]) if c["window"] else j > i
            for h in range(hq):
                p = (s["q"][r0:r1, h].double() @ s["k"][low:r1, h // g].double().T) * d ** -0.5
                p[hidden] = -math.inf
                norm = torch.logsumexp(p, -1)
                lse[r0:r1, h] = norm
                out[r0:r1, h] = torch.exp(p - norm[:, None]) @ s["v"][low:r1, h // g].double()
    return {"out": out, "lse": lse}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "angles":
        return _exact_angles(case, s["first"])
    return _exact_write(s) if case["op"] == "write" else _exact_prompt(s)
