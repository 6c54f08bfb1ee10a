"""The oracle of the calls that take new tokens, tied to things other than itself: the
decode and prefill oracles, complex rotation, and the definition of the microscaled form."""

import numpy as np
import pytest

from mixed_precision_paged_gb300 import workloads as wl
from oracle import decode as od
from oracle import extend as oe
from oracle import micro as om
from oracle import prefill as op

from _extend import cu_of, make_case


def test_one_new_token_is_a_decode():
    c = wl.make_decode_case([5, 33, 100], 8, 2, 64, v_format="mixed", scale_mode=1, seed=1, p_base=0.3, p_compact=0.3)
    out, lse, _, _ = oe.attention(c.q, c, cu_of([1, 1, 1]))
    ref, rl = od.paged_decode(c.q, c.k_pages, c.v_pages, c.v_scales, 1, c.page_mode, c.uniform_mode, c.block_table, c.seq_lens)
    assert np.allclose(out, ref, atol=1e-13) and np.allclose(lse, rl, atol=1e-13)


def test_a_whole_prompt_is_a_prefill():
    rng = np.random.default_rng(2)
    c = wl.make_decode_case([50], 4, 2, 64, v_format="fp16", seed=2, poison=False)
    q = rng.standard_normal((50, 4, 64)).astype(np.float16)
    out, lse, _, _ = oe.attention(q, c, cu_of([50]))
    v = c.v_pages.view("<f2").reshape(-1, 16, 2, 64)
    pages = c.block_table[0, :4]
    ref, rl = op.prefill_attention(q, c.k_pages[pages], v[pages], [0, 50], [0])
    assert np.allclose(out, ref, atol=1e-13) and np.allclose(lse, rl, atol=1e-13)


def test_window_of_one_is_the_own_value_and_a_wide_one_changes_nothing():
    c = make_case([40], 2, 2, 64, "all", seed=3)
    rng = np.random.default_rng(3)
    q = rng.standard_normal((7, 2, 64)).astype(np.float16)
    out, _, _, _ = oe.attention(q, c, cu_of([7]), window=1)
    _, V = oe.sequence_kv(0, c, 40)
    assert np.allclose(out, V[33:], atol=1e-14)
    a, b = oe.attention(q, c, cu_of([7])), oe.attention(q, c, cu_of([7]), window=40)
    assert np.array_equal(a[0], b[0])


@pytest.mark.parametrize("style", [0, 1])
def test_rotation_is_a_complex_product(style):
    rng = np.random.default_rng(4)
    x, ang = rng.standard_normal(64), rng.standard_normal(16)
    y = oe.rotate(x, np.cos(ang), np.sin(ang), style)
    a, b = (slice(0, 16), slice(16, 32)) if style == 0 else (slice(0, 32, 2), slice(1, 32, 2))
    z = (x[a] + 1j * x[b]) * np.exp(1j * ang)
    assert np.allclose(y[a], z.real) and np.allclose(y[b], z.imag) and np.array_equal(y[32:], x[32:])


def test_micro_codes_are_the_nearest_and_the_scale_the_least():
    rng = np.random.default_rng(5)
    for scale in (1e-7, 1e-3, 1.0, 300.0, 2e4):
        x = (rng.standard_normal((20, 32)) * scale).clip(-65504, 65504).astype(np.float16).astype(np.float64)
        for row in x:
            c, k = om.encode_block(row)
            c2, k2 = om.encode_rows(row[None])
            assert np.array_equal(c, c2[0]) and k == k2[0, 0]
            a = np.abs(row).max()
            assert (a <= 6 * 2.0 ** k or k == om.K_MAX) and (k == om.K_MIN or a > 6 * 2.0 ** (k - 1))
            v = np.where(c & 8, -1, 1) * om.VALUES[c & 7] * 2.0 ** k
            if a <= 6 * 2.0 ** k:
                assert np.all(np.abs(v - row) <= 2.0 ** k)          # half of the widest step
            assert np.array_equal(v.astype(np.float16).astype(np.float64), v)   # an fp16 value


def test_micro_ties_signs_and_ends():
    x = np.zeros(32)
    x[:10] = [6, .25, .75, 1.25, 1.75, 2.5, 3.5, 5, -.25, -0.0]
    c, k = om.encode_block(x)
    assert k == 0 and list(c[:10]) == [7, 0, 2, 2, 4, 4, 6, 6, 8, 8]
    assert om.encode_block(np.zeros(32))[1] == -24
    assert om.encode_block(np.full(32, 65504.0)) [1] == 13
    assert om.encode_block(np.full(32, 49152.0)) [1] == 13 and om.encode_block(np.full(32, 24576.0))[1] == 12
    c, k = om.encode_block(np.r_[np.inf, -np.inf, np.nan, np.ones(29)])
    assert k == 13 and list(c[:3]) == [7, 15, 7]


def test_micro_round_trip_keeps_its_values():
    rng = np.random.default_rng(6)
    x = (rng.standard_normal((3, 16, 2, 64)) * [[[[1e-6]]], [[[1.0]]], [[[1e3]]]]).astype(np.float16)
    v = np.full((3, 2 * 16 * 2 * 64 + 16), 0xAB, np.uint8)
    v[:, :-16] = x.reshape(3, -1).view(np.uint8)
    a, mode, bad = om.demote_pages(v, [0, 2], np.zeros(3, np.uint8), 2, 64)
    assert list(mode) == [3, 0, 3] and bad == [] and np.array_equal(a[1], v[1])
    b, mode = om.expand_pages(a, [0, 1, 2], mode, 2, 64)
    assert not mode.any()
    again, mode2, _ = om.demote_pages(b, [0, 2], mode, 2, 64)
    c, _ = om.expand_pages(again, [0, 2], mode2, 2, 64)
    assert np.array_equal(b, c) and np.all(b[:, -16:] == 0xAB)


def test_append_then_attention_reads_the_rotated_tokens():
    rng = np.random.default_rng(7)
    lens, new = np.array([20, 3, 40], np.int32), [4, 3, 1]
    c = make_case(lens, 4, 2, 64, "all", seed=7)
    cu = cu_of(new)
    q, k, v = (rng.standard_normal((8, h, 64)).astype(np.float16) for h in (4, 2, 2))
    rope = np.concatenate([np.cos(a := rng.standard_normal((64, 16))), np.sin(a)], 1).astype(np.float32)
    qo, kp, vp = oe.append(q, k, v, rope, 0, c.k_pages, c.v_pages, c.v_scales, 1, c.page_mode, 0, c.block_table, lens, cu)
    same = np.ones(kp.shape[:2], bool)
    for i, b, t in oe.places(lens, cu):
        page = c.block_table[b, t // 16]
        same[page, t % 16] = False
        assert np.allclose(np.linalg.norm(kp[page, t % 16]), np.linalg.norm(k[i].astype(np.float64)))
    assert np.array_equal(kp[same].astype(np.float16), c.k_pages[same], equal_nan=True)
    assert same.sum() == same.size - 8
