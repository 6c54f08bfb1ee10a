"""The oracle of a prompt's way into the cache, tied to things other than itself: whole-number turns, the demotion and
decode oracles, torch's normalisation and attention."""

import math

import numpy as np
import pytest

from oracle import demote
from oracle import e4m3
from oracle import extend as oe
from oracle import prompt as op

from _extend import cu_of, make_case


def test_angles_are_powers_of_theta_and_scaling_divides_them():
    w = op.turns(64, 1e4)
    assert np.allclose(w * 2 * math.pi, 1e4 ** (-np.arange(32) / 32.0), rtol=1e-14)
    assert np.allclose(op.turns(64, 1e4, op.LINEAR, 4.0), w / 4, rtol=1e-15)
    for kind in (op.BY_TURNS, op.BY_DIMS):
        s = op.turns(128, 1e4, kind, 8.0, 8192, 1.0, 4.0) / op.turns(128, 1e4)
        r = 8192 * op.turns(128, 1e4)
        assert np.all(np.diff(s) <= 1e-15) and math.isclose(s[0], 1.0) and math.isclose(s[-1], 1 / 8)
        mid = (s < 1 - 1e-12) & (s > 1 / 8 + 1e-12)
        slack = 1.0 if kind == op.BY_TURNS else 2 * 1e4 ** (2 / 128)     # (ends moved out to whole pairs)
        assert mid.any() and np.all(r[mid] < 4 * slack) and np.all(r[mid] > 1 / slack)


def test_table_rows_are_unit_rotations_of_their_magnitude():
    t = op.rope_table(5, 40, 32, magnitude=1.25, theta=500.0)
    assert np.allclose(np.hypot(t[:, :16], t[:, 16:]), 1.25)
    z = (t[:, :16] + 1j * t[:, 16:]) / 1.25
    assert np.allclose(z[1:] / z[:-1], np.exp(2j * math.pi * op.turns(32, 500.0)))


def test_norm_is_torch_rms_norm():
    torch = pytest.importorskip("torch")
    rng = np.random.default_rng(1)
    x, w = rng.standard_normal((5, 3, 64)), rng.standard_normal(64)
    ref = torch.nn.functional.rms_norm(torch.from_numpy(x), (64,), torch.from_numpy(w), 1e-3).numpy()
    assert np.allclose(op.normed(x, w, 1e-3), ref, atol=1e-13)
    assert np.array_equal(op.normed(x, None, 1e-3), x)


def test_whole_pages_get_the_scales_and_codes_of_a_demotion():
    rng = np.random.default_rng(2)
    lens = np.array([48], np.int32)
    case = make_case(lens, 2, 2, 64, "e4m3", 1, 3)
    v = (rng.standard_normal((48, 2, 64)) * 3).astype(np.float16)
    zero = np.zeros((48, 2, 64), np.float16)
    _, _, vp, sc = op.append(zero, zero, v, None, None, 1.0, np.zeros((48, 0), np.float32), 0, case.k_pages, case.v_pages,
                             case.v_scales, 1, 1, None, 1, case.block_table, lens, cu_of([48]))
    for j, p in enumerate(case.block_table[0, :3]):
        x = v[16 * j:16 * j + 16]
        s = demote.page_scales(x)
        assert np.array_equal(sc[p], s) and np.array_equal(vp[p, :2048], demote.quantise_page(x, s).reshape(-1))


def test_growth_keeps_values_and_covers_what_comes():
    """Token after token: every value within half a step of the final scale and one rounding of the growth; the scale
    at most twice what the largest value needs."""
    rng = np.random.default_rng(4)
    case = make_case(np.array([16], np.int32), 1, 1, 64, "e4m3", 1, 5)
    v = (rng.standard_normal((16, 1, 64)) * np.exp2(rng.integers(-3, 4, (16, 1, 1)))).astype(np.float16)
    vp, sc = case.v_pages, case.v_scales
    for t in range(16):
        one = np.zeros((1, 1, 64), np.float16)
        _, _, vp, sc = op.append(one, one, v[t:t + 1], None, None, 1.0, np.zeros((16, 0), np.float32), 0, case.k_pages, vp, sc,
                                 1, 1, None, 1, case.block_table, np.array([t + 1]), cu_of([1]))
    p = case.block_table[0, 0]
    s, a = float(sc[p, 0]), np.abs(v.astype(np.float64))
    got = e4m3.decode(vp[p, :1024]).reshape(16, 1, 64) * s
    assert a.max() / 448 <= s * (1 + 2.0 ** -23) and s <= 2 * a.max() / 448
    assert np.all(np.abs(got - v) <= 2 * 2.0 ** -4 * a + 4 * 2.0 ** -10 * s)


@pytest.mark.parametrize("window", [0, 1, 7, 64])
def test_attention_is_torch_attention_per_prompt(window):
    torch = pytest.importorskip("torch")
    rng = np.random.default_rng(6)
    cu = cu_of([5, 0, 30, 1])
    q, k, v = (rng.standard_normal((38, h, 64)) for h in (4, 2, 2))
    out, lse, _, _ = op.attention(q, k, v, cu, window)
    assert np.all(out[36:] == 0) and np.all(np.isneginf(lse[36:]))
    for a, b in zip(cu, cu[1:]):
        if a == b:
            continue
        i = torch.arange(int(b - a))
        seen = (i <= i[:, None]) & (i > i[:, None] - (window or 1000))
        x, y, z = (torch.from_numpy(np.repeat(t[a:b], 4 // t.shape[1], 1)).transpose(0, 1) for t in (q, k, v))
        ref = torch.nn.functional.scaled_dot_product_attention(x, y, z, attn_mask=seen)
        assert np.allclose(out[a:b], ref.transpose(0, 1).numpy(), atol=1e-12)


def test_a_prompt_written_and_extended_is_its_attention():
    rng = np.random.default_rng(7)
    lens = np.array([20, 33], np.int32)
    case = make_case(lens, 4, 2, 64, "fp16", 0, 8)
    cu, T = cu_of(lens), 53
    q, k, v = (rng.standard_normal((T, h, 64)).astype(np.float16) for h in (4, 2, 2))
    w = (1 + 0.1 * rng.standard_normal(64)).astype(np.float16)
    rope = op.rope_table(0, 33, 64, theta=1e4).astype(np.float32)
    qo, kp, vp, _ = op.append(q, k, v, w, w, 1e-6, rope, 0, case.k_pages, case.v_pages, None, 0, 0, None, 0, case.block_table, lens, cu)
    case.k_pages, case.v_pages = kp, vp
    kr = np.concatenate([[kp[case.block_table[b][t // 16], t % 16] for t in range(n)] for b, n in enumerate(lens)])
    a, b = op.attention(qo, kr, v, cu), oe.attention(qo, case, cu)
    assert np.allclose(a[0], b[0], atol=1e-12) and np.allclose(a[1], b[1], atol=1e-12)
