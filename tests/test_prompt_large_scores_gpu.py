"""ekv_prompt_attention with scores up to the stated end of their range, 2^23, where an fp32 step is one: whole-number scores, so that
the products are exact, in both tile forms, with maxima that move by small and by large steps."""

import numpy as np
import pytest

from _extend import cu_of

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("hq,hkv,d,lens,window", [(4, 2, 64, [300, 1, 129], 0), (4, 2, 128, [300, 129], 100), (2, 1, 128, [4100], 0)])
@pytest.mark.parametrize("size", [64000, 16000, 250])
def test_scores_near_the_end_of_their_range(ekv_lib, sign, hq, hkv, d, lens, window, size):
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    rng = np.random.default_rng(260)
    cu, T = cu_of(lens), sum(lens)
    q, k = np.zeros((T, hq, d)), np.zeros((T, hkv, d))
    # every 150 keys the scores move by `size`, among them they differ by 0 .. 12
    at = np.concatenate([np.arange(n) for n in lens])
    q[..., 0], k[..., 0] = size, sign * np.minimum(127, 120 + at // 150)[:, None]
    q[..., 1], k[..., 1] = 1, rng.integers(0, 7, (T, hkv))
    q[..., 2], k[..., 2] = rng.integers(0, 3, (T, hq)), rng.integers(0, 4, (T, hkv))
    v = rng.standard_normal((T, hkv, d))
    q, k, v = (torch.from_numpy(x.astype(np.float16)).cuda() for x in (q, k, v))
    ctx = ekv_lib.Context(hq, hkv, d, len(lens))
    out, lse = torch.empty_like(q), torch.empty((T, hq), device="cuda")
    ekv_lib.ekv_prompt_attention(ctx.handle, q, k, v, hq * d, hkv * d, hkv * d, torch.from_numpy(cu).cuda(), len(lens), T, window, 1.0, out, lse)
    assert ctx.error() == (0, 0)
    g = hq // hkv
    for a, b in zip(cu, cu[1:]):
        i = torch.arange(int(b - a), device="cuda")
        seen = (i <= i[:, None]) & (i > i[:, None] - (window or T))
        for h in range(hq):
            s = (q[a:b, h].double() @ k[a:b, h // g].double().T).masked_fill(~seen, -np.inf)
            assert s[seen].abs().max() < 2 ** 23
            p = torch.softmax(s, -1)
            ref, big = p @ v[a:b, h // g].double(), p @ v[a:b, h // g].double().abs()
            # Weights 2^(s c - m), c = log2 e: c is off by 2^-24 of itself, the same for all scores, so by 2^-24 of their differences;
            # s c - m, below 32 where a weight counts, is rounded once; with the exponential and the sums below 2^-16 of a weight. Weights
            # and results are rounded to fp16 by 2^-11. lse: c, m's sum with the logarithm, 1 / c and the product, 2^-24 each.
            assert ((out[a:b, h].double() - ref).abs() <= 2.0 ** -11 * ref.abs() + 2.0 ** -10.5 * big + 2.0 ** -24).all()
            l = torch.logsumexp(s, -1)
            assert ((lse[a:b, h].double() - l).abs() <= 2.0 ** -22 * l.abs() + 1e-4).all()
