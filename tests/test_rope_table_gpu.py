"""ekv_rope_table against the oracle: every scaling, far positions, odd sizes, tables made in pieces; refusals."""

import ctypes
import math

import numpy as np
import pytest

from oracle import prompt as op

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch_cuda():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return torch


def make(ekv, torch, first, n, dim, theta=1e4, scaling=0, factor=1.0, original_len=8192.0, slow=1.0, fast=4.0, magnitude=1.0):
    ctx = ekv.Context(4, 2, 64, 1)
    table = torch.full((n + 1, dim), float("nan"), dtype=torch.float32, device="cuda")
    cfg = ekv.ekv_rope_config(theta, scaling, factor, original_len, slow, fast, magnitude)
    ekv.ekv_rope_table(ctx.handle, cfg, table, first, n, dim)
    assert ctx.error() == (0, 0)
    assert torch.isnan(table[n]).all()                    # the row behind the last
    return table[:n].cpu().numpy().astype(np.float64)


def check(got, first, dim, magnitude, **cfg):
    """Within a quarter turn a sine or cosine is good to its argument's rounding (2^-24 relative), the function's (one
    unit, 2^-23) and the product's (2^-24): 2^-22 of the value. The angle itself: w to 2^-64 turns and the
    roundings of its 64-bit value and of its product with the position, in the oracle too."""
    n = len(got)
    ref, w = op.rope_table(first, n, dim, magnitude, **cfg), op.turns(dim, **cfg)
    t = np.arange(first, first + n, dtype=np.float64)[:, None] + 1
    angle = 2 * math.pi * t * (2.0 ** -64 + 8 * 2.0 ** -53 * np.concatenate([w, w]))
    err = np.abs(got - ref)
    assert np.all(err <= 2.0 ** -22 * np.abs(ref) + angle * abs(magnitude)), err.max()


@pytest.mark.parametrize("scaling", [0, 1, 2, 3])
@pytest.mark.parametrize("first,n,dim", [(0, 1, 16), (0, 700, 64), (3, 333, 48), (4000, 1000, 128), (1 << 20, 77, 112),
                                         ((1 << 31) - 101, 100, 96), (0, 3000, 32)])
def test_against_the_oracle(ekv_lib, torch_cuda, scaling, first, n, dim):
    cfg = dict(theta=1e4, scaling=scaling, factor=8.0, original_len=4096.0, slow=1.0, fast=32.0)
    got = make(ekv_lib, torch_cuda, first, n, dim, magnitude=1.2, **cfg)
    check(got, first, dim, float(np.float32(1.2)), **cfg)


@pytest.mark.parametrize("theta,factor,original,slow,fast,m", [(1.0001, 1.0, 10.0, 0.1, 0.2, 1.0), (5e5, 32.0, 1e6, 1.0, 4.0, -0.5),
                                                               (1e7, 1e6, 3.0, 1e-3, 1e3, 1.0), (2.0, 3.0, 1e-9, 1.0, 2.0, 0.0)])
def test_odd_configurations(ekv_lib, torch_cuda, theta, factor, original, slow, fast, m):
    for scaling in (2, 3):
        cfg = dict(theta=theta, scaling=scaling, factor=factor, original_len=original, slow=slow, fast=fast)
        check(make(ekv_lib, torch_cuda, 5, 300, 64, magnitude=m, **cfg), 5, 64, float(np.float32(m)), **cfg)


def test_pieces_are_the_whole(ekv_lib, torch_cuda):
    whole = make(ekv_lib, torch_cuda, 0, 5000, 128)
    assert np.array_equal(np.concatenate([make(ekv_lib, torch_cuda, a, b - a, 128) for a, b in ((0, 1), (1, 4097), (4097, 5000))]),
                          whole)


def test_refusals(ekv_lib, torch_cuda):
    torch = torch_cuda
    ctx = ekv_lib.Context(4, 2, 64, 1)
    table = torch.zeros((8, 64), device="cuda")
    good = dict(theta=1e4, scaling=3, factor=2.0, original_len=100.0, slow=1.0, fast=2.0, magnitude=1.0)
    inf, nan = math.inf, math.nan
    for bad in (dict(theta=1.0), dict(theta=nan), dict(theta=inf), dict(scaling=4), dict(scaling=-1), dict(factor=0.5),
                dict(factor=inf), dict(factor=nan), dict(original_len=0.0), dict(original_len=nan), dict(original_len=inf), dict(slow=0.0),
                dict(slow=2.0), dict(slow=nan), dict(fast=inf), dict(magnitude=nan), dict(magnitude=inf)):
        with pytest.raises(ekv_lib.EkvError) as e:
            ekv_lib.ekv_rope_table(ctx.handle, ekv_lib.ekv_rope_config(**{**good, **bad}), table, 0, 8, 64)
        assert e.value.status == ekv_lib.EKV_ERR_INVALID_ARG, bad
    cfg = ekv_lib.ekv_rope_config(**good)
    for bad in (dict(ctx=None), dict(cfg=None), dict(table=None), dict(table=table.data_ptr() + 4), dict(first=-1), dict(rope_len=-1),
                dict(first=(1 << 31) - 8), dict(rope_dim=0), dict(rope_dim=24), dict(rope_dim=144)):
        with pytest.raises(ekv_lib.EkvError) as e:
            ekv_lib.ekv_rope_table(**{**dict(ctx=ctx.handle, cfg=cfg, table=table, first=0, rope_len=8, rope_dim=64), **bad})
        assert e.value.status == ekv_lib.EKV_ERR_INVALID_ARG, bad
    ekv_lib.ekv_rope_table(ctx.handle, cfg, None, 0, 0, 64)
    plain = ekv_lib.ekv_rope_config(1e4, 0, 0.0, 0.0, 0.0, 0.0, 1.0)   # what PLAIN does not look at
    ekv_lib.ekv_rope_table(ctx.handle, plain, table, 0, 8, 64)
    assert ctx.error() == (0, 0) and bool(torch.isfinite(table).all()) and ctypes.sizeof(plain) == 56
