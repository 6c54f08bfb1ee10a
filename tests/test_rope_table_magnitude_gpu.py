"""ekv_rope_table with magnitudes at the ends of fp32's range: what fp32 holds is used, what it does not is refused."""

import numpy as np
import pytest

from oracle import prompt as op

pytestmark = pytest.mark.gpu

LARGEST = float(np.finfo(np.float32).max)


@pytest.fixture(scope="module")
def table_of(ekv_lib):
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    ctx = ekv_lib.Context(4, 2, 64, 1)

    def make(magnitude):
        table = torch.full((50, 64), 7.0, device="cuda")
        ekv_lib.ekv_rope_table(ctx.handle, ekv_lib.ekv_rope_config(1e4, 0, 1.0, 1.0, 1.0, 2.0, magnitude), table, 3, 50, 64)
        assert ctx.error() == (0, 0)
        return table.cpu().numpy()
    return make


@pytest.mark.parametrize("m", [LARGEST, -LARGEST, 2.0 ** -126, 2.0 ** -100, 1e30])
def test_magnitudes_that_fp32_holds(table_of, m):
    """2^-22 of the value (see test_rope_table_gpu.check), the angle's 2^-40 of the magnitude at these positions, and the least
    fp32 step."""
    m = float(np.float32(m))
    ref = op.rope_table(3, 50, 64, m, theta=1e4)
    err = np.abs(table_of(m).astype(np.float64) - ref)
    assert np.all(err <= 2.0 ** -22 * np.abs(ref) + 2.0 ** -40 * abs(m) + 2.0 ** -149), err.max()


@pytest.mark.parametrize("m", [1e39, -1e39, 3.5e38, 1e300])
def test_magnitudes_that_fp32_does_not_hold_are_refused(ekv_lib, table_of, m):
    with pytest.raises(ekv_lib.EkvError) as e:
        table_of(m)
    assert e.value.status == ekv_lib.EKV_ERR_INVALID_ARG
