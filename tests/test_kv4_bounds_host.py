"""How far the numbers that 4-bit codes stand for are from what was quantised
(no GPU; the kernel's codes are these bit for bit)."""
import numpy as np
import pytest

from tests import kv4_ref as ref


def half_ulp16(y):
    """Half the distance of fp16 numbers at y."""
    e = np.floor(np.log2(np.maximum(np.abs(y), 2.0 ** -14)))
    return 2.0 ** (np.maximum(e, -14) - 11)


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("offset", [0, 3, -3, 100, -100, 1000, -1000, -1023.9,
                                    6000, -6000])
@pytest.mark.parametrize("sigma", [0.001, 0.1, 1.0, 30.0])
def test_groups_at_any_distance_from_zero(group, offset, sigma):
    """Half a step, a's rounding (15 steps by 2^-11, or by 2^-25 near fp16's
    least numbers), b's (half an fp16 step at lo - 64 a) and the number's own;
    the 32-bit steps add less than 2^-10 of these."""
    r = np.random.default_rng(group)
    x = (r.standard_normal((200, 128)) * sigma + offset).astype(np.float32)
    x = np.clip(x, -ref.MOST, ref.MOST)
    n, pair = ref.quantise(x, group)
    g = x.reshape(200, -1, group).astype(np.float64)
    lo, hi = g.min(-1), g.max(-1)
    step = (hi - lo) / 15
    tol = step * (0.5 + 15 * 2.0 ** -11) + 15 * 2.0 ** -25 + \
        half_ulp16(lo - 64 * pair[..., 0])
    own = half_ulp16(np.abs(g).max(-1) + tol)
    err = np.abs(ref.values(n, pair).reshape(g.shape) - g).max(-1)
    assert (err <= (tol + own) * (1 + 2.0 ** -10)).all()
    # where the group's offset is large its term is more than a step
    if sigma == 0.1 and abs(offset) >= 1000:
        assert (half_ulp16(lo - 64 * pair[..., 0]) > step).any()
