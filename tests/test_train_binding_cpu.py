"""What the fine-tuning entry points and their Python calls check on the host, beyond tests/test_train_abi_cpu.py: nothing here
needs a GPU, and no pointer is followed."""
import math

import pytest

from test_train_abi_cpu import P, qg  # noqa: F401  (qg: the fixture)


@pytest.mark.parametrize("zp", [math.nan, math.inf, -math.inf, 65505.0, -1e6])
@pytest.mark.parametrize("sizes", [(4, 32, 64), (0, 32, 64), (4, 0, 64)])
def test_uniform_zero_points_as_in_the_forward_pass(qg, zp, sizes):
    """A zero point that fp16 does not hold is refused by both passes, whatever the sizes."""
    M, N, K = sizes
    ws = (P, 1 << 30, None)
    assert qg.lib().qgemm_nbits_uniform_zp(P, qg.QG_F16, P, P, zp, P, qg.QG_F16, M, N, K, 4, 32, *ws) == qg.QG_ERR_INVALID_ARG
    assert qg.lib().qgemm_nbits_uniform_zp_dgrad(P, qg.QG_F16, P, P, zp, P, qg.QG_F16, M, N, K, 4, 32, *ws) == qg.QG_ERR_INVALID_ARG


def test_uniform_zero_points_at_the_ends(qg):
    for zp in (65504.0, -65504.0, 7.5):
        assert qg.lib().qgemm_nbits_uniform_zp_dgrad(P, qg.QG_F16, P, P, zp, P, qg.QG_F16, 0, 32, 64, 4, 32, None, 0, None) == qg.QG_OK
