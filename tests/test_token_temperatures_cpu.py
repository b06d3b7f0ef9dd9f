"""What qg_token_logprobs refuses of inv_temperature, on the host."""
import math

from test_token_ops_cpu import gradient, qg, scores  # noqa: F401  (qg: the fixture)


def test_temperatures(qg):
    assert scores(qg, it=2.4e38) == qg.QG_ERR_UNSUPPORTED and scores(qg, it=3.4e38) == qg.QG_ERR_UNSUPPORTED
    for it in (2.2e38, 1e-45, 3.4e37):
        assert scores(qg, it=it, T=0) == qg.QG_OK
    assert gradient(qg, it=3.4e38, T=0) == qg.QG_OK and gradient(qg, it=math.inf, T=0) == qg.QG_ERR_INVALID_ARG
