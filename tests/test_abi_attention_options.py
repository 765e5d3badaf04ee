"""Options that no formula can use, without a GPU: infinite scales and caps."""
import pytest

from test_abi_attention import BOTH, EINVAL

INF = float("inf")


@pytest.mark.parametrize("call", BOTH)
@pytest.mark.parametrize("opt", [dict(scale=INF), dict(softcap=INF), dict(scale=-INF), dict(softcap=-INF),
                                 dict(scale=1e300), dict(softcap=1e300)])
def test_infinite_scale_or_cap(call, opt):
    """Beyond float's range counts as infinite."""
    assert call(opt=opt) == EINVAL
