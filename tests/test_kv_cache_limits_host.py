"""Ends of the argument ranges of the paged-cache calls, refused on the host."""
import pytest

from test_kv_cache_host import EINVAL, attention, mass, ptr


@pytest.mark.parametrize("call,other", [(attention, dict(out=ptr(0x20000))), (mass, {})])
def test_a_scale_that_overflows_in_base_two(call, other):
    """Scores are kept in units of log 2: an infinite factor makes 0 * inf of a score of 0."""
    for scale in (3.0e38, 2.4e38):
        assert call(scale=scale, **other) == EINVAL
    assert call(scale=2.3e38, n_tokens=0, **other) != EINVAL
