"""Ends of the argument ranges of the paged-cache calls, refused on the host."""
import pytest

from test_kv_cache_host import EINVAL, attention, mass, ptr


@pytest.mark.parametrize("call,other", [(attention, dict(out=ptr(0x20000))), (mass, {})])
def test_a_scale_that_overflows_in_base_two(call, other):
    """Scores are kept in units of log 2: an infinite factor makes 0 * inf of a score of 0."""
    for scale in (3.0e38, 2.4e38):
        assert call(scale=scale, **other) == EINVAL


def test_a_scale_just_below():
    assert attention(scale=2.3e38, out=ptr(0x20000), n_tokens=0) == 0    # (nothing is enqueued)
