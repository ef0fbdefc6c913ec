"""More refusals of the ragged-batch calls, answered on the host before anything is enqueued."""
import pytest

from test_ragged_host import INVALID, NO_DEVICE, _append, _no_gpu, lib  # noqa: F401 (fixtures)


@pytest.mark.parametrize("theta,code", [(1e4, NO_DEVICE), (float("inf"), INVALID), (1e39, INVALID),
                                        (float("nan"), INVALID), (-1e4, INVALID)])
def test_append_takes_a_finite_theta(lib, theta, code):  # noqa: F811
    assert _append(lib, theta=theta) == code
