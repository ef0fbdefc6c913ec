"""More refusals of the ragged-batch calls, answered on the host before anything is enqueued."""
import pytest

from test_ragged_host import INVALID, NO_DEVICE, P, SAME, _append, _evict, _no_gpu, lib  # noqa: F401 (fixtures)


@pytest.mark.parametrize("theta,code", [(1e4, NO_DEVICE), (float("inf"), INVALID), (1e39, INVALID),
                                        (float("nan"), INVALID), (-1e4, INVALID)])
def test_append_takes_a_finite_theta(lib, theta, code):  # noqa: F811
    assert _append(lib, theta=theta) == code


# k, v: 2 * 64 * 2 rows of 256 bytes = 1 << 16; k_out, v_out: 1 << 15; kept: 2 * 2 * 32 * 4 = 512
@pytest.mark.parametrize("over,code", [
    (dict(SAME, v=P, vo=P), INVALID),                            # in place, keys and values one tensor
    (dict(vo=5 * P), INVALID), (dict(vo=5 * P + (1 << 15) - 16), INVALID), (dict(vo=5 * P + (1 << 15)), NO_DEVICE),
    (dict(ko=P + (1 << 16) - 16), INVALID), (dict(ko=P + (1 << 16)), NO_DEVICE), (dict(ko=P - (1 << 15) + 16), INVALID),
    (dict(ko=2 * P + 256), INVALID), (dict(so=3 * P + 4), INVALID), (dict(SAME, so=3 * P + 4), INVALID),
    (dict(kept=4 * P), INVALID), (dict(kept=8 * P), INVALID), (dict(kept=8 * P + 8), NO_DEVICE),
    (dict(kept=4 * P - 512), NO_DEVICE), (dict(nl=4 * P + 4), INVALID), (dict(st=8 * P), INVALID),
    (dict(st=8 * P + 8), NO_DEVICE), (dict(v=P), NO_DEVICE)])
def test_evict_outputs_overlap_nothing(lib, over, code):  # noqa: F811
    assert _evict(lib, **over) == code
