"""More host checks of the operators whose weights each row picks (no device is
touched: every call here is refused)."""
import pytest

from test_rows_cpu import A, experts, lib, lora, route  # noqa: F401


def linear_lora(lib, x=A, ids=A, y=A, N=256, K=256, nbytes=1 << 40):
    return lib.egopq_w4a8_linear_lora(x, A, A, A, A, None, ids, 4, N, K, 128, 4, 16, y, A, nbytes,
                                      0, None)


# Ids and picks' weights that start at any of their elements are accepted: the
# call is refused for what comes after their check.
@pytest.mark.parametrize("at", [4, 8, 12])
def test_picks_may_start_at_any_row(lib, at):
    assert route(lib, ids=A + at, weights=A + at, bias=A + 8) == -3
    assert lib.egopq_last_error_string().startswith(b"bias")
    assert experts(lib, ids=A + at, w=A + at, nbytes=100) == -1
    assert b"workspace" in lib.egopq_last_error_string()
    assert lora(lib, ids=A + at, ranks=A + 4) == -3
    assert lib.egopq_last_error_string().startswith(b"ranks")
    assert linear_lora(lib, ids=A + at, nbytes=100) == -1
    assert b"workspace" in lib.egopq_last_error_string()


@pytest.mark.parametrize("at", [1, 2, 7])
def test_picks_between_their_elements_are_refused(lib, at):
    assert route(lib, ids=A + at) == -3 and route(lib, weights=A + at) == -3
    assert experts(lib, ids=A + at) == -3 and experts(lib, w=A + at) == -3
    assert lora(lib, ids=A + at) == -3 and linear_lora(lib, ids=A + at) == -3
