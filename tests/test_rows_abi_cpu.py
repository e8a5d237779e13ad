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


# x [4][256], y [4][N]: bytes 2 * 4 * 256 and 2 * 4 * N from their addresses
@pytest.mark.parametrize("x,y_in,out,N", [
    (A, 4 * A, A, 256), (A, 4 * A, A + 2032, 256), (A + 2032, 4 * A, A, 256),
    (A + 4096 - 16, 4 * A, A, 512), (4 * A, A, A + 16, 256), (4 * A, A + 2032, A, 256),
    (A, A, A, 256)])
def test_adapters_refuse_an_output_that_lies_on_what_is_read(lib, x, y_in, out, N):
    assert lora(lib, x=x, y=y_in, out=out, N=N) == -1
    assert b"overlap" in lib.egopq_last_error_string()


@pytest.mark.parametrize("x,y,N", [(A, A, 256), (A, A + 2032, 256), (A + 4080, A, 512)])
def test_linear_with_adapters_refuses_an_output_that_lies_on_x(lib, x, y, N):
    assert linear_lora(lib, x=x, y=y, N=N) == -1
    assert b"overlap" in lib.egopq_last_error_string()


def test_adapters_accept_an_output_in_place_or_apart(lib):
    """Neighbours that touch are apart: such a call gets to the device check (or,
    on a machine that has one, would run: only shapes of no rows here)."""
    assert lora(lib, M=0, x=A, y=A, out=A) == 0
    for x, y_in, out in [(A, A + 2048, A + 2048), (A + 2048, A, A), (A, A + 2048, A + 4096)]:
        if lib.egopq_supported(4, 256, 256, 128, 0):
            pytest.skip("a device is there: the addresses here are not")
        assert lora(lib, x=x, y=y_in, out=out) != -1
