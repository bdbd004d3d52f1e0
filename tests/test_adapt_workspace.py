"""A workspace that shares memory with an operand is refused, on the host: the first
kernels would overwrite what later ones read."""
import pytest

from tests.test_adapt_abi import ALIAS, P, SCRATCH, backward, lib, lora  # noqa: F401


# Operands of the calls in test_adapt_abi, by their names there.
@pytest.mark.parametrize("name, at", [("X", 0), ("A", 1), ("B", 2), ("ids", 3), ("s", 4), ("base", 5)])
def test_lora(lib, name, at):  # noqa: F811
    # All of it, a byte of its end, and a workspace that begins inside.
    assert lora(lib, ws=P[at], n=1 << 20) == ALIAS, name
    assert lora(lib, ws=P[at] - 4096, n=4097) == ALIAS
    assert lora(lib, ws=P[at] + 8, n=1 << 20) == ALIAS


@pytest.mark.parametrize("name, at", [("dY", 0), ("X", 1), ("A", 2), ("B", 3), ("H", 4), ("ids", 5), ("s", 6),
                                      ("base", 7)])
def test_backward(lib, name, at):  # noqa: F811
    assert backward(lib, ws=P[at], n=1 << 20) == ALIAS, name
    assert backward(lib, ws=P[at] - 4096, n=4097) == ALIAS
    assert backward(lib, ws=P[at] + 8, n=1 << 20) == ALIAS


def test_beside_is_fine(lib):  # noqa: F811
    """Next to an operand it is too small, not shared."""
    assert backward(lib, ws=P[1] - 2048, n=2048) == SCRATCH
    assert lora(lib, ws=P[0] - 4096, n=4096, M=400, base=None, Y=1 << 50, H=None) == SCRATCH
