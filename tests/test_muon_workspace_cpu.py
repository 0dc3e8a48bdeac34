"""Workspace bytes of single matrices are those that the header states, short sides and vectors included."""
import pytest

import adamw_optimizer_step_apply_amd as A

SHAPES = [(1, 1), (1, 300), (300, 1), (1, 1 << 20), (4, 8192), (16, 768), (16, 2048), (2048, 16), (8, 1 << 24), (64, 64), (65, 64), (65, 65),
          (100, 37), (768, 2304), (2048, 2048), (8192, 2048), (1 << 20, 65)]


def stated(r, c):
    up = lambda n, to: -(-n // to) * to  # noqa: E731
    s, l = (up(x, 64) for x in sorted((r, c)))
    run = up(-(-r * c // 256), 4096)
    runs = -(-r * c // run)
    return 8 * s + 4 * s * l + max(2 * s * l + 4 * s * s, up(4 * r * c, 256)) + up(8 * runs, 256)


@pytest.mark.parametrize("shape", SHAPES)
def test_one_matrix(shape):
    ml = A.MatrixList([shape], [[]])
    head = 256
    assert A.adamw_orthogonalize_workspace_bytes(ml) == A.adamw_orthogonalize_workspace_bytes(ml, least=True) == head + stated(*shape)


def test_a_list_of_both_sorts():
    """All of them at once, or the largest."""
    ml = A.MatrixList(SHAPES[:8], [[]])
    assert A.adamw_orthogonalize_workspace_bytes(ml) == 256 + sum(stated(*s) for s in SHAPES[:8])
    assert A.adamw_orthogonalize_workspace_bytes(ml, least=True) == 256 + max(stated(*s) for s in SHAPES[:8])


def test_bytes_an_element_as_stated():
    for shape, most in (((16, 2048), 24.7), ((4, 8192), 96.7), ((1, 1 << 20), 384.1), ((2048, 2048), 10.1), ((2048, 1 << 17), 8.1)):
        assert 0.98 * most < stated(*shape) / (shape[0] * shape[1]) <= most
