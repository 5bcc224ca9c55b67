"""Workspace sizes of the activation operators, which the library answers without a GPU."""
import pytest

pytest.importorskip("torch")


@pytest.fixture(scope="module")
def lib():
    from allreduce_compatible_gradient_gb300 import _binding, _build
    _build.build_library()
    return _binding.lib()


@pytest.mark.parametrize("rows", [1, 7, 8, 9, 1000, 1016, 1024, 1025, 10 ** 6])
@pytest.mark.parametrize("cols", [8193, 8200, 16384, 50001])
def test_layernorm_of_long_rows(lib, rows, cols):
    """More columns than a block holds: partial rows of the columns' sums, one for 8 rows and 128 at most."""
    assert lib.gq_layernorm_workspace_bytes(rows, cols) == min((rows + 7) // 8, 128) * 2 * cols * 4


def test_layernorm_of_other_rows(lib):
    assert lib.gq_layernorm_workspace_bytes(10 ** 6, 8192) == 1024 * 2 * 8192 * 4
    assert lib.gq_layernorm_workspace_bytes(0, 16384) == 16
