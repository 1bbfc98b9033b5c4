"""Sizes at the edge of what the operators around the attention take (CPU)."""
import pytest

from weight_recurrence_gb300 import build as labuild
from weight_recurrence_gb300 import la


@pytest.fixture(scope="module")
def lib():
    labuild.build()
    return la.lib()


@pytest.mark.parametrize("D", [(1 << 31) - 64, (1 << 31) - 100, 1 << 30, (1 << 29) + 40])
@pytest.mark.parametrize("dtype", [la.LA_DTYPE_F32, la.LA_DTYPE_BF16])
def test_wide_rows_need_no_workspace(lib, D, dtype):
    """Rows this wide fill every SM by themselves: no segments."""
    assert lib.la_recurrence_workspace_bytes(la.la_shape(1, 1, 5000, D, 0, dtype)) == 0


def test_rows_past_the_limit(lib):
    assert lib.la_recurrence_workspace_bytes(la.la_shape(1, 1, 5000, (1 << 31) - 63, 0, la.LA_DTYPE_F32)) == la._SIZE_MAX
