"""Beam selection over vocabularies of a few tokens, whose rows lie inside one vector of the array or
across two, against a sort of all candidates in 64 bits."""
import math

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from tests.test_beam_gpu import check, rows  # noqa: E402


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("V", [2, 3, 4, 5, 6, 7, 8, 9, 11, 17])
@pytest.mark.parametrize("B,K", [(17, 1), (6, 3)])
def test_short_rows(dtype, V, B, K):
    x, s = rows(100 * V + K, B, K, V, dtype)
    check(x, s, 1)
    check(x, s, min(64, K * V + 1))   # all of them, and one place more than there are
    x[1, 0] = -math.inf               # hidden: whole rows, and single columns at their ends
    x[2, :, 0] = -math.inf
    x[3, :, V - 1] = -math.inf
    x[4, 0, V - 1] = math.nan
    check(x, s, min(64, V))
