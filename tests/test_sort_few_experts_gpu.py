"""Entries of few experts sorted by several blocks: more room for parts of their table than it has rows."""
import numpy as np
import pytest

from tests.test_token_rows_gpu import check_sort

pytestmark = pytest.mark.gpu


# 3 to 5 blocks and 128, for 2 to 97 kinds of entries
@pytest.mark.parametrize("entries", [4097, 6144, 6145, 8192, 9000, 262144, 300001])
@pytest.mark.parametrize("experts", [1, 2, 3, 5, 8, 60, 96])
def test_few_experts_and_several_blocks(entries, experts):
    rng = np.random.RandomState(entries + experts)
    check_sort(rng.randint(-1, experts, (entries, 1)), experts)
    # a rank's share, most entries those of others
    check_sort(rng.randint(0, 4 * experts, (entries, 1)), experts, 2 * experts)
