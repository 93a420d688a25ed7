"""An inf or NaN in V of a key that a query does not see (0 times it is NaN): how far before the key it can show."""
import math

import pytest
import torch

from test_gpu_prompt_attn import Batch, msa  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("layout", ["packed", "paged", "fp8"])
@pytest.mark.parametrize("group", [1, 2, 3, 16, 100])
@pytest.mark.parametrize("past", [0, 1, 100])
@pytest.mark.parametrize("key", [383, 700, 1023])
def test_how_far_a_late_value_shows(msa, layout, group, past, key):
    n, far = 1100, 2 * (128 // group) + 126   # an item's tokens, up to the end of its last block
    b = Batch(msa, [n], [past + n], group, 1, layout, seed=key)
    o, lse = b.run()
    b.v[b.rows[0][key]] = 0x7F if layout == "fp8" else math.nan
    o2, lse2 = b.run()
    assert torch.equal(lse, lse2)   # V is no part of it
    at = torch.arange(n, device="cuda") + past
    assert torch.isnan(o2[at >= key]).all()
    assert torch.equal(o[at < key - far], o2[at < key - far])
