"""Sizes beyond what the C calls take are refused in the binding, not cut off on the way."""
import pytest
import torch

from test_many_tokens_abi_cpu import msa  # noqa: F401


@pytest.mark.parametrize("pages", [2 ** 31, 2 ** 64 + 5, -2 ** 64 + 5])
def test_numbers_of_pages(msa, pages):
    with pytest.raises(ValueError, match="num_pages"):
        msa.msa_append_workspace_size(pages)
    with pytest.raises(ValueError, match="num_pages"):
        msa.msa_extend_block_table(torch.zeros(2), torch.zeros(2), torch.zeros(1), torch.zeros(2, 2), 5, num_pages=pages)
