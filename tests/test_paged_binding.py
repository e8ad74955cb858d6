"""The paged cache's binding without a GPU: calls it refuses before it looks at
their device."""
import pytest
import torch

from io_aware_exact_02_gb300 import fa


def test_a_prefix_call_needs_a_prefix():
    x = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    pages = torch.zeros(3, 2, 16, 64, dtype=torch.bfloat16)
    i = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="prefix_pages"):
        fa.fwd_paged_prefix(x, pages, pages, i[None], i, i, None)
