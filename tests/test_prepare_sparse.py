"""prepare() of the sparse call refuses what the call itself refuses, before it packs anything."""
import pytest
import torch

import paged_gqa_decode_kv_gb300 as pgd


@pytest.mark.parametrize("prepared", [False, True])
def test_sparse_attention_without_bounds(prepared):
    q = torch.zeros(1, 8, 128, dtype=torch.bfloat16)
    k = torch.zeros(4, 2, 2, 16, 8, 8, dtype=torch.bfloat16)
    call = pgd.prepare if prepared else pgd.sparse_decode_attention
    name = ("sparse_decode_attention",) if prepared else ()
    with pytest.raises(TypeError, match="bounds must be a tensor"):
        call(*name, q, q, k, k, None, None, None, None, None, None, 1, 2, 0.1,
             workspace=torch.zeros(256, dtype=torch.uint8))
