"""Workspace sizes of the scored decode calls by type (no GPU)."""
import pytest
import torch

import paged_kv_cache_279_gb300 as pkv

size = pkv.paged_attention_decode_scored_workspace_size


@pytest.mark.parametrize("heads,D", [(1, 64), (32, 128), (64, 128)])
def test_a_type_needs_its_own_kernels_workspace(heads, D):
    for S in (1, 64, 256, 8192, 100000):
        for L in (1, 512, 513, 8192, 131072, 2 ** 31 - 1):
            any_, f32, bf16 = size(S, heads, D, L), size(S, heads, D, L, torch.float32), size(S, heads, D, L, torch.bfloat16)
            assert any_ == max(f32, bf16)
            # two partial states a warp of the largest grid (2048 warps of up to 8 heads), and 8 bytes a (sequence, head)
            assert bf16 <= 2 * 2048 * min(heads, 8) * (4 * D + 8) + min(S, 8192) * heads * 8 + 3 * 256
            assert bf16 == size(S, heads, D, 1, torch.bfloat16)       # whatever the length
            assert (f32 == 0) == (L <= 512)                           # contexts that one CTA takes whole need none
    with pytest.raises(TypeError):
        size(1, heads, D, 100, torch.float16)
    assert size(4, heads, D, 0, torch.bfloat16) == 0 and size(0, heads, D, 100, torch.float32) == 0
