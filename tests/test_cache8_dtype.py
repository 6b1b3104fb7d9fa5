"""cache8 makes caches of the two 8-bit types only."""

import pytest
import torch

import grouped_query_attention_attn_b200 as gqa


@pytest.mark.parametrize("dtype", [torch.float8_e4m3fn, torch.int8])
def test_its_types(dtype):
    c = gqa.cache8(3, 2, 64, page=32, block=16, dtype=dtype, device="cpu")
    assert c.k.dtype == c.v.dtype == dtype and c.k.shape == c.v.shape == (3, 2, 32, 64)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32, torch.uint8, torch.float8_e5m2])
def test_other_types_are_refused(dtype):
    # a type of two bytes gave pages of half the head dimension
    with pytest.raises(ValueError, match="dtype"):
        gqa.cache8(3, 2, 64, page=32, block=16, dtype=dtype, device="cpu")
