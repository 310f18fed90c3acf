"""PagedCache4 compares the head size of what it is given with its own."""
import pytest
import torch


def test_heads_of_another_size_than_the_pools():
    """Pages have the same bytes for heads of 72, 80, 88 and 96: the cache compares its own."""
    import speculative_decoding_verification_69_gb300 as sv
    assert sv.cache4_page_bytes(16, 72) == sv.cache4_page_bytes(16, 96)
    cache = sv.PagedCache4(1, 4, 16, 2, 80, 1, 4, device="cpu")
    for D in (72, 96):
        x = torch.zeros((1, 1, 2, D), dtype=torch.bfloat16)
        bounds = torch.zeros((4, 2, 2, D), dtype=torch.bfloat16)
        for call in (lambda: cache.append(0, x, x), lambda: cache.attention(0, x), lambda: cache.summarise(0, bounds),
                     lambda: cache.select(0, x, bounds, 2)):
            with pytest.raises(ValueError, match="80"):
                call()
