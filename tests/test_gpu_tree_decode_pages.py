"""examples/tree_decode.py over a cache in 4 bits and over selected pages."""
import pytest

import test_gpu_tree_decode as plain

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("slots,prompt,page", [(1, 2, 8), (4, 150, 16)])
def test_all_pages_selected_change_nothing(slots, prompt, page):
    ex = plain._example()
    for bits in (16, 4):
        seqs, emitted, worst = ex.run(slots, 8, prompt, page, bits=bits)
        again = ex.run(slots, 8, prompt, page, bits=bits, keep=100)
        assert again[0] == seqs and again[1] == emitted and again[2] == worst
        assert all(len(s) >= prompt + 8 for s in seqs)


@pytest.mark.parametrize("bits", [4, 16])
def test_few_pages_run(bits):
    seqs, emitted, _ = plain._example().run(3, 8, 150, 16, bits=bits, keep=3)
    assert 1.0 <= emitted <= 5.0 and all(len(s) >= 158 for s in seqs)
