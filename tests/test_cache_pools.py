"""Which layouts of a pool are taken, on the host before any CUDA call: a view of
any dense tensor, but none in which two elements share a place."""
import ctypes
import itertools
import random
import struct

import pytest
import torch

FAKE = ctypes.c_void_p(0x10000)  # never dereferenced: the calls below fail at a later check


@pytest.fixture(scope="module")
def lib():
    import speculative_decoding_verification_69_gb300 as sv
    return sv.load_library()


def _status(lib, layers, pages, page, heads, D, strides):
    """1: refused; 4: the pool is taken and the missing workspace found."""
    p = struct.pack("PPiiiiiiqqqq", 0x10000, 0x10000, 1, layers, pages, page, heads, D, *strides)
    return lib.spec_cache_fork(p, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, 2, 4, 8, None, 0, None, None)


def test_overlapping_strides_are_refused(lib):
    L, P, T, H, D = 2, 5, 8, 3, 16
    dense = (P * T * H * D, T * H * D, H * D, D)
    assert _status(lib, L, P, T, H, D, dense) == 4
    for i, low in itertools.product(range(4), (0, 8)):
        if dense[i] - 8 > 0:
            s = list(dense)
            s[i] = dense[i] - 8 if low else 0
            assert _status(lib, L, P, T, H, D, s) == 1, (i, s)
    for i, j in itertools.combinations(range(4), 2):  # equal strides of two dimensions
        s = list(dense)
        s[i] = s[j]
        assert _status(lib, L, P, T, H, D, s) == 1, s
    assert _status(lib, L, P, T, H, D, (2 ** 62, 2 ** 62, 48, 16)) == 1
    for i, extent in enumerate((1, P, T, H)):  # a dimension of one element is not stepped over
        s = list(dense)
        if extent == 1:
            s[i] = 0
            assert _status(lib, 1, P, T, H, D, s) == 4


@pytest.mark.parametrize("seed", range(40))
def test_views_of_dense_tensors_are_taken(lib, seed):
    """Any order of the dimensions in memory, with others between them and slices of them."""
    r = random.Random(seed)
    shape = [r.choice([1, 2, 3]), r.choice([1, 4, 7]), r.choice([8, 16]), r.choice([1, 2, 5])]
    D = 8 * r.randint(1, 4)
    order = r.sample(range(4), 4)
    base = torch.empty([shape[i] * r.choice([1, 1, 2]) + r.choice([0, 1]) for i in order] + [D + 8 * r.choice([0, 1])],
                       dtype=torch.bfloat16, device="meta")
    view = base.permute([order.index(i) for i in range(4)] + [4])[..., :D]
    for d in range(4):
        step = 2 if view.shape[d] >= 2 * shape[d] else 1
        view = view.narrow(d, 0, step * (shape[d] - 1) + 1)[(slice(None),) * d + (slice(None, None, step),)]
    assert list(view.shape) == shape + [D]
    assert _status(lib, *shape, D, view.stride()[:4]) == 4
