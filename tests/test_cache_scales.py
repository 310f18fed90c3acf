"""The scales that the attentions take, checked on the host before any CUDA call."""
import ctypes
import math
import struct

import pytest
import torch

FAKE = ctypes.c_void_p(0x10000)  # never dereferenced: validation fails first


@pytest.fixture(scope="module")
def lib():
    import speculative_decoding_verification_69_gb300 as sv
    return sv.load_library()


def _calls(lib):
    """(calls by scale, factor on the scale): refused with 1, or with 4 for want of a workspace."""
    p4 = struct.pack("Piiiiiqqq", 0x10000, 1, 10, 16, 2, 64, 21760, 2176, 1088)

    def four(scale, dtype):
        return lib.spec_tree_attention4(FAKE, dtype, 1024, 256, 64, p4, FAKE, 0, FAKE, None, None, 2, 4, 4, 8, scale, 0, 0,
                                        FAKE, None, None, 0, None, None)

    def sixteen(scale, dtype, f):
        p = struct.pack("PPiiiiiiqqqq", 0x10000, 0x10000, dtype, 1, 10, 16, 2, 64, 20480, 2048, 128, 64)
        return f(FAKE, 1024, 256, 64, p, FAKE, FAKE, None, None, 2, 4, 4, 8, scale, 0, 0, FAKE, None, None, 0, None, None)
    return [(lambda s: four(s, 1), 1.0), (lambda s: four(s, 2), 4.0),
            (lambda s: sixteen(s, 1, lib.spec_tree_attention), 1.0), (lambda s: sixteen(s, 2, lib.spec_tree_attention), 1.0),
            (lambda s: sixteen(s, 1, lib.spec_sparse_attention), 1.0)]


def test_scales_that_float32_holds_in_base_2(lib):
    """The kernels multiply by scale * log2(e), the 4-bit one by four times that in float16: an infinite factor would make
    NaN of a score of 0.  The largest scale that is taken and the smallest that is refused, and the smallest of all."""
    for call, factor in _calls(lib):
        edge = torch.tensor(torch.finfo(torch.float32).max / factor / math.log2(math.e), dtype=torch.float64)
        below, above = float((edge * (1 - 2.0 ** -22)).float()), float((edge * (1 + 2.0 ** -22)).float())
        assert call(below) == 4 and call(above) == 1 and call(3e38) == 1 and call(2.0 ** -126) == 4
        assert call(0.0) == 1 and call(math.inf) == 1 and call(math.nan) == 1 and call(-1.0) == 1
