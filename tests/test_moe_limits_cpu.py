"""The last sizes that the entry points around the experts' products count: refused
past them before any HIP call."""
import os

import pytest

import fp4_precision_gemms_amd as F

A = 0x10000          # a fake 16-byte aligned device address (never dereferenced)
ERR_NULL, ERR_SHAPE = 1, 2


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(F.LIB_PATH):
        pytest.skip("libfp4.so not built")
    return F.lib()


def test_choices_of_a_token_that_end_past_32_bits(L):
    """The kernels take a token's choices 64 at a time: with k past 2^31 - 65 the
    first of the next 64 is no 32-bit integer."""
    def calls(k, out):
        return (L.fp4_moe_gather(A, None, A, 1, k, 8, 64, out, None, None),
                L.fp4_moe_gather(A, A, A, 1, k, 8, 64, out, A, None),
                L.fp4_moe_combine(A, A, A, 1, k, 8, 64, out, None),
                L.fp4_moe_combine_backward(A, A, A, A, 1, k, 8, 64, out, A, None))

    for k in (2 ** 31 - 64, 2 ** 31 - 4, 2 ** 31 - 1):
        assert set(calls(k, None)) == {ERR_SHAPE}, k
    assert set(calls(2 ** 31 - 65, None)) == {ERR_NULL}          # the size is taken: the next check refuses
