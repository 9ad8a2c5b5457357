"""A pytest plugin for runs on the bounds-checked library: after each test the
block operators' kernels must have recorded no access outside their operands."""
import ctypes

import pytest


def recorded():
    """What the kernels recorded since the last call (0: nothing), cleared by it; waits for them."""
    from communication_compressed_sign_gb300 import block
    word = ctypes.c_int32(-1)
    assert block.load().lioncub_block_checked_word(ctypes.byref(word)) == 0, block.load().lioncub_block_last_error()
    return word.value


@pytest.fixture(autouse=True)
def nothing_recorded():
    yield
    assert recorded() == 0, "an access lay outside its operands"
