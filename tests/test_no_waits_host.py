"""No kernel's result rests on a wait for another workgroup (host only: read from the sources). One that waits holds a
compute unit that the one it waits for may need while other launches hold the rest; a wait that gives up and goes on
all the same gives wrong results. Looking a bounded time, with a way to finish whatever is found, is neither."""
import os

import pytest

import w4a16_nvfp4_dense_amd as ffn

CSRC = os.path.join(ffn.PKG_DIR, "csrc")


@pytest.mark.parametrize("name", ["smallm_gemm.h", "w4a4.hip", "mfma_gemm.h"])
def test_no_wait(name):
    with open(os.path.join(CSRC, name)) as f:
        text = f.read()
    assert "wait_ready" not in text and "s_sleep" not in text


def test_nothing_to_wait_with():
    """The one loop that sleeps looks a bounded number of times and returns what it found."""
    for name in sorted(os.listdir(CSRC)):
        with open(os.path.join(CSRC, name)) as f:
            text = f.read()
        assert "wait_ready" not in text, name
        assert text.count("s_sleep") == (1 if name == "part_words_device.h" else 0), name
