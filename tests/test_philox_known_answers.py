"""The random words of the 8-bit optimizer states against Philox4x32-7's published known answers (the test vectors that
accompany Salmon, Moraes, Dror and Shaw, "Parallel random numbers: as easy as 1, 2, 3", 2011)."""

import numpy as np
import pytest

from oracle import block_oracle as O


@pytest.mark.parametrize("counter,key,want", [
    ([0] * 4, 0, [0x5F6FB709, 0x0D893F64, 0x4F121F81, 0x4F730A48]),
    ([0xFFFFFFFF] * 4, 0xFFFFFFFFFFFFFFFF, [0x5207DDC2, 0x45165E59, 0x4D8EE751, 0x8C52F662]),
    ([0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344], 0x299F31D0A4093822, [0x4DFCCABA, 0x190A87F0, 0xC47362BA, 0xB6B5242A])])
def test_known_answers(counter, key, want):
    assert O.philox7(np.array([counter], np.uint32), key)[0].tolist() == want
