"""The random numbers behind dropout's reference against the published known answers of Philox4x32-10 (those that
accompany Salmon, Moraes, Dror and Shaw, 2011: counter, key, words), so that the kernels, which are compared with that
reference, are compared with the published function."""
from __future__ import annotations

import numpy as np
import pytest

from tests import rows_parity as rp

KNOWN = [
    ((0, 0, 0, 0), (0, 0), (0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8)),
    ((0xFFFFFFFF,) * 4, (0xFFFFFFFF,) * 2, (0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD)),
    ((0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344), (0xA4093822, 0x299F31D0),
     (0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1)),
]


@pytest.mark.parametrize("counter,key,words", KNOWN)
def test_known_answers(counter, key, words):
    got = rp.philox([np.array([c], np.uint32) for c in counter], key)
    assert tuple(int(w[0]) for w in got) == words


def test_words_in_the_order_that_dropout_takes_them():
    """Block 0 of row 0 of site, offset and seed 0 is the first known answer: half-words from the low end of word 0 on."""
    halves = [h for w in KNOWN[0][2] for h in (w & 0xFFFF, w >> 16)]
    for t in (0x6628, 0x9B00, 0xE16A):
        f = rp.drop_factors(1, 8, t / 65536, 0, 0, 0)[0]
        assert [float(v) for v in f] == [0.0 if h < t else 65536 / (65536 - t) for h in halves]

