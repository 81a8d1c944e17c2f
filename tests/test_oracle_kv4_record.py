"""A record of the 4-bit cache written out by hand: which byte and which half of
it holds what, and what the bytes stand for."""
import numpy as np
import pytest

from oracle import kv4


@pytest.mark.parametrize("D,size", [(64, 80), (128, 144)])
def test_a_record_by_hand(D, size):
    k, v = np.zeros(D), np.zeros(D)
    # first group of the key: largest magnitude 6 x 0.25, so the scale is 2^-2, byte (13 << 3); -1.5 is code 7 with its
    # sign, 0.125 code 1, 0.75 code 5 (3 x 0.25)
    k[0], k[1], k[5] = -1.5, 0.125, 0.75
    # last group of the value: largest magnitude 6 x 1.125, byte (15 << 3) + 1; 1.6875 = 1.5 x 1.125 is code 3
    v[D - 1], v[D - 2] = 6.75, 1.6875
    # second group of the key: 3 x 2^-17 lies between the scales 0 and 2^-17 times 6, and goes to the even byte, 0
    k[16], k[17] = 3 * 2.0 ** -17, -(2.0 ** -17)
    # third group: the smallest scale above that, 2 x 2^-17; an element a quarter of it (between the codes 0 and 0.5) is 0
    k[32], k[33] = 12 * 2.0 ** -17, 2.0 ** -18
    rec = kv4.records(k, v)
    want = np.zeros(size, np.uint8)
    want[0] = 0xF | 1 << 4                      # dimensions 0 (low half) and 1
    want[2] = 5 << 4                            # dimension 5
    want[8] = 0x80                              # dimension 17: a zero with its sign
    want[16] = 7                                # dimension 32; 33 is 0
    want[D - 1] = 3 | 7 << 4                    # value, dimensions D - 2 and D - 1
    want[D], want[D + 2] = 13 << 3, 2
    want[D + D // 8 - 1] = (15 << 3) + 1
    np.testing.assert_array_equal(rec, want)
    kk, vv = kv4.values(want, D)
    k[16] = k[17] = k[33] = 0                   # what the format does not hold
    np.testing.assert_array_equal(kk, k)
    np.testing.assert_array_equal(vv, v)
