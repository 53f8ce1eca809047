"""The generator's oracle against its published known answers, and the mask's share."""
import numpy as np

import oracle


def test_known_answers():
    # the test vectors published with the generator: counter, key -> words
    for counter, key, words in (
            ((0, 0, 0, 0), (0, 0), (0x6627e8d5, 0xe169c58d, 0xbc57ac4c, 0x9b00dbd8)),
            ((0xffffffff,) * 4, (0xffffffff,) * 2, (0x408f276d, 0x41c83b0e, 0xa20bc7c6, 0x6d5451fd)),
            ((0x243f6a88, 0x85a308d3, 0x13198a2e, 0x03707344), (0xa4093822, 0x299f31d0),
             (0xd16cfe09, 0x94fdcceb, 0x5001e420, 0x24126ea1))):
        assert tuple(oracle.philox4x32(np.array([counter], np.uint32), key)[0].tolist()) == words


def test_mask():
    n = 1 << 20
    for p in (0.0, 0.1, 0.5, 0.9, 1.0):
        keep = oracle.dropout_keep((1024, 1024), p, seed=123456789012345, offset=7)
        q = 1 - oracle.dropout_threshold(p) / 65536
        # six standard deviations of a binomial share
        assert abs(keep.mean() - q) <= 6 * np.sqrt(q * (1 - q) / n)
    a, b = oracle.dropout_bits(4096, 1, 0), oracle.dropout_bits(4096, 1, 1)
    assert (a != b).mean() > 0.99 and (a == oracle.dropout_bits(8192, 1, 0)[:4096]).all()
    assert (oracle.dropout_bits(64, 1, 0, first=1024) == oracle.dropout_bits(2048, 1, 0)[1024:1088]).all()
