"""The dropout oracle against the generator's published vectors and against what
a mask has to be."""
import numpy as np

from oracle import dropout as D


def test_generator_gives_its_published_vectors():
    # the known answers that the generator's authors publish for philox4x32-10
    known = [
        ([0] * 4, [0] * 2, [0x6627e8d5, 0xe169c58d, 0xbc57ac4c, 0x9b00dbd8]),
        ([0xffffffff] * 4, [0xffffffff] * 2, [0x408f276d, 0x41c83b0e, 0xa20bc7c6, 0x6d5451fd]),
        ([0x243f6a88, 0x85a308d3, 0x13198a2e, 0x03707344], [0xa4093822, 0x299f31d0],
         [0xd16cfe09, 0x94fdcceb, 0x5001e420, 0x24126ea1]),
    ]
    for counter, key, want in known:
        assert D.philox(counter, key) == want


def test_bits_are_the_generators_words_in_order():
    seed, offset = 0x1234567890ABCDEF, 0xFEDCBA0987654321
    for first in (0, 3, 8, 2 ** 35 + 5):  # the block's number passes 32 bits
        got = D.bits(first, 21, seed, offset)
        for i, v in enumerate(got):
            block, e = divmod(first + i, 8)
            w = D.philox([block & D.WORD, block >> 32, offset & D.WORD, offset >> 32], [seed & D.WORD, seed >> 32])
            assert v == (w[e // 2] >> 16 if e % 2 else w[e // 2] & 0xFFFF)


def test_share_scale_and_edges():
    n = 1 << 18
    x = np.ones(n)
    for p in (0.1, 0.5, 0.9):
        y = D.dropout(x, p, 7, 3)
        share = (y == 0).mean()
        assert abs(share - p) < 5 * np.sqrt(p * (1 - p) / n)   # five standard deviations
        assert abs(y.mean() - 1) < 5 * np.sqrt(p / (1 - p) / n)
    assert (D.dropout(x, 0.0, 7, 3) == 1).all() and (D.dropout(x, 1.0, 7, 3) == 0).all()
    bad = np.full(64, np.nan)
    y = D.dropout(bad, 0.5, 1, 1, residual=np.ones(64))
    assert ((y == 1) | np.isnan(y)).all() and (y == 1).any() and np.isnan(y).any()


def test_masks_of_other_seeds_and_offsets_are_unrelated():
    n = 1 << 16
    a = D.bits(0, n, 1, 0) < 32768
    for seed, offset in ((2, 0), (1, 1), (1 << 32, 0), (1, 1 << 32)):
        b = D.bits(0, n, seed, offset) < 32768
        assert abs((a == b).mean() - 0.5) < 5 * 0.5 / np.sqrt(n)
