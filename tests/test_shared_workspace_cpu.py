"""Where the 4-bit decode counts the arrivals of a cut unit's pieces (csrc/decode_fp4.cu, Arrivals): in the
workspace's 256-byte header, five bits a CTA, or a whole word for units of 32 CTAs and more."""
import random

import pytest

from gqa_attention_paged_b200 import binding

CTAS = 320  # 160 SMs x 2


def field(c0, c1):
    """(word, shift, bits) of the count of the unit from CTA c0 to c1."""
    small = c1 - c0 + 1 < 32
    return (c0 // 6 + (not small), c0 % 6 * 5 if small else 0, 5 if small else 32)


def cuts(r, ctas, longest):
    """Units that cross CTAs, in order: each begins at or behind the CTA in which the last one ends."""
    units, c = [], r.randrange(3)
    while True:
        n = r.choice([1, 1, 2, 3, r.randint(1, 12), r.randint(1, longest)])
        if c + n >= ctas:
            return units
        units.append((c, c + n))
        c += n + r.choice([0, 0, 0, 1, 5])


@pytest.mark.parametrize("longest", [5, 40, 330])
def test_counts_have_their_bits_to_themselves(longest):
    r = random.Random(longest)
    for _ in range(400):
        units = cuts(r, CTAS, longest)
        used = set()
        for c0, c1 in units:
            word, shift, bits = field(c0, c1)
            assert c1 - c0 + 1 < 1 << bits          # the last arrival carries into no other field
            assert 4 * (1 + word) < 256 and shift + bits <= 32
            mine = {(word, b) for b in range(shift, shift + bits)}
            assert not mine & used, (c0, c1)
            used |= mine


def test_every_span():
    """Any unit beside any unit that may follow or precede it."""
    for n in range(1, CTAS):
        for c0 in range(0, CTAS - n):
            word, shift, bits = field(c0, c0 + n)
            assert n + 1 < 1 << bits and 4 * (1 + word) < 256
            if bits == 32:  # the word's CTAs lie inside the unit
                assert c0 < 6 * word and 6 * word + 5 < c0 + n


def test_pieces_leave_the_other_decodes_counters_alone():
    """With the same heads, a workspace that the balanced bf16 decode fits in keeps its B * Hq counters in front
    of the 4-bit decode's pieces, which lie at the end."""
    size = binding.load().gqa_paged_decode_workspace_size
    for D in (64, 128):
        for Hk, g in ((1, 1), (8, 1), (8, 4), (2, 7), (8, 8), (4, 12), (4, 16), (1, 64)):
            four = size(1, g * Hk, Hk, D, 16, 4096, 2, 0)
            assert four % 256 == 0
            pieces = four - 256
            for B in (1, 33, 256, 2048):
                total = max(four, size(B, g * Hk, Hk, D, 16, 4096, 0, -1))
                assert (total - pieces) // 256 * 256 >= 256 + 4 * B * g * Hk
