"""The most that gqa_paged_read_kv takes, 2^43 elements: one row or page more is refused on the host (nothing is
launched), and up to there the grid of its kernel fits an int."""
import ctypes

import pytest

from gqa_attention_paged_b200 import binding

INT_MAX = 2 ** 31 - 1


def most(Hk, D):
    return INT_MAX * 256 // (Hk * (D // 16))


@pytest.mark.parametrize("Hk", [1, 3, 8, 64, 65535])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("P,paged", [(16, 0), (16, 1), (64, 1)])
def test_largest_read(Hk, D, P, paged):
    rows = most(Hk, D) // (P if paged else 1) * (P if paged else 1)
    total = rows // (P if paged else 1) + 1
    p = ctypes.c_void_p(0x10000)
    assert binding.load().gqa_paged_read_kv(p, p, None, None, 2, p, 8, None, p, p, 2, Hk, D, P, 16, total, paged,
                                            p, p, p, None) == -2
    rows = min(rows, INT_MAX * (P if paged else 1))
    per_cta = 16 if Hk >= 8 else 16 * -(-8 // Hk)
    assert -(-rows // per_cta) <= INT_MAX
    assert per_cta * Hk >= 128
