"""Both quantised writes over scales whose quotients by bf16 values come closest to the codes' ties (24-bit
integers next to multiples of 2^20, from 2^23 to just below 2^24): e4m3 under given page scales, 4 bits under
head factors, byte for byte what a division gives."""
import numpy as np
import pytest
import torch

from gqa_attention_paged_b200 import binding
from tests import _fp4 as M
from tests.test_fp4_gpu import DEV, Cache, bf16, check_write, cu_of, dev, rng

pytestmark = pytest.mark.gpu
NEAR = [(k << 20) + d for k in range(8, 17) for d in range(-4, 5) if 1 << 23 <= (k << 20) + d < 1 << 24]


def spread(r, ties, shape):
    """Ties and their bf16 neighbours (2^-8 off), of both signs."""
    return r.choice(ties, shape) * (1 + r.choice([0, 1, -1], shape) * 2.0 ** -8) * r.choice([1, -1], shape)


def test_e4m3_under_given_scales():
    r = rng(61)
    s = np.array([np.float32(n) * np.float32(2.0) ** int(e) for n in NEAR for e in (-24, -37, 3)], np.float32)
    n = len(s)
    ties = np.concatenate([(M.E4M3[1:] + M.E4M3[:-1]) / 2, M.E4M3[1:]])
    x = bf16(s.astype(np.float64)[:, None] * spread(r, ties, (n, 1920)))
    want = M.e4m3_code(M.f32(x.double().numpy() / s.astype(np.float64)[:, None]))
    pages = [torch.zeros(n, 1, 16, 128, dtype=torch.uint8, device=DEV) for _ in range(2)]
    scales = [dev(s[:, None]), dev(s[:, None])]
    rows = x.view(n * 15, 1, 128).to(DEV)
    binding.gqa_paged_write_kv(rows, rows, cu_of([15] * n), *pages, torch.arange(n, dtype=torch.int32, device=DEV)[:, None].contiguous(),
                               torch.full((n,), 16, dtype=torch.int32, device=DEV), 15, k_scale=scales[0], v_scale=scales[1])
    for p in pages:
        got = p[:, 0, 1:].reshape(n, 1920).cpu().numpy()
        assert np.array_equal(got, want), np.argwhere(got != want)[:5]


@pytest.mark.parametrize("D,exp", [(64, 0), (128, -30), (64, 25)])
def test_4_bits_under_head_factors(D, exp):
    """A block's largest value is 6 times a power of two times the factor, so that its scale is that power and
    the step the factor's significand; the others lie at the codes' ties."""
    T, Hk = 24, len(NEAR)
    c = Cache([T], Hk, D, 32, seed=62)
    g = (np.array(NEAR, np.float64) * 2.0 ** (exp - 23)).astype(np.float32)
    c.scale = [g, g[::-1].copy()]
    ties = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 1.0, 3.0, 6.0])
    rows = []
    for f in c.scale:
        x = spread(c.r, ties, (T, Hk, D // 16, 16))
        x[..., 0] = 6.0
        step = np.exp2(c.r.integers(-6, 7, (T, Hk, D // 16, 1)))
        rows.append(bf16((x * step * f.astype(np.float64)[None, :, None, None]).reshape(T, Hk, D)))
    check_write(c, [T], *rows)
