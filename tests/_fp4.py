"""Plain 64-bit model of the quantised cache (include/gqa_paged.h): the 4-bit and e4m3 formats, the
tile layout byte by byte, the chunk write, the read back and dense attention.  numpy only."""
import numpy as np

E2M1 = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])
E4M3 = np.array([(m * 2.0 ** -9) if e == 0 else (8 + m) * 2.0 ** (e - 10) for e in range(16)
                 for m in range(8)][:127])


def to_bf16(x):
    """Nearest bf16 value (ties to even) of float64 values, by way of fp32."""
    u = np.asarray(x, np.float32).view(np.uint32).astype(np.uint64)
    r = ((u + 0x7FFF + ((u >> 16) & 1)) >> 16 << 16).astype(np.uint32)
    r = np.where(np.isnan(x), np.uint32(0x7FC00000), r)
    return r.view(np.float32).astype(np.float64)


def nearest(x, grid):
    """Index of the grid value nearest to |x|, ties to the even index, saturating."""
    m = np.minimum(np.abs(x), grid[-1])
    hi = np.minimum(np.searchsorted(grid, m), len(grid) - 1)
    lo = np.maximum(hi - 1, 0)
    dn, up = m - grid[lo], grid[hi] - m
    return np.where((dn < up) | ((dn == up) & (lo % 2 == 0)), lo, hi)


def f32(x):
    return np.asarray(x, np.float64).astype(np.float32).astype(np.float64)


def quantise_fp4(x, g):
    """x [..., D] fp64 (bf16 values), g the head's factor broadcast to [...]: (codes 0..7 with the sign
    apart as -1 / 1, e4m3 scale codes [..., D / 16], 127 = NaN)."""
    b = x.reshape(*x.shape[:-1], -1, 16)
    g = np.asarray(g, np.float64)[..., None]
    with np.errstate(all="ignore"):
        a = np.abs(b).max(-1)
        t = f32(a / f32(6 * g))
        sf = nearest(t, E4M3)
        s = f32(E4M3[sf] * g)
        s = np.where(np.isnan(t), 0.0, s)[..., None]
        y = np.where(s > 0, f32(b / np.where(s > 0, s, 1.0)), 0.0)
    sf = np.where(np.isnan(t), 127, sf)
    return nearest(y, E2M1).reshape(x.shape), np.where(np.signbit(y), -1, 1).reshape(x.shape), sf


def value_fp4(code, sign, sf, g):
    e = np.append(E4M3, np.nan)
    v = E2M1[code] * sign * np.repeat(e[sf], 16, -1)
    return v * np.asarray(g, np.float64)[..., None]


def addresses(P, D, slot, is_v):
    """Of one token: (code byte [D], high nibble? [D], scale byte [D / 16]) in its (page, kv head) block."""
    d, c, t = np.arange(D), np.arange(D // 16), slot % 16
    base = slot // 16 * 9 * D
    if not is_v:
        return base + t * (D // 2) + d // 2, d % 2, base + 8 * D + t * (D // 16) + c
    C, i = D // 8, t // 2
    return (base + (i // 4) * 4 * D + (d // C) * 4 * C + (i % 4) * C + d % C, np.full(D, t % 2),
            base + 8 * D + i * (D // 8) + c * 2 + t % 2)


def token_fp4(block, P, D, slot, is_v, g):
    """fp64 values [D] of the token at `slot` of a block uint8 [P * 9 D / 16]."""
    at, high, sc = addresses(P, D, slot, is_v)
    n = np.where(high == 1, block[at] >> 4, block[at] & 15).astype(int)
    s = block[sc].astype(int)
    e = np.append(E4M3, np.nan)
    return E2M1[n & 7] * np.where(n < 8, 1, -1) * np.repeat(e[s & 127] * np.where(s < 128, 1, -1), 16) * g


def put_fp4(block, P, D, slot, is_v, x, g):
    """Store token x [D] at `slot` of `block`, in place: its own nibbles and scales only."""
    at, high, sc = addresses(P, D, slot, is_v)
    code, sign, sf = quantise_fp4(x[None], np.array([g]))
    nib = (code[0] | np.where(sign[0] < 0, 8, 0)).astype(np.uint8)
    for k in range(D):
        block[at[k]] = (block[at[k]] & 0x0F) | (nib[k] << 4) if high[k] else (block[at[k]] & 0xF0) | nib[k]
    block[sc] = sf[0]


def signless(blocks, D):
    """4-bit blocks [..., P, 9 D / 16] with every -0 code as 0, for comparing bytes."""
    t = blocks.reshape(*blocks.shape[:-2], blocks.shape[-2] // 16, 9 * D).copy()
    c = t[..., :8 * D]
    c[(c & 0x0F) == 0x08] &= 0xF0
    c[(c & 0xF0) == 0x80] &= 0x0F
    return t


def e4m3_value(code):
    e = np.append(E4M3, np.nan)
    c = code.astype(int)
    return e[c & 127] * np.where(c < 128, 1.0, -1.0)


def e4m3_code(y):
    return (nearest(y, E4M3) | np.where(np.signbit(y), 128, 0)).astype(np.uint8)


def attention(q, k, v, scale):
    """q [Hq, D], k / v [L, Hk, D] -> out [Hq, D], lse [Hq], sum p |v| [Hq, D], max |q| |k| scale [Hq]."""
    Hq, D = q.shape
    L, Hk, _ = k.shape
    if L == 0:
        return np.zeros((Hq, D)), np.full(Hq, -np.inf), np.zeros((Hq, D)), np.zeros(Hq)
    g = Hq // Hk
    qq = q.reshape(Hk, g, D)
    x = np.einsum("jgd,ljd->jgl", qq, k) * scale
    m = x.max(-1, keepdims=True)
    p = np.exp(x - m)
    z = p.sum(-1, keepdims=True)
    p /= z
    big = (np.einsum("jgd,ljd->jgl", np.abs(qq), np.abs(k)) * abs(scale)).max(-1)
    return (np.einsum("jgl,ljd->jgd", p, v).reshape(Hq, D), (m + np.log(z))[..., 0].reshape(Hq),
            np.einsum("jgl,ljd->jgd", p, np.abs(v)).reshape(Hq, D), big.reshape(Hq))
