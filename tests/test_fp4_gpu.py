"""The 4-bit cache on the GPU, against the 64-bit model of tests/_fp4.py: what the write stores (byte
for byte), what the read gives back, the decode over it, and a run of all of them together.

Tolerances.  Stored codes and scales are equal.  Values read back: the fp32 product by the factor
(half a step, 2^-24) and the rounding to bf16 (2^-8), none of which the model's own bf16 rounding may
cross by more than one step: |err| <= 2^-7 |ref|; without a factor they are equal for 4 bits.  Decode:
bf16 output (2^-8 |ref|); f16 weights (2^-11 of every term, so 2^-11 sum p |v|; where a weight is subnormal
half of f16's smallest step, 2^-25, on the scale on which the largest weight is 2^7 at least: 2^-32 sum |v|
beside a largest normalised weight of at most 1); fp32 sums of at
most a few thousand terms and the exponential (2^-17 sum p |v|); a score error e changes every weight by a
relative 2 e at most, with e <= 2^-17 scale sum |q| |k| (D products added in fp32, in any order, and the
scale).  lse: e + 2^-20 (log and exp)."""
import numpy as np
import pytest
import torch

from gqa_attention_paged_b200 import binding, split_kv
from tests import _fp4 as M
from tests._util import bits

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
ROW = {"fp4": lambda D: 9 * D // 16, "e4m3": lambda D: D, "bf16": lambda D: D}


def rng(seed):
    return np.random.default_rng(seed)


def bf16(x):
    return torch.from_numpy(np.asarray(x, np.float32)).to(torch.bfloat16)


def dev(x):
    return None if x is None else torch.as_tensor(x).to(DEV)


class Cache:
    """A shuffled pool with random bytes everywhere (scales of unwritten 4-bit slots are NaN), and its
    64-bit model."""

    def __init__(self, lens, Hk, D, P, kv="fp4", seed=0, factor=False, extra_pages=3):
        r = rng(seed)
        self.r, self.Hk, self.D, self.P, self.kv = r, Hk, D, P, kv
        need = [(n + P - 1) // P for n in lens]
        self.pages = sum(need) + extra_pages
        perm = r.permutation(self.pages)
        self.table = np.full((len(lens), max(1, max(need))), perm[-1], np.int32)
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = perm[at:at + n]
            at += n
        self.lens = np.array(lens, np.int32)
        shape = (self.pages, Hk, P, ROW[kv](D))
        self.raw = [r.integers(0, 256, shape, dtype=np.uint8) for _ in range(2)]
        if kv == "bf16":
            self.raw = [bits(bf16(r.normal(size=shape))) for _ in range(2)]
        if kv == "fp4":
            for x in self.raw:
                x.reshape(self.pages, Hk, P // 16, 9 * D)[..., 8 * D:] = 0x7F
            self.scale = [r.uniform(0.3, 3, Hk).astype(np.float32) if factor else None for _ in range(2)]
        elif kv == "e4m3":
            self.scale = [r.uniform(0.005, 0.02, (self.pages, Hk)).astype(np.float32) for _ in range(2)]
        else:
            self.scale = [None, None]

    def g(self, i, j):
        return 1.0 if self.scale[i] is None else float(self.scale[i][j])

    def place(self, b, t):
        return int(self.table[b, t // self.P]), t % self.P

    def write(self, b, t0, k, v):
        """Model: rows k / v [n][Hk][D] become tokens t0 .. of sequence b."""
        for i, rows in enumerate((k, v)):
            rows = np.asarray(rows, np.float64)
            n = rows.shape[0]
            if self.kv == "e4m3":
                for p in range(t0 // self.P, (t0 + n - 1) // self.P + 1):
                    lo, hi = max(t0, p * self.P), min(t0 + n, (p + 1) * self.P)
                    if lo == p * self.P:
                        big = np.abs(rows[lo - t0:hi - t0]).max((0, 2))
                        self.scale[i][self.table[b, p]] = np.where(
                            big > 0, big.astype(np.float32) / np.float32(448), np.float32(1))
            for x in range(n):
                page, slot = self.place(b, t0 + x)
                for j in range(self.Hk):
                    if self.kv == "fp4":
                        M.put_fp4(self.raw[i][page, j].reshape(-1), self.P, self.D, slot, i == 1, rows[x, j],
                                  self.g(i, j))
                    elif self.kv == "e4m3":
                        s = float(self.scale[i][page, j])
                        self.raw[i][page, j, slot] = M.e4m3_code(M.f32(rows[x, j] / s))
                    else:
                        self.raw[i][page, j, slot] = bits(bf16(rows[x, j]))

    def values(self, b, i, t0=0, t1=None):
        """fp64 [n][Hk][D] of tokens t0 .. t1 of sequence b."""
        t1 = int(self.lens[b]) if t1 is None else t1
        out = np.zeros((max(0, t1 - t0), self.Hk, self.D))
        for t in range(t0, t1):
            page, slot = self.place(b, t)
            for j in range(self.Hk):
                if self.kv == "fp4":
                    out[t - t0, j] = M.token_fp4(self.raw[i][page, j].reshape(-1), self.P, self.D, slot, i == 1,
                                                 self.g(i, j))
                elif self.kv == "e4m3":
                    out[t - t0, j] = M.e4m3_value(self.raw[i][page, j, slot]) * float(self.scale[i][page, j])
                else:
                    out[t - t0, j] = (self.raw[i][page, j, slot].astype(np.uint32) << 16).view(np.float32)
        return out

    def fill(self):
        """Every token of every sequence, in the model."""
        for b, n in enumerate(self.lens):
            if n:
                shape = (int(n), self.Hk, self.D)
                self.write(b, 0, bf16(self.r.normal(size=shape)).double(), bf16(self.r.normal(size=shape)).double())
        return self

    def to_gpu(self):
        k, v = (dev(x.view(np.int16)).view(torch.bfloat16) if self.kv == "bf16" else dev(x) for x in self.raw)
        return dict(k_pages=k, v_pages=v, page_table=dev(self.table), seq_lens=dev(self.lens),
                    k_scale=dev(self.scale[0]), v_scale=dev(self.scale[1]))

    def assert_same(self, d):
        for i, name in enumerate(("k_pages", "v_pages")):
            got, want = bits(d[name]), self.raw[i]
            if self.kv == "fp4":
                got, want = M.signless(got, self.D), M.signless(want, self.D)
            assert np.array_equal(got, want), f"{name}: {int((got != want).sum())} bytes differ"
        if self.kv == "e4m3":
            assert np.array_equal(d["k_scale"].cpu().numpy(), self.scale[0])
            assert np.array_equal(d["v_scale"].cpu().numpy(), self.scale[1])


def rows_for(c, counts, spread=1.0):
    n = int(sum(counts))
    x = c.r.normal(size=(2, n, c.Hk, c.D)) * np.exp(c.r.normal(size=(2, n, c.Hk, 1)) * spread)
    return bf16(x[0]), bf16(x[1])


def cu_of(counts, dtype=torch.int32):
    cu = torch.zeros(len(counts) + 1, dtype=dtype)
    cu[1:] = torch.cumsum(torch.tensor([int(x) for x in counts]), 0)
    return cu.to(DEV)


def check_write(c, counts, k, v, strided=False):
    d = c.to_gpu()
    if strided:  # rows of a fused projection, with something else in front
        wide = torch.full((k.shape[0], 3 * c.Hk, c.D), 7.0, dtype=torch.bfloat16)
        wide[:, c.Hk:2 * c.Hk], wide[:, 2 * c.Hk:] = k, v
        wide = wide.to(DEV)
        kd, vd = wide[:, c.Hk:2 * c.Hk], wide[:, 2 * c.Hk:]
    else:
        kd, vd = k.to(DEV), v.to(DEV)
    ws = binding.gqa_paged_write_kv(kd, vd, cu_of(counts), d["k_pages"], d["v_pages"], d["page_table"],
                                    d["seq_lens"], max(counts), k_scale=d["k_scale"], v_scale=d["v_scale"])
    assert binding.gqa_get_error(ws) == 0
    at = 0
    for b, n in enumerate(counts):
        if n:
            c.write(b, int(c.lens[b]) - n, k[at:at + n].double().numpy(), v[at:at + n].double().numpy())
        at += n
    c.assert_same(d)


# ------------------------------------------------------------------------------------ writing

@pytest.mark.parametrize("kv", ["fp4", "e4m3", "bf16"])
@pytest.mark.parametrize("D,P,Hk", [(128, 16, 2), (64, 32, 3), (128, 64, 1), (64, 16, 1)])
def test_write_is_bit_exact(kv, D, P, Hk):
    # whole, partial and continued pages; chunks that begin and end on the odd token of a pair;
    # one token, none, and a whole new sequence
    lens, counts = [37, P + 1, 3 * P, 20, 5, 0, 2 * P + 7], [37, 1, 2 * P + 3, 7, 0, 0, 2]
    c = Cache(lens, Hk, D, P, kv, seed=D + P, factor=(D == 64))
    check_write(c, counts, *rows_for(c, counts), strided=(P == 32))


def test_write_special_values():
    c = Cache([16], 1, 128, 16, "fp4", seed=5)
    x = np.zeros((16, 1, 128))
    ties = [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0]  # halfway between codes at scale 1
    x[0, 0, :16] = ties + [-t for t in ties]
    x[1] = 1e-30                       # the scale rounds to 0
    x[2, 0, 3] = np.inf
    x[2, 0, 4] = 1.0
    x[3, 0, 40] = np.nan               # one block of the token is NaN
    x[4] = 3e38                        # the scale saturates
    x[5, 0, ::2] = -0.0
    x[6, 0] = c.r.normal(size=128) * 1e-3   # subnormal scales
    x[7, 0, :16] = [6.375] + [1.0] * 15     # a / 6 is halfway between two e4m3 scales
    x[8:] = c.r.normal(size=(8, 1, 128)) * 100
    k = bf16(x)
    check_write(c, [16], k, k.flip(0).contiguous())


def test_write_of_one_token_is_the_append():
    for kv in ("fp4", "e4m3", "bf16"):
        lens = [1, 17, 32, 0, 40, 50]
        counts = [1, 1, 1, 0, 1, 1]
        c = Cache(lens, 2, 128, 16, kv, seed=9)
        k, v = rows_for(c, [1] * 6)
        a, w = c.to_gpu(), c.to_gpu()
        ws = binding.gqa_paged_append_kv(k.to(DEV), v.to(DEV), **a)
        pick = [b for b in range(6) if counts[b]]
        binding.gqa_paged_write_kv(k[pick].to(DEV), v[pick].to(DEV), cu_of(counts), w["k_pages"], w["v_pages"],
                                   w["page_table"], w["seq_lens"], 1, k_scale=w["k_scale"], v_scale=w["v_scale"])
        assert binding.gqa_get_error(ws) == 0
        for n in ("k_pages", "v_pages", "k_scale", "v_scale"):
            assert a[n] is None or np.array_equal(a[n].view(torch.uint8).cpu(), w[n].view(torch.uint8).cpu()), n
        for b in pick:
            c.write(b, lens[b] - 1, k[b:b + 1].double().numpy(), v[b:b + 1].double().numpy())
        c.assert_same(a)


@pytest.mark.parametrize("kv", ["fp4", "e4m3"])
def test_write_refuses_what_does_not_fit(kv):
    """A bad page, a chunk longer than its sequence, longer than max_q_len, rows past total_q and a sequence
    past the page table are recorded and not written; the others are."""
    for bad in range(5):
        c = Cache([40, 20, 30], 1, 64, 16, kv, seed=11)
        counts = [10, 20, 8]
        k, v = rows_for(c, counts)
        d, cu, mq = c.to_gpu(), cu_of(counts), 20
        before = [bits(d["k_pages"]).copy(), bits(d["v_pages"]).copy()]
        if bad == 0:
            d["page_table"][1, 0] = c.pages + 3
        elif bad == 1:
            d["seq_lens"][1] = 19
        elif bad == 2:
            mq = 19
        elif bad == 3:
            cu[2:] += 20       # sequence 1's rows end past the others', sequence 2's past total_q
            cu[3] = 1 << 20
        else:
            d["seq_lens"][1] = 16 * d["page_table"].shape[1] + 1
        ws = binding.gqa_paged_write_kv(k.to(DEV), v.to(DEV), cu, d["k_pages"], d["v_pages"], d["page_table"],
                                        d["seq_lens"], mq, k_scale=d["k_scale"], v_scale=d["v_scale"])
        assert binding.gqa_get_error(ws) == -7, bad
        assert binding.gqa_get_error(ws) == 0
        # sequence 0 is written whatever befell the others
        c.write(0, 30, k[:10].double().numpy(), v[:10].double().numpy())
        for i, name in enumerate(("k_pages", "v_pages")):
            pages = c.table[0, :3]
            got, want = bits(d[name])[pages], c.raw[i][pages]
            if kv == "fp4":
                got, want = M.signless(got, 64), M.signless(want, 64)
            assert np.array_equal(got, want), bad
            if bad in (1, 2, 4):  # nothing of sequence 1
                assert np.array_equal(bits(d[name])[c.table[1, :2]], before[i][c.table[1, :2]]), bad


def test_write_of_many_sequences():
    """More sequences than a CTA keeps one by one; chunks of none to a few tokens."""
    r = rng(17)
    counts = [int(x) for x in r.integers(0, 4, 300)]
    lens = [n + int(x) for n, x in zip(counts, r.integers(0, 20, 300))]
    for kv in ("fp4", "e4m3"):
        c = Cache(lens, 1, 64, 16, kv, seed=18)
        check_write(c, counts, *rows_for(c, counts))


def test_quotients_are_a_divisions():
    """e4m3 codes under given page scales: bf16 values at and around every tie of the codes, over scales whose
    quotients come closest to one (24-bit integers next to multiples of 2^20), random ones, and ones at the
    ends of the range, negative and zero."""
    r = rng(19)
    near = [(k << 20) + d for k in range(8, 16) for d in range(-4, 5)]
    s = [np.float32(x) * np.float32(2.0) ** int(e) for x, e in zip(near, r.integers(-40, 20, len(near)))]
    s += list(r.uniform(0.5, 2, 60).astype(np.float32) * np.exp2(r.integers(-30, 30, 60)).astype(np.float32))
    s += [np.float32(x) for x in (0, 1e-45, 3e-41, 1.2e-38, 2.0 ** -61, 2.0 ** 61, 1e30, 3e38, -0.37, -1e-20)]
    s = np.array(s, np.float32)
    n = len(s)
    ties = np.concatenate([(M.E4M3[1:] + M.E4M3[:-1]) / 2, M.E4M3[1:], [480.0, 1e6, 1e30]])
    with np.errstate(over="ignore"):
        t = np.abs(s.astype(np.float64))[:, None] * r.choice(ties, (n, 1920)) * (1 + r.choice([0, 1, -1], (n, 1920)) * 2.0 ** -8)
    x = np.clip(t, 2.0 ** -126, 3e38) * r.choice([1, -1], (n, 1920))
    x[:, 0], x[:, 1] = 0.0, -0.0
    x = bf16(x)
    xs = x.double().numpy()
    with np.errstate(all="ignore"):
        y = (xs.astype(np.float32) / s[:, None]).astype(np.float64)
    keep = ~np.isnan(y)  # 0 / 0
    want = M.e4m3_code(np.where(keep, y, 0.0))
    pages = [torch.zeros(n, 1, 16, 128, dtype=torch.uint8, device=DEV) for _ in range(2)]
    scales = [dev(s[:, None]), dev(s[:, None])]
    table = torch.arange(n, dtype=torch.int32, device=DEV)[:, None].contiguous()
    rows = x.view(n * 15, 1, 128).to(DEV)
    binding.gqa_paged_write_kv(rows, rows, cu_of([15] * n), *pages, table, torch.full((n,), 16, dtype=torch.int32, device=DEV),
                               15, k_scale=scales[0], v_scale=scales[1])
    for p, sc in zip(pages, scales):
        got = p[:, 0, 1:].reshape(n, 1920).cpu().numpy()
        assert np.array_equal(got[keep], want[keep]), np.argwhere((got != want) & keep)[:5]
        assert np.array_equal(sc.cpu().numpy()[:, 0], s)


# ------------------------------------------------------------------------------------ reading

@pytest.mark.parametrize("kv", ["fp4", "e4m3", "bf16"])
@pytest.mark.parametrize("D,P,Hk", [(128, 16, 2), (64, 32, 3), (128, 64, 1)])
@pytest.mark.parametrize("paged", [False, True])
def test_read_gives_the_stored_values(kv, D, P, Hk, paged):
    lens, starts = [P + 5, 0, 1, 3 * P, 17, 40], [3, 0, 0, P, 17, 0]
    c = Cache(lens, Hk, D, P, kv, seed=D * P, factor=(Hk == 3)).fill()
    d = c.to_gpu()
    first = [s // P for s in starts]
    counts = [(n + P - 1) // P - f if n > s else 0 for n, s, f in zip(lens, starts, first)] if paged else \
        [n - s for n, s in zip(lens, starts)]
    total = sum(counts)
    shape = (total, Hk, P, D) if paged else (total, Hk, D)
    mark = [torch.full(shape, 123.0, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    ws = binding.new_workspace(256, DEV)
    got = binding.gqa_paged_read_kv(d["k_pages"], d["v_pages"], d["page_table"], d["seq_lens"],
                                    cu_of(counts, torch.int64), total, starts=dev(np.array(starts, np.int32)),
                                    k_scale=d["k_scale"], v_scale=d["v_scale"], paged=paged, k_out=mark[0],
                                    v_out=mark[1], workspace=ws)
    assert binding.gqa_get_error(ws) == 0
    for i in range(2):
        want = np.full(shape, 123.0)
        at = 0
        for b, n in enumerate(counts):
            if n and paged:
                for t in range(starts[b], lens[b]):
                    want[at + t // P - first[b], :, t % P] = c.values(b, i, t, t + 1)[0]
            elif n:
                want[at:at + n] = c.values(b, i, starts[b])
            at += n
        o = got[i].double().cpu().numpy()
        if kv == "e4m3" or c.scale[i] is not None:
            assert np.all(np.abs(o - want) <= 2.0 ** -7 * np.abs(want))
        else:
            assert np.array_equal(o, want)


def test_read_records_rows_past_the_sequence():
    c = Cache([20, 16], 1, 64, 16, seed=3).fill()
    d = c.to_gpu()
    ws = binding.new_workspace(256, DEV)
    k, _ = binding.gqa_paged_read_kv(d["k_pages"], d["v_pages"], d["page_table"], d["seq_lens"],
                                     cu_of([20, 17], torch.int64), 37, workspace=ws,
                                     k_out=torch.full((37, 1, 64), 5.0, dtype=torch.bfloat16, device=DEV))
    assert binding.gqa_get_error(ws) == -7
    assert torch.all(k[36] == 5.0)
    assert np.array_equal(k[20:36].double().cpu().numpy(), c.values(1, 0))
    d["page_table"][0, 0] = -1
    binding.gqa_paged_read_kv(d["k_pages"], d["v_pages"], d["page_table"], d["seq_lens"],
                              cu_of([20, 16], torch.int64), 36, workspace=ws)
    assert binding.gqa_get_error(ws) == -7


# ------------------------------------------------------------------------------------- decode

def expect(c, q, scale):
    B = q.shape[0]
    res = [M.attention(q[b].double().numpy(), c.values(b, 0), c.values(b, 1), scale) for b in range(B)]
    sv = [np.repeat(np.abs(c.values(b, 1)).sum(0), q.shape[1] // c.Hk, 0) for b in range(B)]
    return [np.stack([x[i] for x in res]) for i in range(4)] + [np.stack(sv)]


def close(out, lse, ref, f32_out=False):
    o, l, pv, big, sv = ref
    got = out.double().cpu().numpy()
    e = 2.0 ** -17 * big
    tol = (0 if f32_out else 2.0 ** -8) * np.abs(o) + (2.0 ** -11 + 2.0 ** -17 + 2 * e[..., None]) * pv \
        + 2.0 ** -32 * sv + 1e-30
    bad = ~(np.abs(got - o) <= tol)
    assert not bad.any(), f"{int(bad.sum())} of {bad.size}: worst {np.nanmax(np.abs(got - o) / tol):.2f} times the tolerance"
    if lse is not None:
        g = lse.double().cpu().numpy()
        fin = np.isfinite(l)
        assert np.array_equal(fin, np.isfinite(g))
        assert np.all(g[~fin] == -np.inf)
        assert np.all(np.abs(g[fin] - l[fin]) <= (e + 2.0 ** -20 + 2.0 ** -23 * np.abs(l))[fin])


def queries(c, B, Hq, seed=1):
    return bf16(rng(seed).normal(size=(B, Hq, c.D)))


CASES = [
    # Hq, Hk, D, P, lens
    (8, 2, 64, 16, [37, 100]),
    (8, 2, 128, 16, [1, 2, 15, 16, 17, 31, 33, 0]),
    (4, 1, 128, 64, [200, 0, 65, 64]),
    (3, 3, 128, 32, [50, 7]),             # one query head per kv head
    (14, 2, 64, 32, [129, 300, 5]),       # groups of 7
    (16, 1, 128, 16, [90, 260]),          # groups of 16
    (24, 1, 128, 16, [77, 150]),          # groups of 24: more than one block of heads
    (40, 2, 64, 64, [64, 191]),           # groups of 20
    (12, 1, 128, 16, [400]),              # groups of 12
    (8, 1, 128, 16, [2100]),              # one long sequence
    (2, 1, 64, 16, [16] * 70 + [0] * 5 + [33] * 3),   # many short ones
    # a sequence above 1024 tokens: the whole batch is cut into equal shares, units between CTAs
    (8, 2, 64, 16, [37, 1100, 0, 1]),
    (16, 1, 128, 16, [1300, 90, 31]),
    (24, 1, 128, 32, [16, 0, 1100]),
    (14, 2, 64, 32, [1200, 5]),
    (4, 1, 128, 64, [0, 1030, 65, 64]),
    (4, 2, 64, 16, [1025] * 3),
    (4, 2, 64, 16, [1024, 1023, 993, 992, 33, 32]),   # 32 steps and just below: a CTA per unit
]


@pytest.mark.parametrize("case", range(len(CASES)))
def test_decode_matches_the_model(case):
    Hq, Hk, D, P, lens = CASES[case]
    c = Cache(lens, Hk, D, P, seed=case, factor=case % 2 == 1).fill()
    q, scale = queries(c, len(lens), Hq), D ** -0.5
    ref = expect(c, q, scale)
    d = c.to_gpu()
    ws = binding.new_workspace(binding.gqa_paged_decode_workspace_size(
        len(lens), Hq, Hk, D, P, d["page_table"].shape[1] * P, 2, 0), DEV)
    out, lse = binding.gqa_paged_decode(q.to(DEV), scale=scale, workspace=ws, **d)
    close(out, lse, ref)
    assert binding.gqa_get_error(ws) == 0
    # again on the same workspace: the same bits; without lse; on request balanced; one head a block
    again, _ = binding.gqa_paged_decode(q.to(DEV), scale=scale, workspace=ws, want_lse=False, num_splits=-1, **d)
    assert torch.equal(out.view(torch.int16), again.view(torch.int16))
    one, lse1 = binding.gqa_paged_decode(q.to(DEV), scale=scale, workspace=ws, pack_gqa=False, **d)
    close(one, lse1, ref)
    part, lsep = binding.gqa_paged_decode_partial(q.to(DEV), scale=scale, workspace=ws, **d)
    assert part.dtype == torch.float32
    close(part, lsep, ref, f32_out=True)
    stat, lses = binding.gqa_paged_decode_static_scratch(q.to(DEV), scale=scale, **d)
    assert torch.equal(stat.view(torch.int16), out.view(torch.int16)) and torch.equal(lses, lse)


@pytest.mark.parametrize("B,per", [(257, 7), (700, 40)])
def test_decode_of_many_sequences(B, per):
    """More sequences than the kernel keeps one by one: runs of them, empty ones inside and at the ends."""
    r = rng(B)
    lens = [int(x) if x > 2 else 0 for x in r.integers(0, per, B)]
    lens[0] = lens[-1] = lens[255] = 0
    c = Cache(lens, 1, 64, 16, seed=B).fill()
    q, scale = queries(c, B, 2), 0.125
    out, lse = binding.gqa_paged_decode(q.to(DEV), scale=scale, **c.to_gpu())
    close(out, lse, expect(c, q, scale))


LARGE = [
    # B, Hq, Hk, D, P, longest, share of empty sequences: several steps for every warp of the GPU
    (128, 32, 8, 128, 16, 2500, 0.1),
    (600, 32, 8, 128, 16, 700, 0.4),      # runs of sequences
    (90, 56, 8, 64, 64, 4000, 0.0),
    (48, 64, 4, 128, 32, 3000, 0.05),     # two blocks of heads
    (3, 64, 8, 128, 64, 33000, 0.0),
    (256, 8, 8, 128, 16, 1100, 0.9),
]


@pytest.mark.parametrize("case", range(len(LARGE)))
def test_decode_of_large_batches_is_the_bf16_decode_of_what_is_read_back(case):
    """Code times scale is a bf16 value, so the cache read back is exact and the bf16 decode over it says the
    same.  Both outputs are rounded to bf16 (2^-8 of each), the weights here are f16 (2^-11, and fp32 work of
    2^-15) and there two bf16 terms (2^-15); a score error of 2^-17 scale sum |q| |k| on either side."""
    B, Hq, Hk, D, P, most, none = LARGE[case]
    r = rng(100 + case)
    lens = r.integers(1, most + 1, B)
    lens[r.uniform(size=B) < none] = 0
    lens[-1] = max(lens[-1], 1)
    need = (lens + P - 1) // P
    pages = int(need.sum()) + 3
    perm = r.permutation(pages).astype(np.int32)
    table = np.full((B, max(1, int(need.max()))), -1, np.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = perm[at:at + n]
        at += n
    gen = torch.Generator(DEV).manual_seed(case)
    pools = []
    for _ in range(2):
        x = torch.randint(0, 256, (pages, Hk, P // 16, 9 * D), generator=gen, device=DEV, dtype=torch.uint8)
        x[..., 8 * D:] = torch.randint(0x20, 0x39, x[..., 8 * D:].shape, generator=gen, device=DEV, dtype=torch.uint8)
        pools.append(x.view(pages, Hk, P, 9 * D // 16))
    table, sl = dev(table), dev(lens.astype(np.int32))
    q = torch.randn(B, Hq, D, generator=gen, device=DEV).to(torch.bfloat16)
    scale = 0.5 * D ** -0.5
    ws = binding.new_workspace(16 << 20, DEV)
    out, lse = binding.gqa_paged_decode(q, *pools, table, sl, scale, workspace=ws)
    cu = cu_of(need, torch.int64)
    kb, vb = binding.gqa_paged_read_kv(*pools, table, sl, cu, int(need.sum()), paged=True, workspace=ws,
                                       k_out=torch.zeros(int(need.sum()), Hk, P, D, dtype=torch.bfloat16, device=DEV),
                                       v_out=torch.zeros(int(need.sum()), Hk, P, D, dtype=torch.bfloat16, device=DEV))
    assert binding.gqa_get_error(ws) == 0
    cols = torch.arange(table.shape[1], device=DEV)
    back = (cu[:-1, None] + cols).to(torch.int32).clamp(max=int(need.sum()) - 1).contiguous()
    ref, lref = binding.gqa_paged_decode(q, kb, vb, back, sl, scale)
    pv, _ = binding.gqa_paged_decode(q, kb, vb.abs(), back, sl, scale)
    o, got, pv = ref.double(), out.double(), pv.double() * (1 + 2.0 ** -7)
    e = 2 * 2.0 ** -17 * scale * (q.abs().double().sum(-1) * kb.abs().max().double())
    tol = 2.0 ** -7 * o.abs() + (2.0 ** -11 + 2.0 ** -14 + 2 * e[..., None]) * pv + 1e-30
    assert bool(((got - o).abs() <= tol).all()), float(((got - o).abs() / tol).max())
    fin = torch.isfinite(lref)
    assert torch.equal(fin, torch.isfinite(lse)) and torch.equal(fin, (sl > 0)[:, None].expand_as(fin))
    assert bool(((lse - lref).abs() <= e.float() + 2.0 ** -18 + 2.0 ** -21 * lref.abs())[fin].all())


def test_one_workspace_for_changing_batches():
    """Batch sizes and head counts in turn on one workspace that was zeroed once."""
    ws = binding.new_workspace(16 << 20, DEV)
    shapes = [([1300], 8, 2, 128), ([200, 90, 310] * 4, 8, 2, 128), ([1700], 16, 1, 64), ([5] * 40 + [1400], 4, 2, 128)]
    batches = []
    for i, (lens, Hq, Hk, D) in enumerate(shapes):
        c = Cache(lens, Hk, D, 16, seed=70 + i).fill()
        q = queries(c, len(lens), Hq)
        batches.append((c.to_gpu(), q.to(DEV), expect(c, q, 0.1)))
    for i in (0, 1, 2, 3, 1, 0, 3, 2):
        d, q, ref = batches[i]
        out, lse = binding.gqa_paged_decode(q, scale=0.1, workspace=ws, **d)
        close(out, lse, ref)
    assert binding.gqa_get_error(ws) == 0


def test_two_decodes_at_once():
    """Two streams, a workspace each."""
    c = Cache([1100, 300], 2, 128, 16, seed=81).fill()
    d, ref = c.to_gpu(), None
    q = queries(c, 2, 8)
    ref, qd = expect(c, q, 0.1), q.to(DEV)
    streams = [torch.cuda.Stream() for _ in range(2)]
    bufs = [(torch.empty_like(qd), torch.empty(2, 8, device=DEV), binding.new_workspace(4 << 20, DEV)) for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(20):
        for s, (out, lse, ws) in zip(streams, bufs):
            binding.gqa_paged_decode(qd, scale=0.1, out=out, lse=lse, workspace=ws, stream=s, **d)
    torch.cuda.synchronize()
    for out, lse, ws in bufs:
        close(out, lse, ref)


@pytest.mark.parametrize("what", ["large q", "small q", "mixed heads", "large scale", "negative scale", "zero scale"])
def test_decode_score_ranges(what):
    c = Cache([70, 33], 2, 128, 16, seed=21).fill()
    q, scale = queries(c, 2, 8).double().numpy(), 128 ** -0.5
    if what == "large q":
        q *= 2.0 ** 100
        scale *= 2.0 ** -99
    elif what == "small q":
        q *= 2.0 ** -100
        scale *= 2.0 ** 98
    elif what == "mixed heads":  # heads of one group 2^60 apart
        q *= np.exp2(np.linspace(-30, 3, 8)).reshape(1, 8, 1)
    elif what == "large scale":
        scale = 3.0
    elif what == "negative scale":
        scale = -scale
    else:
        scale = 0.0
    q = bf16(q)
    ref = expect(c, q, scale)
    out, lse = binding.gqa_paged_decode(q.to(DEV), scale=scale, **c.to_gpu())
    close(out, lse, ref)


def test_decode_of_extreme_blocks():
    """The largest and smallest scales, zero blocks, codes of both signs; a NaN stays in its sequence and
    kv head."""
    c = Cache([40, 40, 40], 2, 64, 16, seed=23)
    x = c.r.normal(size=(2, 120, 2, 64))
    x[:, :40] *= 2688 / 6
    x[:, 40:80] *= 2.0 ** -7
    x[:, 85:90] = 0
    k, v = bf16(x[0]), bf16(x[1])
    for b in range(3):
        c.write(b, 0, k[40 * b:40 * b + 40].double().numpy(), v[40 * b:40 * b + 40].double().numpy())
    q, scale = queries(c, 3, 8), 2.0 ** -12
    ref = expect(c, q, scale)
    d = c.to_gpu()
    out, lse = binding.gqa_paged_decode(q.to(DEV), scale=scale, **d)
    close(out, lse, ref)
    page, slot = c.place(1, 37)
    c.raw[1][page, 1].reshape(-1)[M.addresses(16, 64, slot, True)[2][0]] = 0x7F
    d = c.to_gpu()
    got, _ = binding.gqa_paged_decode(q.to(DEV), scale=scale, **d)
    bad = torch.isnan(got.float())
    assert bad[1, 4:, :16].all() and int(bad.sum()) == 4 * 16
    keep = ~bad
    assert torch.equal(got[keep], out[keep])


def test_decode_shared_pages_and_masked_table():
    """A prefix page shared by all sequences, the same page twice in one; entries past a sequence's pages
    are not read."""
    c = Cache([48, 40, 33], 1, 128, 16, seed=25).fill()
    c.table[1:, 0] = c.table[0, 0]
    c.table[2, 1] = c.table[2, 0]
    q, scale = queries(c, 3, 4), 0.09
    ref = expect(c, q, scale)
    wide = np.full((3, 9), -5, np.int32)
    wide[:, :3] = c.table
    d = dict(c.to_gpu(), page_table=dev(wide))
    ws = binding.new_workspace(1 << 24, DEV)
    out, lse = binding.gqa_paged_decode(q.to(DEV), scale=scale, workspace=ws, **d)
    assert binding.gqa_get_error(ws) == 0
    close(out, lse, ref)


def test_decode_records_bad_pages_and_lengths():
    c = Cache([48, 40], 1, 128, 16, seed=26).fill()
    q = queries(c, 2, 4).to(DEV)
    ref = expect(c, q.cpu(), 0.09)
    ws = binding.new_workspace(1 << 24, DEV)
    for what in ("high", "negative", "long", "below"):
        d = c.to_gpu()
        if what == "high":
            d["page_table"][1, 1] = c.pages
        elif what == "negative":
            d["page_table"][1, 1] = -1
        elif what == "long":
            d["seq_lens"][1] = 49
        else:
            d["seq_lens"][1] = -3
        out, _ = binding.gqa_paged_decode(q, scale=0.09, workspace=ws, **d)
        assert binding.gqa_get_error(ws) == -7, what
        close(out[:1], None, [x[:1] for x in ref])
    ws.zero_()
    out, lse = binding.gqa_paged_decode(q, scale=0.09, workspace=ws, **c.to_gpu())
    close(out, lse, ref)


def test_decode_offsets_past_32_bits():
    """Pools of more than 2^32 bytes, the tokens in their last pages."""
    D, P, Hk = 128, 64, 8
    pages = (1 << 32) // (Hk * P * 72) + 40
    small = Cache([150, 70], Hk, D, P, seed=27).fill()
    q = queries(small, 2, 16)
    ref = expect(small, q, 0.09)
    d = small.to_gpu()
    for n in ("k_pages", "v_pages"):
        big = torch.empty(pages, Hk, P, 72, dtype=torch.uint8, device=DEV)
        big[pages - small.pages:] = d[n]
        d[n] = big
    d["page_table"] += pages - small.pages
    out, lse = binding.gqa_paged_decode(q.to(DEV), scale=0.09, **d)
    close(out, lse, ref)
    k, v = rows_for(small, [3, 2])
    binding.gqa_paged_write_kv(k.to(DEV), v.to(DEV), cu_of([3, 2]), d["k_pages"], d["v_pages"], d["page_table"],
                               d["seq_lens"], 3)
    small.write(0, 147, k[:3].double().numpy(), v[:3].double().numpy())
    small.write(1, 68, k[3:].double().numpy(), v[3:].double().numpy())
    rk, rv = binding.gqa_paged_read_kv(d["k_pages"], d["v_pages"], d["page_table"], d["seq_lens"],
                                       cu_of([150, 70], torch.int64), 220)
    for got, i in ((rk, 0), (rv, 1)):
        assert np.array_equal(got.double().cpu().numpy(), np.concatenate([small.values(0, i), small.values(1, i)]))


def test_calls_refuse_another_device(monkeypatch):
    """The current stream belongs to the current device: tensors of another one are refused."""
    c = Cache([20, 16], 1, 64, 16, seed=3).fill()
    d, q = c.to_gpu(), queries(c, 2, 4).to(DEV)
    k = torch.zeros(2, 1, 64, dtype=torch.bfloat16, device=DEV)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    for call in (lambda: binding.gqa_paged_decode(q, scale=0.1, **d),
                 lambda: binding.gqa_paged_decode_partial(q, scale=0.1, **d),
                 lambda: binding.gqa_paged_decode_static_scratch(q, scale=0.1, **d),
                 lambda: binding.gqa_paged_append_kv(k, k, **d),
                 lambda: binding.gqa_paged_append_decode(q, k, k, scale=0.1, **d),
                 lambda: binding.gqa_paged_write_kv(k, k, cu_of([1, 1]), d["k_pages"], d["v_pages"], d["page_table"],
                                                    d["seq_lens"], 1),
                 lambda: binding.gqa_paged_read_kv(d["k_pages"], d["v_pages"], d["page_table"], d["seq_lens"],
                                                   cu_of([20, 16], torch.int64), 36)):
        with pytest.raises(ValueError, match="current device"):
            call()


def test_binding_refuses_what_does_not_fit():
    c = Cache([20, 16], 2, 64, 16, seed=3).fill()
    d, q = c.to_gpu(), queries(c, 2, 4).to(DEV)
    k = torch.zeros(2, 2, 64, dtype=torch.bfloat16, device=DEV)
    cu, cu64 = cu_of([1, 1]), cu_of([20, 16], torch.int64)
    pools = (d["k_pages"], d["v_pages"], d["page_table"], d["seq_lens"])
    bad = torch.ones(3, device=DEV)
    with pytest.raises(ValueError, match="k_scale"):
        binding.gqa_paged_decode(q, *pools, 0.1, k_scale=bad)
    with pytest.raises(ValueError, match="v_scale"):
        binding.gqa_paged_write_kv(k, k, cu, *pools, 1, v_scale=bad)
    with pytest.raises(ValueError, match="head_dim"):
        binding.gqa_paged_decode(torch.zeros(2, 4, 128, dtype=torch.bfloat16, device=DEV), *pools, 0.1)
    with pytest.raises(ValueError, match="contiguous"):
        wide = torch.zeros(2, 2, 128, dtype=torch.bfloat16, device=DEV)
        binding.gqa_paged_write_kv(wide[..., :64], k, cu, *pools, 1)
    with pytest.raises(ValueError, match="shape"):
        binding.gqa_paged_write_kv(k, k[:, :1], cu, *pools, 1)
    with pytest.raises(TypeError):
        binding.gqa_paged_write_kv(k.float(), k, cu, *pools, 1)
    with pytest.raises(TypeError):
        binding.gqa_paged_read_kv(*pools, cu, 36)
    with pytest.raises(ValueError, match="shape"):
        binding.gqa_paged_read_kv(*pools, cu64, 36, k_out=k, v_out=k)
    with pytest.raises(ValueError, match="workspace"):
        binding.gqa_paged_read_kv(*pools, cu64, 36, workspace=torch.zeros(64, dtype=torch.uint8, device=DEV))
    with pytest.raises(binding.GQAError):
        binding.gqa_paged_decode(q, *pools, 0.1, num_splits=2)
    with pytest.raises(binding.GQAError):
        binding.gqa_paged_decode(q, *pools, 0.1, workspace=torch.zeros(256, dtype=torch.uint8, device=DEV))
    # rows of one token need no contiguous stride
    one = torch.zeros(4, 2, 64, dtype=torch.bfloat16, device=DEV)[::4]
    binding.gqa_paged_write_kv(one, one, cu_of([1, 0]), *pools, 1)


def test_compiled_calls_take_valid_tensors_only():
    """The compiled half of the binding makes the calls that Python's checks would make, and no other."""
    c = Cache([20, 16], 2, 64, 16, seed=3, factor=True).fill()
    d, q = c.to_gpu(), queries(c, 2, 4).to(DEV)
    k = torch.zeros(2, 2, 64, dtype=torch.bfloat16, device=DEV)
    out, lse, ws = torch.empty_like(q), torch.empty(2, 4, device=DEV), binding.new_workspace(1 << 24, DEV)
    cu, cu64 = cu_of([1, 1]), cu_of([20, 16], torch.int64)
    rows = torch.empty(36, 2, 64, dtype=torch.bfloat16, device=DEV)
    pools = [d[n] for n in ("k_pages", "v_pages", "page_table", "seq_lens", "k_scale", "v_scale")]
    end = (0, torch.cuda.current_stream().cuda_stream)
    calls = {
        "decode": [False, q, *pools, 0.1, 0, True, out, lse, ws, *end],
        "append_kv": [k, k, *pools, ws, *end],
        "append_decode": [q, k, k, *pools, 0.1, 0, True, out, lse, ws, *end],
        "write_kv": [k, k, cu, *pools, 1, ws, *end],
        "read_kv": [*pools, None, cu64, 36, False, rows, rows.clone(), ws, *end],
    }
    for name, args in calls.items():
        f = getattr(binding._fast, name)
        assert f(*args) == 0, name
        for i, a in enumerate(args):
            if not isinstance(a, torch.Tensor):
                continue
            wrong = [a.cpu(), a.double() if a.dtype == torch.bfloat16 else a.to(torch.float16), a.unsqueeze(0), "no", 3]
            if a.dim() > 1:
                # (rows of any stride are what the chunk write takes)
                t = a.transpose(0, 1).contiguous().transpose(0, 1) if a.dim() == 2 else a.transpose(-1, -2).contiguous().transpose(-1, -2)
                wrong.append(t)
            for w in wrong:
                assert f(*args[:i], w, *args[i + 1:]) is None, (name, i, type(w))
            if a.numel() > 300 or a.dim() > 1:
                continue
            assert f(*args[:i], torch.cat([a, a]), *args[i + 1:]) is None, (name, i)
        assert f(*args[:-2], 1, args[-1]) is None
    # and Python says what the library answers
    with pytest.raises(binding.GQAError):
        binding.gqa_paged_decode(q, *pools[:4], 0.1, num_splits=3, out=out, lse=lse, workspace=ws)
    got, none = binding.gqa_paged_decode(q, *pools[:4], 0.1, out=out, lse=None, workspace=ws, want_lse=False)
    assert got is out and none is None


# ----------------------------------------------------------------------- streams, graphs, all together

@pytest.mark.parametrize("lens", [[90, 0, 260, 16], [90, 0, 1060, 16]])
def test_decode_in_a_graph_and_on_another_stream(lens):
    c = Cache(lens, 2, 128, 16, seed=31).fill()
    q, scale = queries(c, 4, 16).to(DEV), 0.09
    ref = expect(c, q.cpu(), scale)
    d = c.to_gpu()
    ws = binding.new_workspace(binding.gqa_paged_decode_workspace_size(4, 16, 2, 128, 16, 1072, 2, 0), DEV)
    out, lse = torch.zeros(4, 16, 128, dtype=torch.bfloat16, device=DEV), torch.zeros(4, 16, device=DEV)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    binding.gqa_paged_decode(q, scale=scale, out=out, lse=lse, workspace=ws, stream=s, **d)
    s.synchronize()
    close(out, lse, ref)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        binding.gqa_paged_decode(q, scale=scale, out=out, lse=lse, workspace=ws, **d)
        first = out.clone()
        binding.gqa_paged_decode(q, scale=scale, out=out, lse=lse, workspace=ws, **d)
    for _ in range(3):
        out.zero_(), lse.zero_()
        graph.replay()
    torch.cuda.synchronize()
    close(out, lse, ref)
    assert torch.equal(first.view(torch.int16), out.view(torch.int16))
    # other contents and lengths under the same graph
    q.copy_(-q)
    d["seq_lens"].copy_(torch.tensor([3, 90, 0, 1], dtype=torch.int32))
    d["page_table"][1] = d["page_table"][2]
    c.table[1], c.lens = c.table[2].copy(), np.array([3, 90, 0, 1], np.int32)
    graph.replay()
    close(out, lse, expect(c, q.cpu(), scale))
    assert binding.gqa_get_error(ws) == 0


@pytest.mark.parametrize("D,P,Hq,Hk", [(128, 16, 8, 2), (64, 64, 16, 1)])
def test_prefill_chunks_then_decode_steps(D, P, Hq, Hk):
    """A serving run: prompts written in two chunks (the second's prior context read back as bf16 pages and
    attended by the prefill), then decode steps that append a token and attend, on one 4-bit cache."""
    prompts, cut, steps = [45, 7, 80], [20, 7, 33], 4
    c = Cache([n + steps for n in prompts], Hk, D, P, seed=41, factor=True)
    d = c.to_gpu()
    scale, B = D ** -0.5, 3
    ws = binding.new_workspace(1 << 24, DEV)
    done = [0] * B
    for chunk in range(2):
        counts = cut if chunk == 0 else [n - m for n, m in zip(prompts, cut)]
        now = [a + b for a, b in zip(done, counts)]
        k, v = rows_for(c, counts, 0.3)
        sl = dev(np.array(now, np.int32))
        binding.gqa_paged_write_kv(k.to(DEV), v.to(DEV), cu_of(counts), d["k_pages"], d["v_pages"],
                                   d["page_table"], sl, max(counts), k_scale=d["k_scale"], v_scale=d["v_scale"],
                                   workspace=ws)
        at = 0
        for b, n in enumerate(counts):
            if n:
                c.write(b, done[b], k[at:at + n].double().numpy(), v[at:at + n].double().numpy())
            at += n
        done = now
        # attention of the chunk over what the cache holds
        npg = [(n + P - 1) // P for n in done]
        cup = cu_of(npg, torch.int64)
        kp, vp = binding.gqa_paged_read_kv(d["k_pages"], d["v_pages"], d["page_table"], sl, cup, sum(npg),
                                           k_scale=d["k_scale"], v_scale=d["v_scale"], paged=True, workspace=ws)
        pt = torch.zeros(B, max(npg), dtype=torch.int32)
        for b in range(B):
            pt[b, :npg[b]] = torch.arange(npg[b]) + int(cup[b])
        q = bf16(c.r.normal(size=(sum(counts), Hq, D)))
        out, _ = binding.gqa_paged_prefill(q.to(DEV), cu_of(counts), kp, vp, pt.to(DEV), sl, scale, max(counts))
        at = 0
        for b, n in enumerate(counts):
            if n:
                kk, vv = (M.to_bf16(c.values(b, i, 0, done[b])) for i in range(2))
                o, _, _, _ = M.attention(q[at + n - 1].double().numpy(), kk, vv, scale)
                got = out[at + n - 1].double().cpu().numpy()
                assert np.all(np.abs(got - o) <= 2e-3 + 1e-2 * np.abs(o))  # the prefill's own gate
            at += n
    for _ in range(steps):
        done = [n + 1 for n in done]
        k, v = rows_for(c, [1] * B, 0.3)
        q, sl = bf16(c.r.normal(size=(B, Hq, D))), dev(np.array(done, np.int32))
        for b in range(B):
            c.write(b, done[b] - 1, k[b:b + 1].double().numpy(), v[b:b + 1].double().numpy())
        c.lens = np.array(done, np.int32)
        out, lse = binding.gqa_paged_append_decode(q.to(DEV), k.to(DEV), v.to(DEV), d["k_pages"], d["v_pages"],
                                                   d["page_table"], sl, scale, k_scale=d["k_scale"],
                                                   v_scale=d["v_scale"], workspace=ws)
        close(out, lse, expect(c, q, scale))
    assert binding.gqa_get_error(ws) == 0
    c.assert_same(d)


def test_ranks_of_a_split_sequence():
    """The page-range partition of split_kv over a 4-bit cache: partial decodes merged by lse_combine."""
    c = Cache([300, 40, 0, 129], 2, 128, 16, seed=43).fill()
    q, scale = queries(c, 4, 8), 0.09
    ref = expect(c, q, scale)
    d = c.to_gpu()
    parts = []
    for rank in range(3):
        p0, p1 = split_kv.rank_page_range(d["page_table"].shape[1], 3, rank)
        mine = dict(d, page_table=split_kv.local_page_table(d["page_table"], p0, p1),
                    seq_lens=split_kv.local_seq_lens(d["seq_lens"], 16, p0, p1))
        parts.append(binding.gqa_paged_decode_partial(q.to(DEV), scale=scale, **mine))
    o = torch.stack([p[0].view(32, 128) for p in parts])
    out, lse = binding.lse_combine(o, torch.stack([p[1].view(32) for p in parts]))
    close(out.view(4, 8, 128), lse.view(4, 8), ref)
