"""One workspace, zeroed once, for calls of every kind in turn: what a prefill, a split or balanced bf16
decode or a sparse selection leaves in it must not reach the 4-bit decode's count of its pieces, and the
4-bit decode must leave alone what the balanced bf16 decode counts in.  Outputs are compared bit for bit
with those of the same call on a workspace of its own (pieces are merged in a fixed order), the 4-bit ones
with the 64-bit model too."""
import pytest
import torch

from gqa_attention_paged_b200 import binding, inputs
from tests.test_fp4_gpu import Cache, close, expect, queries

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def same(a, b):
    return torch.equal(a.view(torch.int16), b.view(torch.int16))


def fp4_case(lens, Hq, Hk, D, P, seed):
    c = Cache(lens, Hk, D, P, seed=seed).fill()
    q = queries(c, len(lens), Hq)
    d, qd, ref = c.to_gpu(), q.to(DEV), expect(c, q, 0.1)

    def call(ws):
        out = torch.full((len(lens), Hq, D), float("nan"), dtype=torch.bfloat16, device=DEV)
        lse = torch.full((len(lens), Hq), float("nan"), device=DEV)
        binding.gqa_paged_decode(qd, scale=0.1, out=out, lse=lse, workspace=ws, **d)
        close(out, lse, ref)
        return out
    return call


def bf16_case(B, Hq, Hk, D, ctx, splits, seed):
    case = inputs.make_decode_case(B, Hq, Hk, D, 16, [ctx] * B, seed=seed)
    kv = case.kv
    a = [t.to(DEV) for t in (case.q, kv.k_pages, kv.v_pages, kv.page_table, kv.seq_lens)]

    def call(ws):
        out = torch.full((B, Hq, D), float("nan"), dtype=torch.bfloat16, device=DEV)
        lse = torch.full((B, Hq), float("nan"), device=DEV)
        binding.gqa_paged_decode(*a, case.scale, num_splits=splits, out=out, lse=lse, workspace=ws)
        return out
    return call


def prefill_case(seed):
    case = inputs.make_prefill_case(3, 8, 2, 64, 16, [0, 20, 45], [170, 100, 240], seed=seed)
    kv = case.kv
    a = [t.to(DEV) for t in (case.q, case.cu_q, kv.k_pages, kv.v_pages, kv.page_table, kv.seq_lens)]
    return lambda ws: binding.gqa_paged_prefill(*a, case.scale, max_q_len=case.max_q_len, workspace=ws)[0]


def sparse_case(seed, decode):
    case = inputs.make_decode_case(3, 8, 2, 64, 16, [900, 337, 1290], seed=seed)
    kv = case.kv
    q, k, v, pt, sl = [t.to(DEV) for t in (case.q, kv.k_pages, kv.v_pages, kv.page_table, kv.seq_lens)]
    kt = binding.gqa_paged_kt_build(k, pt, sl)
    if decode:
        return lambda ws: binding.gqa_paged_sparse_decode(q, k, v, kt, pt, sl, case.scale, 4, 32, workspace=ws)[0]
    return lambda ws: binding.gqa_paged_sparse_select(q, kt, k, pt, sl, 4, 32, workspace=ws)[2].view(torch.int16)


OTHERS = {
    "prefill": lambda: prefill_case(1),
    "split bf16 decode": lambda: bf16_case(8, 8, 2, 64, 500, 3, 2),
    "balanced bf16 decode of a small batch": lambda: bf16_case(2, 8, 2, 64, 900, -1, 3),
    "sparse selection": lambda: sparse_case(4, False),
    "sparse decode": lambda: sparse_case(5, True),
}


@pytest.mark.parametrize("other", list(OTHERS))
def test_4_bit_decode_after_other_calls(other):
    ws = binding.new_workspace(16 << 20, DEV)
    before = OTHERS[other]()
    # units of 2 to over 31 CTAs, of head_dim 64 and 128
    calls = [fp4_case([1300, 40, 900], 8, 2, 64, 16, 1), fp4_case([2600], 8, 1, 128, 16, 2),
             fp4_case([200, 90, 310] * 4 + [1100], 8, 2, 128, 32, 3)]
    own = [f(binding.new_workspace(16 << 20, DEV)) for f in calls]
    want = before(binding.new_workspace(16 << 20, DEV))
    for f, o in zip(calls, own):
        assert same(before(ws), want)
        assert same(f(ws), o)
        assert same(f(ws), o)
    assert binding.gqa_get_error(ws) == 0


def test_balanced_bf16_decode_after_4_bit_decode():
    """The same heads; the bf16 decode counts its pieces in more than the first 320 places."""
    B, Hq, Hk, D = 200, 8, 4, 64
    bf = bf16_case(B, Hq, Hk, D, 700, -1, 7)
    four = fp4_case([1300, 40, 900, 33], Hq, Hk, D, 16, 8)
    size = binding.gqa_paged_decode_workspace_size
    need = max(size(B, Hq, Hk, D, 16, 704, 0, -1), size(4, Hq, Hk, D, 16, 1312, 2, 0))
    want, own = bf(binding.new_workspace(need, DEV)), four(binding.new_workspace(need, DEV))
    for total in (need, 16 << 20):
        ws = binding.new_workspace(total, DEV)
        for _ in range(2):
            assert same(four(ws), own)
            assert same(bf(ws), want)
        assert binding.gqa_get_error(ws) == 0


@pytest.mark.parametrize("Hq,D,lens", [(8, 128, [9000]), (4, 64, [20000, 5, 700]), (16, 128, [1, 6000, 40] * 3)])
def test_units_of_many_ctas_on_one_workspace(Hq, D, lens):
    """Units that span from 2 to hundreds of CTAs, again and again on one workspace: every count returns to
    zero."""
    f = fp4_case(lens, Hq, 1, D, 16, 11)
    ws = binding.new_workspace(16 << 20, DEV)
    first = f(ws)
    for _ in range(5):
        assert same(f(ws), first)
    assert binding.gqa_get_error(ws) == 0
    assert int(ws[:256].count_nonzero()) == 0
