"""Calls on another stream than the current one that make their own buffers: the workspace's zeros and the
outputs belong to the stream that the call runs on.  The current stream is kept busy meanwhile, and the memory
that a buffer could be made of holds other bytes."""
import pytest
import torch

from gqa_attention_paged_b200 import binding, inputs
from tests._util import bf16_tol_ok, oracle_decode
from tests.test_fp4_gpu import Cache, close, cu_of, expect, queries, rows_for

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def busy(*sizes):
    """Free blocks of these sizes that hold ones, and a current stream that is behind."""
    held = [torch.full((n,), 0xFF, dtype=torch.uint8, device=DEV) for n in sizes]
    torch.cuda.synchronize()
    del held
    torch.cuda._sleep(200_000_000)


@pytest.mark.parametrize("raw", [False, True])
def test_4_bit_calls(raw):
    c = Cache([1300, 90], 2, 128, 16, seed=51, factor=True).fill()
    d, q = c.to_gpu(), queries(c, 2, 8)
    qd, ref = q.to(DEV), expect(c, q, 0.1)
    need = binding.gqa_paged_decode_workspace_size(2, 8, 2, 128, 16, d["page_table"].shape[1] * 16, 2, 0)
    need = (need + 255) // 256 * 256
    s = torch.cuda.Stream()
    on = s.cuda_stream if raw else s
    sizes = (need, 256, 2 * 8 * 128 * 2, 2 * 8 * 128 * 4, 2 * 8 * 4)
    torch.cuda.synchronize()
    for call, f32 in ((binding.gqa_paged_decode, False), (binding.gqa_paged_decode_partial, True)):
        busy(*sizes)
        out, lse = call(qd, scale=0.1, stream=on, **d)
        s.synchronize()
        with torch.cuda.stream(s):
            close(out, lse, ref, f32_out=f32)
    # the write's error word, then what it wrote, read back
    k, v = rows_for(c, [3, 1])
    kd, vd, cu, cu_out = k.to(DEV), v.to(DEV), cu_of([3, 1]), cu_of([1300, 90], torch.int64)
    torch.cuda.synchronize()
    busy(*sizes)
    ws = binding.gqa_paged_write_kv(kd, vd, cu, d["k_pages"], d["v_pages"], d["page_table"], d["seq_lens"], 3,
                                    k_scale=d["k_scale"], v_scale=d["v_scale"], stream=on)
    assert binding.gqa_get_error(ws, stream=on) == 0
    rk, _ = binding.gqa_paged_read_kv(d["k_pages"], d["v_pages"], d["page_table"], d["seq_lens"], cu_out, 1390,
                                      k_scale=d["k_scale"], v_scale=d["v_scale"], stream=on)
    with torch.cuda.stream(s):
        got = rk[1297:1300].double().cpu().numpy()
    c.write(0, 1297, k[:3].double().numpy(), v[:3].double().numpy())
    want = c.values(0, 0, 1297)
    assert (abs(got - want) <= 2.0 ** -7 * abs(want)).all()


def test_bf16_decode():
    case = inputs.make_decode_case(40, 8, 4, 64, 16, [700] * 40, seed=9)
    kv = case.kv
    a = [t.to(DEV) for t in (case.q, kv.k_pages, kv.v_pages, kv.page_table, kv.seq_lens)]
    need = binding.gqa_paged_decode_workspace_size(40, 8, 4, 64, 16, kv.page_table.shape[1] * 16, 0, -1)
    ref, _ = oracle_decode(case)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    busy((need + 255) // 256 * 256, 40 * 8 * 64 * 2, 40 * 8 * 4)
    out, _ = binding.gqa_paged_decode(*a, case.scale, num_splits=-1, stream=s)
    s.synchronize()
    with torch.cuda.stream(s):
        ok, bad = bf16_tol_ok(out.float().cpu().numpy(), ref)
    assert ok, int(bad.sum())
