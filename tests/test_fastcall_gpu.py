"""Without the binding's compiled half the same calls give the same results."""
import pytest
import torch

from gqa_attention_paged_b200 import binding
from tests.test_fp4_gpu import DEV, Cache, cu_of, queries, rows_for

pytestmark = pytest.mark.gpu


def run(kv):
    c = Cache([70, 33], 2, 128, 16, kv, seed=71, factor=kv == "fp4").fill()
    d, q = c.to_gpu(), queries(c, 2, 8).to(DEV)
    pools = [d[n] for n in ("k_pages", "v_pages", "page_table", "seq_lens")]
    scales = dict(k_scale=d["k_scale"], v_scale=d["v_scale"])
    ws = binding.new_workspace(1 << 24, DEV)
    k, v = (x.to(DEV) for x in rows_for(c, [3, 1]))
    res = []
    binding.gqa_paged_write_kv(k, v, cu_of([3, 1]), *pools, 3, workspace=ws, **scales)
    binding.gqa_paged_append_kv(k[:2], v[:2], *pools, workspace=ws, **scales)
    for fn, t in ((binding.gqa_paged_decode, torch.bfloat16), (binding.gqa_paged_decode_partial, torch.float32)):
        o, l = torch.empty(2, 8, 128, dtype=t, device=DEV), torch.empty(2, 8, device=DEV)
        names = ("out", "lse") if t is torch.bfloat16 else ("o_part", "lse_part")
        res += fn(q, *pools, 0.1, num_splits=-1, workspace=ws, **dict(zip(names, (o, l))), **scales)
    o, l = torch.empty(2, 8, 128, dtype=torch.bfloat16, device=DEV), torch.empty(2, 8, device=DEV)
    res += binding.gqa_paged_append_decode(q, k[2:], v[2:], *pools, 0.1, num_splits=-1, out=o, lse=l, workspace=ws, **scales)
    rows = [torch.empty(103, 2, 128, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    res += binding.gqa_paged_read_kv(*pools, cu_of([70, 33], torch.int64), 103, k_out=rows[0], v_out=rows[1],
                                     workspace=ws, **scales)
    assert binding.gqa_get_error(ws) == 0
    return res + [d["k_pages"], d["v_pages"]]


@pytest.mark.parametrize("kv", ["bf16", "e4m3", "fp4"])
def test_both_halves_agree(kv, monkeypatch):
    binding.load()
    assert binding._fast is not None
    want = run(kv)
    monkeypatch.setattr(binding, "_fast", None)
    for a, b in zip(want, run(kv)):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
