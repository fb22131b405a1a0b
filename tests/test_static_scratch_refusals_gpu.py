"""What gqa_paged_decode_static_scratch refuses in Python, as gqa_paged_decode does: a page table that is not
[B][pt_stride] (the kernel would read past it), and scales of another shape or type, for every kind of pool."""
import pytest
import torch

from gqa_attention_paged_b200 import binding

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
FNS = (binding.gqa_paged_decode, binding.gqa_paged_decode_static_scratch)


def one(fn, kv, **kw):
    pool = {"bf16": lambda: torch.zeros(4, 2, 16, 128, dtype=torch.bfloat16, device=DEV),
            "e4m3": lambda: torch.zeros(4, 2, 16, 128, dtype=torch.uint8, device=DEV),
            "fp4": lambda: binding.new_fp4_pool(4, 2, 16, 128, DEV)}[kv]()
    args = dict(q=torch.zeros(2, 4, 128, dtype=torch.bfloat16, device=DEV), k_pages=pool, v_pages=pool,
                page_table=torch.zeros(2, 2, dtype=torch.int32, device=DEV),
                seq_lens=torch.full((2,), 20, dtype=torch.int32, device=DEV), scale=0.1)
    if kv == "e4m3":
        args["k_scale"] = args["v_scale"] = torch.ones(4, 2, device=DEV)
    args.update(kw)
    return fn(**args)


@pytest.mark.parametrize("kv", ["bf16", "e4m3", "fp4"])
def test_valid_calls_agree(kv):
    out, lse = one(FNS[0], kv)
    out2, lse2 = one(FNS[1], kv)
    assert torch.equal(out, out2) and torch.equal(lse, lse2)


@pytest.mark.parametrize("kv", ["bf16", "e4m3", "fp4"])
@pytest.mark.parametrize("fn", FNS)
def test_page_table(kv, fn):
    for table in (torch.zeros(1, 2, dtype=torch.int32), torch.zeros(4, dtype=torch.int32),
                  torch.zeros(2, 2, 1, dtype=torch.int32), torch.zeros(3, 2, dtype=torch.int32)):
        with pytest.raises(ValueError, match="page_table"):
            one(fn, kv, page_table=table.to(DEV))
    with pytest.raises(TypeError, match="page_table"):
        one(fn, kv, page_table=torch.zeros(2, 2, dtype=torch.int64, device=DEV))


@pytest.mark.parametrize("fn", FNS)
def test_scales(fn):
    with pytest.raises(ValueError, match="scale"):
        one(fn, "e4m3", k_scale=None)
    with pytest.raises(ValueError, match="v_scale"):
        one(fn, "e4m3", v_scale=torch.ones(2, device=DEV))
    with pytest.raises(TypeError, match="k_scale"):
        one(fn, "e4m3", k_scale=torch.ones(4, 2, dtype=torch.bfloat16, device=DEV))
    with pytest.raises(ValueError, match="k_scale"):
        one(fn, "fp4", k_scale=torch.ones(4, 2, device=DEV))
    with pytest.raises(ValueError, match="CUDA"):
        one(fn, "fp4", v_scale=torch.ones(2))
