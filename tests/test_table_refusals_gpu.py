"""Calls whose page table does not have a row per sequence, or whose KT cache is not that of the new keys, are
refused in Python: the kernels would go past the end of them."""
import pytest
import torch

from gqa_attention_paged_b200 import binding

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def i32(*shape):
    return torch.zeros(*shape, dtype=torch.int32, device=DEV)


def bf16(*shape):
    return torch.zeros(*shape, dtype=torch.bfloat16, device=DEV)


def calls():
    pool, kt, lens = bf16(4, 2, 16, 64), bf16(4, 2, 64, 2), i32(3)
    cu, cu64 = i32(4), torch.zeros(4, dtype=torch.int64, device=DEV)
    return {
        "prefill": lambda t: binding.gqa_paged_prefill(bf16(3, 4, 64), cu, pool, pool, t, lens, 0.1, 1),
        "gather": lambda t: binding.gqa_paged_gather(pool, pool, t, lens, cu64, 1),
        "kt_build": lambda t: binding.gqa_paged_kt_build(pool, t, lens),
        "kt_append": lambda t: binding.gqa_paged_kt_append(bf16(3, 2, 64), t, lens, kt, 16),
    }


@pytest.mark.parametrize("name", ["prefill", "gather", "kt_build", "kt_append"])
def test_page_table(name):
    call = calls()[name]
    call(i32(3, 2))
    for t in (i32(2, 2), i32(6), i32(3, 2, 1), i32(4, 2)):
        with pytest.raises(ValueError, match="page_table"):
            call(t)


@pytest.mark.parametrize("shape", [(4, 1, 64, 2), (4, 2, 32, 2), (4, 2, 64), (4, 2, 64, 1)])
def test_kt_cache(shape):
    with pytest.raises(ValueError, match="kt"):
        binding.gqa_paged_kt_append(bf16(3, 2, 64), i32(3, 2), i32(3), bf16(*shape), 16)
