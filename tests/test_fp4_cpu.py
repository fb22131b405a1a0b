"""The 4-bit cache without a GPU: the refusals of its calls, the sizes the host computes, and the 64-bit
model the GPU tests compare with."""
import ctypes

import numpy as np
import pytest
import torch

from gqa_attention_paged_b200 import binding
from tests import _fp4 as M


def _fake(n=0x10000):
    return ctypes.c_void_p(n)


def _decode(fn="gqa_paged_decode", **kw):
    args = dict(q=_fake(), k=_fake(), v=_fake(), ks=None, vs=None, kvd=2, pt=_fake(), pts=8, sl=_fake(), B=2,
                Hq=8, Hk=2, D=64, P=16, npg=16, scale=0.125, S=0, pack=1, out=_fake(), lse=_fake(), ws=_fake(),
                wsb=1 << 26, st=None)
    args.update(kw)
    return getattr(binding.load(), fn)(*args.values())


@pytest.mark.parametrize("fn", ["gqa_paged_decode", "gqa_paged_decode_partial"])
@pytest.mark.parametrize("kw,status", [
    (dict(q=None), -1), (dict(ws=None), -1), (dict(D=96), -2), (dict(P=8), -2), (dict(Hq=6, Hk=4), -2),
    (dict(npg=1 << 30), -2), (dict(B=65535, pts=1 << 14), -2), (dict(Hq=1 << 30, B=4), -2), (dict(kvd=3), -3), (dict(S=1), -4), (dict(S=64), -4), (dict(S=-2), -4),
    (dict(wsb=256), -5), (dict(ws=_fake(0x10010)), -5), (dict(k=_fake(0x10008)), -9),
    (dict(ks=_fake(0x10002)), -9), (dict(vs=_fake(0x10001)), -9),
])
def test_decode_refuses_on_the_host(fn, kw, status):
    assert _decode(fn, **kw) == status


def test_append_decode_refuses_before_writing():
    def call(**kw):
        args = dict(q=_fake(), kn=_fake(), vn=_fake(), k=_fake(), v=_fake(), ks=None, vs=None, kvd=2, pt=_fake(),
                    pts=8, sl=_fake(), B=2, Hq=8, Hk=2, D=64, P=16, npg=16, scale=0.125, S=0, pack=1, out=_fake(),
                    lse=None, ws=_fake(), wsb=1 << 26, st=None)
        args.update(kw)
        return binding.load().gqa_paged_append_decode(*args.values())
    assert call(S=2) == -4
    assert call(wsb=256) == -5
    assert call(kn=_fake(0x10008)) == -9
    assert call(ks=_fake(0x10002)) == -9
    assert call(D=32) == -2
    assert call(B=65535, pts=1 << 14) == -2


def _write(**kw):
    args = dict(kn=_fake(), vn=_fake(), kst=128, vst=128, cu=_fake(), k=_fake(), v=_fake(), ks=None, vs=None, kvd=2,
                pt=_fake(), pts=8, sl=_fake(), B=2, Hk=2, D=64, P=16, npg=16, tq=10, mq=5, ws=_fake(), st=None)
    args.update(kw)
    return binding.load().gqa_paged_write_kv(*args.values())


@pytest.mark.parametrize("kw,status", [
    (dict(kn=None), -1), (dict(v=None), -1), (dict(pt=None), -1), (dict(ws=None), -1),
    (dict(kvd=3), -3), (dict(kvd=1), -3), (dict(kvd=1, ks=_fake()), -3),
    (dict(D=96), -2), (dict(P=24), -2), (dict(B=-1), -2), (dict(B=70000), -2), (dict(Hk=0), -2), (dict(npg=0), -2),
    (dict(tq=-1), -2), (dict(mq=-1), -2), (dict(kst=120), -2), (dict(vst=64), -2), (dict(npg=1 << 30), -2),
    (dict(cu=None), -2), (dict(cu=None, tq=2, mq=2), -2),   # without cu_q: one row per sequence
    (dict(tq=1 << 30, Hk=8192, kst=1 << 20, vst=1 << 20, npg=1), -2),
    (dict(kst=132), -9), (dict(vst=130), -9), (dict(kn=_fake(0x10008)), -9), (dict(k=_fake(0x10008)), -9),
    (dict(cu=_fake(0x10002)), -9), (dict(ws=_fake(0x10010)), -9), (dict(ks=_fake(0x10002)), -9),
    (dict(tq=0), 0), (dict(B=0), 0), (dict(mq=0), 0),       # nothing to do: nothing is launched
])
def test_write_refuses_on_the_host(kw, status):
    assert _write(**kw) == status


def _read(**kw):
    args = dict(k=_fake(), v=_fake(), ks=None, vs=None, kvd=2, pt=_fake(), pts=8, st0=None, sl=_fake(), cu=_fake(),
                B=2, Hk=2, D=64, P=16, npg=16, total=10, paged=0, ko=_fake(), vo=_fake(), ws=_fake(), st=None)
    args.update(kw)
    return binding.load().gqa_paged_read_kv(*args.values())


@pytest.mark.parametrize("kw,status", [
    (dict(k=None), -1), (dict(cu=None), -1), (dict(vo=None), -1), (dict(ws=None), -1),
    (dict(kvd=9), -3), (dict(kvd=1, vs=_fake()), -3),
    (dict(D=48), -2), (dict(P=8), -2), (dict(B=-1), -2), (dict(total=-1), -2), (dict(total=1 << 40), -2),
    (dict(total=1 << 31, paged=1), -2), (dict(pts=0), -2),
    (dict(ko=_fake(0x10008)), -9), (dict(cu=_fake(0x10004)), -9), (dict(st0=_fake(0x10001)), -9),
    (dict(ws=_fake(0x10010)), -9),
    (dict(total=0), 0), (dict(B=0), 0),
])
def test_read_refuses_on_the_host(kw, status):
    assert _read(**kw) == status


def test_host_policy():
    lib = binding.load()
    ws = lib.gqa_paged_decode_workspace_size
    for B in (1, 64, 5000, 65535):
        # the same for every batch, context and for the two names of the one schedule; room for a counter
        # and two pieces of 4 heads of every CTA
        assert ws(B, 32, 8, 128, 16, 2048, 2, 0) == ws(1, 32, 8, 128, 64, 32768, 2, -1) >= 256 + 320 * (4 + 2 * 4 * 130 * 4)
    assert ws(64, 64, 2, 128, 16, 2048, 2, 0) <= binding.new_workspace(16 << 20, "cpu").numel()
    assert lib.gqa_pick_splits(1, 8, 32768, 16, 2) == 1
    assert binding.gqa_paged_decode_kernel_launches(4, 64, 8, 128, 64, 32768, 2, 0) == 1
    assert binding.gqa_paged_decode_kernel_launches(4, 64, 8, 128, 64, 32768, 2, 4) == 0


def test_binding_tells_the_pools_apart():
    z = lambda row, t=torch.uint8: torch.zeros(2, 3, 16, row, dtype=t)  # noqa: E731
    assert binding._kv_layout(z(72)) == (binding.GQA_KV_FP4, 128)
    assert binding._kv_layout(z(36)) == (binding.GQA_KV_FP4, 64)
    assert binding._kv_layout(z(128)) == (binding.GQA_KV_FP8_E4M3, 128)
    assert binding._kv_layout(z(64, torch.bfloat16)) == (binding.GQA_KV_BF16, 64)
    assert binding._kv_layout(z(72, torch.bfloat16)) == (binding.GQA_KV_BF16, 72)
    with pytest.raises(ValueError):
        binding._kv_layout(torch.zeros(4, 72, dtype=torch.uint8))
    p = binding.new_fp4_pool(5, 2, 32, 128, "cpu")
    assert p.shape == (5, 2, 32, 72) and p.dtype == torch.uint8
    with pytest.raises(ValueError):
        binding.new_fp4_pool(5, 2, 32, 96, "cpu")


def test_binding_refuses_cpu_tensors():
    p = binding.new_fp4_pool(4, 2, 16, 64, "cpu")
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
    x = torch.zeros(3, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        binding.gqa_paged_write_kv(x, x, i32(3), p, p, i32(2, 4), i32(2), 3)
    with pytest.raises(ValueError, match="CUDA"):
        binding.gqa_paged_read_kv(p, p, i32(2, 4), i32(2), torch.zeros(3, dtype=torch.int64), 4)
    with pytest.raises(ValueError, match="CUDA"):
        binding.gqa_paged_decode(x, p, p, i32(3, 4), i32(3), 0.1)


# -------------------------------------------------------------------------- the model itself

def test_model_grids():
    assert list(M.E4M3[:3]) == [0, 2.0 ** -9, 2.0 ** -8] and M.E4M3[126] == 448 and len(M.E4M3) == 127
    codes = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(codes, M.E4M3)
    x = np.concatenate([np.random.default_rng(0).uniform(-500, 500, 4000), (M.E4M3[1:] + M.E4M3[:-1]) / 2])
    want = torch.from_numpy(x).clamp(-448, 448).float().to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(M.e4m3_code(x), want)
    # e2m1: nearest of the eight, ties to the even code
    y = np.linspace(0, 7, 2801)
    d = np.abs(y[:, None] - M.E2M1)
    best = d.min(1)
    for v, code, row in zip(y, M.nearest(y, M.E2M1), d):
        near = np.flatnonzero(row == best[np.flatnonzero(y == v)[0]])
        assert code in near and (len(near) == 1 or code % 2 == 0)
    assert np.array_equal(M.to_bf16(x), torch.from_numpy(x).float().to(torch.bfloat16).double().numpy())


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("is_v", [False, True])
def test_model_layout_covers_every_byte_once(D, is_v):
    P = 32
    seen = np.zeros(P * 9 * D // 16, int)
    for slot in range(P):
        at, high, sc = M.addresses(P, D, slot, is_v)
        np.add.at(seen, at, np.where(high == 1, 16, 1))
        np.add.at(seen, sc, 17)
    assert np.all(seen == 17)


def test_model_put_then_read():
    r = np.random.default_rng(1)
    for is_v in (False, True):
        block = r.integers(0, 256, 16 * 72, dtype=np.uint8)
        x = M.to_bf16(r.normal(size=(16, 128)))
        for slot in r.permutation(16):
            M.put_fp4(block, 16, 128, slot, is_v, x[slot], 0.7)
        for slot in range(16):
            y = M.token_fp4(block, 16, 128, slot, is_v, 0.7)
            step = np.repeat(np.abs(x[slot]).reshape(8, 16).max(1), 16) / 6
            # half the widest gap between codes (4 to 6, one step of the block's scale) and what
            # the e4m3 scale is off by (2^-4 of it, times the code)
            assert np.all(np.abs(y - x[slot]) <= step * (1 + 6 * 2.0 ** -4) + 1e-9)


def test_compiled_calls_leave_the_rest_to_python():
    """Whatever is not a valid call on CUDA tensors returns None and runs nothing."""
    binding.load()
    f = binding._fast
    p = binding.new_fp4_pool(4, 2, 16, 64, "cpu")
    i32 = torch.zeros(2, 4, dtype=torch.int32)
    for name, n in (("decode", 16), ("append_kv", 11), ("append_decode", 17), ("write_kv", 13), ("read_kv", 15)):
        call = getattr(f, name)
        assert call() is None
        assert call(*[None] * n) is None
        assert call(*[None] * (n - 2), 0, 0) is None
        assert call(*[p] * (n - 2), 0, 0) is None
        assert call(*[p] * (n - 2), -1, 0) is None
        assert call(*[i32] * (n - 2), 0, "stream") is None
    with pytest.raises(TypeError):
        f.init(1, 2)
    with pytest.raises(ValueError):
        f.init(torch.Tensor, 0, 0, 0, 0, 0, 0)
