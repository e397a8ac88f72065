"""GPU tests of the cache operators' ranges: sizes that are refused, buffers beside one another, every plan of the
decodes, scores and probes far from those of the other tests."""
import math

import numpy as np
import pytest
import torch

import oracle

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def plx():
    from local_linear_attention_streamed_b200 import plx as mod
    assert torch.cuda.is_available()
    return mod


@pytest.fixture(autouse=True)
def no_device_error(plx):
    yield
    assert plx.get_device_status() == 0


def raw(t):
    """Bytes of a tensor's rows, so that NaN compare too: [B, Hkv, L, row bytes]."""
    return t.contiguous().view(torch.uint8).reshape(*t.shape[:3], -1).cpu().numpy()


# ---------------------------------------------------------------- refusals


@pytest.mark.parametrize("d", [32, 96, 2048, 2050, 4096])
def test_unsupported_head_sizes_raise(plx, d):
    """The binding asks for the workspace's size before the call checks the sizes."""
    B, Hkv, L = 1, 2, 5
    q = torch.zeros((B, Hkv, d), dtype=torch.bfloat16, device="cuda")
    K = torch.zeros((B, Hkv, L, d), dtype=torch.bfloat16, device="cuda")
    codes = torch.zeros((B, Hkv, L, d // 2), dtype=torch.uint8, device="cuda")
    params = torch.zeros((B, Hkv, L, 2), dtype=torch.bfloat16, device="cuda")
    w = torch.zeros((B, Hkv, L), device="cuda")
    sl = torch.full((B,), L, dtype=torch.int32, device="cuda")
    for call in (lambda: plx.decode_weights(q, q, K, K, sl, w),
                 lambda: plx.decode_int4kv_weights(q, q, codes, params, codes, params, sl, w),
                 lambda: plx.decode_int4kv(q, q, codes, params, codes, params, sl)):
        with pytest.raises(plx.PlxError) as e:
            call()
        assert e.value.code == -2


def test_numbers_beyond_32_bits_are_refused(plx):
    """A C int would take their low 32 bits: here a valid budget, valid sinks, a valid length."""
    g = torch.Generator().manual_seed(12)
    w, rows = torch.rand((1, 2, 20), generator=g), torch.randn((1, 2, 20, 128), generator=g).to(torch.bfloat16)
    t, wd = rows.cuda(), w.cuda()
    sl = torch.tensor([20], dtype=torch.int32, device="cuda")
    for kw in (dict(budget=(1 << 32) + 4), dict(budget=4, sinks=(1 << 32) + 1), dict(budget=4, sinks=1 - (1 << 32)),
               dict(budget=4, recent=1 - (1 << 32)), dict(budget=4 - (1 << 32))):
        with pytest.raises(ValueError):
            plx.cache_evict([t], wd, sl, **kw)
    assert torch.equal(t.cpu(), rows) and torch.equal(wd.cpu(), w)
    long = torch.empty((1, 1, (1 << 32) + 20), device="cuda")
    with pytest.raises(ValueError):
        plx.cache_evict([], long, sl, 4)


# ---------------------------------------------------------------- eviction


def test_neighbouring_buffers_are_not_overlaps(plx):
    """Caches, totals and lengths cut out of one buffer, each ending where the next begins."""
    B, Hkv, L, budget = 2, 2, 64, 16
    g = torch.Generator().manual_seed(11)
    w, rows = torch.rand((B, Hkv, L), generator=g), torch.randn((B, Hkv, L, 128), generator=g).to(torch.bfloat16)
    sizes = [B * Hkv * L * 256, B * Hkv * budget * 256, B * Hkv * L * 4, B * Hkv * budget * 4, B * 4, B * 4]
    buf = torch.zeros(sum(sizes), dtype=torch.uint8, device="cuda")
    at = [sum(sizes[:i]) for i in range(len(sizes))]
    part = [buf[a:a + n] for a, n in zip(at, sizes)]
    src, dst = (p.view(torch.bfloat16).view(B, Hkv, -1, 128) for p in part[:2])
    wd, wo = (p.view(torch.float32).view(B, Hkv, -1) for p in part[2:4])
    sl, new = (p.view(torch.int32) for p in part[4:])
    src.copy_(rows), wd.copy_(w), sl.copy_(torch.tensor([64, 40]))
    kept, got = plx.cache_evict([src], wd, sl, budget, 1, 2, caches_out=[dst], weights_out=wo, seqlens_out=new)
    assert got is new and new.tolist() == [16, 16] and sl.tolist() == [64, 40]
    assert np.array_equal(raw(src), raw(rows)) and torch.equal(wd.cpu(), w)
    for b, n in enumerate([64, 40]):
        for h in range(Hkv):
            ids = oracle.evict_ref(w[b, h].tolist(), n, budget, 1, 2)
            assert kept[b, h].tolist() == ids.tolist()
            assert np.array_equal(raw(dst)[b, h], raw(rows)[b, h, ids])
            assert torch.equal(wo[b, h].cpu(), w[b, h, ids])
    with pytest.raises(plx.PlxError):  # new lengths over the totals
        plx.cache_evict([src], wd, sl, budget, 1, 2, caches_out=[dst], weights_out=wo,
                        seqlens_out=wd.view(torch.int32).view(-1)[:B])
