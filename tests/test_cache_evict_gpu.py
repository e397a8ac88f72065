"""GPU parity of the eviction by attention weight: positions, lengths and rows are exact."""
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


def make(seed, B, Hkv, L):
    g = torch.Generator().manual_seed(seed)
    w = torch.exp(2 * torch.randn((B, Hkv, L), generator=g))
    caches = [torch.randn((B, Hkv, L, 128), generator=g).to(torch.bfloat16),          # 256 bytes
              torch.randint(0, 256, (B, Hkv, L, 32), generator=g, dtype=torch.uint8),  # 32 bytes
              torch.randn((B, Hkv, L, 2), generator=g).to(torch.bfloat16),            # 4 bytes
              torch.randn((B, Hkv, L), generator=g),                                  # 4 bytes, no trailing axis
              torch.randint(0, 256, (B, Hkv, L, 7), generator=g, dtype=torch.uint8)]   # 7 bytes
    return w, caches


def check(plx, w, caches, lens, budget, sinks, recent, in_place, L_out=None):
    B, Hkv, L = w.shape
    src = [t.cuda() for t in caches]
    wd, sl = w.cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda")
    if in_place:
        dst, wo = src, wd
        before = [raw(t) for t in src]
        kept, new = plx.cache_evict(src, wd, sl, budget, sinks, recent)
    else:
        L_out = L_out or min(budget, L)
        g = torch.Generator().manual_seed(1)
        dst = [torch.randint(0, 256, (B, Hkv, L_out, raw(t).shape[-1]), generator=g, dtype=torch.uint8)
               .view(t.dtype).reshape(B, Hkv, L_out, *t.shape[3:]).cuda() for t in caches]
        before = [raw(t) for t in dst]
        wo = torch.full((B, Hkv, L_out), 5.0, device="cuda")
        kept, new = plx.cache_evict(src, wd, sl, budget, sinks, recent, caches_out=dst, weights_out=wo)
        for t, s in zip(caches, src):
            assert np.array_equal(raw(t), raw(s))
        assert np.array_equal(raw(w), raw(wd))
    assert new.tolist() == [min(n, budget) for n in lens] and sl.tolist() == list(lens)
    assert kept.shape == (B, Hkv, min(budget, L)) and kept.dtype == torch.int32
    kept, wn = kept.cpu().numpy(), w.numpy()
    for b, n in enumerate(lens):
        m = min(n, budget)
        for h in range(Hkv):
            ids = oracle.evict_ref(wn[b, h].tolist(), n, budget, sinks, recent)
            assert np.array_equal(kept[b, h, :m], ids)
            assert (kept[b, h, m:] == -1).all()
            assert np.array_equal(raw(wo)[b, h, :m], raw(w)[b, h, ids])
            assert not raw(wo)[b, h, m:].any()
            for t, out, old in zip(caches, dst, before):
                assert np.array_equal(raw(out)[b, h, :m], raw(t)[b, h, ids])
                assert np.array_equal(raw(out)[b, h, m:], old[b, h, m:])


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("L,budget,sinks,recent", [
    (1, 1, 0, 0), (7, 3, 1, 1), (64, 64, 4, 8), (65, 64, 0, 0), (130, 1, 0, 0), (130, 5, 5, 0), (130, 5, 0, 5),
    (130, 9, 4, 5), (1000, 333, 1, 32), (1025, 1024, 4, 128), (2100, 128, 3, 0), (500, 900, 4, 16),
])
def test_sizes(plx, L, budget, sinks, recent, in_place):
    B, Hkv = 3, 2
    w, caches = make(L + budget, B, Hkv, L)
    check(plx, w, caches, [L, (L + 1) // 2, max(1, L - 1)], budget, sinks, recent, in_place)


@pytest.mark.parametrize("L", [4096, 33000, 70001])
def test_long(plx, L):
    w, caches = make(L, 1, 2, L)
    check(plx, w, caches[2:4], [L], L // 8, 4, 100, False)
    check(plx, w, caches[1:2], [L - 5], L // 2, 0, 1, True)


def test_larger_output_and_no_caches(plx):
    w, caches = make(3, 2, 2, 50)
    check(plx, w, caches, [50, 20], 16, 2, 2, False, L_out=40)
    check(plx, w, [], [50, 20], 16, 2, 2, False)


@pytest.mark.parametrize("values", [
    [1.0], [0.0, -0.0], [math.nan, 1.0, -math.inf], [math.nan], [math.inf, 1.0, math.inf, -1.0],
    [1e-45, -1e-45, 0.0, 1e-38], [1.0, 1.0 + 2 ** -23, 1.0 - 2 ** -24],
])
@pytest.mark.parametrize("in_place", [False, True])
def test_ties_and_special_weights(plx, values, in_place):
    L = 300
    _, caches = make(4, 2, 1, L)
    rng = np.random.default_rng(len(values))
    w = torch.from_numpy(rng.choice(np.array(values, dtype=np.float32), (2, 1, L)))
    for budget in (1, 40, 150, 299):
        check(plx, w, caches[1:2], [L, L - 3], budget, 0, 0, in_place)
        check(plx, w, caches[1:2], [L, L - 3], budget, min(3, budget), max(0, min(10, budget - 3)), in_place)


def test_misaligned_rows(plx):
    """Caches whose first byte is not on a 16- or 4-byte boundary are moved in smaller pieces."""
    L, B, Hkv = 90, 1, 2
    w, _ = make(5, B, Hkv, L)
    for off in (1, 4, 8):
        buf = torch.randint(0, 256, (off + B * Hkv * L * 32,), dtype=torch.uint8, device="cuda")
        t = buf[off:].view(B, Hkv, L, 32)
        want = raw(t)
        sl = torch.tensor([L], dtype=torch.int32, device="cuda")
        kept, _ = plx.cache_evict([t], w.cuda(), sl, 30)
        kept = kept.cpu().numpy()
        for h in range(Hkv):
            assert np.array_equal(raw(t)[0, h, :30], want[0, h, kept[0, h]])
            assert np.array_equal(raw(t)[0, h, 30:], want[0, h, 30:])


def test_lengths_in_place_and_bad_lengths(plx):
    B, Hkv, L = 3, 2, 40
    w, caches = make(6, B, Hkv, L)
    t, wd = caches[0].cuda(), w.cuda()
    sl = torch.tensor([40, 0, 41], dtype=torch.int32, device="cuda")
    before = raw(t)
    kept, new = plx.cache_evict([t], wd, sl, 10, 1, 1, seqlens_out=sl)
    assert plx.get_device_status() == -6
    assert new is sl and sl.tolist() == [10, 0, 0]
    assert (kept[1:] == -1).all() and not wd[1:].any() and np.array_equal(raw(t)[1:], before[1:])
    ids = oracle.evict_ref(w[0, 1].tolist(), 40, 10, 1, 1)
    assert kept[0, 1].tolist() == ids.tolist()


def test_lengths_in_place_with_many_caches(plx):
    """New lengths are written while other CTAs still compact: nothing may depend on which comes first."""
    B, Hkv, L, budget = 16, 8, 700, 100
    w, caches = make(9, B, Hkv, L)
    lens = [700 - 13 * b for b in range(B)]
    for _ in range(5):
        t, wd = [c.cuda() for c in caches], w.cuda()
        sl = torch.tensor(lens, dtype=torch.int32, device="cuda")
        kept, new = plx.cache_evict(t, wd, sl, budget, 1, 8, seqlens_out=sl)
        assert sl.tolist() == [budget] * B
        at = kept.long()
        for c, d in zip(caches, t):
            idx = at.view(*at.shape, *([1] * (c.dim() - 3))).expand(*at.shape, *c.shape[3:])
            assert np.array_equal(raw(d[:, :, :budget]), raw(torch.gather(c.cuda(), 2, idx)))
            assert np.array_equal(raw(d[:, :, budget:]), raw(c[:, :, budget:]))
        assert torch.equal(wd[..., :budget], torch.gather(w.cuda(), 2, at)) and not wd[..., budget:].any()


@pytest.mark.parametrize("B,L", [(1, 5000), (2, 32768), (1, 40000), (160, 4200), (150, 17000), (150, 33000)])
def test_every_select(plx, B, L):
    """Clusters and single CTAs, totals in registers or read again, with many ties."""
    g = torch.Generator(device="cuda").manual_seed(L)
    w = torch.randint(0, 40, (B, 1, L), generator=g, device="cuda").float()
    lens = torch.randint(L // 2, L + 1, (B,), generator=g, device="cuda").to(torch.int32)
    lens[0] = L
    budget, sinks, recent = L // 3, 4, 50
    kept, new = plx.cache_evict([], w, lens, budget, sinks, recent, caches_out=[],
                                weights_out=torch.empty((B, 1, budget), device="cuda"))
    pos = torch.arange(L, device="cuda")
    must = (pos < sinks) | ((pos >= lens[:, None, None] - recent) & (pos < lens[:, None, None]))
    rank = torch.where(must, 1e9, torch.where(pos < lens[:, None, None], w, -1.0))
    want = torch.sort(torch.sort(-rank, stable=True).indices[..., :budget]).values
    assert torch.equal(kept.long(), want) and (new == budget).all()


def test_graph_replays_with_new_lengths(plx):
    B, Hkv, L, budget = 2, 2, 200, 64
    w, caches = make(7, B, Hkv, L)
    src, wd = [t.cuda() for t in caches[:2]], w.cuda()
    dst = [torch.zeros((B, Hkv, budget, *t.shape[3:]), dtype=t.dtype, device="cuda") for t in src]
    wo = torch.zeros((B, Hkv, budget), device="cuda")
    sl = torch.tensor([200, 30], dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kept, new = plx.cache_evict(src, wd, sl, budget, 1, 8, caches_out=dst, weights_out=wo)
    for lens in ([200, 30], [65, 200], [64, 1]):
        sl.copy_(torch.tensor(lens, dtype=torch.int32))
        wd.copy_(wd.roll(1, -1))
        graph.replay()
        torch.cuda.synchronize()
        for b, n in enumerate(lens):
            for h in range(Hkv):
                ids = oracle.evict_ref(wd[b, h].tolist(), n, budget, 1, 8)
                m = len(ids)
                assert kept[b, h, :m].tolist() == ids.tolist() and (kept[b, h, m:] == -1).all()
                assert torch.equal(dst[0][b, h, :m], src[0][b, h, torch.from_numpy(ids).cuda()])


def test_refusals(plx):
    w, caches = make(8, 1, 2, 20)
    t, wd = caches[0].cuda(), w.cuda()
    sl = torch.tensor([20], dtype=torch.int32, device="cuda")
    for kw in (dict(budget=0), dict(budget=4, sinks=3, recent=2), dict(budget=4, sinks=-1), dict(budget=4, recent=-1)):
        with pytest.raises(plx.PlxError):
            plx.cache_evict([t], wd, sl, **kw)
    with pytest.raises(plx.PlxError):  # room for fewer rows than the budget
        plx.cache_evict([t], wd, sl, 10, caches_out=[t[:, :, :5].clone()], weights_out=wd[..., :5].clone())
    with pytest.raises(plx.PlxError):  # overlapping, not in place
        buf = torch.zeros(2 * 20 * 128 + 128, dtype=torch.bfloat16, device="cuda")
        plx.cache_evict([buf[:-128].view_as(t)], wd, sl, 10, caches_out=[buf[128:].view_as(t)],
                        weights_out=torch.zeros_like(wd))
    with pytest.raises(plx.PlxError):  # more caches than a call takes
        plx.cache_evict([t.clone() for _ in range(9)], wd, sl, 10)
    with pytest.raises(plx.PlxError):  # one buffer twice: its rows would move twice
        plx.cache_evict([t, t], wd, sl, 10)
    for args in (([t], wd.double(), sl, 10), ([t.cpu()], wd, sl, 10), ([t], wd, sl.long(), 10),
                 ([t[:, :, :10]], wd, sl, 10), ([t.transpose(2, 3)], wd, sl, 10)):
        with pytest.raises(ValueError):
            plx.cache_evict(*args)
    with pytest.raises(ValueError):
        plx.cache_evict([t], wd, sl, 10, caches_out=[t])
    with pytest.raises(ValueError):
        plx.cache_evict([t], wd, sl, 10, caches_out=[], weights_out=wd)
