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


@pytest.mark.parametrize("in_place", [False, True])
def test_eviction_beyond_32_bit_offsets(plx, in_place):
    """Rows of the second head lie more than 2^32 bytes into their cache, and kept ones up to its end."""
    L, budget, sinks, recent = 70_000_000, 5000, 3, 60
    cache = torch.empty((1, 2, L, 64), dtype=torch.uint8, device="cuda")
    w = torch.rand((1, 2, L), device="cuda", generator=torch.Generator(device="cuda").manual_seed(1))
    g = torch.Generator(device="cuda").manual_seed(2)
    heavy = torch.stack([torch.randperm(L - recent - sinks, generator=g, device="cuda")[:budget - sinks - recent]
                         for _ in range(2)]).sort(-1).values + sinks
    w.scatter_(2, heavy[None], 2.0 + torch.rand(heavy.shape, generator=g, device="cuda")[None])
    ends = torch.arange(sinks, device="cuda"), torch.arange(L - recent, L, device="cuda")
    want = torch.stack([torch.cat((ends[0], h, ends[1])) for h in heavy])
    rows = torch.randint(0, 256, (2, budget, 64), generator=g, device="cuda", dtype=torch.uint8)
    for h in range(2):
        cache[0, h, want[h]] = rows[h]
    totals = torch.gather(w[0], 1, want)
    to, w_to = (cache, w) if in_place else (torch.empty_like(cache[:, :, :budget]), torch.empty_like(w[:, :, :budget]))
    sl = torch.tensor([L], dtype=torch.int32, device="cuda")
    kept, new = plx.cache_evict([cache], w, sl, budget, sinks, recent, caches_out=[to], weights_out=w_to)
    assert L * 64 > 2 ** 32 and new.tolist() == [budget]
    assert torch.equal(kept[0].long(), want)
    assert torch.equal(to[0, :, :budget], rows) and torch.equal(w_to[0, :, :budget], totals)
    assert not w_to[0, :, budget:].any()


# ---------------------------------------------------------------- decodes


def f64(t):
    return t.detach().double().cpu().numpy()


def quantised(plx, X):
    """(device codes, device params, float64 values) of bf16 rows."""
    codes, params = plx.kv_quantize_int4(X.cuda())
    return codes, params, oracle.kv_dequantize_int4_ref(codes.cpu().numpy(), f64(params)[..., 0], f64(params)[..., 1])


def check_out(got, q, r, K, V, sl):
    """The bound of test_cache_int4_gpu.py: one rounding to bf16, and 2^-13 of the terms' sizes."""
    want = oracle.decode_gqa_ref(q, r, K, V, sl)
    mag = oracle.decode_magnitude(q, r, K, V, sl)
    err = np.abs(f64(got) - want) - 2.0 ** -8 * np.abs(want) - 2.0 ** -13 * mag
    assert err.max() <= 0, err.max()


def check_weights(got, q, r, K, V, sl, w, before):
    """Also of test_cache_int4_gpu.py."""
    _, want = oracle.decode_weights_ref(q, r, K, V, sl, f64(w))
    got = f64(got)
    for b, n in enumerate(sl):
        err = np.abs(got[b, :, :n] - want[b, :, :n])
        p = want[b, :, :n] - f64(w)[b, :, :n]
        assert (err <= 2.0 ** -23 * np.abs(want[b, :, :n]) + 2.0 ** -15 * p).all()
        assert np.array_equal(got[b, :, n:], f64(before)[b, :, n:])


def random_case(seed, B, Hkv, G, L, d):
    g = torch.Generator().manual_seed(seed)
    H = Hkv * G

    def rms(*shape):
        x = torch.randn(shape, generator=g)
        return x / x.square().mean(-1, keepdim=True).sqrt()

    return dict(q=(1.5 * rms(B, H, d)).to(torch.bfloat16),
                r=(0.25 * torch.randn((B, H, d), generator=g)).to(torch.bfloat16),
                K=rms(B, Hkv, L, d).to(torch.bfloat16), V=torch.randn((B, Hkv, L, d), generator=g).to(torch.bfloat16),
                w=torch.rand((B, Hkv, L), generator=g), g=g)


def in_shares(plx, B, Hkv, G, L, d, weights):
    """Whether the decode cuts the keys in shares: that form alone keeps partial records in the workspace."""
    H = Hkv * G
    if not weights:
        return plx.decode_int4kv_workspace_bytes(B, H, Hkv, L, d) > 0
    alone = sum((n + 255) // 256 * 256 for n in (8 * B * H, 4 * B * H * L))  # statistics and scores
    return plx.decode_weights_workspace_bytes(B, H, Hkv, L, d) > alone


@pytest.mark.parametrize("B,Hkv,G,L,d,shares", [
    (300, 3, 1, 70, 64, False), (300, 3, 2, 50, 128, False), (230, 4, 4, 40, 128, False), (84, 8, 8, 60, 64, False),
    (135, 5, 8, 33, 128, False), (900, 1, 4, 65, 64, False),
    (200, 2, 1, 1100, 64, True), (140, 2, 2, 300, 128, True), (130, 1, 8, 400, 64, True), (3, 2, 4, 5000, 128, True),
    (1, 1, 8, 20000, 128, True),
])
def test_both_plans_of_the_decodes_with_weights(plx, B, Hkv, G, L, d, shares):
    """bf16 and 4-bit: one CTA a KV head, and shares (with batches of more than 128 sequences); bad lengths among
    them (first, last, around the 128th); repeatable."""
    assert in_shares(plx, B, Hkv, G, L, d, True) == shares
    c = random_case(B + L, B, Hkv, G, L, d)
    sl = torch.randint(1, L + 1, (B,), generator=c["g"], dtype=torch.int32)
    sl[-1] = L
    bad = [] if B < 100 else [b for b in (0, 1, 127, 128, 129, B - 2) if b < B]
    for i, b in enumerate(bad):
        sl[b] = (0, L + 1, -1)[i % 3]
    good = [b for b in range(B) if b not in bad]
    q, r, w = c["q"].cuda(), c["r"].cuda(), c["w"].cuda()
    Kc, Kp, K4 = quantised(plx, c["K"])
    Vc, Vp, V4 = quantised(plx, c["V"])
    for call, cache, K, V in ((plx.decode_weights, (c["K"].cuda(), c["V"].cuda()), f64(c["K"]), f64(c["V"])),
                              (plx.decode_int4kv_weights, (Kc, Kp, Vc, Vp), K4, V4)):
        first = None
        for _ in range(2):
            wo = torch.full_like(w, -3.0)
            out = call(q, r, *cache, sl.cuda(), w, weights_out=wo, out=torch.ones_like(q))
            assert plx.get_device_status() == (-6 if bad else 0)
            assert first is None or (torch.equal(first[0], out) and torch.equal(first[1], wo))
            first = out, wo
        assert not out[bad].any() and (wo[bad] == -3).all()
        args = f64(q)[good], f64(r)[good], K[good], V[good], sl[good].tolist()
        check_out(out[good], *args)
        check_weights(wo[good], *args, w[good], torch.full_like(w, -3.0)[good])


@pytest.mark.parametrize("B,Hkv,G,L,d,shares", [
    (64, 8, 4, 430, 128, True), (32, 8, 8, 860, 128, True), (64, 8, 2, 430, 128, True), (32, 8, 8, 1650, 64, True),
    (16, 4, 4, 3500, 128, True), (8, 4, 8, 7000, 128, True), (16, 4, 1, 3500, 128, True), (2, 2, 2, 17000, 64, True),
    (300, 3, 4, 50, 128, False), (84, 8, 8, 60, 128, False), (1, 2, 8, 3000, 128, False), (2, 3, 4, 2500, 64, False),
])
def test_both_plans_of_the_decode(plx, B, Hkv, G, L, d, shares):
    """4-bit: shares merged by few and by many threads a head, one CTA a KV head, clusters; ragged, repeatable."""
    assert in_shares(plx, B, Hkv, G, L, d, False) == shares
    c = random_case(B + L, B, Hkv, G, L, d)
    sl = torch.randint(1, L + 1, (B,), generator=c["g"], dtype=torch.int32)
    sl[0] = L
    Kc, Kp, K = quantised(plx, c["K"])
    Vc, Vp, V = quantised(plx, c["V"])
    args = (c["q"].cuda(), c["r"].cuda(), Kc, Kp, Vc, Vp, sl.cuda())
    out = plx.decode_int4kv(*args)
    assert torch.equal(out, plx.decode_int4kv(*args))
    check_out(out, f64(c["q"]), f64(c["r"]), K, V, sl.tolist())


@pytest.mark.parametrize("B,G,L,d", [(512, 1, 40000, 64), (300, 2, 70000, 128), (400, 8, 20000, 64)])
def test_one_long_sequence_among_hundreds(plx, B, G, L, d):
    """Nearly all shares, so nearly all records, belong to one KV head; the others have one key or a few."""
    H = G
    g = torch.Generator(device="cuda").manual_seed(B)
    lens = [1 + b % 3 for b in range(B)]
    lens[B // 2] = L
    codes = [torch.empty((B, 1, L, d // 2), dtype=torch.uint8, device="cuda") for _ in range(2)]
    params = [torch.empty((B, 1, L, 2), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    w = torch.rand((B, 1, L), generator=g, device="cuda")
    values = []
    for i in range(2):
        rows = torch.randn((B - 1, 1, 3, d), generator=g, device="cuda").to(torch.bfloat16)
        long = torch.randn((1, 1, L, d), generator=g, device="cuda").to(torch.bfloat16)
        (c0, p0, v0), (c1, p1, v1) = quantised(plx, rows), quantised(plx, long)
        others = [b for b in range(B) if b != B // 2]
        codes[i][others, :, :3], params[i][others, :, :3] = c0, p0
        codes[i][B // 2], params[i][B // 2] = c1[0], p1[0]
        values.append((v0, v1, others))
    q = (1.5 * torch.randn((B, H, d), generator=g, device="cuda")).to(torch.bfloat16)
    r = (0.25 * torch.randn((B, H, d), generator=g, device="cuda")).to(torch.bfloat16)
    sl = torch.tensor(lens, dtype=torch.int32, device="cuda")
    cache = (codes[0], params[0], codes[1], params[1])
    assert in_shares(plx, B, 1, G, L, d, False) and in_shares(plx, B, 1, G, L, d, True)
    wo = torch.full_like(w, -3.0)
    outs = plx.decode_int4kv(q, r, *cache, sl), plx.decode_int4kv_weights(q, r, *cache, sl, w, weights_out=wo)
    (ks, kl, others), (vs, vl, _) = values
    at = [B // 2]
    for out in outs:
        check_out(out[at], f64(q)[at], f64(r)[at], kl, vl, [L])
        check_out(out[others], f64(q)[others], f64(r)[others], ks, vs, [lens[b] for b in others])
    check_weights(wo[at], f64(q)[at], f64(r)[at], kl, vl, [L], w[at], torch.full_like(w, -3.0)[at])
    for i, b in enumerate(others):
        check_weights(wo[b:b + 1, :, :3], f64(q)[b:b + 1], f64(r)[b:b + 1], ks[i:i + 1], vs[i:i + 1], [lens[b]],
                      w[b:b + 1, :, :3], torch.full_like(w, -3.0)[b:b + 1, :, :3])
        assert (wo[b, :, 3:] == -3).all()


def whole_rows(g, *shape):
    """Rows of the integers -7..8, both ends in each: held in 4 bits with scale 1 and zero point 7, exactly."""
    x = torch.randint(-7, 9, shape, generator=g).double()
    x[..., -1], x[..., -2] = -7, 8
    return x


@pytest.mark.parametrize("G", [1, 2, 4, 8])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("rising", [True, False])
@pytest.mark.parametrize("scale_v", [1.0, 2.0 ** -80, 2.0 ** 80])
def test_large_scores(plx, G, d, rising, scale_v):
    """Scores up to 2^20 log2 units, 500 or more apart or equal: what the softmax has to give is known although a score
    of this size is off by more than its last bits would allow.

    Keys are integers and queries integers times 2^12, so q.k is exact in fp32 and equal scores are equal bits.  A score
    q.k log2(e) / sqrt(d) is rounded three more times, by 3 * 2^20 * 2^-24 < 0.2 log2 units; keys that do not have the
    largest score are 2^12 log2(e) / sqrt(128) > 500 units behind it, so their weights are 0 in fp32 and below 2^-499 in
    the formula.  The largest score belongs to several keys (equal in the dims that q sees), so t and tbar count, too.
    With `rising` scores grow along the sequence and the reference is raised in nearly every tile.  The bounds are those
    of check_out and check_weights (equal weights have no score error): V is small integers times a power of two, and a
    term keeps its 16 bits down to 2^-133."""
    B, Hkv, L = 2, 2, 300
    g = torch.Generator().manual_seed(17 * G + d)
    H = Hkv * G
    K, V = whole_rows(g, B, Hkv, L, d), whole_rows(g, B, Hkv, L, d) * scale_v
    q = torch.zeros((B, H, d), dtype=torch.float64)
    q[..., :d // 2] = torch.randint(-3, 4, (B, 1, d // 2), generator=g).double()  # heads of a group agree on the order
    q *= 2.0 ** 12
    r = torch.randint(-4, 5, (B, H, d), generator=g).double() / 16
    for b in range(B):
        for h in range(Hkv):
            order = torch.argsort(K[b, h] @ q[b, h * G], stable=True)
            if rising:
                K[b, h] = K[b, h, order].clone()
            top = K[b, h, -1 if rising else order[-1], :d // 2].clone()
            for j in (L - 1, L - 2, L - 40, L - 41, L - 75) if rising else (L - 1, L - 2, L - 40, 77, 12):
                K[b, h, j, :d // 2] = top
    q, r, K, V = (x.to(torch.bfloat16) for x in (q, r, K, V))
    sl = torch.full((B,), L, dtype=torch.int32, device="cuda")
    Kc, Kp, K4 = quantised(plx, K)
    Vc, Vp, V4 = quantised(plx, V)
    assert np.array_equal(K4, f64(K)) and np.array_equal(V4, f64(V))
    q64, r64, K64, V64, lens = f64(q), f64(r), f64(K), f64(V), [L] * B
    s = np.einsum("bgd,bgld->bgl", q64[:, ::G], K64)
    assert (np.sort(s, -1)[..., -5:] == s.max(-1, keepdims=True)).all()
    # What is checked tells wrong answers apart: nothing, the wrong sign, no probe, another key.
    want = oracle.decode_gqa_ref(q64, r64, K64, V64, lens)
    allowed = 2.0 ** -8 * np.abs(want) + 2.0 ** -13 * oracle.decode_magnitude(q64, r64, K64, V64, lens)
    for wrong in (0 * want, -want, oracle.decode_gqa_ref(q64, 0 * r64, K64, V64, lens),
                  oracle.decode_gqa_ref(q64, r64, K64[:, :, :-1], V64[:, :, :-1], [L - 1] * B)):
        assert ((np.abs(wrong - want) > 2 * allowed).any(-1)).all()
    w = torch.rand((B, Hkv, L), generator=g).cuda()
    qd, rd = q.cuda(), r.cuda()
    check_out(plx.decode_int4kv(qd, rd, Kc, Kp, Vc, Vp, sl), q64, r64, K64, V64, lens)
    for call, cache in ((plx.decode_int4kv_weights, (Kc, Kp, Vc, Vp)), (plx.decode_weights, (K.cuda(), V.cuda()))):
        wo = torch.empty_like(w)
        check_out(call(qd, rd, *cache, sl, w, weights_out=wo), q64, r64, K64, V64, lens)
        check_weights(wo, q64, r64, K64, V64, lens, w, w)


def spread(q, r, K, V, seqlens):
    """sum_j p_j (1 + |t_j - tbar|) |v_j|: what rounding errors of the terms p_j (1 - (t_j - tbar)) v_j scale with."""
    B, H, d = q.shape
    G = H // K.shape[1]
    out = np.zeros((B, H, d))
    for b in range(B):
        n = int(seqlens[b])
        for h in range(H):
            k, v = K[b, h // G, :n], V[b, h // G, :n]
            p = oracle.softmax_weights_row(q[b, h], k)
            t = k @ r[b, h]
            out[b, h] = (p * (1 + np.abs(t - p @ t))) @ np.abs(v)
    return out


@pytest.mark.parametrize("B,Hkv,G,L,d", [
    (2, 2, 1, 300, 128), (2, 1, 2, 300, 64), (2, 2, 4, 100, 128), (1, 2, 8, 2000, 64), (1, 1, 1, 17000, 64),
    (1, 1, 4, 17000, 128), (300, 3, 1, 20, 64), (1, 2, 2, 1500, 128), (900, 1, 2, 33, 128),
])
@pytest.mark.parametrize("common", [2.0 ** 15, -2.0 ** 12, 0.0])
def test_a_direction_that_all_keys_share(plx, B, Hkv, G, L, d, common):
    """t = rho.k is about `common` for every key, with differences of a few units between them.

    Taking one number off all t changes nothing in the formula, so errors may scale with the differences alone:
    |g - o| <= 2^-8 |o| + 2^-13 sum p (1 + |t - tbar|) |v|.  Keys are integers -7..8 and the probe multiples of 1/8, so
    t is exact in fp32 (multiples of 1/8 below 2^17); t less its reference and the sums over it are then rounded
    relative to the differences: 2^-16 (bf16 pairs) and a few 2^-23, as in check_out."""
    g = torch.Generator().manual_seed(L + G)
    H = Hkv * G
    K, V = whole_rows(g, B, Hkv, L, d), torch.randn((B, Hkv, L, d), generator=g)
    K[..., :8] = 8
    q = 0.05 * torch.randn((B, H, d), generator=g)
    r = torch.randint(-2, 3, (B, H, d), generator=g).double() / 8
    r[..., :8] = common / 64
    q, r, K, V = (x.to(torch.bfloat16) for x in (q, r, K, V))
    lens = torch.randint(1, L + 1, (B,), generator=g).tolist()
    lens[0] = L
    sl = torch.tensor(lens, dtype=torch.int32, device="cuda")
    Kc, Kp, K4 = quantised(plx, K)
    Vc, Vp, V4 = quantised(plx, V)
    assert np.array_equal(K4, f64(K))
    q64, r64, K64, w = f64(q), f64(r), f64(K), torch.zeros((B, Hkv, L), device="cuda")
    qd, rd = q.cuda(), r.cuda()
    outs = ((plx.decode_int4kv(qd, rd, Kc, Kp, Vc, Vp, sl), V4),
            (plx.decode_int4kv_weights(qd, rd, Kc, Kp, Vc, Vp, sl, w), V4),
            (plx.decode_weights(qd, rd, K.cuda(), V.cuda(), sl, w), f64(V)))
    for out, V64 in outs:
        want = oracle.decode_gqa_ref(q64, r64, K64, V64, lens)
        err = np.abs(f64(out) - want) - 2.0 ** -8 * np.abs(want) - 2.0 ** -13 * spread(q64, r64, K64, V64, lens)
        assert err.max() <= 0, err.max()


@pytest.mark.parametrize("G,d", [(1, 128), (2, 64), (4, 128), (8, 64)])
@pytest.mark.parametrize("scale", [2.0 ** 119, 2.0 ** -110])
@pytest.mark.parametrize("int4", [True, False])
def test_probes_of_extreme_size(plx, G, d, scale, int4):
    """Probes next to 2^120, the largest that is computed with, and tiny ones.  t, about 2^6 scale for every key, is an
    integer times scale / 4, and exact; a sum of 32 of the large ones passes fp32's range.  Values are 2^-20 where t is
    large, so that outputs are bf16 numbers.  Bounds as in test_a_direction_that_all_keys_share."""
    B, Hkv, L = 2, 2, 300
    g = torch.Generator().manual_seed(G + d)
    H = Hkv * G
    K, V = whole_rows(g, B, Hkv, L, d), torch.randn((B, Hkv, L, d), generator=g) * min(1.0, 2.0 ** 99 / scale)
    K[..., :8] = 8
    q = 0.05 * torch.randn((B, H, d), generator=g)
    r = torch.zeros((B, H, d), dtype=torch.float64)
    r[..., 8:-2] = torch.randint(-1, 2, (B, H, d - 10), generator=g).double() / 4
    r[..., :8] = 1
    q, r, K, V = (x.to(torch.bfloat16) for x in (q, r * scale, K, V))
    lens = [L, 77]
    sl = torch.tensor(lens, dtype=torch.int32, device="cuda")
    qd, rd, w = q.cuda(), r.cuda(), torch.zeros((B, Hkv, L), device="cuda")
    if int4:
        Kc, Kp, K64 = quantised(plx, K)
        Vc, Vp, V64 = quantised(plx, V)
        assert np.array_equal(K64, f64(K))
        outs = [plx.decode_int4kv(qd, rd, Kc, Kp, Vc, Vp, sl), plx.decode_int4kv_weights(qd, rd, Kc, Kp, Vc, Vp, sl, w)]
    else:
        K64, V64 = f64(K), f64(V)
        outs = [plx.decode_weights(qd, rd, K.cuda(), V.cuda(), sl, w)]
    want = oracle.decode_gqa_ref(f64(q), f64(r), K64, V64, lens)
    allowed = 2.0 ** -8 * np.abs(want) + 2.0 ** -13 * spread(f64(q), f64(r), K64, V64, lens)
    for out in outs:
        err = np.abs(f64(out) - want) - allowed
        assert err.max() <= 0, err.max()


def test_decode_with_weights_beyond_32_bit_offsets(plx):
    """bf16 rows of the last head lie more than 2^32 bytes into their cache, its scores more than 2^31 into theirs."""
    B, Hkv, G, L, d, n = 1, 2, 8, 36_000_000, 64, 500
    c = random_case(70, B, Hkv, G, n, d)
    K, V = (torch.empty((B, Hkv, L, d), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    K[:, :, :n], V[:, :, :n] = c["K"].cuda(), c["V"].cuda()
    w = torch.zeros((B, Hkv, L), device="cuda")
    w[:, :, :n] = c["w"].cuda()
    sl = torch.tensor([n], dtype=torch.int32, device="cuda")
    out = plx.decode_weights(c["q"].cuda(), c["r"].cuda(), K, V, sl, w)
    args = f64(c["q"]), f64(c["r"]), f64(c["K"]), f64(c["V"]), [n]
    check_out(out, *args)
    check_weights(w[:, :, :n], *args, c["w"], c["w"])
    assert not w[:, :, n:].any()


def test_two_graphs_at_once_with_their_inputs_held(plx):
    """Captured decodes and evictions of two sizes, replayed on two streams at the same time, eager calls on a third;
    every tensor that a graph reads lives as long as the graph."""
    runs = []
    for i, (B, Hkv, G, L, d) in enumerate([(1, 2, 2, 9000, 128), (3, 2, 1, 4000, 64)]):
        c = random_case(60 + i, B, Hkv, G, L, d)
        Kc, Kp, _ = quantised(plx, c["K"])
        Vc, Vp, _ = quantised(plx, c["V"])
        sl = torch.full((B,), L - 5, dtype=torch.int32, device="cuda")
        args, w = (c["q"].cuda(), c["r"].cuda(), Kc, Kp, Vc, Vp, sl), c["w"].cuda()
        want_w = w.clone()
        want = plx.decode_int4kv_weights(*args, want_w)
        wo = torch.zeros_like(w)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = plx.decode_int4kv_weights(*args, w, weights_out=wo)
            small = [torch.zeros((B, Hkv, 500, *t.shape[3:]), dtype=t.dtype, device="cuda") for t in (Kc, Kp)]
            small_w = torch.empty((B, Hkv, 500), device="cuda")
            kept, _ = plx.cache_evict([Kc, Kp], wo, sl, 500, 2, 16, caches_out=small, weights_out=small_w)
        runs.append((graph, torch.cuda.Stream(), args, w, out, wo, want, want_w, kept, small, small_w, L))
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(8):
        for graph, stream, *_ in runs:
            with torch.cuda.stream(stream):
                graph.replay()
        other = plx.decode_int4kv(*runs[0][2], stream=side)
    torch.cuda.synchronize()
    assert torch.equal(other, plx.decode_int4kv(*runs[0][2]))
    for _, _, args, w, out, wo, want, want_w, kept, small, small_w, L in runs:
        n = L - 5
        assert torch.equal(out, want) and torch.equal(wo[..., :n], want_w[..., :n])
        at = kept.long()[..., None]
        assert torch.equal(small[0], torch.gather(args[2], 2, at.expand(*at.shape[:3], args[2].shape[-1])))
        assert torch.equal(small_w, torch.gather(want_w, 2, kept.long()))
        for b in range(kept.shape[0]):
            for h in range(kept.shape[1]):
                assert kept[b, h].tolist() == oracle.evict_ref(want_w[b, h].tolist(), n, 500, 2, 16).tolist()
