"""GPU parity of the 4-bit KV cache and of the decodes that collect attention weight.

Rows: codes, scales and zero points are integer decisions, bit for bit those of exact arithmetic.

Outputs of a decode: |g - o| <= 2^-8 |o| + 2^-13 A with A = sum_j p_j (1 + |t_j| + |tbar|) |v_j|.  The first term is
the one rounding to bf16.  The second covers the arithmetic: the weights enter the value sums as bf16 hi + lo pairs
(relative 2^-16), scores and t are fp32 sums over d <= 128 products (at most 2^-24 a term of a sum of about 12 in units
of the softmax argument, so below 2^-16 relative in p, and 2^-24 * 100 absolute in t against the 1 in A), exp2f and
the merges are a few 2^-23: together below 2^-15, with a factor 4 left.

Weights: |g - o| <= 2^-23 |o| + 2^-15 p for the sum p of the head's softmax weights (the same score error, and the
additions in fp32).
"""
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


def f64(t):
    return t.detach().double().cpu().numpy()


def rms_rows(g, *shape):
    x = torch.randn(shape, generator=g)
    return (x / x.square().mean(-1, keepdim=True).sqrt()).to(torch.bfloat16)


def case(seed, B, Hkv, G, L, d):
    g = torch.Generator().manual_seed(seed)
    H = Hkv * G
    return dict(q=(1.5 * rms_rows(g, B, H, d)).to(torch.bfloat16), r=(0.25 * torch.randn((B, H, d), generator=g)).to(torch.bfloat16),
                K=rms_rows(g, B, Hkv, L, d), V=torch.randn((B, Hkv, L, d), generator=g).to(torch.bfloat16),
                w=torch.rand((B, Hkv, L), generator=g))


def quantised(plx, X):
    """(device codes, device params, float64 values) of bf16 rows on the CPU."""
    codes, params = plx.kv_quantize_int4(X.cuda())
    return codes, params, oracle.kv_dequantize_int4_ref(codes.cpu().numpy(), f64(params)[..., 0], f64(params)[..., 1])


def check_out(got, q, r, K, V, sl):
    want = oracle.decode_gqa_ref(q, r, K, V, sl)
    mag = oracle.decode_magnitude(q, r, K, V, sl)
    err = np.abs(f64(got) - want) - 2.0 ** -8 * np.abs(want) - 2.0 ** -13 * mag
    assert err.max() <= 0, err.max()


def check_weights(got, q, r, K, V, sl, w, before):
    _, want = oracle.decode_weights_ref(q, r, K, V, sl, f64(w))
    got = f64(got)
    for b, n in enumerate(sl):
        err = np.abs(got[b, :, :n] - want[b, :, :n])
        p = want[b, :, :n] - f64(w)[b, :, :n]
        assert (err <= 2.0 ** -23 * np.abs(want[b, :, :n]) + 2.0 ** -15 * p).all()
        assert np.array_equal(got[b, :, n:], f64(before)[b, :, n:])


# ---------------------------------------------------------------- rows


@pytest.mark.parametrize("d", [64, 128])
def test_rows_are_bit_exact(plx, d):
    rng = np.random.default_rng(d)
    rows = [rng.standard_normal(d) * np.exp(rng.uniform(-60, 60)) for _ in range(200)]
    rows += [rng.standard_normal(d) + rng.uniform(-6, 6) for _ in range(200)]
    rows += [np.zeros(d), np.full(d, 3.0), np.full(d, -2.0), np.abs(rng.standard_normal(d)), np.full(d, 2.0 ** -133)]
    ties = np.resize(np.arange(-14, 17) / 2.0, d)
    rows += [ties, ties * 2.0 ** -120, ties * 2.0 ** 100]  # the scale is 1 here: quotients are half integers
    tiny = np.resize([2.0 ** -133 * k for k in range(40)], d)
    rows += [tiny, -tiny, np.resize([3e38, 1e38, -3e37], d)]
    X = torch.from_numpy(np.stack(rows)).to(torch.bfloat16)
    codes, params = plx.kv_quantize_int4(X.cuda())
    want_c, want_s, want_z = oracle.kv_quantize_int4_ref(X.double().numpy())
    assert np.array_equal(f64(params)[:, 0], want_s)
    assert np.array_equal(f64(params)[:, 1], want_z)
    assert np.array_equal(codes.cpu().numpy(), want_c)
    back = plx.kv_dequantize_int4(codes, params)
    want = torch.from_numpy(oracle.kv_dequantize_int4_ref(want_c, want_s, want_z)).to(torch.bfloat16)
    assert torch.equal(back.cpu(), want)


def test_rows_with_infinities_and_nan(plx):
    X = torch.zeros((6, 64), dtype=torch.bfloat16)
    X[0, 3], X[1, 60], X[2, 0], X[3, 1] = math.inf, -math.inf, math.nan, -math.nan
    X[4, 5], X[4, 6] = math.inf, -math.inf
    X[5] = 1.0
    codes, params = plx.kv_quantize_int4(X.cuda())
    back = plx.kv_dequantize_int4(codes, params)
    assert back[:5].isnan().all() and torch.equal(back[5].cpu(), X[5])


@pytest.mark.parametrize("rows", [1, 2, 3, 31, 1000])
@pytest.mark.parametrize("d", [64, 128])
def test_row_counts_and_neighbours(plx, rows, d):
    """Buffers longer than the rows keep what lies behind them."""
    X = torch.randn((rows, d), generator=torch.Generator().manual_seed(rows)).to(torch.bfloat16).cuda()
    codes = torch.full((rows + 5, d // 2), 0xAB, dtype=torch.uint8, device="cuda")
    params = torch.full((rows + 5, 2), 7.0, dtype=torch.bfloat16, device="cuda")
    out = torch.full((rows + 5, d), 9.0, dtype=torch.bfloat16, device="cuda")
    plx.kv_quantize_int4(X, codes=codes[:rows], params=params[:rows])
    plx.kv_dequantize_int4(codes[:rows], params[:rows], out=out[:rows])
    assert (codes[rows:] == 0xAB).all() and (params[rows:] == 7).all() and (out[rows:] == 9).all()
    c, s, z = oracle.kv_quantize_int4_ref(f64(X))
    assert np.array_equal(codes[:rows].cpu().numpy(), c)
    assert np.array_equal(f64(out[:rows]), f64(torch.from_numpy(oracle.kv_dequantize_int4_ref(c, s, z)).to(torch.bfloat16)))


@pytest.mark.parametrize("B,Hkv,L,d", [(1, 1, 1, 128), (3, 5, 17, 64), (4, 2, 33, 128)])
def test_append_is_a_row_of_the_cache(plx, B, Hkv, L, d):
    c = case(5, B, Hkv, 1, L, d)
    Kc, Kp, _ = quantised(plx, c["K"])
    Vc, Vp, _ = quantised(plx, c["V"])
    k, v = c["q"].cuda(), c["r"].cuda()  # [B, Hkv, d] with groups of one
    sl = torch.tensor([L, 1, (L + 1) // 2, 2][:B], dtype=torch.int32)
    before = [t.clone() for t in (Kc, Kp, Vc, Vp)]
    k_out, v_out = torch.empty_like(k), torch.empty_like(v)
    plx.kv_append_int4(k, v, Kc, Kp, Vc, Vp, sl.cuda(), k_out=k_out, v_out=v_out)
    for new, back, (codes, params), (codes0, params0) in ((k, k_out, (Kc, Kp), before[:2]), (v, v_out, (Vc, Vp), before[2:])):
        nc, np_ = plx.kv_quantize_int4(new)
        assert torch.equal(back, plx.kv_dequantize_int4(nc, np_))
        for b in range(B):
            codes0[b, :, sl[b] - 1], params0[b, :, sl[b] - 1] = nc[b], np_[b]
        assert torch.equal(codes, codes0) and torch.equal(params.view(torch.int16), params0.view(torch.int16))
    plx.kv_append_int4(k, v, Kc, Kp, Vc, Vp, sl.cuda())  # without the values
    assert torch.equal(Kc, before[0])


# ---------------------------------------------------------------- decode


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("G,Hkv", [(1, 3), (2, 2), (4, 1), (8, 2)])
def test_decode_lengths(plx, G, Hkv, d):
    """Lengths at the edges of the 16-key blocks, the 32-key tiles and the warps' turns; both caches."""
    lens = [1, 2, 15, 16, 17, 31, 32, 33, 127, 128, 129, 500, 601]
    B, L = len(lens), 601
    c = case(10 * G + d, B, Hkv, G, L, d)
    sl = torch.tensor(lens, dtype=torch.int32)
    Kc, Kp, K = quantised(plx, c["K"])
    Vc, Vp, V = quantised(plx, c["V"])
    q, r, w = c["q"].cuda(), c["r"].cuda(), c["w"].cuda()
    q64, r64 = f64(q), f64(r)
    check_out(plx.decode_int4kv(q, r, Kc, Kp, Vc, Vp, sl.cuda()), q64, r64, K, V, lens)
    wo = torch.full_like(w, -3.0)
    out = plx.decode_int4kv_weights(q, r, Kc, Kp, Vc, Vp, sl.cuda(), w, weights_out=wo)
    check_out(out, q64, r64, K, V, lens)
    check_weights(wo, q64, r64, K, V, lens, w, torch.full_like(w, -3.0))
    wo = w.clone()
    out = plx.decode_weights(q, r, c["K"].cuda(), c["V"].cuda(), sl.cuda(), wo)  # in place
    check_out(out, q64, r64, f64(c["K"]), f64(c["V"]), lens)
    check_weights(wo, q64, r64, f64(c["K"]), f64(c["V"]), lens, w, w)


@pytest.mark.parametrize("B,Hkv,G,L,d", [
    (1, 1, 1, 5000, 128), (1, 2, 4, 9001, 64), (2, 1, 8, 4099, 128), (1, 1, 2, 40000, 64), (40, 3, 1, 700, 128),
    (300, 4, 1, 40, 64), (7, 8, 2, 129, 128), (200, 2, 1, 1100, 64), (1, 1, 8, 150000, 64), (1, 1, 1, 5, 128),
    (225, 4, 4, 70, 128), (20, 4, 8, 900, 128),
])
def test_decode_splits(plx, B, Hkv, G, L, d):
    """Every way a sequence is cut: many CTAs merged through the workspace, clusters, one CTA; repeatable."""
    c = case(B + L, B, Hkv, G, L, d)
    g = torch.Generator().manual_seed(3)
    sl = torch.randint(max(1, L // 3), L + 1, (B,), generator=g, dtype=torch.int32)
    sl[0] = L
    Kc, Kp, K = quantised(plx, c["K"])
    Vc, Vp, V = quantised(plx, c["V"])
    q, r, w = c["q"].cuda(), c["r"].cuda(), c["w"].cuda()
    args = (q, r, Kc, Kp, Vc, Vp, sl.cuda())
    out = plx.decode_int4kv(*args)
    check_out(out, f64(q), f64(r), K, V, sl.tolist())
    assert torch.equal(out, plx.decode_int4kv(*args))
    need = plx.decode_int4kv_workspace_bytes(B, Hkv * G, Hkv, L, d)
    ws = torch.full((max(need, 1),), 0xFF, dtype=torch.uint8, device="cuda")
    assert torch.equal(out, plx.decode_int4kv(*args, workspace=ws))
    wo = w.clone()
    plx.decode_int4kv_weights(*args, wo)
    check_weights(wo, f64(q), f64(r), K, V, sl.tolist(), w, w)
    wo2 = w.clone()
    ws = torch.full((plx.decode_weights_workspace_bytes(B, Hkv * G, Hkv, L, d),), 0xFF, dtype=torch.uint8, device="cuda")
    out2 = plx.decode_int4kv_weights(*args, wo2, workspace=ws)
    assert torch.equal(wo, wo2)
    check_out(out2, f64(q), f64(r), K, V, sl.tolist())


@pytest.mark.parametrize("d", [64, 128])
def test_what_lies_behind_a_sequence_does_not_matter(plx, d):
    B, Hkv, G, L = 3, 2, 2, 90
    c = case(1, B, Hkv, G, L, d)
    sl = [1, 33, 90]
    t = torch.tensor(sl, dtype=torch.int32, device="cuda")
    Kc, Kp, K = quantised(plx, c["K"])
    Vc, Vp, V = quantised(plx, c["V"])
    K16, V16 = c["K"].cuda(), c["V"].cuda()
    q, r, w = c["q"].cuda(), c["r"].cuda(), c["w"].cuda()
    first = plx.decode_int4kv(q, r, Kc, Kp, Vc, Vp, t), plx.decode_weights(q, r, K16, V16, t, w.clone())
    for b, n in enumerate(sl):
        for x in (Kp, Vp, K16, V16):
            x[b, :, n:] = math.nan
        for x in (Kc, Vc):
            x[b, :, n:] = 0xFF
    w2 = w.clone()
    for b, n in enumerate(sl):
        w2[b, :, n:] = math.nan
    again = plx.decode_int4kv(q, r, Kc, Kp, Vc, Vp, t), plx.decode_weights(q, r, K16, V16, t, w2)
    assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])
    for b, n in enumerate(sl):
        assert w2[b, :, n:].isnan().all() and w2[b, :, :n].isfinite().all()


def test_a_nan_row_reaches_its_own_heads_only(plx):
    B, Hkv, G, L, d = 2, 2, 4, 70, 128
    c = case(2, B, Hkv, G, L, d)
    c["K"][1, 0, 5, 3] = math.inf
    c["V"][0, 1, 69, 3] = math.nan
    Kc, Kp, _ = quantised(plx, c["K"])
    Vc, Vp, _ = quantised(plx, c["V"])
    sl = torch.full((B,), L, dtype=torch.int32, device="cuda")
    out = plx.decode_int4kv(c["q"].cuda(), c["r"].cuda(), Kc, Kp, Vc, Vp, sl)
    nan = out.isnan().all(-1).view(B, Hkv, G).all(-1)
    assert nan.tolist() == [[False, True], [True, False]]
    assert out.view(B, Hkv, G, d)[0, 0].isfinite().all() and out.view(B, Hkv, G, d)[1, 1].isfinite().all()


@pytest.mark.parametrize("scale_q,scale_v", [(40.0, 1.0), (1e-20, 1e-20), (1.0, 1e30), (1e4, 1e-25)])
def test_wide_ranges(plx, scale_q, scale_v):
    """Scores far apart (one key takes all, the reference is raised often), tiny and huge values."""
    B, Hkv, G, L, d = 2, 2, 2, 800, 64
    c = case(3, B, Hkv, G, L, d)
    c["q"] = (c["q"].double() * scale_q).to(torch.bfloat16)
    c["r"] = (c["r"].double() * 0.1).to(torch.bfloat16)
    c["V"] = (c["V"].double() * scale_v).to(torch.bfloat16)
    c["K"] *= torch.linspace(0.1, 2.0, L)[:, None].to(torch.bfloat16)
    Kc, Kp, K = quantised(plx, c["K"])
    Vc, Vp, V = quantised(plx, c["V"])
    sl = torch.full((B,), L, dtype=torch.int32, device="cuda")
    out = plx.decode_int4kv(c["q"].cuda(), c["r"].cuda(), Kc, Kp, Vc, Vp, sl)
    q, r = f64(c["q"]), f64(c["r"])
    want = oracle.decode_gqa_ref(q, r, K, V, [L] * B)
    mag = oracle.decode_magnitude(q, r, K, V, [L] * B)
    # A score error is relative to the scores (2^-21 of the sum of |q k| over sqrt d, in units of the argument).
    ds = np.abs(q).max() * np.abs(K).max() * d ** 0.5 * 2.0 ** -21
    # Underflow, absolute: with the reference 2^8 above the largest score, a weight below 2^-118 of the largest is less
    # than the smallest normal fp32, and w s_v (w t s_v) keeps no bits below the smallest bf16, 2^-133.  So a key's
    # term loses at most 15 * 2^-133 + 15 s_v 2^-126, times 2^8 / omega <= 2^9 at the end, for O1 and for O2 (times |t|).
    t = 1 + 2 * np.abs(r).max() * np.abs(K).max() * d
    lost = L * t * 2.0 ** 13 * (2.0 ** -133 + 2.0 ** -126 * np.abs(V).max())
    assert (np.abs(f64(out) - want) <= 2.0 ** -8 * np.abs(want) + (2.0 ** -13 + 2 * ds) * mag + lost).all()


def test_rows_beyond_32_bit_offsets(plx):
    """Codes of the last heads lie more than 2^32 bytes into their cache."""
    B, Hkv, G, L, d, n = 2, 2, 1, 36_000_000, 128, 100
    c = case(4, B, Hkv, G, n, d)
    caches = []
    for X in (c["K"], c["V"]):
        small = quantised(plx, X)
        codes = torch.empty((B, Hkv, L, d // 2), dtype=torch.uint8, device="cuda")
        params = torch.empty((B, Hkv, L, 2), dtype=torch.bfloat16, device="cuda")
        codes[:, :, :n], params[:, :, :n] = small[0], small[1]
        caches.append((codes, params, small[2]))
    sl = torch.tensor([n, n], dtype=torch.int32, device="cuda")
    (Kc, Kp, K), (Vc, Vp, V) = caches
    assert (B * Hkv - 1) * L * d // 2 > 2 ** 32
    out = plx.decode_int4kv(c["q"].cuda(), c["r"].cuda(), Kc, Kp, Vc, Vp, sl)
    check_out(out, f64(c["q"]), f64(c["r"]), K, V, [n, n])
    k = c["K"][:, :, 0].cuda()
    plx.kv_append_int4(k, k, Kc, Kp, Vc, Vp, torch.tensor([n, L], dtype=torch.int32, device="cuda"))
    want_c, want_p = plx.kv_quantize_int4(k)
    assert torch.equal(Kc[1, :, L - 1], want_c[1]) and torch.equal(Vp[1, :, L - 1], want_p[1])
    assert torch.equal(Kc[0, :, n - 1], want_c[0])


# ---------------------------------------------------------------- errors, streams, graphs


def test_bad_lengths_are_reported(plx):
    B, Hkv, G, L, d = 3, 2, 2, 40, 64
    c = case(6, B, Hkv, G, L, d)
    Kc, Kp, K = quantised(plx, c["K"])
    Vc, Vp, V = quantised(plx, c["V"])
    q, r, w = c["q"].cuda(), c["r"].cuda(), c["w"].cuda()
    for bad in (0, -5, L + 1, 2 ** 31 - 1):
        t = torch.tensor([L, bad, 3], dtype=torch.int32, device="cuda")
        wo = w.clone()
        out = plx.decode_int4kv_weights(q, r, Kc, Kp, Vc, Vp, t, wo)
        assert plx.get_device_status() == -6
        assert not out[1].any() and torch.equal(wo[1], w[1])
        check_out(out[[0, 2]], f64(q)[[0, 2]], f64(r)[[0, 2]], K[[0, 2]], V[[0, 2]], [L, 3])
        out = plx.decode_int4kv(q, r, Kc, Kp, Vc, Vp, t)
        assert plx.get_device_status() == -6 and not out[1].any()
        before = [x.clone() for x in (Kc, Vc)]
        k = torch.ones((B, Hkv, d), dtype=torch.bfloat16, device="cuda")
        k_out = torch.full_like(k, 5.0)
        plx.kv_append_int4(k, k, Kc, Kp, Vc, Vp, t, k_out=k_out)
        assert plx.get_device_status() == -6
        assert torch.equal(Kc[1], before[0][1]) and torch.equal(Vc[1], before[1][1])
        assert not k_out[1].any() and (k_out[0] == 1).all()
        Kc, Kp, K = quantised(plx, c["K"])
        Vc, Vp, V = quantised(plx, c["V"])


@pytest.mark.parametrize("B,Hkv,L", [(200, 2, 1100), (300, 3, 50)])
def test_bad_lengths_in_a_large_batch(plx, B, Hkv, L):
    """Every kind of launch skips the bad sequences and serves the others (first, last and neighbours among the bad)."""
    d, G = 64, 1
    c = case(8, B, Hkv, G, L, d)
    Kc, Kp, K = quantised(plx, c["K"])
    Vc, Vp, V = quantised(plx, c["V"])
    q, r, w = c["q"].cuda(), c["r"].cuda(), c["w"].cuda()
    g = torch.Generator().manual_seed(5)
    sl = torch.randint(1, L + 1, (B,), generator=g, dtype=torch.int32)
    bad = [0, 1, 63, 127, 128, 129, B - 1]
    for i, b in enumerate(bad):
        sl[b] = (0, L + 1, -1)[i % 3]
    good = [b for b in range(B) if b not in bad]
    wo = w.clone()
    outs = [plx.decode_int4kv(q, r, Kc, Kp, Vc, Vp, sl.cuda(), out=torch.ones_like(q)),
            plx.decode_int4kv_weights(q, r, Kc, Kp, Vc, Vp, sl.cuda(), wo, out=torch.ones_like(q))]
    assert plx.get_device_status() == -6
    for out in outs:
        assert not out[bad].any()
        check_out(out[good], f64(q)[good], f64(r)[good], K[good], V[good], sl[good].tolist())
    assert torch.equal(wo[bad], w[bad])
    check_weights(wo[good], f64(q)[good], f64(r)[good], K[good], V[good], sl[good].tolist(), w[good], w[good])
    none = torch.zeros((B,), dtype=torch.int32, device="cuda")
    out = plx.decode_int4kv_weights(q, r, Kc, Kp, Vc, Vp, none, wo)
    assert plx.get_device_status() == -6 and not out.any()


def test_binding_refuses(plx):
    B, Hkv, G, L, d = 2, 2, 2, 24, 64
    c = case(7, B, Hkv, G, L, d)
    Kc, Kp, _ = quantised(plx, c["K"])
    Vc, Vp, _ = quantised(plx, c["V"])
    q, r, w = c["q"].cuda(), c["r"].cuda(), c["w"].cuda()
    K16, V16 = c["K"].cuda(), c["V"].cuda()
    sl = torch.full((B,), L, dtype=torch.int32, device="cuda")
    ok = (q, r, Kc, Kp, Vc, Vp, sl)
    for i, wrong in ((0, q.float()), (1, r[:, :2]), (2, Kc.view(torch.int8)), (3, Kp.float()), (4, Vc[..., :16]),
                     (5, Vp.transpose(2, 3)), (6, sl.long()), (6, sl[:1]), (6, sl.cpu()), (2, Kc.cpu())):
        args = list(ok)
        args[i] = wrong
        with pytest.raises(ValueError):
            plx.decode_int4kv(*args)
        with pytest.raises(ValueError):
            plx.decode_int4kv_weights(*args, w)
    with pytest.raises(ValueError):
        plx.decode_int4kv(q.transpose(0, 1).contiguous().transpose(0, 1), *ok[1:])
    with pytest.raises(ValueError):
        plx.decode_weights(q, r, K16, V16, sl, w.double())
    with pytest.raises(ValueError):
        plx.decode_weights(q, r, K16.float(), V16.float(), sl, w)
    with pytest.raises(plx.PlxError):
        plx.decode_weights(q, r, K16, V16, sl, w, workspace=torch.empty(64, dtype=torch.uint8, device="cuda"))
    flat = torch.zeros(w.numel() + 8, device="cuda")
    with pytest.raises(plx.PlxError):  # weights and weights_out overlap
        plx.decode_weights(q, r, K16, V16, sl, flat[:-8].view_as(w), weights_out=flat[8:].view_as(w))
    shifted = torch.zeros(q.numel() + 1, dtype=torch.bfloat16, device="cuda")[1:].view_as(q)
    with pytest.raises(plx.PlxError):  # not 16-byte aligned
        plx.decode_int4kv(shifted, *ok[1:])
    with pytest.raises(plx.PlxError):  # workspace not 256-byte aligned
        plx.decode_weights(q, r, K16, V16, sl, w, workspace=torch.empty(1 << 22, dtype=torch.uint8, device="cuda")[8:])
    with pytest.raises(plx.PlxError):  # group of three
        plx.decode_int4kv(torch.cat((q, q[:, :2]), 1), torch.cat((r, r[:, :2]), 1), *ok[2:])
    with pytest.raises(ValueError):
        plx.kv_append_int4(q[:, :2].float(), q[:, :2], Kc, Kp, Vc, Vp, sl)
    with pytest.raises(plx.PlxError):
        plx.kv_quantize_int4(torch.zeros((4, 32), dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(ValueError):
        plx.kv_quantize_int4(torch.zeros((4, 64), device="cuda"))
    with pytest.raises(ValueError):
        plx.kv_quantize_int4(torch.zeros((4, 64), dtype=torch.bfloat16))


def test_two_streams_at_once(plx):
    """Calls on two streams share nothing, whatever the sizes."""
    sizes = [(1, 2, 4, 6000, 128), (2, 1, 1, 9000, 64)]
    runs = []
    for i, (B, Hkv, G, L, d) in enumerate(sizes):
        c = case(20 + i, B, Hkv, G, L, d)
        Kc, Kp, _ = quantised(plx, c["K"])
        Vc, Vp, _ = quantised(plx, c["V"])
        sl = torch.full((B,), L, dtype=torch.int32, device="cuda")
        args = (c["q"].cuda(), c["r"].cuda(), Kc, Kp, Vc, Vp, sl)
        w = c["w"].cuda()
        want_w = w.clone()
        want = plx.decode_int4kv_weights(*args, want_w)
        runs.append((torch.cuda.Stream(), args, w, plx.decode_int4kv(*args), want, want_w))
    torch.cuda.synchronize()
    results = []
    for _ in range(10):
        for stream, args, w, *_ in runs:
            wo = torch.empty_like(w)
            wo.record_stream(stream)
            stream.wait_stream(torch.cuda.current_stream())
            results.append((plx.decode_int4kv(*args, stream=stream),
                            plx.decode_int4kv_weights(*args, w, weights_out=wo, stream=stream), wo))
    torch.cuda.synchronize()
    for i, (a, b, wo) in enumerate(results):
        _, _, _, step, want, want_w = runs[i % 2]
        assert torch.equal(a, step) and torch.equal(b, want) and torch.equal(wo, want_w)


def test_two_graphs_and_eager_calls_between(plx):
    sizes = [(1, 2, 4, 5000, 128), (2, 1, 1, 300, 64)]
    graphs = []
    for i, (B, Hkv, G, L, d) in enumerate(sizes):
        c = case(30 + i, B, Hkv, G, L, d)
        Kc, Kp, _ = quantised(plx, c["K"])
        Vc, Vp, _ = quantised(plx, c["V"])
        sl = torch.full((B,), L - 3, dtype=torch.int32, device="cuda")
        q, r, w = c["q"].cuda(), c["r"].cuda(), c["w"].cuda()
        k = c["K"][:, :, 0].cuda().contiguous()
        out, wo = torch.empty_like(q), torch.zeros_like(w)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            plx.kv_append_int4(k, k, Kc, Kp, Vc, Vp, sl)
            plx.decode_int4kv(q, r, Kc, Kp, Vc, Vp, sl, out=out)
            out2 = plx.decode_int4kv_weights(q, r, Kc, Kp, Vc, Vp, sl, w, weights_out=wo)
        graphs.append((graph, q, r, Kc, Kp, Vc, Vp, sl, w, k, out, wo, out2))
    for turn in range(3):
        for graph, q, r, Kc, Kp, Vc, Vp, sl, w, k, out, wo, out2 in graphs:
            q.copy_(q.roll(1, 0))
            k.mul_(1.25)
            sl += 1
            out.zero_()
            wo.zero_()
        for g in graphs:
            g[0].replay()
        big = case(40, 1, 1, 1, 20000, 64)  # an eager call with a larger workspace in between
        K = quantised(plx, big["K"])
        plx.decode_int4kv(big["q"].cuda(), big["r"].cuda(), K[0], K[1], K[0], K[1],
                          torch.tensor([20000], dtype=torch.int32, device="cuda"))
        torch.cuda.synchronize()
        for graph, q, r, Kc, Kp, Vc, Vp, sl, w, k, out, wo, out2 in graphs:
            K, V = (oracle.kv_dequantize_int4_ref(x.cpu().numpy(), f64(p)[..., 0], f64(p)[..., 1])
                    for x, p in ((Kc, Kp), (Vc, Vp)))
            nc, _ = plx.kv_quantize_int4(k)
            for b, n in enumerate(sl.tolist()):
                assert torch.equal(Kc[b, :, n - 1], nc[b])
            check_out(out, f64(q), f64(r), K, V, sl.tolist())
            check_out(out2, f64(q), f64(r), K, V, sl.tolist())
            check_weights(wo, f64(q), f64(r), K, V, sl.tolist(), w, torch.zeros_like(w))


def test_two_graphs_at_once(plx):
    """Captured calls of two sizes, replayed on two streams at the same time, with other calls on a third."""
    runs = []
    for i, (B, Hkv, G, L, d) in enumerate([(1, 2, 2, 9000, 128), (3, 2, 1, 4000, 64)]):
        c = case(60 + i, B, Hkv, G, L, d)
        Kc, Kp, _ = quantised(plx, c["K"])
        Vc, Vp, _ = quantised(plx, c["V"])
        sl = torch.full((B,), L - 5, dtype=torch.int32, device="cuda")
        args = (c["q"].cuda(), c["r"].cuda(), Kc, Kp, Vc, Vp, sl)
        w = c["w"].cuda()
        want_w = w.clone()
        want = plx.decode_int4kv_weights(*args, want_w)
        wo, kept = torch.zeros_like(w), None
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = plx.decode_int4kv_weights(*args, w, weights_out=wo)
            small = [torch.zeros((B, Hkv, 500, *t.shape[3:]), dtype=t.dtype, device="cuda") for t in (Kc, Kp)]
            kept, _ = plx.cache_evict([Kc, Kp], wo, sl, 500, 2, 16, caches_out=small,
                                      weights_out=torch.empty((B, Hkv, 500), device="cuda"))
        runs.append((graph, torch.cuda.Stream(), args, out, wo, want, want_w, kept, small, L))
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(8):
        for graph, stream, *_ in runs:
            with torch.cuda.stream(stream):
                graph.replay()
        other = plx.decode_int4kv(*runs[0][2], stream=side)
    torch.cuda.synchronize()
    assert torch.equal(other, plx.decode_int4kv(*runs[0][2]))
    for _, _, args, out, wo, want, want_w, kept, small, L in runs:
        assert torch.equal(out, want)
        n = L - 5
        assert torch.equal(wo[..., :n], want_w[..., :n])
        at = kept.long()[..., None]
        assert torch.equal(small[0], torch.gather(args[2], 2, at.expand(*at.shape[:3], args[2].shape[-1])))
        for b in range(kept.shape[0]):
            for h in range(kept.shape[1]):
                assert kept[b, h].tolist() == oracle.evict_ref(want_w[b, h].tolist(), n, 500, 2, 16).tolist()


@pytest.mark.parametrize("int4", [False, True])
def test_a_serving_loop(plx, int4):
    """Steps that append, attend and collect weight; an eviction in place; more steps on the thinned cache."""
    B, Hkv, G, L, d, budget = 2, 2, 2, 64, 64, 24
    c = case(50 + int4, B, Hkv, G, L, d)
    n = [40, 17]
    g = torch.Generator().manual_seed(9)
    if int4:
        (Kc, Kp, K), (Vc, Vp, V) = quantised(plx, c["K"]), quantised(plx, c["V"])
        caches = [Kc, Kp, Vc, Vp]
    else:
        caches = [c["K"].cuda(), c["V"].cuda()]
        K, V = f64(c["K"]), f64(c["V"])
    w = torch.zeros((B, Hkv, L), device="cuda")
    w64 = np.zeros((B, Hkv, L))
    p_sum = np.zeros((B, Hkv, L))
    sl = torch.tensor(n, dtype=torch.int32, device="cuda")
    for step in range(12):
        if step == 6:  # totals of the GPU decide; they are checked against the oracle's before
            kept, sl = plx.cache_evict(caches, w, sl, budget, sinks=2, recent=4)
            want = [[oracle.evict_ref(before_w[b, h], n[b], budget, 2, 4) for h in range(Hkv)] for b in range(B)]
            n = [min(x, budget) for x in n]
            assert sl.tolist() == n
            for b in range(B):
                for h in range(Hkv):
                    ids = want[b][h]
                    assert kept[b, h, :n[b]].tolist() == ids.tolist()
                    for x in (K, V):
                        x[b, h, :n[b]] = x[b, h, ids]
                    w64[b, h, :n[b]] = w64[b, h, ids]
                    p_sum[b, h, :n[b]] = p_sum[b, h, ids]
                    w64[b, h, n[b]:] = p_sum[b, h, n[b]:] = 0
                    assert not w[b, h, n[b]:].any()
        n = [x + 1 for x in n]
        sl += 1
        k = rms_rows(g, B, Hkv, d).cuda()
        v = torch.randn((B, Hkv, d), generator=g).to(torch.bfloat16).cuda()
        q, r = ((s * rms_rows(g, B, Hkv * G, d)).to(torch.bfloat16).cuda() for s in (1.5, 0.25))
        if int4:
            plx.kv_append_int4(k, v, *caches, sl)
            new = [plx.kv_quantize_int4(x) for x in (k, v)]
            new = [oracle.kv_dequantize_int4_ref(a.cpu().numpy(), f64(p)[..., 0], f64(p)[..., 1]) for a, p in new]
            out = plx.decode_int4kv_weights(q, r, *caches, sl, w)
        else:
            for b in range(B):
                caches[0][b, :, n[b] - 1], caches[1][b, :, n[b] - 1] = k[b], v[b]
            new = [f64(k), f64(v)]
            out = plx.decode_weights(q, r, *caches, sl, w)
        for b in range(B):
            K[b, :, n[b] - 1], V[b, :, n[b] - 1] = new[0][b], new[1][b]
        check_out(out, f64(q), f64(r), K, V, n)
        _, total = oracle.decode_weights_ref(f64(q), f64(r), K, V, n, w64)
        p_sum += total - w64
        w64 = total
        assert (np.abs(f64(w) - w64) <= 12 * 2.0 ** -24 * np.abs(w64) + 2.0 ** -15 * p_sum).all()
        before_w = f64(w).copy()
