"""The serving operators over a compressed KV cache: their plain forms and the calls a user makes.

Four operators, in the order a serving loop meets them:

* write: rows of bf16 keys or values become 4-bit codes with one (scale, zero
  point) pair for each row, and are read back as the bf16 values they stand for;
* step: the new token's key and value rows are appended to a 4-bit cache (and
  given back as the values they now stand for), and the token's query attends
  over the cache (one decode step);
* weigh: one decode step that also adds every key's softmax weight, summed over
  the query heads that share the key's head, to a running total;
* evict: the rows with the largest totals move to a smaller cache, in the order
  of their positions, the first and the last few rows always among them.

``own`` False runs the operators in elementary torch operations; True makes the
framework's calls on the same inputs.
"""
import math

import torch

own = False

# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------


def listed():
    return [
        # A prompt of the prefill workload, its keys of all layers' heads written once into a 4-bit cache.
        dict(name="write_prompt", op="write", B=8, Hkv=16, L=4096, d=128),
        # A short prompt with odd sizes and narrow heads.
        dict(name="write_odd", op="write", B=3, Hkv=5, L=1001, d=64),
        # One user waiting for the next token: the smallest call, where latency counts.
        dict(name="step_one_user", op="step", B=1, Hkv=2, G=4, L=1000, d=128, ragged=False),
        # The decode workload: a full batch with one key head for each query head.
        dict(name="step_batch", op="step", B=64, Hkv=16, G=1, L=4096, d=128, ragged=False),
        # The grouped decode workload, sequences of different lengths.
        dict(name="step_grouped_ragged", op="step", B=64, Hkv=8, G=4, L=4096, d=128, ragged=True),
        # Long documents with narrow heads, eight query heads to a key head.
        dict(name="step_long_narrow", op="step", B=4, Hkv=8, G=8, L=16384, d=64, ragged=True),
        # The grouped decode workload over a bf16 cache that will be thinned out.
        dict(name="weigh_bf16_grouped", op="weigh", cache="bf16", B=64, Hkv=8, G=4, L=4096, d=128, ragged=True),
        # A small batch with odd sizes and narrow heads.
        dict(name="weigh_bf16_odd", op="weigh", cache="bf16", B=3, Hkv=5, G=2, L=777, d=64, ragged=True),
        # One long document in a 4-bit cache.
        dict(name="weigh_4bit_long", op="weigh", cache="4bit", B=1, Hkv=16, G=1, L=32768, d=128, ragged=False),
        # A full batch cut to a quarter of its bf16 cache.
        dict(name="evict_bf16_batch", op="evict", cache="bf16", B=64, Hkv=8, L=4096, d=128, budget=1024, sinks=4,
             recent=128, ragged=False),
        # One long document in a 4-bit cache cut to an eighth.
        dict(name="evict_4bit_long", op="evict", cache="4bit", B=1, Hkv=16, L=32768, d=128, budget=4096, sinks=4,
             recent=512, ragged=False),
        # A small batch with odd sizes; some sequences are within the budget already.
        dict(name="evict_bf16_odd", op="evict", cache="bf16", B=3, Hkv=5, L=1001, d=64, budget=333, sinks=1,
             recent=32, ragged=True),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["write", "step", "step", "weigh", "weigh", "evict"])
    d = rng.choice([64, 128])
    Hkv = rng.choice([1, 2, 3, 5, 8, 16])
    B = _log_int(rng, 1, 64)
    L = _log_int(rng, 1 if op in ("step", "weigh") else 16, 32768)
    most = {"write": 1 << 19, "step": 1 << 22, "weigh": 1 << 21, "evict": 1 << 21}[op]  # cache rows, as the listed cases
    while B * Hkv * L > most:
        if B > 1:
            B = (B + 1) // 2
        elif Hkv > 1:
            Hkv = (Hkv + 1) // 2
        else:
            L = most
    if op == "write":
        return dict(op=op, B=B, Hkv=Hkv, L=L, d=d)
    if op == "step":
        return dict(op=op, B=B, Hkv=Hkv, G=rng.choice([1, 2, 4, 8]), L=L, d=d, ragged=rng.random() < 0.7)
    if op == "weigh":
        return dict(op=op, cache=rng.choice(["bf16", "4bit"]), B=B, Hkv=Hkv, G=rng.choice([1, 2, 4, 8]), L=L, d=d,
                    ragged=rng.random() < 0.7)
    budget = max(1, int(L * rng.uniform(0.05, 0.9)))
    sinks = rng.choice([0, 1, 4]) if budget > 16 else 0
    recent = int((budget - sinks) * rng.choice([0.0, 0.125, 0.5]))
    return dict(op=op, cache=rng.choice(["bf16", "4bit"]), B=B, Hkv=Hkv, L=L, d=d, budget=budget, sinks=sinks,
                recent=recent, ragged=rng.random() < 0.7)


def work(case):
    B, Hkv, L, d = case["B"], case["Hkv"], case["L"], case["d"]
    rows = B * Hkv * L
    # Ragged lengths are uniform between half the capacity and all of it.
    seen = rows * (0.75 if case.get("ragged") else 1.0)
    row4, row16 = d // 2 + 4, 2 * d
    if case["op"] == "write":  # bf16 in, codes out; codes in, bf16 out
        return {"bytes": rows * 2 * (row16 + row4), "flops": rows * d * 4}
    H = Hkv * case.get("G", 1)
    heads = 3 * B * H * d * 2  # q, rho, out
    flops = 8.0 * d * seen * case.get("G", 1)
    if case["op"] == "step":
        return {"bytes": seen * 2 * row4 + heads + B * Hkv * 2 * (2 * row16 + row4), "flops": flops}
    row = row4 if case["cache"] == "4bit" else row16
    if case["op"] == "weigh":  # the totals are read and written
        return {"bytes": seen * (2 * row + 8) + heads, "flops": flops}
    kept = B * Hkv * min(case["budget"], L)
    back = 2 * (row4 + row16) if case["cache"] == "4bit" else 0  # 4-bit rows are read back as values
    return {"bytes": seen * 4 + kept * (4 * row + 8 + back), "flops": seen}


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------


def _round_up_bf16(x64):
    """The smallest bf16 at or above a non-negative float64 value."""
    c = x64.to(torch.bfloat16)
    return torch.where(c.double() < x64, (c.view(torch.int16) + 1).view(torch.bfloat16), c)


def _quantise(X):
    """4-bit codes (two to a byte, the even element in the low half) and (scale, zero point) rows of X [..., d]."""
    lo = X.amin(-1).double().clamp(max=0)
    hi = X.amax(-1).double().clamp(min=0)
    s = _round_up_bf16((hi - lo) / 15)
    safe = torch.where(s > 0, s, torch.ones_like(s)).float()
    zero = torch.round(-lo.float() / safe)
    c = (torch.round(X.float() / safe[..., None]) + zero[..., None]).clamp(0, 15).to(torch.uint8)
    return c[..., 0::2] | (c[..., 1::2] << 4), torch.stack((s, zero.to(torch.bfloat16)), -1)


def _values(codes, params):
    """The fp32 values that 4-bit rows stand for."""
    c = torch.stack((codes & 15, codes >> 4), -1).flatten(-2).float()
    p = params.float()
    return (c - p[..., 1:]) * p[..., :1]


def _rms_rows(g, shape):
    x = torch.randn(shape, generator=g, device="cuda")
    return x / x.square().mean(-1, keepdim=True).sqrt()


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 7919 + 17)
    B, Hkv, L, d = case["B"], case["Hkv"], case["L"], case["d"]
    st = {"case": case}
    if case["op"] == "write":
        st["X"] = _rms_rows(g, (B, Hkv, L, d)).to(torch.bfloat16)
        return st
    lens = torch.full((B,), L, device="cuda")
    if case["ragged"]:
        lens = torch.randint((L + 1) // 2, L + 1, (B,), generator=g, device="cuda")
    st["seqlens"] = lens.to(torch.int32)
    # Keys are RMS-normalised rows and values are normal, as a layer makes them.
    K = _rms_rows(g, (B, Hkv, L, d)).to(torch.bfloat16)
    V = torch.randn((B, Hkv, L, d), generator=g, device="cuda").to(torch.bfloat16)
    if case["op"] == "evict":
        # Totals over many decode steps: a few heavy keys and a long tail.
        st["weights"] = torch.exp(2.0 * torch.randn((B, Hkv, L), generator=g, device="cuda"))
        keep = min(case["budget"], L)
        st["weights_to"] = torch.zeros((B, Hkv, keep), device="cuda")
    else:
        H = Hkv * case["G"]
        st["q"] = (1.5 * _rms_rows(g, (B, H, d))).to(torch.bfloat16)
        st["r"] = (0.25 * torch.randn((B, H, d), generator=g, device="cuda")).to(torch.bfloat16)
        st["out"] = torch.empty_like(st["q"])
    if case["op"] == "step":
        st["k"] = _rms_rows(g, (B, Hkv, d)).to(torch.bfloat16)
        st["v"] = torch.randn((B, Hkv, d), generator=g, device="cuda").to(torch.bfloat16)
        st["k_to"], st["v_to"] = torch.empty_like(st["k"]), torch.empty_like(st["v"])
    if case["op"] == "weigh":
        st["weights"] = torch.rand((B, Hkv, L), generator=g, device="cuda")
        st["weights_to"] = torch.zeros_like(st["weights"])
    if case["op"] == "step" or case["cache"] == "4bit":
        # Rows are written in slices: the 64-bit intermediates of a whole cache are large.
        parts = [[_quantise(x) for x in X.flatten(0, 1).split(max(1, (1 << 19) // L))] for X in (K, V)]
        st["cache"] = tuple(torch.cat([p[i] for p in part]).unflatten(0, (B, Hkv)) for part in parts for i in (0, 1))
    else:
        st["cache"] = (K, V)
    if case["op"] == "evict":
        st["cache_to"] = tuple(torch.zeros_like(t[:, :, :keep]) for t in st["cache"])
    return st


# ---------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------


def _attend(q, r, K, V, seqlens):
    """out and softmax weights [B, Hkv, G, L] of one decode step over fp32 keys and values."""
    B, H, d = q.shape
    Hkv, L = K.shape[1], K.shape[2]
    seen = torch.arange(L, device=q.device) < seqlens[:, None, None, None]
    q4, r4 = (x.float().view(B, Hkv, H // Hkv, d) for x in (q, r))
    s = torch.matmul(q4, K.transpose(2, 3)) / math.sqrt(d)
    s = torch.where(seen, s, torch.full_like(s, -math.inf))
    p = torch.exp(s - s.amax(-1, keepdim=True))
    p = p / p.sum(-1, keepdim=True)
    t = torch.where(seen, torch.matmul(r4, K.transpose(2, 3)), torch.zeros_like(s))
    tbar = (p * t).sum(-1, keepdim=True)
    out = torch.matmul(p * (1 - (t - tbar)), V)
    return out.view(B, H, d).to(q.dtype), p


def _run_plain(st):
    case = st["case"]
    op = case["op"]
    if op == "write":
        return _values(*_quantise(st["X"])).to(torch.bfloat16)
    seqlens = st["seqlens"]
    if op == "step":
        Kc, Kp, Vc, Vp = st["cache"]
        b, last = torch.arange(case["B"], device="cuda"), seqlens.long() - 1
        k, v = _quantise(st["k"]), _quantise(st["v"])
        (Kc[b, :, last], Kp[b, :, last]), (Vc[b, :, last], Vp[b, :, last]) = k, v
        out = _attend(st["q"], st["r"], _values(Kc, Kp), _values(Vc, Vp), seqlens)[0]
        return (out, *_shown(k + v))
    if op == "weigh":
        if case["cache"] == "4bit":
            Kc, Kp, Vc, Vp = st["cache"]
            K, V = _values(Kc, Kp), _values(Vc, Vp)
        else:
            K, V = (t.float() for t in st["cache"])
        out, p = _attend(st["q"], st["r"], K, V, seqlens)
        seen = torch.arange(case["L"], device="cuda") < seqlens[:, None, None]
        return out, torch.where(seen, st["weights"] + p.sum(2), st["weights_to"])
    # evict
    L, sinks, recent = case["L"], case["sinks"], case["recent"]
    keep = min(case["budget"], L)
    n = seqlens.long()[:, None, None]
    pos = torch.arange(L, device="cuda")
    must = (pos < sinks) | ((pos >= n - recent) & (pos < n))
    rank = torch.where(must, math.inf, torch.where(pos < n, st["weights"], -math.inf))
    order = torch.argsort(rank, dim=-1, descending=True, stable=True)[..., :keep]
    kept = torch.sort(torch.where(order < n, order, L), dim=-1).values
    real = kept < L
    at = kept.clamp(max=L - 1)
    moved = tuple(torch.where(real[..., None], torch.gather(t, 2, at[..., None].expand(*at.shape, t.shape[-1])), to)
                  for t, to in zip(st["cache"], st["cache_to"]))
    weights = torch.where(real, torch.gather(st["weights"], 2, at), 0.0)
    kept = torch.where(real, kept, -1).to(torch.int32)
    return kept, seqlens.clamp(max=case["budget"]), weights, _shown(moved)


def _shown(caches):
    """A cache as bf16 values: 4-bit rows read back as what they stand for."""
    if len(caches) == 2:
        return caches
    return _values(*caches[:2]).to(torch.bfloat16), _values(*caches[2:]).to(torch.bfloat16)


def _run_own(st):
    from local_linear_attention_streamed_b200 import plx
    case = st["case"]
    op = case["op"]
    if op == "write":
        return plx.kv_dequantize_int4(*plx.kv_quantize_int4(st["X"]))
    if op == "step":
        plx.kv_append_int4(st["k"], st["v"], *st["cache"], st["seqlens"], k_out=st["k_to"], v_out=st["v_to"])
        out = plx.decode_int4kv(st["q"], st["r"], *st["cache"], st["seqlens"], out=st["out"])
        return out, st["k_to"], st["v_to"]
    if op == "weigh":
        call = plx.decode_int4kv_weights if case["cache"] == "4bit" else plx.decode_weights
        out = call(st["q"], st["r"], *st["cache"], st["seqlens"], st["weights"], weights_out=st["weights_to"],
                   out=st["out"])
        return out, st["weights_to"]
    kept, lens = plx.cache_evict(st["cache"], st["weights"], st["seqlens"], case["budget"], sinks=case["sinks"],
                                 recent=case["recent"], caches_out=st["cache_to"], weights_out=st["weights_to"])
    to = st["cache_to"]
    if len(to) == 4:
        to = (plx.kv_dequantize_int4(*to[:2]), plx.kv_dequantize_int4(*to[2:]))
    return kept, lens, st["weights_to"], to


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ---------------------------------------------------------------------------
# The same outputs in 64 bits, from the definitions
# ---------------------------------------------------------------------------


def _exact_rows(X):
    """float64 values and (scale, zero point) of rows X [n, d] held in 4 bits: the scale is the smallest bf16 that
    spans the row (zero included) in 15 steps, the zero point and the codes are the nearest integers, ties to even."""
    x = X.double()
    top = torch.maximum(x.max(-1).values, torch.zeros((), dtype=x.dtype, device=x.device))
    low = torch.minimum(x.min(-1).values, torch.zeros((), dtype=x.dtype, device=x.device))
    step = (top - low) / 15
    s32 = step.float()
    s32 = torch.where(s32.double() < step, torch.nextafter(s32, torch.full_like(s32, math.inf)), s32)
    bits = (s32.view(torch.int32) + 0xFFFF) & ~0xFFFF
    s = bits.view(torch.float32).double()
    unit = torch.where(s == 0, torch.ones_like(s), s)
    zero = (-low / unit).round()
    code = ((x / unit[:, None]).round() + zero[:, None]).clamp(0, 15)
    return s[:, None] * (code - zero[:, None])


def _exact_cache(codes, params, n):
    """float64 values [n, d] of the first n rows of one head's 4-bit cache."""
    c = codes[:n].long()
    c = torch.stack((c % 16, c // 16), -1).reshape(n, -1).double()
    return params[:n, 0, None].double() * (c - params[:n, 1, None].double())


def _exact_step(q, r, K, V):
    """One query group [G, d] over one head's visible keys [n, d]: softmax attention minus the covariance of values
    and keys applied to the probe; and the softmax weights [G, n]."""
    q, r = q.double(), r.double()
    p = torch.softmax(q @ K.T / math.sqrt(K.shape[1]), -1)
    vbar, kbar = p @ V, p @ K
    probe = r @ K.T - (r * kbar).sum(-1, keepdim=True)
    pp = p * probe
    return vbar - (pp @ V - pp.sum(-1, keepdim=True) * vbar), p


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "write":
        return _exact_rows(st["X"].flatten(0, 2)).view(st["X"].shape)
    B, Hkv, L = case["B"], case["Hkv"], case["L"]
    lens = st["seqlens"].tolist()
    if op in ("step", "weigh"):
        G, d = case["G"], case["d"]
        out = torch.empty((B, Hkv, G, d), dtype=torch.float64, device="cuda")
        total = st["weights_to"].double() if op == "weigh" else None
        if op == "step":
            k, v = (_exact_rows(st[x].flatten(0, 1)).view(B, Hkv, d) for x in ("k", "v"))
        q, r = st["q"].view(B, Hkv, G, d), st["r"].view(B, Hkv, G, d)
        for b in range(B):
            n = lens[b]
            for h in range(Hkv):
                if len(st["cache"]) == 4:
                    Kc, Kp, Vc, Vp = (t[b, h] for t in st["cache"])
                    K, V = _exact_cache(Kc, Kp, n), _exact_cache(Vc, Vp, n)
                else:
                    K, V = (t[b, h, :n].double() for t in st["cache"])
                if op == "step":
                    K[n - 1], V[n - 1] = k[b, h], v[b, h]
                out[b, h], p = _exact_step(q[b, h], r[b, h], K, V)
                if op == "weigh":
                    total[b, h, :n] = st["weights"][b, h, :n].double() + p.sum(0)
        out = out.view(B, Hkv * G, d)
        return (out, total) if op == "weigh" else (out, k, v)
    # evict: whole numbers, moved totals, and moved rows as the values they stand for
    budget, sinks, recent = case["budget"], case["sinks"], case["recent"]
    room = min(budget, L)
    kept = torch.full((B, Hkv, room), -1, dtype=torch.int32)
    weights = torch.zeros((B, Hkv, room), dtype=torch.float64, device="cuda")
    K = torch.zeros((B, Hkv, room, case["d"]), dtype=torch.float64, device="cuda")
    V = torch.zeros_like(K)
    totals = st["weights"].cpu()
    for b in range(B):
        n = lens[b]
        for h in range(Hkv):
            ids = torch.arange(n)
            if n > budget:
                middle = torch.arange(sinks, n - recent)
                best = torch.sort(-totals[b, h, sinks:n - recent], stable=True).indices[:budget - sinks - recent]
                ids = torch.cat((torch.arange(sinks), middle[best].sort().values, torch.arange(n - recent, n)))
            m = len(ids)
            kept[b, h, :m] = ids.to(torch.int32)
            at = ids.cuda()
            weights[b, h, :m] = st["weights"][b, h, at].double()
            if len(st["cache"]) == 4:
                Kc, Kp, Vc, Vp = (t[b, h, at] for t in st["cache"])
                K[b, h, :m], V[b, h, :m] = _exact_cache(Kc, Kp, m), _exact_cache(Vc, Vp, m)
            else:
                K[b, h, :m], V[b, h, :m] = (t[b, h, at].double() for t in st["cache"])
    new = torch.tensor([min(n, budget) for n in lens], dtype=torch.int32)
    return kept.cuda(), new.cuda(), weights, (K, V)
