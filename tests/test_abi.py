"""C ABI of libplx.so on the CPU: it loads, exports what include/*.h declares,
and rejects bad arguments on the host before any CUDA call."""
import ctypes
import os
import re

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PKG = os.path.join(ROOT, "local_linear_attention_streamed_b200")


def _declared(header):
    text = open(os.path.join(ROOT, "include", header)).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    return sorted(set(re.findall(r"\b(plx_\w+)\s*\(", text)))


@pytest.fixture(scope="module")
def lib():
    from local_linear_attention_streamed_b200 import plx
    return plx.lib


@pytest.mark.parametrize("header,so", [("plx.h", "libplx.so"), ("plx_synth.h", "libplx_synth.so")])
def test_exports_every_declared_symbol(header, so):
    names = _declared(header)
    assert names, header
    dll = ctypes.CDLL(os.path.join(PKG, so))
    missing = [n for n in names if not hasattr(dll, n)]
    assert not missing, f"{so} lacks {missing}"


def test_binding_covers_header(lib):
    from local_linear_attention_streamed_b200 import plx
    assert set(_declared("plx.h")) == set(plx.SIGNATURES)


def test_version_and_status_strings(lib):
    assert lib.plx_abi_version() == 1
    for code in (0, -1, -2, -3, -4, -5, -6, -7):
        s = lib.plx_status_string(code).decode()
        assert s and s != "unknown status code"
    assert lib.plx_status_string(-99).decode() == "unknown status code"


A = 0x10000  # aligned fake device addresses: validation fails before they are used


def test_prefill_rejects_bad_arguments(lib):
    ok = [A, A, A, A, A]
    assert lib.plx_prefill_ex(None, A, A, A, A, 1, 1, 8, 64, 1, 1, None) == -1
    assert lib.plx_prefill_ex(*ok, 0, 1, 8, 64, 1, 1, None) == -1
    assert lib.plx_prefill_ex(*ok, 1, 1, 0, 64, 1, 1, None) == -1
    assert lib.plx_prefill_ex(*ok, 1, 1, 8, 64, 1, 7, None) == -1
    assert lib.plx_prefill_ex(*ok, 1, 1, 8, 96, 1, 1, None) == -2   # bf16 needs d in {64, 128}
    assert lib.plx_prefill_ex(*ok, 1, 1, 8, 160, 1, 0, None) == -2  # f32 needs d <= 128
    assert lib.plx_prefill_ex(*ok, 1, 1, 8, 48, 1, 0, None) == -2   # f32 needs d % 32 == 0
    assert lib.plx_prefill_ex(A, A + 2, A, A, A, 1, 1, 8, 64, 1, 1, None) == -3


def test_decode_rejects_bad_arguments(lib):
    ok = [A] * 6
    assert lib.plx_decode_ex(A, A, A, A, None, A, 1, 1, 8, 128, 1, None, 0, None) == -1
    assert lib.plx_decode_ex(*ok, 1, 0, 8, 128, 1, None, 0, None) == -1
    assert lib.plx_decode_ex(*ok, 1, 1, 8, 32, 1, None, 0, None) == -2
    assert lib.plx_decode_ex(A, A, A, A + 8, A, A, 1, 1, 8, 128, 1, None, 0, None) == -3
    assert lib.plx_decode_ex(A, A, A, A, A + 2, A, 1, 1, 8, 128, 1, None, 0, None) == -3


def test_decode_size_bounds_are_shared(lib):
    """Every decode entry point rejects the same oversized problems on the host:
    more than 2^24 query (b, h) pairs, or cache rows (B * KV heads * L) that
    reach 2^31 once a 128-key block is added."""
    ok = [A] * 6
    big_bh = (1 << 24) // 16 + 1
    assert lib.plx_decode_ex(*ok, big_bh, 16, 8, 128, 1, None, 0, None) == -2
    assert lib.plx_decode_noalloc(*ok, big_bh, 16, 8, 128, None) == -2
    rows_L = ((1 << 31) - 128) // 64       # B * Hkv = 64: B*Hkv*L + 128 just reaches 2^31
    assert lib.plx_decode_ex(*ok, 4, 16, rows_L, 128, 1, None, 0, None) == -2
    assert lib.plx_decode_noalloc(*ok, 4, 16, rows_L, 128, None) == -2
    assert lib.plx_decode_gqa(*ok, 4, 64, 16, rows_L, 128, None, 0, None) == -2
    assert lib.plx_decode_window(*ok, 4, 64, 16, rows_L, 128, 1024, 1, None, 0, None) == -2


def test_decode_gqa_rejects_bad_arguments(lib):
    ok = [A] * 6
    assert lib.plx_decode_gqa(A, A, A, A, None, A, 1, 8, 2, 64, 128, None, 0, None) == -1
    assert lib.plx_decode_gqa(*ok, 1, 8, 3, 64, 128, None, 0, None) == -1   # H not a multiple of Hkv
    assert lib.plx_decode_gqa(*ok, 1, 6, 2, 64, 128, None, 0, None) == -2   # group of 3
    assert lib.plx_decode_gqa(*ok, 1, 32, 2, 64, 128, None, 0, None) == -2  # group of 16
    assert lib.plx_decode_gqa(*ok, 1, 8, 2, 64, 96, None, 0, None) == -2
    assert lib.plx_decode_gqa(A, A, A, A + 8, A, A, 1, 8, 2, 64, 128, None, 0, None) == -3
    assert lib.plx_decode_gqa_workspace_bytes(1, 8, 3, 64, 128) == 0
    # Two (b, KV head) pairs over 8192 keys: the split plan takes the most
    # chunks it allows (L / 256) for one or two CTAs per SM alike, so the
    # ungrouped plan of the same pairs gives the grouped decode's count.
    S = lib.plx_decode_num_splits(1, 2, 8192, 128)
    assert S > 1
    assert lib.plx_decode_gqa_workspace_bytes(1, 8, 2, 8192, 128) == 8 * S * (2 * 128 + 4) * 4
    assert lib.plx_decode_gqa_workspace_bytes(1, 16, 2, 8192, 128) > 0


def test_decode_kernel_choice(lib):
    """The ungrouped bf16 decode's size rule, as plx_decode_uses_tc reports it
    (1 = tensor-core kernel, 0 = warp-MMA kernel): at d = 128 long caches,
    or enough (b, h) with medium ones; at d = 64 head pairs for long caches
    over few heads only."""
    cells = {(64, 16, 4096, 128): 1, (1, 16, 32768, 128): 1, (8, 16, 4096, 128): 0,
             (64, 16, 1024, 128): 1, (256, 16, 16384, 128): 1, (2048, 16, 128, 128): 0,
             (16, 16, 2048, 128): 1, (8, 16, 2048, 128): 0, (256, 16, 1024, 128): 0,
             (1, 32, 32768, 64): 1, (64, 32, 4096, 64): 0, (1, 31, 32768, 64): 0, (4, 32, 16384, 64): 0}
    for (B, H, L, d), want in cells.items():
        assert lib.plx_decode_uses_tc(B, H, L, d) == want, (B, H, L, d)
    assert lib.plx_decode_uses_tc(1, 16, 4096, 96) == -1


def test_fp8_cache_calls_reject_bad_arguments(lib):
    # plx_kv_quantize_fp8(X, codes, scales, rows, d, stream)
    assert lib.plx_kv_quantize_fp8(None, A, A, 4, 128, None) == -1
    assert lib.plx_kv_quantize_fp8(A, A, A, 0, 128, None) == -1
    assert lib.plx_kv_quantize_fp8(A, A, A, 4, 96, None) == -2
    assert lib.plx_kv_quantize_fp8(A + 8, A, A, 4, 128, None) == -3
    assert lib.plx_kv_quantize_fp8(A, A, A + 2, 4, 128, None) == -3      # scales need 4 bytes
    # plx_decode_fp8kv(q, r, Kc, Ks, Vc, Vs, seqlens, out, B, H, Hkv, L, d, ws, ws_bytes, stream)
    ok = [A] * 8
    assert lib.plx_decode_fp8kv(A, A, A, None, A, A, A, A, 1, 8, 2, 64, 128, None, 0, None) == -1
    assert lib.plx_decode_fp8kv(*ok, 1, 8, 3, 64, 128, None, 0, None) == -1   # H not a multiple of Hkv
    assert lib.plx_decode_fp8kv(*ok, 1, 6, 2, 64, 128, None, 0, None) == -2   # group of 3
    assert lib.plx_decode_fp8kv(*ok, 1, 32, 2, 64, 128, None, 0, None) == -2  # group of 16
    assert lib.plx_decode_fp8kv(*ok, 1, 8, 2, 64, 64, None, 0, None) == -2    # d = 128 only
    assert lib.plx_decode_fp8kv(A + 4, A, A, A, A, A, A, A, 1, 8, 2, 64, 128, None, 0, None) == -3
    assert lib.plx_decode_fp8kv(A, A, A, A + 4, A, A, A, A, 1, 8, 2, 64, 128, None, 0, None) == -3  # scales 16 B
    assert lib.plx_decode_fp8kv(A, A, A, A, A, A, A + 2, A, 1, 8, 2, 64, 128, None, 0, None) == -3  # seqlens 4 B
    assert lib.plx_decode_fp8kv(*ok, 1 << 22, 8, 8, 64, 128, None, 0, None) == -2  # B*H above 2^24
    assert lib.plx_decode_fp8kv_workspace_bytes(1, 8, 3, 64, 128) == 0
    S = lib.plx_decode_num_splits(1, 2, 8192, 128)
    assert S > 1 and lib.plx_decode_fp8kv_workspace_bytes(1, 8, 2, 8192, 128) == 8 * S * (2 * 128 + 4) * 4


def test_dilated_prefill_rejects_bad_arguments(lib):
    # plx_prefill_dilated(Q, K, V, R, out, B, H, Hkv, N, d, dilation, window, stream)
    ok = [A] * 5
    assert lib.plx_prefill_dilated(None, A, A, A, A, 1, 4, 2, 256, 128, 2, 0, None) == -1
    assert lib.plx_prefill_dilated(*ok, 1, 4, 2, 256, 128, 0, 0, None) == -1      # dilation >= 1
    assert lib.plx_prefill_dilated(*ok, 1, 4, 2, 256, 128, 2, -1, None) == -1     # window >= 0
    assert lib.plx_prefill_dilated(*ok, 1, 4, 3, 256, 128, 2, 0, None) == -1      # H not a multiple of Hkv
    assert lib.plx_prefill_dilated(*ok, 1, 4, 2, 300, 128, 7, 0, None) == -2      # ragged classes
    assert lib.plx_prefill_dilated(*ok, 1, 4, 2, 256, 96, 2, 0, None) == -2
    assert lib.plx_prefill_dilated(A, A, A + 8, A, A, 1, 4, 2, 256, 128, 2, 0, None) == -3
    assert lib.plx_prefill_dilated(*ok, 1 << 20, 16, 16, 256, 128, 2, 0, None) == -2  # B*H*r above 2^24


def test_layer_and_norm_rope_reject_bad_arguments(lib):
    assert lib.plx_qkr_norm_rope(None, A, 1, 8, 2, 128, 1e-6, 1e4, None) == -1
    assert lib.plx_qkr_norm_rope(A, A, 1, 8, 2, 96, 1e-6, 1e4, None) == -2
    assert lib.plx_qkr_norm_rope(A, A, 1, 8, 2, 128, -1.0, 1e4, None) == -1
    assert lib.plx_layer_forward(*([A] * 6), None, 1, 8, 2, 128, None, 0, None) == -1
    assert lib.plx_layer_forward(*([A] * 7), 1, 8, 2, 32, None, 0, None) == -2
    assert lib.plx_layer_forward(*([A] * 6), A + 4, 1, 8, 2, 128, None, 0, None) == -3


def test_decode_split_plan(lib):
    # Sizes on both sides of the kernel choice (tensor-core decode: one CTA
    # per SM; warp-MMA decode: two), whose split plans differ.
    for (B, H, L) in [(64, 16, 4096), (1, 16, 32768), (2048, 16, 4096), (1, 1, 1), (3, 5, 1000),
                      (1, 16, 128), (8, 16, 16384), (64, 16, 1024), (256, 16, 1024), (16, 16, 2048),
                      (8, 16, 2048), (1, 16, 16384), (3, 7, 20000)]:
        S = lib.plx_decode_num_splits(B, H, L, 128)
        assert 1 <= S <= max(1, L // 256) + 1
        ws = lib.plx_decode_workspace_bytes(B, H, L, 128)
        if S == 1:
            assert ws == 0
        else:
            assert ws == B * H * S * (2 * 128 + 4) * 4
    # Small batches split the context; large ones do not need to.
    assert lib.plx_decode_num_splits(1, 16, 32768, 128) > 8
    assert lib.plx_decode_num_splits(2048, 16, 4096, 128) == 1


def test_layer_workspace_slots_match_the_binding():
    """The caller workspace of plx_layer_forward holds nine 256-byte-aligned
    slots; the binding's views of the layer's own attention inputs and output
    are slots 4..8, [B, H, N, d] bf16 each."""
    import torch
    from local_linear_attention_streamed_b200 import plx
    for (B, N, H, d) in [(1, 1, 1, 64), (2, 100, 3, 64), (4, 8192, 16, 128), (3, 7, 5, 128)]:
        slot = -(-(B * N * H * d * 2) // 256) * 256
        assert plx.layer_workspace_bytes(B, N, H, d) == 9 * slot
        if B * N * H * d > 1 << 20:
            continue
        ws = torch.zeros(9 * slot, dtype=torch.uint8)
        views = plx.layer_workspace_views(ws, B, N, H, d)
        base = ws.data_ptr()
        for i, name in enumerate(("q", "k", "v", "rho", "attn")):
            t = views[name]
            assert t.dtype == torch.bfloat16 and tuple(t.shape) == (B, H, N, d)
            assert t.data_ptr() - base == (4 + i) * slot


def test_int4_cache_calls_reject_bad_arguments(lib):
    # plx_kv_quantize_int4(X, codes, params, rows, d, stream)
    for call in (lib.plx_kv_quantize_int4, lib.plx_kv_dequantize_int4):
        assert call(None, A, A, 4, 128, None) == -1
        assert call(A, A, A, 0, 128, None) == -1
        assert call(A, A, A, 4, 96, None) == -2
        assert call(A + 8, A, A, 4, 128, None) == -3
    assert lib.plx_kv_quantize_int4(A, A, A + 2, 4, 128, None) == -3
    # plx_kv_append_int4(k, v, Kc, Kp, Vc, Vp, seqlens, k_out, v_out, B, Hkv, L, d, stream)
    ok = [A] * 9
    assert lib.plx_kv_append_int4(A, A, A, A, A, None, A, None, None, 1, 2, 8, 128, None) == -1
    assert lib.plx_kv_append_int4(*ok, 1, 0, 8, 128, None) == -1
    assert lib.plx_kv_append_int4(*ok, 1, 2, 8, 32, None) == -2
    assert lib.plx_kv_append_int4(A, A, A, A, A, A, A, A + 8, None, 1, 2, 8, 128, None) == -3
    assert lib.plx_kv_append_int4(*ok, 1 << 20, 16, 200, 128, None) == -2


def test_cache_decodes_reject_bad_arguments(lib):
    # plx_decode_int4kv(q, r, Kc, Kp, Vc, Vp, seqlens, out, B, H, Hkv, L, d, ws, ws_bytes, stream)
    tail = (None, 0, None)
    ok8, ok10 = [A] * 8, [A] * 9 + [A]
    B5 = 0x500000  # a second array apart from the first
    w10 = [A] * 7 + [A, B5, A]    # ... seqlens, weights, weights_out, out
    w8 = [A] * 5 + [A, B5, A]
    for call, ok in ((lib.plx_decode_int4kv, ok8), (lib.plx_decode_int4kv_weights, w10), (lib.plx_decode_weights, w8)):
        for i in range(len(ok)):
            assert call(*ok[:i], None, *ok[i + 1:], 1, 8, 2, 64, 128, *tail) == -1
        assert call(*ok, 1, 8, 3, 64, 128, *tail) == -1    # H not a multiple of Hkv
        assert call(*ok, 0, 8, 2, 64, 128, *tail) == -1
        assert call(*ok, 1, 6, 2, 64, 128, *tail) == -2    # group of 3
        assert call(*ok, 1, 32, 2, 64, 128, *tail) == -2   # group of 16
        assert call(*ok, 1, 8, 2, 64, 96, *tail) == -2
        assert call(*ok, 1 << 22, 8, 8, 64, 128, *tail) == -2
        assert call(*ok, 4, 64, 16, ((1 << 31) - 128) // 64, 128, *tail) == -2
        assert call(A + 8, *ok[1:], 1, 8, 2, 64, 128, *tail) == -3
    assert lib.plx_decode_int4kv(A, A, A, A + 2, A, A, A, A, 1, 8, 2, 64, 128, *tail) == -3   # params 4 B
    # weights and weights_out overlap without being the same
    assert lib.plx_decode_weights(*[A] * 6, A + 64, A, 1, 8, 2, 64, 128, *tail) == -1
    assert lib.plx_decode_int4kv_workspace_bytes(1, 8, 3, 64, 128) == 0
    assert lib.plx_decode_weights_workspace_bytes(1, 8, 2, 64, 128) >= 8 * 64 * 4
    assert lib.plx_decode_int4kv_workspace_bytes(1, 8, 2, 1000, 128) == 0
    assert lib.plx_decode_int4kv_workspace_bytes(1, 1, 1, 1 << 20, 128) > 0


def test_cache_evict_rejects_bad_arguments(lib):
    """Checked on the host: sizes, the rule's numbers, overlaps of caches, totals and outputs."""
    vp, it = ctypes.c_void_p, ctypes.c_int

    def call(src=(A,), dst=(0x900000,), row=(256,), w=0x2000000, wo=0x3000000, B=1, Hkv=2, L=64, Lout=16, budget=16,
             sinks=1, recent=2, count=None, sl=A, kept=A):
        n = len(src)
        return lib.plx_cache_evict(n if count is None else count, (vp * max(n, 1))(*src), (vp * max(n, 1))(*dst),
                                   (it * max(n, 1))(*row), w, wo, sl, sl, kept, B, Hkv, L, Lout, budget, sinks,
                                   recent, None)

    for kw in (dict(w=None), dict(wo=None), dict(sl=None), dict(kept=None), dict(count=-1), dict(B=0), dict(L=0),
               dict(budget=0), dict(sinks=-1), dict(recent=-1), dict(sinks=10, recent=7), dict(Lout=15),
               dict(row=(0,)), dict(src=(None,)), dict(dst=(None,)),
               dict(sinks=2 ** 31 - 1, recent=2 ** 31 - 1),
               dict(dst=(A,)),                                   # in place needs L_out = L
               dict(dst=(A + 256,)), dict(wo=0x2000000 + 4),     # partly over itself
               dict(src=(A, A), dst=(A, A), row=(4, 4), Lout=64),  # one buffer twice
               dict(src=(A, 0x700000), dst=(0x900000, 0x900010), row=(256, 256)),
               dict(dst=(0x2000000,))):                          # over the totals
        assert call(**kw) == -1, kw
    assert call(row=(65537,), dst=(0x90000000,)) == -2
    assert call(src=[A * 16 * i for i in range(1, 10)], dst=[A * 4096 * i for i in range(1, 10)], row=[4] * 9,
                w=0x200000000, wo=0x300000000) == -2
    assert call(B=1 << 20, Hkv=32, w=0x20000000000, wo=0x30000000000) == -2
    assert call(w=0x2000002) == -3


def test_cache_decode_size_queries_of_refused_sizes(lib):
    """0 for every size that the calls refuse, a head size beyond 2048 among them (in a process of its own: a query
    that divides by zero ends it)."""
    import subprocess
    import sys
    refused = [(1, 1, 1, 64, 96), (1, 1, 1, 64, 2048), (1, 1, 1, 64, 2049), (1, 1, 1, 64, 4096), (2, 4, 1, 7, 1 << 24),
               (1, 3, 1, 64, 128), (1, 16, 1, 64, 128), (1, 64, 1, 64, 64), (1 << 20, 32, 32, 64, 128),
               (4, 64, 16, ((1 << 31) - 128) // 64, 128), ((1 << 31) - 1,) * 5, (1, 8, 0, 64, 128), (1, 8, 2, 0, 128)]
    code = f"""
import ctypes
lib = ctypes.CDLL({os.path.join(PKG, 'libplx.so')!r})
for name in ("plx_decode_int4kv_workspace_bytes", "plx_decode_weights_workspace_bytes"):
    query = getattr(lib, name)
    query.restype, query.argtypes = ctypes.c_size_t, [ctypes.c_int] * 5
    for sizes in {refused!r}:
        assert query(*sizes) == 0, (name, sizes)
    assert query(1, 8, 2, 1 << 20, 128) > 0 and query(1, 1, 1, 1 << 20, 64) > 0
"""
    done = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=120)
    assert done.returncode == 0, (done.returncode, done.stderr[-2000:])


def test_cache_evict_rejects_overlaps_of_positions_and_lengths(lib):
    """kept and seqlens_out are outputs too: apart from every cache, the totals, the lengths and each other."""
    vp, it = ctypes.c_void_p, ctypes.c_int
    B, Hkv, L, Lout, budget = 2, 2, 64, 16, 16
    src, dst, w, wo = 0x1000000, 0x2000000, 0x3000000, 0x4000000      # 256-byte rows: 0x10000 and 0x4000 bytes
    sl, slo, kept = 0x5000000, 0x6000000, 0x7000000                    # 8, 8 and 256 bytes

    def call(**kw):
        a = dict(src=src, dst=dst, w=w, wo=wo, sl=sl, slo=slo, kept=kept)
        a.update(kw)
        return lib.plx_cache_evict(1, (vp * 1)(a["src"]), (vp * 1)(a["dst"]), (it * 1)(256), a["w"], a["wo"], a["sl"],
                                   a["slo"], a["kept"], B, Hkv, L, Lout, budget, 1, 2, None)

    spans = dict(src=(src, 0x10000), dst=(dst, 0x4000), w=(w, B * Hkv * L * 4), wo=(wo, B * Hkv * Lout * 4),
                 sl=(sl, 8), slo=(slo, 8), kept=(kept, 256))
    for out in ("kept", "slo"):
        for name, (at, size) in spans.items():
            if name == out:
                continue
            for x in (at, at + size - 4, at - spans[out][1] + 4):
                if out == "slo" and name == "sl" and x == at:
                    continue  # new lengths over the old ones are allowed
                assert call(**{out: x}) == -1, (out, name, hex(x))
    for name in ("dst", "wo"):  # rows and totals written over the lengths that are read meanwhile
        at, size = spans[name]
        for x in (at, at + size - 4, at - 4):
            assert call(sl=x) == -1, (name, hex(x))
    assert call(sl=src + 64, slo=src + 64) == -1  # new lengths over the old ones, inside of a cache
    assert call(sl=w, slo=w) == -1


def test_cache_calls_refuse_lengths_next_to_2_31(lib):
    """The kernels count rows in 32 bits, a block's turn past the last one."""
    vp, it = ctypes.c_void_p, ctypes.c_int
    most = (1 << 31) - 4096
    far = [1 << 44, 2 << 44, 3 << 44, 4 << 44, 5 << 44, 6 << 44]
    for L in (most + 1, (1 << 31) - 2047, (1 << 31) - 129):
        for Lout in (16, L):
            assert lib.plx_cache_evict(0, (vp * 1)(), (vp * 1)(), (it * 1)(), far[0], far[1], far[2], far[3], far[4],
                                       1, 1, L, Lout, 16, 1, 2, None) == -2
        assert lib.plx_cache_evict(0, (vp * 1)(), (vp * 1)(), (it * 1)(), far[0], far[1], far[2], far[3], far[4],
                                   1, 1, 64, L, 16, 1, 2, None) == -2
        tail = (1, 1, 1, L, 64, None, 0, None)
        assert lib.plx_decode_weights(*far[:4], far[4], A, A + (1 << 40), far[5], *tail) == -2
        assert lib.plx_decode_int4kv_weights(*far, A, A, A + (1 << 40), A, *tail) == -2
        assert lib.plx_decode_int4kv(*far, A, A, *tail) == -2
        assert lib.plx_decode_weights_workspace_bytes(1, 1, 1, L, 64) == 0
    assert lib.plx_decode_weights_workspace_bytes(1, 1, 1, most, 64) > 4 * most
