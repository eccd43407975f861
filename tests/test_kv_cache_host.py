"""Host-side checks of the paged 8-bit key/value cache: refusals of the C ABI
and of the binding (no GPU, no compute calls), and pins of the numpy reference
the GPU tests compare with."""

import ctypes
import math

import numpy as np
import pytest
import torch

import int8_quantized_matmul_absmax_amd as i8
from int8_quantized_matmul_absmax_amd import _lib
from oracle import kv_cache as R

A = 0x10000       # aligned, never dereferenced
MIS = 0x10008     # not 16-byte aligned
ODD = 0x10002     # not 4-byte aligned


@pytest.fixture(scope="module")
def lib():
    return i8.ensure_built()


def cache(**kw):
    f = dict(k_codes=A, k_absmax=A, v_codes=A, v_absmax=A, num_pages=8, page_tokens=64, kv_heads=2,
             head_dim=64)
    f.update(kw)
    return ctypes.byref(_lib.KVCacheStruct(**f))


def batch(**kw):
    f = dict(page_table=A, seq_lens=A, cu_tokens=A, num_seqs=2, max_pages=4, total_tokens=6,
             max_tokens=4, max_len=256)
    f.update(kw)
    return ctypes.byref(_lib.KVBatchStruct(**f))


def rotary(**kw):
    f = dict(cos=A, sin=A, dim=64, positions=256, interleaved=0)
    f.update(kw)
    return ctypes.byref(_lib.RotaryStruct(**f))


BAD_SIZES = [
    (dict(num_pages=-1), {}, _lib.I8MM_EINVAL),
    (dict(page_tokens=0), {}, _lib.I8MM_EINVAL),
    (dict(page_tokens=24), {}, _lib.I8MM_EALIGN),
    (dict(page_tokens=1 << 20), {}, _lib.I8MM_EINVAL),
    (dict(kv_heads=0), {}, _lib.I8MM_EINVAL),
    (dict(kv_heads=70000), {}, _lib.I8MM_EINVAL),
    (dict(head_dim=72), {}, _lib.I8MM_EINVAL),
    (dict(num_pages=1 << 30), {}, _lib.I8MM_EINVAL),
    ({}, dict(num_seqs=-1), _lib.I8MM_EINVAL),
    ({}, dict(num_seqs=70000), _lib.I8MM_EINVAL),
    ({}, dict(max_pages=-1), _lib.I8MM_EINVAL),
    ({}, dict(total_tokens=-1), _lib.I8MM_EINVAL),
    ({}, dict(total_tokens=1 << 32), _lib.I8MM_EINVAL),
    ({}, dict(max_tokens=-1), _lib.I8MM_EINVAL),
    ({}, dict(max_len=-1), _lib.I8MM_EINVAL),
    ({}, dict(max_len=1 << 40, max_pages=1 << 30), _lib.I8MM_EINVAL),
    ({}, dict(cu_tokens=None), _lib.I8MM_EINVAL),
]
BAD_POINTERS = [
    (dict(k_codes=None), {}, _lib.I8MM_EINVAL),
    (dict(v_codes=MIS), {}, _lib.I8MM_EALIGN),
    (dict(k_absmax=MIS), {}, _lib.I8MM_EALIGN),
    (dict(v_absmax=None), {}, _lib.I8MM_EINVAL),
    ({}, dict(page_table=None), _lib.I8MM_EINVAL),
    ({}, dict(seq_lens=None), _lib.I8MM_EINVAL),
    ({}, dict(page_table=ODD), _lib.I8MM_EALIGN),
    ({}, dict(seq_lens=ODD), _lib.I8MM_EALIGN),
    ({}, dict(cu_tokens=ODD), _lib.I8MM_EALIGN),
]


def call_append(lib, c, b, r=None, k=A, v=A, strides=(128, 64, 128, 64)):
    return lib.int8_kv_cache_append(k, strides[0], strides[1], v, strides[2], strides[3], c, b, r, None)


def call_attention(lib, c, b, r=None, q=A, strides=(256, 64), heads=4, scale=0.125, causal=1, window=0,
                   slopes=None, out=A, ws=A, wn=1 << 40):
    return lib.int8_kv_cache_attention(q, strides[0], strides[1], heads, c, b, r, scale, causal, window,
                                       slopes, out, ws, wn, None)


@pytest.mark.parametrize("ck,bk,status", BAD_SIZES + BAD_POINTERS)
def test_refused_cache_or_batch(lib, ck, bk, status):
    c, b = cache(**ck), batch(**bk)
    assert call_append(lib, c, b) == status
    assert lib.i8mm_last_error().startswith(b"int8_kv_cache_append: ")
    assert call_attention(lib, c, b) == status
    assert lib.int8_kv_cache_read(c, b, A, A, None) == status


def test_refused_null_structs(lib):
    assert call_append(lib, None, batch()) == _lib.I8MM_EINVAL
    assert call_attention(lib, cache(), None) == _lib.I8MM_EINVAL
    assert lib.int8_kv_cache_read(None, None, A, A, None) == _lib.I8MM_EINVAL
    assert lib.int8_kv_cache_attention_workspace_bytes(None, batch(), 4) == 0


@pytest.mark.parametrize("rk,status", [
    (dict(dim=0), _lib.I8MM_EINVAL), (dict(dim=24), _lib.I8MM_EINVAL),
    (dict(dim=80), _lib.I8MM_EINVAL), (dict(positions=255), _lib.I8MM_EINVAL),
    (dict(cos=None), _lib.I8MM_EINVAL), (dict(sin=MIS), _lib.I8MM_EALIGN)])
def test_refused_rotary(lib, rk, status):
    assert call_append(lib, cache(), batch(), rotary(**rk)) == status
    assert call_attention(lib, cache(), batch(), rotary(**rk)) == status


@pytest.mark.parametrize("kw,status", [
    (dict(k=None), _lib.I8MM_EINVAL), (dict(v=MIS), _lib.I8MM_EALIGN),
    (dict(strides=(132, 64, 128, 64)), _lib.I8MM_EALIGN),
    (dict(strides=(128, 64, 128, 12)), _lib.I8MM_EALIGN),
    (dict(strides=(128, 64, -128, 64)), _lib.I8MM_EINVAL)])
def test_refused_append(lib, kw, status):
    assert call_append(lib, cache(), batch(), **kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(q=None), _lib.I8MM_EINVAL), (dict(q=MIS), _lib.I8MM_EALIGN),
    (dict(strides=(260, 64)), _lib.I8MM_EALIGN), (dict(strides=(256, -64)), _lib.I8MM_EINVAL),
    (dict(heads=0), _lib.I8MM_EINVAL), (dict(heads=3), _lib.I8MM_EINVAL),
    (dict(heads=1 << 20), _lib.I8MM_EINVAL),
    (dict(scale=math.nan), _lib.I8MM_EINVAL), (dict(scale=math.inf), _lib.I8MM_EINVAL),
    (dict(scale=0.0), _lib.I8MM_EINVAL), (dict(scale=-1.0), _lib.I8MM_EINVAL),
    (dict(causal=2), _lib.I8MM_EINVAL), (dict(window=-1), _lib.I8MM_EINVAL),
    (dict(window=5, causal=0), _lib.I8MM_EINVAL), (dict(slopes=ODD), _lib.I8MM_EALIGN),
    (dict(out=None), _lib.I8MM_EINVAL), (dict(out=MIS), _lib.I8MM_EALIGN)])
def test_refused_attention(lib, kw, status):
    assert call_attention(lib, cache(), batch(), **kw) == status


def test_refused_rows_beyond_int32(lib):
    """The queries of a sequence that share a head are numbered in int32."""
    b = batch(total_tokens=1 << 28, max_tokens=1 << 28)
    assert lib.int8_kv_cache_attention_workspace_bytes(cache(), b, 20) == 0
    assert call_attention(lib, cache(), b, heads=20) == _lib.I8MM_EINVAL


def test_attention_workspace(lib):
    """A long cache with few rows needs one; it is refused when missing, short
    or misaligned."""
    c, b = cache(), batch(max_pages=1 << 12, max_len=1 << 17)
    need = lib.int8_kv_cache_attention_workspace_bytes(c, b, 4)
    assert need > 0
    assert call_attention(lib, c, b, ws=None, wn=0) == _lib.I8MM_EWORKSPACE
    assert call_attention(lib, c, b, wn=need - 1) == _lib.I8MM_EWORKSPACE
    assert call_attention(lib, c, b, ws=A + 64) == _lib.I8MM_EALIGN
    assert lib.int8_kv_cache_attention_workspace_bytes(c, b, 3) == 0
    assert lib.int8_kv_cache_attention_workspace_bytes(c, b, 0) == 0


def test_nothing_to_do_needs_no_device(lib):
    none = dict(page_table=None, seq_lens=None, cu_tokens=None, num_seqs=0, total_tokens=0)
    assert call_append(lib, cache(), batch(**none), k=None, v=None) == 0
    assert call_attention(lib, cache(), batch(**none), q=None, out=None, ws=None, wn=0) == 0
    assert lib.int8_kv_cache_read(cache(), batch(**none), None, None, None) == 0


def test_binding_refuses_host_and_misshapen_tensors():
    with pytest.raises(ValueError, match="GPU"):
        i8.Int8KVCache(2, 2, 64, device="cpu")
    with pytest.raises(ValueError):
        i8.Int8KVCache(2, 2, 72, device="cpu")
    with pytest.raises(ValueError):
        i8.Int8KVCache(2, 2, 64, page_tokens=24, device="cpu")
    codes, absmax = torch.zeros((2, 2, 4, 4, 16, 16), dtype=torch.int8), torch.zeros((2, 2, 4))
    for bad in [(codes[..., 0], absmax, codes, absmax), (codes, absmax[:1], codes, absmax),
                (codes, absmax, codes[:1], absmax), (codes[:, :, :, :3], absmax, codes, absmax)]:
        with pytest.raises(ValueError):
            i8.Int8KVCache.from_tensors(*bad)
    with pytest.raises(TypeError):
        i8.Int8KVCache.from_tensors(codes.int(), absmax, codes, absmax)
    i32 = torch.int32
    table, lens, cu = torch.zeros((2, 3), dtype=i32), torch.zeros(2, dtype=i32), torch.zeros(3, dtype=i32)
    for args, kw in [((table[0], lens), {}), ((table, lens[:1]), {}), ((table, lens, cu[:2]), {}),
                     ((table, lens, cu), {}), ((table, lens), {"total_tokens": 5}),
                     ((table, lens), {"max_tokens": 2}), ((table, lens), {})]:
        with pytest.raises(ValueError):
            i8.KVBatch(*args, **kw)
    with pytest.raises(TypeError):
        i8.KVBatch(table.long(), lens)
    with pytest.raises(ValueError):
        i8.Rotary(torch.zeros((4, 8)), torch.zeros((4, 9)))


# ------------------------------------------------------------------ reference

def empty(pages=4, heads=2, dim=64, page=32):
    slots = page // 16
    c = {}
    for w in "kv":
        c[w + "_codes"] = np.full((pages, heads, slots, dim // 16, 16, 16), 55, np.int8)
        c[w + "_absmax"] = np.full((pages, heads, slots), np.nan, np.float32)
    return c


def test_reference_append_rounds_to_the_nearest_code():
    """Against 64-bit quotients: code - x * 127 / a is at most a half, plus the
    binary32 roundings of 127 / a and of the product: each 2^-24 of at most 127,
    so 2^-16 in all."""
    rng = np.random.default_rng(1)
    c, b = empty(), (np.array([[2, 0]]), [50], [50])
    k, v = rng.normal(0, 1, (2, 50, 2, 64)).astype(np.float16)
    R.append(c, k, v, b)
    for which, x in (("k", k), ("v", v)):
        for t in range(50):
            page, slot, row = R.place(c, b[0][0], t)
            block = x[t // 16 * 16:t // 16 * 16 + 16].astype(np.float64)
            top = np.abs(block).max(axis=(0, 2))
            assert np.array_equal(c[which + "_absmax"][page, :, slot], top.astype(np.float32))
            code = R.get_rows(c, which, page, slot)[:, row]
            assert np.abs(code - x[t] * (127.0 / top[:, None])).max() <= 0.5 + 2.0 ** -16


def test_reference_tile_layout():
    """Token t and feature f of a block stand where the header says."""
    c, b = empty(1, 1, 64, 16), (np.array([[0]]), [16], [16])
    k = np.zeros((16, 1, 64), np.float16)
    k[5, 0, 37] = 1
    R.append(c, k, 2 * k, b)
    assert c["k_codes"].sum() == 127 and c["k_codes"][0, 0, 0, 2, 5, 5] == 127   # 37 = 2 * 16 + 5
    k[5, 0, 37], k[11, 0, 50] = 0, 1
    R.append(c, k, k, b)
    assert c["k_codes"][0, 0, 0, 3, 11, 2] == 127 and c["v_codes"][0, 0, 0, 3, 2, 11] == 127


def test_reference_rotation_keeps_products_of_equal_distance():
    """<rot(q, p), rot(k, t)> depends on p - t alone, in both pairings."""
    rng = np.random.default_rng(2)
    half = 32
    ang = np.arange(30)[:, None] * (100.0 ** (-np.arange(half) / half))
    cos, sin = np.cos(ang).astype(np.float32), np.sin(ang).astype(np.float32)
    q, k = rng.normal(0, 1, (2, 1, 64)).astype(np.float32)
    for inter in (False, True):
        dots = [float((R.rotate(q, p + 7, cos, sin, inter) * R.rotate(k, p, cos, sin, inter)).sum())
                for p in range(20)]
        assert np.ptp(dots) < 1e-4 and abs(dots[0] - float((q * k).sum())) > 1e-3


def test_reference_attention_closed_forms():
    """One visible token returns its value; a zero query averages; a slope far
    above every logit picks the nearest token; nothing visible gives 0."""
    rng = np.random.default_rng(3)
    c, b = empty(), (np.array([[1, 3]]), [40], [40])
    k, v = rng.normal(0, 1, (2, 40, 2, 64)).astype(np.float16)
    R.append(c, k, v, b)
    vals = np.array([R.values(c, "v", b[0][0], t) for t in range(40)], np.float64)
    q = rng.normal(0, 1, (40, 2, 64)).astype(np.float16)
    out, bound = R.attention(c, q, b)
    assert np.allclose(out[0], vals[0], atol=1e-12) and (bound > 0).all() and bound.max() < 0.1
    assert np.allclose(R.attention(c, 0 * q, b)[0][-1], vals.mean(axis=0), atol=1e-12)
    assert np.allclose(R.attention(c, q, b, window=1)[0], vals, atol=1e-12)
    assert np.allclose(R.attention(c, q, b, slopes=[1e4, 1e4])[0], vals, atol=1e-9)
    absent = (np.array([[-1, 9]]), [40], [40])
    assert not R.attention(c, q, absent)[0].any()
    o2, _ = R.attention(c, q, b, causal=False)
    assert np.allclose(o2[-1], out[-1]) and not np.allclose(o2[0], out[0])


def test_cached_attention_layer_refusals():
    with pytest.raises(ValueError):
        i8.Int8CachedAttention(256, 4, 3, device="cpu")
    with pytest.raises(ValueError):
        i8.Int8CachedAttention(256, 0, device="cpu")
    with pytest.raises(ValueError):
        i8.Int8CachedAttention(256, 6, device="cpu")
    layer = i8.Int8CachedAttention(256, 4, 2, device="cpu")
    assert (layer.qkv.out_features, layer.out.in_features, layer.head_dim) == (512, 256, 64)

    class Sizes:
        kv_heads, head_dim, total_tokens = 2, 80, 3
    with pytest.raises(ValueError):     # another cache's head size
        layer(torch.zeros((3, 256), dtype=torch.float16), Sizes, Sizes)
    Sizes.head_dim = 64
    with pytest.raises(ValueError):     # rows that the batch does not have
        layer(torch.zeros((2, 256), dtype=torch.float16), Sizes, Sizes)
