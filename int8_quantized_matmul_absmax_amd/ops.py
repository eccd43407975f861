"""Torch-tensor wrappers of the C ABI, one per entry point, with the same names.

Argument marshalling only: every step of the layer runs in the HIP kernels of
libi8mm.so. torch provides device memory and the current stream. Inputs must
be contiguous tensors on one gfx950 GPU; outputs are allocated here with torch
unless passed in.

Pages cited: [HF-blog] Hugging Face blog "A Gentle Introduction to 8-bit Matrix
Multiplication for transformers at scale using Hugging Face Transformers,
Accelerate and bitsandbytes"; [Summary] paper summary page "LLM.int8(): 8-Bit
Matrix Multiplication for Transformers at Scale".
"""

import ctypes
import math

import torch

from . import _lib

DEFAULT_THRESHOLD = 6.0  # [HF-blog] "Inside the MatMul": magnitude 6 or more


def outlier_ld(n):
    """Row stride (in halfs) of the gathered outlier columns: n rounded up to 32."""
    return (int(n) + 31) // 32 * 32


def _ptr(t):
    return ctypes.c_void_p(t.data_ptr()) if t is not None else ctypes.c_void_p(0)


def _raw_stream(device):
    # (the handle alone: a Stream object costs 2 us a call)
    return torch._C._cuda_getCurrentRawStream(device.index)


def _run(device, call, *args):
    """call(*args, the current stream of `device`), checked, with `device` current."""
    if torch._C._cuda_getDevice() == device.index:
        return _lib.check(call(*args, _raw_stream(device)))
    with torch.cuda.device(device):
        return _lib.check(call(*args, _raw_stream(device)))


def _need(t, name, dtype, ndim=None, shape=None, min_numel=None):
    """Type, dtype, contiguity and size of one tensor argument (no device check:
    _on_gpu does that for all arguments of a call together)."""
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch.Tensor" % name)
    if t.dtype != dtype:
        raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    if ndim is not None and t.dim() != ndim:
        raise ValueError("%s must have %d dims, got %d" % (name, ndim, t.dim()))
    if shape is not None and t.shape != shape and tuple(t.shape) != tuple(shape):
        raise ValueError("%s must have shape %s, got %s" % (name, tuple(shape), tuple(t.shape)))
    if min_numel is not None and t.numel() < min_numel:
        raise ValueError("%s must hold at least %d elements, got %d" % (name, min_numel, t.numel()))


def _on_gpu(**tensors):
    """Every given tensor (None = absent) is on one GPU; returns that device.
    The path runs on the GPU only: a host tensor is an error, not a fallback."""
    dev = None
    for name, t in tensors.items():
        if t is None:
            continue
        if not t.is_cuda:
            raise ValueError("%s must be on a GPU (the path runs on the GPU only)" % name)
        if dev is None:
            dev = t.device
        elif t.device != dev:
            raise ValueError("%s is on %s, the other arguments on %s" % (name, t.device, dev))
    return dev


def _flatten_tokens(X):
    """[..., K] -> [M, K] (tokens of all leading dims are the rows)."""
    if X.dim() < 2:
        raise ValueError("X must be at least 2-D")
    return X.reshape(math.prod(X.shape[:-1]), X.shape[-1])   # (-1 is ambiguous when K == 0)


def int8_quantize_colwise_weight(W, Wq=None, sw=None):
    """Per-output-row absmax quantization of W [N, K] fp16 -> (Wq int8 [N, K], sw fp32 [N])."""
    lib = _lib.load_library()
    _need(W, "W", torch.float16, 2)
    N, K = W.shape
    if Wq is not None:
        _need(Wq, "Wq", torch.int8, shape=(N, K))
    if sw is not None:
        _need(sw, "sw", torch.float32, shape=(N,))
    dev = _on_gpu(W=W, Wq=Wq, sw=sw)
    Wq = Wq if Wq is not None else torch.empty((N, K), dtype=torch.int8, device=dev)
    sw = sw if sw is not None else torch.empty((N,), dtype=torch.float32, device=dev)
    _run(dev, lib.int8_quantize_colwise_weight, _ptr(W), N, K, _ptr(Wq), _ptr(sw))
    return Wq, sw


def int8_quantize_rowwise(X, outlier_bitmap=None, Xq=None, sx=None):
    """Row-wise absmax quantization of X [M, K] fp16 over its non-outlier columns
    -> (Xq int8 [M, K], sx fp32 [M])."""
    lib = _lib.load_library()
    _need(X, "X", torch.float16)
    X2 = _flatten_tokens(X)
    M, K = X2.shape
    if outlier_bitmap is not None:
        _need(outlier_bitmap, "outlier_bitmap", torch.int32, 1, min_numel=(K + 31) // 32)
    if Xq is not None:
        _need(Xq, "Xq", torch.int8, shape=(M, K))
    if sx is not None:
        _need(sx, "sx", torch.float32, shape=(M,))
    dev = _on_gpu(X=X, outlier_bitmap=outlier_bitmap, Xq=Xq, sx=sx)
    Xq = Xq if Xq is not None else torch.empty((M, K), dtype=torch.int8, device=dev)
    sx = sx if sx is not None else torch.empty((M,), dtype=torch.float32, device=dev)
    _run(dev, lib.int8_quantize_rowwise, _ptr(X2), M, K, _ptr(outlier_bitmap), _ptr(Xq), _ptr(sx))
    return Xq, sx


def outlier_detect_gather(X, threshold=DEFAULT_THRESHOLD, gather=True):
    """Outlier columns of X [M, K] fp16.

    Returns (bitmap int32 [ceil(K/32)] (bit patterns of the uint32 words),
    cols int32 [K] (first n valid, ascending), n int32 [1] on the device,
    Xo fp16 flat buffer of capacity M * outlier_ld(K) holding [M, outlier_ld(n)]
    or None).
    """
    lib = _lib.load_library()
    _need(X, "X", torch.float16)
    X2 = _flatten_tokens(X)
    M, K = X2.shape
    dev = _on_gpu(X=X)
    bitmap = torch.empty(((K + 31) // 32,), dtype=torch.int32, device=dev)
    cols = torch.empty((max(K, 1),), dtype=torch.int32, device=dev)
    n = torch.empty((1,), dtype=torch.int32, device=dev)
    Xo = torch.empty((max(M * outlier_ld(K), 1),), dtype=torch.float16, device=dev) if gather else None
    _run(dev, lib.outlier_detect_gather, _ptr(X2), M, K, float(threshold), _ptr(bitmap), _ptr(cols),
         _ptr(n), _ptr(Xo))
    return bitmap, cols, n, Xo


def outlier_detect_quantize(X, threshold=DEFAULT_THRESHOLD, workspace=None):
    """The activation side of linear_int8_mixed alone (detection, gather and
    row quantization, the same two kernels) into a layer workspace. Returns
    the workspace; workspace_views(workspace, M, K) gives bitmap, cols, n, sx,
    Xq and Xo, which int8_mm_dequant takes."""
    lib = _lib.load_library()
    _need(X, "X", torch.float16)
    X2 = _flatten_tokens(X)
    M, K = X2.shape
    if workspace is not None:
        _need(workspace, "workspace", torch.uint8, 1, min_numel=workspace_bytes(M, K))
    dev = _on_gpu(X=X, workspace=workspace)
    if workspace is None:
        workspace = torch.empty((max(workspace_bytes(M, K), 1),), dtype=torch.uint8, device=dev)
    _run(dev, lib.outlier_detect_quantize, _ptr(X2), M, K, float(threshold), _ptr(workspace),
         workspace.numel())
    return workspace


def int8_mm_dequant(Xq, Wq, sx, sw, Xo=None, cols=None, n=None, bias=None, want_y=True,
                    want_int32=False, out=None):
    """int8 GEMM (int32 accumulation) with the fused dequantization, fp16 outlier
    product and bias. Returns Y fp16 [M, N] and/or C int32 [M, N].

    Xo, cols, n come together (from outlier_detect_gather or a layer
    workspace): Xo fp16 of capacity >= M * outlier_ld(K) (the count n is only
    known on the device, so room for every column is required), cols int32
    with >= K entries, n int32 [1] on the device."""
    lib = _lib.load_library()
    _need(Xq, "Xq", torch.int8, 2)
    M, K = Xq.shape
    _need(Wq, "Wq", torch.int8, 2)
    N = Wq.shape[0]
    _need(Wq, "Wq", torch.int8, shape=(N, K))
    _need(sx, "sx", torch.float32, shape=(M,))
    _need(sw, "sw", torch.float32, shape=(N,))
    given = [t is not None for t in (Xo, cols, n)]
    if any(given) and not all(given):
        raise ValueError("Xo, cols and n must be given together")
    if Xo is not None:
        _need(Xo, "Xo", torch.float16, min_numel=M * outlier_ld(K))
        _need(cols, "cols", torch.int32, min_numel=K)
        _need(n, "n", torch.int32, shape=(1,))
    if bias is not None:
        _need(bias, "bias", torch.float16, shape=(N,))
    if out is not None:
        _need(out, "out", torch.float16, shape=(M, N))
    if not (want_y or want_int32):
        raise ValueError("nothing requested: want_y and want_int32 are both False")
    dev = _on_gpu(Xq=Xq, Wq=Wq, sx=sx, sw=sw, Xo=Xo, cols=cols, n=n, bias=bias, out=out)
    Y = None
    if want_y:
        Y = out if out is not None else torch.empty((M, N), dtype=torch.float16, device=dev)
    C = torch.empty((M, N), dtype=torch.int32, device=dev) if want_int32 else None
    _run(dev, lib.int8_mm_dequant, _ptr(Xq), _ptr(Wq), _ptr(sx), _ptr(sw), M, N, K, _ptr(Xo),
         _ptr(cols), _ptr(n), _ptr(bias), _ptr(Y), _ptr(C))
    if want_y and want_int32:
        return Y, C
    return Y if want_y else C


def workspace_bytes(M, K, N=None):
    """Workspace bytes of linear_int8_mixed for M tokens and K features; with N
    (output features) given, the size with a region of recovered outlier
    weights with room for 512 columns, which speeds up 17 to 512 outlier
    columns; without it every outlier count still takes a second GEMM loop.
    Any larger workspace has room for floor(extra / (2 N) / 32) * 32 columns
    (see workspace_bytes_all_outliers)."""
    lib = _lib.load_library()
    if N is None:
        return int(lib.linear_int8_mixed_workspace_bytes(int(M), int(K)))
    return int(lib.linear_int8_mixed_workspace_bytes_many_outliers(int(M), int(K), int(N)))


def workspace_bytes_all_outliers(M, K, N):
    """Workspace bytes whose outlier weight region has room for every outlier
    count (K columns): the fastest layer at any count, for N * outlier_ld(K)
    * 2 extra bytes."""
    base = workspace_bytes(M, K)
    return base + int(N) * outlier_ld(int(K)) * 2 if base else 0


def outlier_region_cols(workspace_bytes_, M, K, N):
    """Outlier columns a workspace of workspace_bytes_ bytes has room for in
    its recovered-weight region (0 means none)."""
    extra = int(workspace_bytes_) - workspace_bytes(M, K)
    if extra <= 0 or N <= 0:
        return 0
    return min(extra // (2 * int(N)) // 32 * 32, outlier_ld(int(K)))


def workspace_layout(M, K):
    """Byte offsets of bitmap, cols, n, sx, Xq, Xo in the workspace, and its size."""
    lib = _lib.load_library()
    off = (ctypes.c_int64 * 7)()
    _lib.check(lib.i8mm_workspace_layout(int(M), int(K), off))
    keys = ("bitmap", "cols", "n", "sx", "Xq", "Xo", "total")
    return dict(zip(keys, [int(v) for v in off]))


def _layer_buffers(X, N, bias, workspace, out, K_w, W_name):
    """Shared argument checks of the two layer calls; returns (X2, M, K, dev,
    workspace, Y, lead)."""
    lead = X.shape[:-1]
    X2 = _flatten_tokens(X)
    M, K = X2.shape
    if K_w != K:
        raise ValueError("%s has %d input features, X has %d" % (W_name, K_w, K))
    if bias is not None:
        _need(bias, "bias", torch.float16, shape=(N,))
    if workspace is not None:
        _need(workspace, "workspace", torch.uint8, 1, min_numel=workspace_bytes(M, K))
    if out is not None:
        _need(out, "out", torch.float16)
        if out.numel() != M * N:
            raise ValueError("out must hold M * N = %d elements, got %d" % (M * N, out.numel()))
    return X2, M, K, lead


def linear_int8_mixed(X, Wq, sw, bias=None, threshold=DEFAULT_THRESHOLD, workspace=None, out=None):
    """The whole layer: Y = X . W^T with outlier decomposition, for an int8 weight
    (Wq, sw) from int8_quantize_colwise_weight. X [..., K] fp16 -> Y [..., N] fp16.
    Without a workspace, one of workspace_bytes(M, K, N) bytes is allocated."""
    lib = _lib.load_library()
    _need(X, "X", torch.float16)
    _need(Wq, "Wq", torch.int8, 2)
    N = Wq.shape[0]
    _need(sw, "sw", torch.float32, shape=(N,))
    X2, M, K, lead = _layer_buffers(X, N, bias, workspace, out, Wq.shape[1], "Wq")
    dev = _on_gpu(X=X, Wq=Wq, sw=sw, bias=bias, workspace=workspace, out=out)
    if workspace is None:
        workspace = torch.empty((max(workspace_bytes(M, K, N), 1),), dtype=torch.uint8, device=dev)
    Y = out if out is not None else torch.empty((M, N), dtype=torch.float16, device=dev)
    _run(dev, lib.linear_int8_mixed, _ptr(X2), M, K, _ptr(Wq), _ptr(sw), N, _ptr(bias),
         float(threshold), _ptr(Y), _ptr(workspace), workspace.numel())
    return Y.reshape(*lead, N)


def linear_int8_mixed_fp16_weights(X, W, Wq, sw, quantize_weight=True, bias=None,
                                   threshold=DEFAULT_THRESHOLD, workspace=None, out=None):
    """The whole layer for a weight kept in fp16 (has_fp16_weights=True).
    W [N, K] fp16; Wq [N, K] int8 and sw [N] fp32 are caller-owned buffers that
    receive W's codes when quantize_weight (else they must already hold them).
    The outlier product uses W's own columns. X [..., K] fp16 -> Y [..., N]."""
    lib = _lib.load_library()
    _need(X, "X", torch.float16)
    _need(W, "W", torch.float16, 2)
    N, K_w = W.shape
    _need(Wq, "Wq", torch.int8, shape=(N, K_w))
    _need(sw, "sw", torch.float32, shape=(N,))
    X2, M, K, lead = _layer_buffers(X, N, bias, workspace, out, K_w, "W")
    dev = _on_gpu(X=X, W=W, Wq=Wq, sw=sw, bias=bias, workspace=workspace, out=out)
    if workspace is None:
        workspace = torch.empty((max(workspace_bytes(M, K, N), 1),), dtype=torch.uint8, device=dev)
    Y = out if out is not None else torch.empty((M, N), dtype=torch.float16, device=dev)
    _run(dev, lib.linear_int8_mixed_fp16_weights, _ptr(X2), M, K, _ptr(W), N, _ptr(Wq), _ptr(sw),
         1 if quantize_weight else 0, _ptr(bias), float(threshold), _ptr(Y), _ptr(workspace),
         workspace.numel())
    return Y.reshape(*lead, N)


def gelu_f16(X, out=None):
    """Exact-erf GELU in fp32 on an fp16 tensor (glue between MLP layers)."""
    lib = _lib.load_library()
    _need(X, "X", torch.float16)
    if out is not None:
        _need(out, "out", torch.float16, min_numel=X.numel())
    dev = _on_gpu(X=X, out=out)
    Y = out if out is not None else torch.empty_like(X)
    _run(dev, lib.i8mm_gelu_f16, _ptr(X), X.numel(), _ptr(Y))
    return Y


# ---- paged 8-bit key/value cache (cache, batch, rotary: kv_cache.Int8KVCache,
# KVBatch and Rotary, which check and hold their own tensors)

KV_BLOCK = 16   # I8MM_KV_BLOCK


def _need_heads(t, name, tokens, heads, dim, device):
    """fp16 [tokens, heads, dim] on device, features contiguous, 16-byte rows."""
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch.Tensor" % name)
    if t.dtype != torch.float16:
        raise TypeError("%s must be torch.float16, got %s" % (name, t.dtype))
    shape = t.shape
    if len(shape) != 3 or shape[0] != tokens or shape[2] != dim or heads not in (None, shape[1]):
        raise ValueError("%s must have shape %s, got %s"
                         % (name, (tokens, "heads" if heads is None else heads, dim),
                            tuple(shape)))
    if t.device != device:
        raise ValueError("%s is on %s, the cache on %s" % (name, t.device, device))
    ts, hs, fs = t.stride()
    if fs != 1 and t.numel() > 0:
        raise ValueError("the features of %s must be contiguous" % name)
    return t.data_ptr(), ts, hs


def _kv_args(cache, batch, rotary):
    if batch.device != cache.device:
        raise ValueError("the batch is on %s, the cache on %s" % (batch.device, cache.device))
    if rotary is None:
        return None
    if rotary.device != cache.device:
        raise ValueError("the rotary tables are on %s, the cache on %s"
                         % (rotary.device, cache.device))
    return rotary.ref


def _scratch(workspace, dev, size, *args):
    """A workspace of size(*args) bytes, its address and its size: `workspace` is a
    uint8 tensor, or a function of the device and a number of bytes that gives one, or
    None (allocated here). The caller keeps the tensor until its call returns: memory
    that nothing holds could be given to another thread's call, or back to the device,
    before the kernels that use it are on the stream."""
    if workspace is None or callable(workspace):
        need = size(*args)
        if not need:
            return None, None, 0
        workspace = workspace(dev, need) if workspace else \
            torch.empty((need,), dtype=torch.uint8, device=dev)
    else:
        _need(workspace, "workspace", torch.uint8, 1)
        if workspace.device != dev:
            raise ValueError("workspace is on %s, the call on %s" % (workspace.device, dev))
    return workspace, workspace.data_ptr(), workspace.numel()


def int8_kv_cache_append(k, v, cache, batch, rotary=None):
    """Quantize new keys (rotated first when `rotary` is given) and values into
    the cache. k, v fp16 [total_tokens, kv_heads, D]; the token and head strides
    are free (multiples of 8)."""
    lib = _lib.load_library()
    rot = _kv_args(cache, batch, rotary)
    kp, kts, khs = _need_heads(k, "k", batch.total_tokens, cache.kv_heads, cache.head_dim,
                               cache.device)
    vp, vts, vhs = _need_heads(v, "v", batch.total_tokens, cache.kv_heads, cache.head_dim,
                               cache.device)
    _run(cache.device, lib.int8_kv_cache_append, kp, kts, khs, vp, vts, vhs, cache.ref, batch.ref,
         rot)


def int8_kv_cache_attention_workspace_bytes(cache, batch, q_heads):
    """Bytes of workspace int8_kv_cache_attention needs."""
    return _lib.load_library().int8_kv_cache_attention_workspace_bytes(cache.ref, batch.ref,
                                                                       int(q_heads))


def int8_kv_cache_attention(q, cache, batch, rotary=None, scale=None, causal=True, window=0,
                            alibi_slopes=None, workspace=None, out=None):
    """Attention of the queries q fp16 [total_tokens, q_heads, D] (rotated here
    when `rotary` is given) over the cached tokens -> fp16 [total_tokens,
    q_heads, D]. scale defaults to 1 / sqrt(D). workspace: a uint8 tensor, or a
    function of the device and a number of bytes that gives one; allocated here
    when None."""
    lib = _lib.load_library()
    rot = _kv_args(cache, batch, rotary)
    dev, D = cache.device, cache.head_dim
    qp, qts, qhs = _need_heads(q, "q", batch.total_tokens, None, D, dev)
    heads = q.shape[1]
    slopes = None
    if alibi_slopes is not None:
        _need(alibi_slopes, "alibi_slopes", torch.float32, shape=(heads,))
        _on_gpu(q=q, alibi_slopes=alibi_slopes)
        slopes = alibi_slopes.data_ptr()
    if out is None:
        out = q.new_empty(q.shape)
    else:
        _need(out, "out", torch.float16, shape=q.shape)
        _on_gpu(q=q, out=out)
    held, wp, wn = _scratch(workspace, dev, lib.int8_kv_cache_attention_workspace_bytes, cache.ref,
                            batch.ref, heads)
    _run(dev, lib.int8_kv_cache_attention, qp, qts, qhs, heads, cache.ref, batch.ref, rot,
         1.0 / math.sqrt(D) if scale is None else scale, 1 if causal else 0, window, slopes,
         out.data_ptr(), wp, wn)
    return out


def int8_kv_cache_read(cache, batch):
    """The cached keys (rotated, as stored) and values of the batch's tokens:
    two fp16 tensors [total_tokens, kv_heads, D]."""
    lib = _lib.load_library()
    _kv_args(cache, batch, None)
    k, v = torch.empty((2, batch.total_tokens, cache.kv_heads, cache.head_dim),
                       dtype=torch.float16, device=cache.device).unbind(0)
    _run(cache.device, lib.int8_kv_cache_read, cache.ref, batch.ref, k.data_ptr(), v.data_ptr())
    return k, v


def _means_of(cache):
    if cache.k_means is None:
        raise ValueError("the cache holds no mean keys (page_means=True)")
    return cache.k_means.data_ptr()


def int8_kv_cache_page_means(cache, batch):
    """Mean keys (cache.k_means) of the pages that hold the batch's new tokens, after
    their append."""
    lib = _lib.load_library()
    _kv_args(cache, batch, None)
    _run(cache.device, lib.int8_kv_cache_page_means, cache.ref, batch.ref, _means_of(cache))


def int8_kv_cache_select_pages(q, cache, batch, count, rotary=None, first=1, recent=1, out=None):
    """The pages that each new token and key/value head attends to: int32
    [total_tokens, kv_heads, count] numbers of pages in the sequence, ascending, then
    -1. Always the first `first` and the newest `recent`, the others by the product
    of the head's queries (q fp16 [total_tokens, q_heads, D], rotated here when
    `rotary` is given) with the page's mean key."""
    lib = _lib.load_library()
    rot = _kv_args(cache, batch, rotary)
    means = _means_of(cache)
    qp, qts, qhs = _need_heads(q, "q", batch.total_tokens, None, cache.head_dim, cache.device)
    shape = (batch.total_tokens, cache.kv_heads, max(int(count), 0))
    if out is None:
        out = torch.empty(shape, dtype=torch.int32, device=cache.device)
    else:
        _need(out, "out", torch.int32, shape=shape)
        _on_gpu(q=q, out=out)
    _run(cache.device, lib.int8_kv_cache_select_pages, qp, qts, qhs, q.shape[1], cache.ref, means,
         batch.ref, rot, count, first, recent, out.data_ptr())
    return out


def int8_kv_cache_attention_pages(q, pages, cache, batch, rotary=None, scale=None, workspace=None,
                                  out=None):
    """Causal attention of the queries q fp16 [total_tokens, q_heads, D] over the
    tokens of the listed pages: pages int32 [total_tokens, kv_heads, count], as
    int8_kv_cache_select_pages gives them. scale and workspace as for
    int8_kv_cache_attention."""
    lib = _lib.load_library()
    rot = _kv_args(cache, batch, rotary)
    dev, D = cache.device, cache.head_dim
    qp, qts, qhs = _need_heads(q, "q", batch.total_tokens, None, D, dev)
    heads = q.shape[1]
    _need(pages, "pages", torch.int32, 3)
    count = pages.shape[2]
    if pages.shape[:2] != (batch.total_tokens, cache.kv_heads):
        raise ValueError("pages must be [%d, %d, count], got %s"
                         % (batch.total_tokens, cache.kv_heads, tuple(pages.shape)))
    if out is None:
        out = q.new_empty(q.shape)
    else:
        _need(out, "out", torch.float16, shape=q.shape)
    _on_gpu(q=q, pages=pages, out=out)
    held, wp, wn = _scratch(workspace, dev, lib.int8_kv_cache_attention_pages_workspace_bytes,
                            cache.ref, batch.ref, heads, count)
    _run(dev, lib.int8_kv_cache_attention_pages, qp, qts, qhs, heads, cache.ref, batch.ref, rot,
         pages.data_ptr(), count, 1.0 / math.sqrt(D) if scale is None else scale, out.data_ptr(), wp, wn)
    return out


class _PagesStep:
    """What a step of the page tables gives, in one tensor; views of it as they are
    asked for (each costs as much as a call's checks)."""

    def __init__(self, rows, width, device):
        self.rows, self.width = rows, width
        n = rows * width
        self.at = (0, n, n + rows, n + 4 * rows, n + 4 * rows + 2, n + 4 * rows + 3)
        self.out = torch.empty((n + 5 * rows + 3,), dtype=torch.int32, device=device)

    def view(self, i, *shape):
        return self.out.as_strided(shape, (shape[1], 1) if len(shape) == 2 else (1,), self.at[i])

    table = property(lambda self: self.view(0, self.rows, self.width))
    lens = property(lambda self: self.view(1, self.rows))
    copies = property(lambda self: self.view(2, self.rows, 3))
    counts = property(lambda self: self.view(3, 2))
    full = property(lambda self: self.view(4, 1))
    batch_lens = property(lambda self: self.view(5, self.rows))


def _pages_step(page_table, seq_lens, parents, num_pages, page_tokens, new_tokens=1, keep=None,
               workspace=None, max_len=None):
    """kv_pages_step, its results as a _PagesStep."""
    lib = _lib.load_library()
    _need(page_table, "page_table", torch.int32, 2)
    seqs, width = page_table.shape
    _need(seq_lens, "seq_lens", torch.int32, shape=(seqs,))
    _need(parents, "parents", torch.int32)
    rows = parents.numel()
    each, new_all = None, 0
    if isinstance(new_tokens, torch.Tensor):
        _need(new_tokens, "new_tokens", torch.int32)
        each = new_tokens
    else:
        new_all = int(new_tokens)
    if keep is not None:
        _need(keep, "keep", torch.int32)
    for name, t in (("new_tokens", each), ("keep", keep)):
        if t is not None and t.numel() != rows:
            raise ValueError("%s must hold %d numbers, got %d" % (name, rows, t.numel()))
    dev = _on_gpu(page_table=page_table, seq_lens=seq_lens, parents=parents, keep=keep,
                  new_tokens=each)
    step = _PagesStep(rows, width, dev)
    begin = step.out.data_ptr()
    table, lens, copies, counts, full, batch_lens = [begin + 4 * i for i in step.at]
    held, wp, wn = _scratch(workspace, dev, lib.i8mm_kv_pages_workspace_bytes, rows, width, num_pages)
    _run(dev, lib.i8mm_kv_pages_step_batch, page_table.data_ptr(), seq_lens.data_ptr(), seqs, width,
         parents.data_ptr(), None if keep is None else keep.data_ptr(),
         None if each is None else each.data_ptr(), new_all, rows, num_pages, page_tokens,
         1 << 30 if max_len is None else int(max_len), table, lens, batch_lens, full, copies, counts,
         wp, wn)
    return step


def kv_pages_step(page_table, seq_lens, parents, num_pages, page_tokens, new_tokens=1, keep=None,
                  workspace=None, max_len=None, batch=False):
    """The page table of the next step: row i keeps the first keep[i] tokens (None:
    all) of row parents[i] (none for a parent outside the table) and has room for
    new_tokens (an int, or int32 [rows]) after them. All int32 on the GPU.

    Returns the table [rows, max_pages], the lengths [rows] (new tokens included),
    the copies to make before the next append [rows, 3] and counts [2]: copies, and
    pages that were wanting (their tokens are absent). With batch=True also the lengths
    for a KVBatch of the new tokens [rows] (0 for a row that has none, or no room for all
    of them, in the table or below max_len) and how many have no room [1]."""
    s = _pages_step(page_table, seq_lens, parents, num_pages, page_tokens, new_tokens, keep, workspace,
                   max_len)
    found = s.table, s.lens, s.copies, s.counts
    return found + (s.batch_lens, s.full) if batch else found


def kv_pages_compact(page_table, seq_lens, num_pages, page_tokens, workspace=None):
    """The used pages to the front: the table with their new places, the copies to
    make [num_pages // 2, 3] and counts [2]: copies, and used pages."""
    lib = _lib.load_library()
    _need(page_table, "page_table", torch.int32, 2)
    seqs, width = page_table.shape
    _need(seq_lens, "seq_lens", torch.int32, shape=(seqs,))
    dev = _on_gpu(page_table=page_table, seq_lens=seq_lens)
    most = max(int(num_pages) // 2, 0)
    out = torch.empty((seqs * width + 3 * most + 2,), dtype=torch.int32, device=dev)
    table = out.as_strided((seqs, width), (width, 1))
    copies = out.as_strided((most, 3), (3, 1), seqs * width)
    counts = out.as_strided((2,), (1,), seqs * width + 3 * most)
    held, wp, wn = _scratch(workspace, dev, lib.i8mm_kv_pages_workspace_bytes, seqs, width, num_pages)
    _run(dev, lib.i8mm_kv_pages_compact, page_table.data_ptr(), seq_lens.data_ptr(), seqs, width,
         num_pages, page_tokens, table.data_ptr(), copies.data_ptr(), counts.data_ptr(), wp, wn)
    return table, copies, counts


def int8_kv_cache_copy_pages(cache, copies, count):
    """Copy a cache's pages (its mean keys, too, where it holds them): copies int32
    [n, 3] of (page, page to copy it to, tokens that count), of which the first
    `count` (int32, its first element) are made."""
    lib = _lib.load_library()
    _need(copies, "copies", torch.int32, 2)
    if copies.shape[1] != 3:
        raise ValueError("copies must be [n, 3], got %s" % (tuple(copies.shape),))
    _need(count, "count", torch.int32, min_numel=1)
    _on_gpu(cache=cache.k_codes, copies=copies, count=count)
    _run(cache.device, lib.int8_kv_cache_copy_pages, cache.ref,
         None if cache.k_means is None else cache.k_means.data_ptr(), copies.data_ptr(),
         count.data_ptr(), copies.shape[0])


# ---- a beam search over such caches

MAX_BEAM_COUNT = 64    # I8MM_MAX_BEAM_COUNT

def beam_select(logits, scores, live=None, eos=None, count=None, workspace=None):
    """The next beams of a batch of beam searches: of each search the `count`
    (default: beams) best of all its beams' words, by scores + log_softmax(logits),
    equal ones by beam and word.

    logits  fp16 or fp32 [batch, beams, vocab], words contiguous, rows evenly apart
    scores  fp32 [batch, beams]; -inf for a beam that is not there (all but one at
            the start of a search)
    live    int32 [batch, beams], 0 for a beam that has ended: it stands for itself,
            with its score and the word eos. None: all go on
    eos     the word that ends a beam, None if none does
    workspace  as for int8_kv_cache_attention

    Returns scores fp32, tokens, parents (rows search * beams + beam: what
    KVPages.step takes) and live int32, each [batch, count]; -inf, -1, -1 and 0
    where there is no candidate left."""
    lib = _lib.load_library()
    if not isinstance(logits, torch.Tensor):
        raise TypeError("logits must be a torch.Tensor")
    if logits.dtype not in (torch.float16, torch.float32):
        raise TypeError("logits must be torch.float16 or torch.float32, got %s" % logits.dtype)
    if logits.dim() != 3:
        raise ValueError("logits must have 3 dims, got %d" % logits.dim())
    batch, beams, vocab = logits.shape
    _need(scores, "scores", torch.float32, shape=(batch, beams))
    if live is not None:
        _need(live, "live", torch.int32, shape=(batch, beams))
    bs, rs, ws = logits.stride()
    if beams == 1:
        rs = bs
    if batch * beams <= 1:
        rs = max(rs, vocab)
    if logits.numel() and ((vocab > 1 and ws != 1) or (batch > 1 and bs != beams * rs) or rs < vocab):
        raise ValueError("the words of logits must be contiguous and its rows evenly apart")
    dev = _on_gpu(logits=logits, scores=scores, live=live)
    count = beams if count is None else int(count)
    fp32 = 1 if logits.dtype == torch.float32 else 0
    tokens, parents, alive = torch.empty((3, batch, max(count, 0)), dtype=torch.int32,
                                         device=dev).unbind(0)
    out = torch.empty((batch, max(count, 0)), dtype=torch.float32, device=dev)
    held, wp, wn = _scratch(workspace, dev, lib.i8mm_beam_select_workspace_bytes, fp32, batch, beams,
                            vocab, count)
    _run(dev, lib.i8mm_beam_select, logits.data_ptr(), fp32, max(rs, vocab), scores.data_ptr(),
         None if live is None else live.data_ptr(), batch, beams, vocab, count,
         -1 if eos is None else int(eos), out.data_ptr(), tokens.data_ptr(), parents.data_ptr(),
         alive.data_ptr(), wp, wn)
    return out, tokens, parents, alive


OUTLIER_REGION_COLS = 512   # I8MM_OUTLIER_REGION_COLS


def workspace_views(workspace, M, K, N=None):
    """Typed views of the intermediates inside a linear_int8_mixed workspace.
    Given N and a workspace larger than workspace_bytes(M, K), also "Wo": the
    region of fp16 outlier weight columns the tiled path materializes when
    16 < n <= outlier_region_cols(...), N rows outlier_ld(n) halfs apart
    (flat, the region's whole room)."""
    off = workspace_layout(M, K)
    w = workspace
    views = {
        "bitmap": w[off["bitmap"]:off["bitmap"] + ((K + 31) // 32) * 4].view(torch.int32),
        "cols": w[off["cols"]:off["cols"] + K * 4].view(torch.int32),
        "n": w[off["n"]:off["n"] + 4].view(torch.int32),
        "sx": w[off["sx"]:off["sx"] + M * 4].view(torch.float32),
        "Xq": w[off["Xq"]:off["Xq"] + M * K].view(torch.int8).view(M, K),
        "Xo": w[off["Xo"]:off["Xo"] + M * outlier_ld(K) * 2].view(torch.float16),
    }
    if N is not None:
        room = outlier_region_cols(workspace.numel(), M, K, N)
        if room == 0:
            raise ValueError("workspace has no outlier weight region for N=%d" % N)
        end = off["total"] + int(N) * room * 2
        views["Wo"] = w[off["total"]:end].view(torch.float16)
    return views
