"""The operators of a transformer step between the DF11 matrix products.

Thin wrappers, one to one over the C entry points in ``include/df11.h``
("decoding step"): they check what the C calls cannot see (tensor types,
sizes, devices) and marshal arguments.  Every call enqueues on ``stream``
(default: torch's current stream of the output's device) and allocates
nothing.  Index tensors are int32; row strides are free, the last dimension is
contiguous.
"""
from __future__ import annotations

import ctypes

import torch

try:  # the current stream's handle without building a stream object
    from torch._C import _cuda_getCurrentRawStream
except ImportError:
    def _cuda_getCurrentRawStream(device: int) -> int:
        return torch.cuda.current_stream(device).cuda_stream

_U32, _U64, _F, _P = ctypes.c_uint32, ctypes.c_uint64, ctypes.c_float, ctypes.c_void_p

BF16, F32, E4M3 = 0, 1, 2
_TYPES = {torch.bfloat16: BF16, torch.float32: F32}
PAGE_TOKENS = (16, 32, 64, 128, 256)
HEAD_DIMS = (64, 128, 256)


class KvCacheDesc(ctypes.Structure):
    _fields_ = [("pages", _P), ("bytes", _U64), ("page_stride", _U64), ("head_stride", _U64),
                ("n_pages", _U32), ("kv_heads", _U32), ("dim", _U32), ("page_tokens", _U32),
                ("status", _P)]


_CACHE = ctypes.POINTER(KvCacheDesc)
_SIGNATURES = {
    "df11_add_rms_norm": [_P, _U32, _U64, _P, _P, _U32, _U64, _U64, _P, _U32, _F, _P, _U32, _U64,
                          _P, _U32, _U32, _P],
    "df11_silu_mul": [_P, _U64, _P, _U64, _U32, _P, _U64, _U32, _U32, _P],
    "df11_logits": [_P, _U32, _U64, _P, _U64, _P, _U64, _U32, _P, _P, _P, _P, _P, _P, _P, _U64,
                    _U32, _P, _U64, _U32, _U32, _P],
    "df11_rope_append": [_CACHE, _P, _U64, _U64, _P, _U64, _U64, _P, _U64, _U64, _U32, _U32, _P,
                         _U64, _P, _U64, _U32, _U32, _U32, _P, _P, _P, _U64, _U64, _U32, _P],
    "df11_kv_read": [_CACHE, _P, _P, _U64, _U64, _P, _U64, _U64, _U32, _P],
    "df11_attention": [_CACHE, _P, _U64, _U64, _U32, _U32, _P, _P, _U32, _P, _U64, _U32, _U32,
                       _U32, _F, _U32, _U32, _P, _U64, _U64, _P, _P, _U64, _P],
}


_entry = None  # the loaded library with the signatures above


def _lib():
    global _entry
    if _entry is None:
        from . import _load
        lib = _load()
        for name, args in _SIGNATURES.items():
            fn = getattr(lib, name)
            fn.argtypes, fn.restype = args, ctypes.c_int
        lib.df11_kv_block_bytes.argtypes = [_U32, _U32]
        lib.df11_kv_block_bytes.restype = _U64
        lib.df11_attention_workspace_bytes.argtypes = [_CACHE, _U32, _U32, _U32, _U32, _U32]
        lib.df11_attention_workspace_bytes.restype = _U64
        _entry = lib
    return _entry


def _fail(fn: str, status: int) -> None:
    from . import Df11Error
    raise Df11Error(fn, status)


# A call's checks are host work before every launch, so each tensor is looked
# at once, in one helper: about half a microsecond apiece, where a launch takes 3
# to 4.  (torch.cuda.current_stream alone would add 2.)

def _stream(stream, device: int) -> int:
    return _cuda_getCurrentRawStream(device) if stream is None else stream.cuda_stream


def _too_large(name: str, *sizes: int) -> ValueError:
    """The C calls count in 32 bits, and ctypes would cut what does not fit
    (each call looks at all its sizes at once)."""
    return ValueError(f"{name}: sizes must be below 2**32 and not negative, not {sizes}")


def _device(name: str, t) -> int:
    dev = t.get_device()
    if dev < 0:
        raise ValueError(f"{name} must be on the GPU")
    return dev


def _type_of(name: str, t) -> int:
    kind = _TYPES.get(t.dtype)
    if kind is None:
        raise ValueError(f"{name} must be bfloat16 or float32, not {t.dtype}")
    return kind


def _matrix(name: str, t, dev: int, rows: int, cols: int) -> int:
    """The row stride (in elements) of a [rows, cols] matrix with contiguous
    rows on GPU dev; a single row may carry any stride."""
    shape, stride = t.shape, t.stride()
    if len(shape) != 2 or shape[0] != rows or shape[1] != cols or t.get_device() != dev \
            or (stride[1] != 1 and cols > 1):
        raise ValueError(f"{name} must be a [{rows}, {cols}] tensor with contiguous rows on GPU {dev}; "
                         f"it has shape {tuple(shape)}, strides {stride}, device {t.device}")
    return stride[0] if rows > 1 else cols


def _vector(name: str, t, dev: int, n: int, dtype) -> int:
    """The address of a contiguous vector."""
    if t.dtype is not dtype or t.numel() != n or t.dim() != 1 or t.get_device() != dev \
            or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of {n} elements on GPU {dev}")
    return t.data_ptr()


def _heads(name: str, t, dev: int, tokens: int, heads: int, dim: int) -> tuple[int, int]:
    """Token and head strides of a [tokens, heads, dim] tensor with contiguous
    heads; those of a single token or head may be anything."""
    shape, stride = t.shape, t.stride()
    if len(shape) != 3 or shape[0] != tokens or shape[1] != heads or shape[2] != dim \
            or t.get_device() != dev or stride[2] != 1:
        raise ValueError(f"{name} must be a [{tokens}, {heads}, {dim}] tensor with contiguous heads on "
                         f"GPU {dev}; it has shape {tuple(shape)}, strides {stride}, device {t.device}")
    head = stride[1] if heads > 1 else dim
    return (stride[0] if tokens > 1 else heads * dim), head


def df11_add_rms_norm(x, weight, out, eps: float, residual=None, residual_out=None, scales=None,
                      stream=None) -> None:
    """h = x + residual, residual_out = h, out = h / sqrt(mean(h^2) + eps) * weight
    for the rows of x [rows, width] (bfloat16 or float32).  residual and
    residual_out may be one tensor (updated in place; residual_out None means
    that).  out: bfloat16, or float8_e4m3fn with ``scales`` [rows] float32,
    where out * scales[row] stands for the result."""
    dev = _device("x", x)
    if x.dim() != 2:
        raise ValueError("x must be [rows, width]")
    rows, width = x.shape
    xs, xt = _matrix("x", x, dev, rows, width), _type_of("x", x)
    wt = _type_of("weight", weight)
    wp = _vector("weight", weight, dev, width, weight.dtype)
    os = _matrix("out", out, dev, rows, width)
    sp = None
    if out.dtype is torch.bfloat16:
        ot = BF16
        if scales is not None:
            raise ValueError("scales go with a float8_e4m3fn output")
    elif out.dtype is torch.float8_e4m3fn:
        ot = E4M3
        if scales is None:
            raise ValueError("a float8_e4m3fn output needs scales")
        sp = _vector("scales", scales, dev, rows, torch.float32)
    else:
        raise ValueError(f"out must be bfloat16 or float8_e4m3fn, not {out.dtype}")
    rp = rop = None
    rt = rs = ros = 0
    if residual is not None:
        rs, rt, rp = _matrix("residual", residual, dev, rows, width), _type_of("residual", residual), \
            residual.data_ptr()
        ros, rop = rs, rp
        if residual_out is not None:
            ros, rop = _matrix("residual_out", residual_out, dev, rows, width), residual_out.data_ptr()
            if residual_out.dtype is not residual.dtype:
                raise ValueError("residual and residual_out must have one type")
    elif residual_out is not None:
        raise ValueError("residual_out goes with residual")
    if (rows | width) >> 32:
        raise _too_large("x", rows, width)
    status = _lib().df11_add_rms_norm(x.data_ptr(), xt, xs, rp, rop, rt, rs, ros, wp, wt, eps,
                                      out.data_ptr(), ot, os, sp, rows, width, _stream(stream, dev))
    if status:
        _fail("df11_add_rms_norm", status)


def df11_silu_mul(gate, up, out, stream=None) -> None:
    """out = gate / (1 + exp(-gate)) * up for [rows, width] tensors: gate and up
    bfloat16 or float32 (one type), out bfloat16."""
    dev = _device("gate", gate)
    if gate.dim() != 2:
        raise ValueError("gate must be [rows, width]")
    rows, width = gate.shape
    gs, us = _matrix("gate", gate, dev, rows, width), _matrix("up", up, dev, rows, width)
    os, kind = _matrix("out", out, dev, rows, width), _type_of("gate", gate)
    if up.dtype is not gate.dtype or out.dtype is not torch.bfloat16:
        raise ValueError("gate and up must have one type and out be bfloat16")
    if (rows | width) >> 32:
        raise _too_large("gate", rows, width)
    status = _lib().df11_silu_mul(gate.data_ptr(), gs, up.data_ptr(), us, kind, out.data_ptr(), os,
                                  rows, width, _stream(stream, dev))
    if status:
        _fail("df11_silu_mul", status)


def df11_logits(logits, out, tokens=None, lens=None, prompt_lens=None, repetition=None,
                frequency=None, presence=None, bias_ids=None, bias_values=None, mask=None,
                stream=None) -> None:
    """Penalties, bias and mask on logits [rows, vocab] (bfloat16 or float32)
    into out (float32; may be logits itself).  tokens [rows, history] int32
    with lens [rows]: each row's tokens, those from prompt_lens[row] on
    generated; repetition, frequency, presence [rows] float32; bias_ids
    [rows, n] int32 and bias_values [rows, n] float32 (ids outside the
    vocabulary are skipped, of an id listed twice the last value counts); mask [rows, words] int32, bit id % 32 of word
    id / 32 set where the id is allowed."""
    dev = _device("logits", logits)
    if logits.dim() != 2:
        raise ValueError("logits must be [rows, vocab]")
    rows, vocab = logits.shape
    ls, kind = _matrix("logits", logits, dev, rows, vocab), _type_of("logits", logits)
    os = _matrix("out", out, dev, rows, vocab)
    if out.dtype is not torch.float32:
        raise ValueError("out must be float32")
    i32, f32 = torch.int32, torch.float32
    tp = lp = pp = rp = fp = sp = ip = vp = mp = None
    history = ts = n_bias = bs = ms = 0
    if tokens is not None:
        if tokens.dtype is not i32 or tokens.dim() != 2 or lens is None:
            raise ValueError("tokens must be int32 [rows, history], with lens")
        history = tokens.shape[1]
        ts, tp = _matrix("tokens", tokens, dev, rows, history), tokens.data_ptr()
        lp = _vector("lens", lens, dev, rows, i32)
        if prompt_lens is not None:
            pp = _vector("prompt_lens", prompt_lens, dev, rows, i32)
    elif lens is not None or prompt_lens is not None:
        raise ValueError("lens and prompt_lens go with tokens")
    if repetition is not None:
        rp = _vector("repetition", repetition, dev, rows, f32)
    if frequency is not None:
        fp = _vector("frequency", frequency, dev, rows, f32)
    if presence is not None:
        sp = _vector("presence", presence, dev, rows, f32)
    if bias_ids is not None and bias_values is not None:
        if bias_ids.dtype is not i32 or bias_values.dtype is not f32 or bias_ids.dim() != 2:
            raise ValueError("bias_ids must be int32 [rows, n], bias_values float32")
        n_bias = bias_ids.shape[1]
        bs = _matrix("bias_ids", bias_ids, dev, rows, n_bias)
        if _matrix("bias_values", bias_values, dev, rows, n_bias) != bs:
            raise ValueError("bias_ids and bias_values must have one row stride")
        ip, vp = bias_ids.data_ptr(), bias_values.data_ptr()
    elif bias_ids is not None or bias_values is not None:
        raise ValueError("bias_ids and bias_values go together")
    if mask is not None:
        if mask.dtype is not i32 or mask.dim() != 2 or mask.shape[1] * 32 < vocab:
            raise ValueError(f"mask must be int32 [{rows}, at least {-(-vocab // 32)}]")
        ms, mp = _matrix("mask", mask, dev, rows, mask.shape[1]), mask.data_ptr()
    if (rows | vocab | history | n_bias) >> 32:
        raise _too_large("logits", rows, vocab, history, n_bias)
    status = _lib().df11_logits(logits.data_ptr(), kind, ls, out.data_ptr(), os, tp, ts, history, lp,
                                pp, rp, fp, sp, ip, vp, bs, n_bias, mp, ms, rows, vocab,
                                _stream(stream, dev))
    if status:
        _fail("df11_logits", status)


# ------------------------------------------------------------ the 4-bit cache

def kv_block_bytes(page_tokens: int, dim: int) -> int:
    """Bytes of one page of one key head (0 for sizes the cache does not have)."""
    if (page_tokens | dim) >> 32:
        return 0
    return int(_lib().df11_kv_block_bytes(page_tokens, dim))


class KvCache:
    """A paged cache of keys and values in 4 bits over a uint8 GPU tensor
    ``pages`` [n_pages, kv_heads, block bytes] (blocks contiguous, strides free
    multiples of 16), e.g. one layer's part of a larger tensor.  ``status``:
    optional int32 tensor of one element that the kernels add to when an index
    is out of range.  Handing out pages is the caller's."""

    def __init__(self, pages, dim: int, page_tokens: int, status=None):
        if pages.dtype != torch.uint8 or pages.dim() != 3 or not pages.is_cuda \
                or pages.stride(2) != 1:
            raise ValueError("pages must be a uint8 GPU tensor [n_pages, kv_heads, block bytes] "
                             "with contiguous blocks")
        block = kv_block_bytes(page_tokens, dim)
        if block == 0 or pages.shape[2] != block:
            raise ValueError(f"a block of {page_tokens} tokens and {dim} channels has {block} "
                             f"bytes, pages has {pages.shape[2]}")
        if status is not None and (status.dtype != torch.int32 or status.numel() < 1
                                   or status.device != pages.device):
            raise ValueError("status must be an int32 tensor on the pages' device")
        self.pages, self.status, self.device = pages, status, pages.get_device()
        n_pages, kv_heads = pages.shape[:2]
        if (n_pages | kv_heads) >> 32:
            raise _too_large("pages", n_pages, kv_heads)
        # a single head or page may carry any stride
        head = pages.stride(1) if kv_heads > 1 else block
        page = pages.stride(0) if n_pages > 1 else head * kv_heads
        self.desc = KvCacheDesc(
            pages.data_ptr(), page * (n_pages - 1) + head * (kv_heads - 1) + block, page, head,
            n_pages, kv_heads, dim, page_tokens, None if status is None else status.data_ptr())
        self._ref = ctypes.byref(self.desc)
        self.n_pages, self.kv_heads, self.dim, self.page_tokens = n_pages, kv_heads, dim, page_tokens

    @classmethod
    def empty(cls, n_pages: int, kv_heads: int, dim: int, page_tokens: int = 64, device="cuda",
              status=None) -> "KvCache":
        """A cache over newly allocated pages (contents undefined)."""
        block = kv_block_bytes(page_tokens, dim)
        if block == 0:
            raise ValueError(f"page_tokens must be one of {PAGE_TOKENS} and dim one of {HEAD_DIMS}")
        return cls(torch.empty(n_pages, kv_heads, block, dtype=torch.uint8, device=device), dim,
                   page_tokens, status)


def df11_rope_append(cache: KvCache, q, k, v, cos, sin, positions, slots, q_out,
                     adjacent: bool = False, stream=None) -> None:
    """Turn q [tokens, heads, dim] and k [tokens, kv_heads, dim] by their rotary
    positions, write the queries to q_out (bfloat16) and k and v to the cache at
    ``slots`` (negative: not stored).  q, k, v: bfloat16 or float32 (one type),
    e.g. views of a product's rows.  cos, sin: float32 [positions, rot / 2]; the
    first rot channels are turned, in halves or with ``adjacent`` in pairs
    (2i, 2i + 1)."""
    if q.dim() != 3 or cos.dim() != 2:
        raise ValueError("q must be [tokens, heads, dim] and cos [positions, rot / 2]")
    dev, dim, kv_heads = cache.device, cache.dim, cache.kv_heads
    tokens, heads = q.shape[0], q.shape[1]
    n_pos, half = cos.shape
    if (tokens | heads | n_pos | 2 * half) >> 32:
        raise _too_large("q and cos", tokens, heads, n_pos, 2 * half)
    qs, qh = _heads("q", q, dev, tokens, heads, dim)
    ks, kh = _heads("k", k, dev, tokens, kv_heads, dim)
    vs, vh = _heads("v", v, dev, tokens, kv_heads, dim)
    os, oh = _heads("q_out", q_out, dev, tokens, heads, dim)
    kind = _type_of("k", k)
    if q.dtype is not k.dtype or v.dtype is not k.dtype or q_out.dtype is not torch.bfloat16:
        raise ValueError("q, k and v must have one type and q_out be bfloat16")
    cs, ss = _matrix("cos", cos, dev, n_pos, half), _matrix("sin", sin, dev, n_pos, half)
    if cos.dtype is not torch.float32 or sin.dtype is not torch.float32:
        raise ValueError("cos and sin must be float32")
    pp = _vector("positions", positions, dev, tokens, torch.int32)
    sp = _vector("slots", slots, dev, tokens, torch.int32)
    status = _lib().df11_rope_append(
        cache._ref, q.data_ptr(), qs, qh, k.data_ptr(), ks, kh, v.data_ptr(), vs, vh, kind, heads,
        cos.data_ptr(), cs, sin.data_ptr(), ss, n_pos, 2 * half, adjacent, pp, sp, q_out.data_ptr(), os,
        oh, tokens, _stream(stream, dev))
    if status:
        _fail("df11_rope_append", status)


def df11_kv_read(cache: KvCache, slots, k_out, v_out, stream=None) -> None:
    """The values held at ``slots`` into k_out and v_out [tokens, kv_heads, dim]
    (bfloat16, exact)."""
    dev, tokens = cache.device, slots.shape[0]
    if tokens >> 32:
        raise _too_large("slots", tokens)
    sp = _vector("slots", slots, dev, tokens, torch.int32)
    ks, kh = _heads("k_out", k_out, dev, tokens, cache.kv_heads, cache.dim)
    vs, vh = _heads("v_out", v_out, dev, tokens, cache.kv_heads, cache.dim)
    if k_out.dtype is not torch.bfloat16 or v_out.dtype is not torch.bfloat16:
        raise ValueError("k_out and v_out must be bfloat16")
    status = _lib().df11_kv_read(cache._ref, sp, k_out.data_ptr(), ks, kh, v_out.data_ptr(), vs, vh,
                                 tokens, _stream(stream, dev))
    if status:
        _fail("df11_kv_read", status)


def df11_attention_workspace_bytes(cache: KvCache, tokens: int, heads: int, batch: int,
                                   max_queries: int, max_kv: int) -> int:
    """Workspace bytes of df11_attention for these sizes (0: none needed)."""
    if (tokens | heads | batch | max_queries | max_kv) >> 32:
        raise _too_large("workspace", tokens, heads, batch, max_queries, max_kv)
    return int(_lib().df11_attention_workspace_bytes(cache._ref, tokens, heads, batch, max_queries,
                                                     max_kv))


def df11_attention(cache: KvCache, q, q_start, kv_lens, page_table, out, max_queries: int,
                   max_kv: int, scale: float | None = None, causal: bool = True, window: int = 0,
                   lse=None, workspace=None, stream=None) -> None:
    """Attention of q [tokens, heads, dim] (bfloat16) over the cache into out:
    sequence b has queries q_start[b] .. q_start[b + 1] - 1 and kv_lens[b]
    cached tokens in the pages page_table[b]; its queries are its last tokens.
    max_queries and max_kv bound the sequences' lengths.  scale defaults to
    1 / sqrt(dim).  lse: optional float32 [tokens, heads].  workspace: a GPU
    tensor of at least df11_attention_workspace_bytes, None where that is 0."""
    if q.dim() != 3 or page_table.dim() != 2:
        raise ValueError("q must be [tokens, heads, dim] and page_table [sequences, pages]")
    dev, dim = cache.device, cache.dim
    tokens, heads = q.shape[0], q.shape[1]
    qs, qh = _heads("q", q, dev, tokens, heads, dim)
    os, oh = _heads("out", out, dev, tokens, heads, dim)
    if q.dtype is not torch.bfloat16 or out.dtype is not torch.bfloat16:
        raise ValueError("q and out must be bfloat16")
    batch, cols = page_table.shape
    if (tokens | heads | batch | cols) >> 32:
        raise _too_large("q and page_table", tokens, heads, batch, cols)
    kp = _vector("kv_lens", kv_lens, dev, batch, torch.int32)
    sp = _vector("q_start", q_start, dev, batch + 1, torch.int32)
    ts = _matrix("page_table", page_table, dev, batch, cols)
    if page_table.dtype is not torch.int32:
        raise ValueError("page_table must be int32")
    lp = wp = None
    nbytes = 0
    if lse is not None:
        if lse.dtype is not torch.float32 or _matrix("lse", lse, dev, tokens, heads) != heads:
            raise ValueError(f"lse must be a contiguous float32 tensor [{tokens}, {heads}]")
        lp = lse.data_ptr()
    for name, n in (("max_queries", max_queries), ("max_kv", max_kv), ("window", window)):
        if not 0 <= n < 1 << 31:  # (ctypes would cut what does not fit)
            raise ValueError(f"{name} must be in [0, 2**31), not {n}")
    if workspace is not None:
        if not workspace.is_contiguous() or workspace.get_device() != dev:
            raise ValueError(f"workspace must be a contiguous tensor on GPU {dev}")
        wp, nbytes = workspace.data_ptr(), workspace.numel() * workspace.element_size()
    status = _lib().df11_attention(
        cache._ref, q.data_ptr(), qs, qh, tokens, heads, sp, kp, batch, page_table.data_ptr(), ts, cols,
        max_queries, max_kv, dim ** -0.5 if scale is None else scale, causal, window, out.data_ptr(), os,
        oh, lp, wp, nbytes, _stream(stream, dev))
    if status:
        _fail("df11_attention", status)
