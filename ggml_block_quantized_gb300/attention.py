"""Attention around the block-quantized products: the binding of include/qattn.h.

A decoder layer's step in this library:
  q, k, v = the products (qgemv / qgemm)
  kv_append    rotates q and k, writes k and v to a paged cache in 4 bits
  prompt_attend  (a prompt's tokens, on the f16 rows kv_append hands out) or
  kv_attend    (a few new tokens, over the cache)
  the output product.

As in the rest of the package, nothing here computes: tensors are checked,
outputs allocated with torch where none are passed, and the C entry points
called on the current stream (or `stream`).
"""
import ctypes

__all__ = ["KVCache", "kv_cache_bytes", "kv_append", "kv_read", "kv_attend", "kv_attend_workspace_bytes",
           "prompt_attend", "rope_table", "ATTENTION_SYMBOLS"]

# every function declared in include/qattn.h
ATTENTION_SYMBOLS = ("qkv_cache_bytes", "qkv_append", "qkv_read", "qkv_attend_workspace_bytes", "qkv_attend",
                     "qattn_prompt")


class _Cache(ctypes.Structure):
    """qkv_cache."""
    _fields_ = [("data", ctypes.c_void_p), ("n_pages", ctypes.c_int64), ("n_kv_heads", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("page_size", ctypes.c_int32)]


class _AppendArgs(ctypes.Structure):
    """qkv_append_args."""
    _fields_ = [("q", ctypes.c_void_p), ("k", ctypes.c_void_p), ("v", ctypes.c_void_p),
                ("q_stride", ctypes.c_int64), ("k_stride", ctypes.c_int64), ("v_stride", ctypes.c_int64),
                ("slots", ctypes.c_void_p), ("positions", ctypes.c_void_p), ("rope", ctypes.c_void_p),
                ("q_out", ctypes.c_void_p), ("k_out", ctypes.c_void_p), ("v_out", ctypes.c_void_p),
                ("n_tok", ctypes.c_int64), ("n_heads", ctypes.c_int32), ("in_type", ctypes.c_int32),
                ("out_type", ctypes.c_int32), ("n_pos", ctypes.c_int32), ("rot_dim", ctypes.c_int32),
                ("rope_pairs", ctypes.c_int32)]


_attn = None


def _lib():
    """The loaded library with qattn.h's functions declared."""
    global _attn
    if _attn is None:
        from . import lib
        L = lib()
        i64, i32, vp, f32 = ctypes.c_int64, ctypes.c_int, ctypes.c_void_p, ctypes.c_float
        cache = ctypes.POINTER(_Cache)
        L.qkv_cache_bytes.argtypes, L.qkv_cache_bytes.restype = [i64, i32, i32, i32], i64
        L.qkv_append.argtypes, L.qkv_append.restype = [cache, ctypes.POINTER(_AppendArgs), vp], i32
        L.qkv_read.argtypes, L.qkv_read.restype = [cache, vp, i64, vp, vp, vp], i32
        L.qkv_attend_workspace_bytes.argtypes = [i32, i32, i32, i32]
        L.qkv_attend_workspace_bytes.restype = ctypes.c_size_t
        L.qkv_attend.argtypes = [cache, i32, vp, i64, vp, vp, i64, vp, vp, i64, i64, i32, i32, f32, vp,
                                 ctypes.c_size_t, vp]
        L.qkv_attend.restype = i32
        L.qattn_prompt.argtypes = [vp, i64, vp, i64, vp, i64, i32, vp, vp, i64, i64, i32, i32, i32, f32, vp]
        L.qattn_prompt.restype = i32
        _attn = L
    return _attn


# ------------------------------------------------------------ helpers
import torch  # noqa: E402

_TYPE = {torch.float32: 0, torch.float16: 1}  # QG_F32, QG_F16


def _check(st, where):
    if st != 0:
        from . import QGError
        raise QGError(st, where)


def _refuse(t, device, name, dtypes):
    """Raises for what every tensor argument must be; returns where t is that."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.dtype not in dtypes:
        raise TypeError(f"{name} must be {' or '.join(map(str, dtypes))}, got {t.dtype}")
    if t.get_device() != device:
        raise ValueError(f"{name} is on cuda:{t.get_device()}, not on cuda:{device}")


# The checks below ask once for what nearly every call passes, and look for the
# reason of a refusal only then: a step of few tokens is as long as its host code.
# (A CPU tensor's get_device() is -1; what is no tensor has none.)
def _on(t, device, name, dtype):
    """The address of t, a contiguous tensor of `dtype` on `device`."""
    try:
        if t.dtype is dtype and t.get_device() == device and t.is_contiguous():
            return t.data_ptr()
    except AttributeError:
        pass
    _refuse(t, device, name, (dtype,))
    raise ValueError(f"{name} must be contiguous")


def _rows(t, device, name, head_dim, dtypes):
    """(address, stride from token to token, tokens, heads) of [tokens, heads,
    head_dim] with contiguous heads; the tokens may lie apart."""
    try:
        n, heads, d = t.shape
        if d == head_dim and t.dtype in dtypes and t.get_device() == device:
            if t.is_contiguous():
                return t.data_ptr(), heads * d, n, heads
            stride = t.stride()
            if stride[2] == 1 and (stride[1] == d or heads == 1):
                return t.data_ptr(), stride[0] if n > 1 else heads * d, n, heads
    except (AttributeError, ValueError):
        pass
    _refuse(t, device, name, dtypes)
    if t.dim() != 3 or t.shape[2] != head_dim:
        raise ValueError(f"{name} must be [tokens, heads, {head_dim}], got {list(t.shape)}")
    raise ValueError(f"{name}: the heads of a token must be contiguous")


def _out(t, shape, dtypes, device, name):
    """The address of t, contiguous, of `shape` and one of `dtypes`."""
    try:
        if t.shape == shape and t.dtype in dtypes and t.get_device() == device and t.is_contiguous():
            return t.data_ptr()
    except AttributeError:
        pass
    _refuse(t, device, name, dtypes)
    raise ValueError(f"{name} must be contiguous {list(shape)}, got {list(t.shape)}")


def _place(t, name):
    """The device index of t, which must be the current device: the C calls
    plan for and launch on that one."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    device = t.get_device()
    if device != torch._C._cuda_getDevice():
        raise ValueError(f"{name} is not on the current CUDA device")
    return device


def _new(shape, dtype, device, stream):
    """A tensor that work on `stream` may use at once: its memory is that stream's own. (What torch hands out for the
    current stream may still be in use there by work enqueued before.) The current stream, where the caller goes on,
    may use it, too: torch hands the memory out again only after that."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        t = torch.empty(shape, dtype=dtype, device=device)
    t.record_stream(torch.cuda.current_stream(device))
    return t


def _stream(stream, device):
    """The stream's handle; the current stream's without building its object (2.8 us on the host)."""
    return torch._C._cuda_getCurrentRawStream(device) if stream is None else stream.cuda_stream


# ------------------------------------------------------------ the cache
def kv_cache_bytes(n_pages: int, n_kv_heads: int, head_dim: int, page_size: int) -> int:
    return int(_lib().qkv_cache_bytes(n_pages, n_kv_heads, head_dim, page_size))


def _pages(n_bytes, n_kv_heads, head_dim, page_size):
    """How many pages a cache of n_bytes has."""
    page = n_kv_heads * (page_size // 16) * 18 * head_dim  # (as kv_cache_bytes has it)
    n_pages = n_bytes // page if page > 0 else 0
    if kv_cache_bytes(n_pages, n_kv_heads, head_dim, page_size) == n_bytes:
        return n_pages
    if kv_cache_bytes(1, n_kv_heads, head_dim, page_size) < 0:
        raise ValueError(f"no cache of {n_kv_heads} heads of {head_dim} in pages of {page_size}: heads of 64 or 128, "
                         "pages of a multiple of 16 tokens")
    if n_bytes % page:
        raise ValueError(f"data holds {n_bytes} bytes, not a number of pages of {page}")
    raise ValueError(f"data holds {n_pages} pages of {page_size} tokens: a cache has at most 2^31 - 1 tokens")


class KVCache:
    """A paged cache of keys and values held in 4 bits (the layout of
    qkv_cache in include/qattn.h) over `data`, a uint8 CUDA tensor whose size
    says how many pages it has. Allocates and keeps nothing else."""
    __slots__ = ("n_kv_heads", "head_dim", "page_size", "n_pages", "data", "device", "c", "ref")

    def __init__(self, n_kv_heads: int, head_dim: int, page_size: int, data):
        if not isinstance(data, torch.Tensor) or not data.is_cuda or data.dtype != torch.uint8:
            raise TypeError("data must be a uint8 CUDA tensor")
        if not data.is_contiguous():
            raise ValueError("data must be contiguous")
        n_pages = _pages(data.numel(), n_kv_heads, head_dim, page_size)
        self.n_kv_heads, self.head_dim, self.page_size, self.n_pages = n_kv_heads, head_dim, page_size, n_pages
        self.data, self.device = data, data.get_device()
        self.c = _Cache(data.data_ptr(), n_pages, n_kv_heads, head_dim, page_size)
        self.ref = ctypes.byref(self.c)

    @classmethod
    def empty(cls, n_pages: int, n_kv_heads: int, head_dim: int, page_size: int = 64, device="cuda"):
        """A cache over new, uninitialised memory."""
        n = kv_cache_bytes(n_pages, n_kv_heads, head_dim, page_size)
        if n < 0:
            raise ValueError(f"no cache of {n_pages} pages of {page_size}, {n_kv_heads} heads of {head_dim}")
        return cls(n_kv_heads, head_dim, page_size, torch.empty(n, dtype=torch.uint8, device=device))


def rope_table(n_pos: int, rot_dim: int, base: float = 10000.0, device="cuda"):
    """cos and sin of position * base^(-2 i / rot_dim), f32 [n_pos, rot_dim/2, 2],
    computed in 64 bits: the `rope` of kv_append. Scaled or stretched
    rotations are tables of the caller's own."""
    half = rot_dim // 2
    freq = float(base) ** (-torch.arange(half, dtype=torch.float64) / half)
    angle = torch.arange(n_pos, dtype=torch.float64)[:, None] * freq
    return torch.stack([angle.cos(), angle.sin()], -1).float().to(device)


def kv_append(cache: KVCache, k, v, slots, positions=None, rope=None, rope_pairs: bool = False, q=None, q_out=None,
              k_out=None, v_out=None, stream=None):
    """Rotates q and k by `rope` [n_pos, rot/2, 2] at `positions`, writes k and v
    [n_tok, kv heads, D] to the cache's `slots` (int32; < 0: not cached) in 4
    bits, the rotated q to q_out (allocated if q is given and q_out is not, in
    k_out's type or else q's), and the rotated k and v to k_out and v_out where
    given. Inputs float32 or float16, of one type; outputs likewise. Returns q_out."""
    device = _place(k, "k")
    if cache.device != device:
        raise ValueError(f"the cache is on cuda:{cache.device}, not on cuda:{device}")
    d, t = cache.head_dim, k.dtype
    k_ptr, k_stride, n, n_kv = _rows(k, device, "k", d, _TYPE)
    v_ptr, v_stride, n_v, n_kv_v = _rows(v, device, "v", d, (t,))
    if n_kv != cache.n_kv_heads or n_kv_v != n_kv or n_v != n:
        raise ValueError(f"k and v must be [tokens, {cache.n_kv_heads}, {d}]")
    if slots.shape != (n,):
        raise ValueError(f"slots must be [{n}]")
    slots_ptr = _on(slots, device, "slots", torch.int32)
    q_ptr = q_stride = heads = n_pos = rot = 0
    rope_ptr = pos_ptr = None
    if q is not None:
        q_ptr, q_stride, n_q, heads = _rows(q, device, "q", d, (t,))
        if n_q != n or heads < 1 or heads % n_kv:
            raise ValueError(f"q must be [{n}, a multiple of {cache.n_kv_heads}, {d}]")
        if q_out is None:
            q_out = _new(q.shape, (k_out if k_out is not None else q).dtype, q.device, stream)
    elif q_out is not None:
        raise ValueError("q_out without q")
    if rope is not None:
        if positions is None:
            raise ValueError("rope needs positions")
        rope_ptr = _on(rope, device, "rope", torch.float32)
        shape = rope.shape
        if len(shape) != 3 or shape[2] != 2 or shape[1] % 4 or not 4 <= shape[1] <= d // 2:
            raise ValueError(f"rope must be [positions, pairs, 2], pairs a multiple of 4 up to {d // 2}")
        n_pos, rot = shape[0], 2 * shape[1]
        if n > 0 and n_pos == 0:  # (it has no address, and the C call would take it for no rotation)
            raise ValueError("rope holds no position")
        if positions.shape != (n,):
            raise ValueError(f"positions must be [{n}]")
        pos_ptr = _on(positions, device, "positions", torch.int32)
    out_t = q_out_ptr = k_out_ptr = v_out_ptr = None
    if q_out is not None:
        q_out_ptr, out_t = _out(q_out, (n, heads, d), _TYPE, device, "q_out"), q_out.dtype
    if k_out is not None:
        k_out_ptr, out_t = _out(k_out, (n, n_kv, d), _TYPE if out_t is None else (out_t,), device, "k_out"), k_out.dtype
    if v_out is not None:
        v_out_ptr, out_t = _out(v_out, (n, n_kv, d), _TYPE if out_t is None else (out_t,), device, "v_out"), v_out.dtype
    args = _AppendArgs(q_ptr, k_ptr, v_ptr, q_stride, k_stride, v_stride, slots_ptr, pos_ptr, rope_ptr, q_out_ptr,
                       k_out_ptr, v_out_ptr, n, heads, _TYPE[t], _TYPE[out_t or t], n_pos, rot, 1 if rope_pairs else 0)
    st = _lib().qkv_append(cache.ref, ctypes.byref(args), _stream(stream, device))
    if st:
        _check(st, "kv_append")
    return q_out


def kv_read(cache: KVCache, slots, k_out=None, v_out=None, stream=None):
    """The values of the cache's rows `slots`: float32 (k, v), each [n, kv heads, D];
    zeros for a slot < 0. Both are allocated if neither is given; one given
    alone is read alone."""
    device = _place(slots, "slots")
    if cache.device != device:
        raise ValueError(f"the cache is on cuda:{cache.device}, not on cuda:{device}")
    slots_ptr = _on(slots, device, "slots", torch.int32)
    if slots.dim() != 1:
        raise ValueError("slots must be [n]")
    shape = (slots.shape[0], cache.n_kv_heads, cache.head_dim)
    if k_out is None and v_out is None:
        k_out, v_out = (_new(shape, torch.float32, slots.device, stream) for _ in range(2))
    f32 = (torch.float32,)
    st = _lib().qkv_read(cache.ref, slots_ptr, shape[0],
                         _out(k_out, shape, f32, device, "k_out") if k_out is not None else None,
                         _out(v_out, shape, f32, device, "v_out") if v_out is not None else None, _stream(stream, device))
    if st:
        _check(st, "kv_read")
    return k_out, v_out


# ------------------------------------------------------------ attention
def kv_attend_workspace_bytes(cache: KVCache, n_heads: int, max_q_len: int = 1) -> int:
    return int(_lib().qkv_attend_workspace_bytes(cache.head_dim, cache.n_kv_heads, n_heads, max_q_len))


def kv_attend(cache: KVCache, q, table, lengths, q_offsets=None, max_q_len: int = 1, scale=None, out=None,
              workspace=None, stream=None):
    """Attention of new tokens q [n_tok, heads, D] (float32 or float16, rotated)
    over the cache. Sequence s holds lengths[s] tokens (int32, the new ones
    included) in the pages table[s] (int32 [n_seq, pages]); its queries are rows
    q_offsets[s] .. q_offsets[s + 1] - 1 (int32 [n_seq + 1], at most max_q_len a
    sequence), or row s where q_offsets is None, and belong to its last tokens:
    each sees the tokens up to its own. scale: 1 / sqrt(D) by default. Returns
    out [n_tok, heads, D] in q's type; zeros for a row that sees nothing. Rows
    in no sequence are not written, nor those of a sequence with more queries
    than max_q_len (device_error() is 4 then)."""
    device = _place(q, "q")
    if cache.device != device:
        raise ValueError(f"the cache is on cuda:{cache.device}, not on cuda:{device}")
    d = cache.head_dim
    q_ptr, q_stride, n_tok, heads = _rows(q, device, "q", d, _TYPE)
    if heads < 1 or heads % cache.n_kv_heads:
        raise ValueError(f"q must have a multiple of {cache.n_kv_heads} heads")
    table_ptr = _on(table, device, "table", torch.int32)
    len_ptr = _on(lengths, device, "lengths", torch.int32)
    shape, off_ptr = table.shape, None
    if len(shape) != 2 or lengths.shape != shape[:1]:
        raise ValueError("table must be [sequences, pages] and lengths [sequences]")
    n_seq, pages = shape
    if q_offsets is not None:
        off_ptr = _on(q_offsets, device, "q_offsets", torch.int32)
        if q_offsets.shape != (n_seq + 1,):
            raise ValueError(f"q_offsets must be [{n_seq + 1}]")
    elif n_tok != n_seq:
        raise ValueError(f"q holds {n_tok} tokens for {n_seq} sequences: q_offsets is needed")
    if out is None:
        out = _new(q.shape, q.dtype, q.device, stream)
    out_ptr = _out(out, (n_tok, heads, d), (q.dtype,), device, "out")
    L = _lib()
    if workspace is None:
        need = L.qkv_attend_workspace_bytes(d, cache.n_kv_heads, heads, max_q_len)
        workspace = _new((max(need, 16),), torch.uint8, q.device, stream)
    ws_ptr = _on(workspace, device, "workspace", torch.uint8)
    st = L.qkv_attend(cache.ref, _TYPE[q.dtype], q_ptr, q_stride, out_ptr, table_ptr, pages, len_ptr, off_ptr,
                      n_seq, n_tok, heads, max_q_len, d ** -0.5 if scale is None else scale, ws_ptr,
                      workspace.numel(), _stream(stream, device))
    if st:
        _check(st, "kv_attend")
    return out


def prompt_attend(q, k, v, offsets, scale=None, out=None, stream=None):
    """Causal attention over packed prompts: sequence s is rows offsets[s] ..
    offsets[s + 1] - 1 (int32 [n_seq + 1]) of q [n_tok, heads, D] and of k and
    v [n_tok, kv heads, D], float16; each row sees the rows of its sequence up
    to its own. scale: 1 / sqrt(D) by default. Returns out [n_tok, heads, D],
    float16 (or float32 if such an `out` is passed); rows in no sequence are
    not written."""
    device = _place(q, "q")
    d, f16 = q.shape[-1] if q.dim() else 0, (torch.float16,)
    q_ptr, q_stride, n_tok, heads = _rows(q, device, "q", d, f16)
    k_ptr, k_stride, n_k, n_kv = _rows(k, device, "k", d, f16)
    v_ptr, v_stride, n_v, n_kv_v = _rows(v, device, "v", d, f16)
    if n_k != n_tok or n_v != n_k or n_kv_v != n_kv or n_kv < 1 or heads < 1 or heads % n_kv:
        raise ValueError("k and v must be [tokens, kv heads, D], q [tokens, a multiple of the kv heads, D]")
    off_ptr = _on(offsets, device, "offsets", torch.int32)
    ends = offsets.shape
    if len(ends) != 1 or ends[0] < 1:
        raise ValueError("offsets must be [sequences + 1]")
    if out is None:
        out = _new(q.shape, torch.float16, q.device, stream)
    out_ptr = _out(out, (n_tok, heads, d), _TYPE, device, "out")
    st = _lib().qattn_prompt(q_ptr, q_stride, k_ptr, k_stride, v_ptr, v_stride, _TYPE[out.dtype], out_ptr, off_ptr,
                             ends[0] - 1, n_tok, heads, n_kv, d, d ** -0.5 if scale is None else scale,
                             _stream(stream, device))
    if st:
        _check(st, "prompt_attend")
    return out
