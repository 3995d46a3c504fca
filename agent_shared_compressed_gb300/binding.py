"""ctypes binding of include/kvpool.h -- argument marshalling only.

Every function has the C name and returns the C status (0 = KVP_OK,
negative = KVP_ERR_*); all computation happens in the CUDA library.
Arguments that the C API takes as device pointers accept a torch tensor
(its data_ptr()), a plain int address or None (NULL); the page calls, whose
kernels read as much as the counts and types say, refuse tensors that do not
hold it.  Per-layer pointer
lists accept Python sequences of the same.  `stream` accepts a
torch.cuda.Stream, a raw cudaStream_t int, or None (legacy default stream).

The library is loaded from this package's directory (built in-tree by
agent_shared_compressed_gb300.build); if it is missing, load() raises -- there
is no fallback.
"""
import ctypes as C
import os
import re
import struct

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libkvcodec.so")
HEADER = os.path.join(os.path.dirname(_PKG), "include", "kvpool.h")

KVP_OK = 0
KVP_ERR_ARG = -1
KVP_ERR_UNSUPPORTED_D = -2
KVP_ERR_ALIGN = -3
KVP_ERR_SIZE = -4
KVP_ERR_CUDA = -5
KVP_ERR_NONFINITE = -6
KVP_ERR_RANGE = -7
KVP_ERR_BITS = -8
KVP_ERR_HEADER = -9
KVP_ERR_TIMEOUT = -10
KVP_ERR_PAGE = -11
KVP_MAX_LAYERS = 512
KVP_K_PER_TENSOR = 0
KVP_K_Q8_0 = 1
KVP_PAGES_BF16 = 0
KVP_PAGES_K8V8 = 1
KVP_PAGES_K8V4 = 2
KVP_PAGES_K4V4 = 4
KVP_MAX_AXES = 4
KVP_PROMPT_MAX_SEQS = 65536
KVP_PAGES_MAX_SEQS = 4096
KVP_NOALLOC_SCRATCH_BYTES = 262144
KVP_PROBE_STORE = 0
KVP_PROBE_BULK_STORE = 1
KVP_PROBE_COPY = 2


class Shape(C.Structure):
    """kvp_shape: n_layers tensors of [n_kv_heads][n_tokens][head_dim]."""
    _fields_ = [("n_layers", C.c_int32), ("n_kv_heads", C.c_int32),
                ("head_dim", C.c_int32), ("n_tokens", C.c_int32)]

    def __repr__(self):
        return "Shape(L=%d, H=%d, d=%d, T=%d)" % (self.n_layers, self.n_kv_heads, self.head_dim, self.n_tokens)


class CardHeader(C.Structure):
    """kvp_card_header: the first 128 bytes of a CacheCard."""
    _fields_ = [("magic", C.c_uint32), ("version", C.c_uint32), ("seq_len", C.c_int32),
                ("n_layers", C.c_int32), ("n_kv_heads", C.c_int32), ("head_dim", C.c_int32),
                ("group_size", C.c_int32), ("dtype", C.c_int32), ("model_id", C.c_uint64),
                ("pos_offset", C.c_int64), ("off_bits", C.c_uint64), ("off_offsets", C.c_uint64),
                ("off_layers", C.c_uint64), ("layer_stride", C.c_uint64), ("total_bytes", C.c_uint64),
                ("error", C.c_uint32), ("reserved", C.c_uint32 * 9)]


assert C.sizeof(CardHeader) == 128


class PagesConfig(C.Structure):
    """kvp_pages_config: a container of n_pages pages of page_tokens tokens per layer."""
    _fields_ = [("n_layers", C.c_int32), ("n_kv_heads", C.c_int32), ("head_dim", C.c_int32),
                ("page_tokens", C.c_int32), ("n_pages", C.c_int32), ("format", C.c_int32)]

    def __repr__(self):
        return "PagesConfig(L=%d, H=%d, d=%d, P=%d, pages=%d, format=%d)" % (
            self.n_layers, self.n_kv_heads, self.head_dim, self.page_tokens, self.n_pages, self.format)


class PromptShape(C.Structure):
    """kvp_prompt_shape: sequences, rows of q, rows of k and v, heads, head_dim."""
    _fields_ = [("n_seqs", C.c_int32), ("n_q_tokens", C.c_int32), ("n_k_tokens", C.c_int32), ("n_q_heads", C.c_int32),
                ("n_kv_heads", C.c_int32), ("head_dim", C.c_int32)]

    def __repr__(self):
        return "PromptShape(B=%d, n=%d, keys=%d, nq=%d, H=%d, d=%d)" % (
            self.n_seqs, self.n_q_tokens, self.n_k_tokens, self.n_q_heads, self.n_kv_heads, self.head_dim)


class Rows(C.Structure):
    """kvp_rows: a bf16 [tokens][heads][head_dim] tensor with element strides.
    shape: the tensor's, where it was made from one (rows())."""
    _fields_ = [("ptr", C.c_void_p), ("token_stride", C.c_int64), ("head_stride", C.c_int64)]
    shape = None


_vp = C.c_void_p
_SIGS = {
    "kvpool_pool_bytes": (C.c_size_t, [C.POINTER(Shape)]),
    "kvpool_workspace_bytes": (C.c_size_t, [C.POINTER(Shape)]),
    "kvpool_encode": (C.c_int, [C.POINTER(Shape), C.POINTER(_vp), C.POINTER(_vp), _vp, C.c_size_t,
                                _vp, C.c_size_t, _vp]),
    "kvpool_pool_bytes_ex": (C.c_size_t, [C.POINTER(Shape), C.c_int]),
    "kvpool_encode_ex": (C.c_int, [C.POINTER(Shape), C.c_int, C.POINTER(_vp), C.POINTER(_vp), _vp, C.c_size_t,
                                   _vp, C.c_size_t, _vp]),
    "kvpool_decode_into": (C.c_int, [_vp, C.POINTER(Shape), C.c_int, C.c_int, C.c_int,
                                     C.POINTER(_vp), C.POINTER(_vp), _vp]),
    "kvpool_status": (C.c_int, [_vp, _vp]),
    "kvpool_attend_workspace_bytes": (C.c_size_t, [C.POINTER(Shape), C.c_int, C.c_int]),
    "kvpool_attend": (C.c_int, [_vp, C.POINTER(Shape), C.c_int, C.c_int, C.c_int, _vp, C.c_float, _vp, _vp, _vp,
                                C.c_size_t, _vp]),
    "kvpool_attend_lora_workspace_bytes": (C.c_size_t, [C.POINTER(Shape), C.c_int, C.c_int, C.c_int]),
    "kvpool_attend_lora": (C.c_int, [_vp, C.POINTER(Shape), C.c_int, C.c_int, C.c_int, _vp, C.c_float, C.c_int, _vp,
                                     _vp, _vp, _vp, _vp, C.c_size_t, _vp]),
    "kvpool_encode_noalloc": (C.c_int, [C.POINTER(Shape), C.POINTER(_vp), C.POINTER(_vp), _vp, C.c_size_t, _vp]),
    "cachecard_bytes": (C.c_size_t, [C.POINTER(Shape), C.POINTER(C.c_uint8)]),
    "cachecard_pack": (C.c_int, [C.POINTER(Shape), C.c_uint64, C.c_int64, _vp, C.POINTER(_vp),
                                 C.POINTER(_vp), _vp, C.c_size_t, _vp]),
    "cachecard_read_header": (C.c_int, [_vp, C.POINTER(CardHeader), _vp]),
    "cachecard_unpack": (C.c_int, [_vp, C.POINTER(CardHeader), C.POINTER(_vp), C.POINTER(_vp), _vp]),
    "cachecard_unpack_at": (C.c_int, [_vp, C.POINTER(CardHeader), C.c_int64, C.POINTER(C.c_float), C.POINTER(_vp),
                                      C.POINTER(_vp), _vp]),
    "cachecard_status": (C.c_int, [_vp, _vp]),
    "kvpages_bytes": (C.c_size_t, [_vp]),
    "kvpages_init": (C.c_int, [_vp, _vp, C.c_size_t, _vp]),
    "kvpages_append": (C.c_int, [_vp, _vp, C.c_int, C.c_int, C.c_int, _vp, _vp, _vp, _vp, _vp, _vp, _vp, C.c_float,
                                 C.c_int, _vp, _vp, _vp, _vp, _vp]),
    "kvpages_append_axes": (C.c_int, [_vp, _vp, C.c_int, C.c_int, C.c_int, _vp, _vp, _vp, _vp, _vp, C.c_int, _vp, _vp, _vp,
                                      C.c_float, C.c_int, _vp, _vp, _vp, _vp, _vp]),
    "kvpages_read": (C.c_int, [_vp, _vp, C.c_int, C.c_int, _vp, C.c_int, _vp, C.c_int, _vp, _vp, _vp]),
    "kvpages_attend_workspace_bytes": (C.c_size_t, [_vp, C.c_int, C.c_int, C.c_int]),
    "kvpages_attend": (C.c_int, [_vp, _vp, C.c_int, C.c_int, C.c_int, C.c_int, _vp, C.c_float, _vp, C.c_int, _vp, _vp,
                                 _vp, _vp, _vp, _vp, C.c_size_t, _vp]),
    "kvpages_attend_window": (C.c_int, [_vp, _vp, C.c_int, C.c_int, C.c_int, C.c_int, _vp, C.c_float, C.c_int, C.c_int, _vp,
                                        C.c_int, _vp, _vp, _vp, _vp, _vp, _vp, C.c_size_t, _vp]),
    "kvpages_status": (C.c_int, [_vp, _vp]),
    "kvprompt_workspace_bytes": (C.c_size_t, [_vp]),
    "kvprompt_attend": (C.c_int, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, C.c_float, C.c_int, C.c_int, _vp, _vp, _vp, _vp, _vp, _vp,
                                  C.c_size_t, _vp]),
    "kvprompt_status": (C.c_int, [_vp, _vp]),
    "kvp_strerror": (C.c_char_p, [C.c_int]),
    "kvp_launch_count": (C.c_uint64, []),
    "kvp_bandwidth_probe": (C.c_int, [C.c_int, _vp, _vp, C.c_size_t, _vp]),
    "kvp_test_fail_next_encode": (C.c_int, [C.c_int, C.c_uint32]),
    "kvp_test_limit_next_attend": (C.c_int, [C.c_uint32]),
    "kvp_test_limit_next_unpack": (C.c_int, [C.c_uint32]),
    "kvp_test_limit_next_pages_attend": (C.c_int, [C.c_uint32]),
    "kvp_test_limit_next_pages_attend_lanes": (C.c_int, [C.c_uint32, C.c_uint32]),
    "kvp_test_limit_next_prompt": (C.c_int, [C.c_uint32]),
}

_lib = None


def load(path=None):
    """Load the CUDA codec library (raises if it has not been built)."""
    global _lib
    if _lib is not None and path is None:
        return _lib
    p = path or LIB_PATH
    if not os.path.exists(p):
        raise RuntimeError("CUDA codec library not built: %s (run agent_shared_compressed_gb300.build.build())" % p)
    lib = C.CDLL(p)
    for name, (res, args) in _SIGS.items():
        f = getattr(lib, name)
        f.restype = res
        f.argtypes = args
    if path is None:
        _lib = lib
    return lib


def declared_functions(header=HEADER):
    """Names of the functions include/kvpool.h declares."""
    src = open(header).read()
    src = re.sub(r"/\*.*?\*/", "", src, flags=re.S)
    return sorted(set(re.findall(r"\b([a-z_][a-z0-9_]*)\s*\([^;{]*\)\s*;", src)))


# --- marshalling helpers ---------------------------------------------------

def _addr(x):
    if x is None or x.__class__ is int:
        return x
    try:
        return x.data_ptr()
    except AttributeError:
        if isinstance(x, int):
            return x
        raise TypeError("expected a tensor, an int address or None, got %r" % type(x)) from None


def _ptrs(seq):
    seq = list(seq)
    arr = (_vp * max(1, len(seq)))()
    for i, x in enumerate(seq):
        arr[i] = _addr(x)
    return arr


def _stream(s):
    if s is None:
        return None
    if isinstance(s, int):
        return s
    return s.cuda_stream


def _shape(s):
    if isinstance(s, Shape):
        return s
    L, H, d, T = s
    return Shape(L, H, d, T)


# --- C API -----------------------------------------------------------------

def kvpool_pool_bytes(shape):
    return int(load().kvpool_pool_bytes(C.byref(_shape(shape))))


def kvpool_workspace_bytes(shape):
    return int(load().kvpool_workspace_bytes(C.byref(_shape(shape))))


def kvpool_encode(shape, k_layers, v_layers, pool, pool_bytes, ws, ws_bytes, stream=None):
    return load().kvpool_encode(C.byref(_shape(shape)), _ptrs(k_layers), _ptrs(v_layers), _addr(pool),
                                int(pool_bytes), _addr(ws), int(ws_bytes), _stream(stream))


def kvpool_pool_bytes_ex(shape, k_mode):
    return int(load().kvpool_pool_bytes_ex(C.byref(_shape(shape)), int(k_mode)))


def kvpool_encode_ex(shape, k_mode, k_layers, v_layers, pool, pool_bytes, ws, ws_bytes, stream=None):
    """k_mode: KVP_K_PER_TENSOR or KVP_K_Q8_0."""
    return load().kvpool_encode_ex(C.byref(_shape(shape)), int(k_mode), _ptrs(k_layers), _ptrs(v_layers),
                                   _addr(pool), int(pool_bytes), _addr(ws), int(ws_bytes), _stream(stream))


def kvpool_encode_noalloc(shape, k_layers, v_layers, pool, pool_bytes, stream=None):
    """kvpool_encode with the library's own scratch array as workspace (for
    callers that cannot allocate device memory)."""
    return load().kvpool_encode_noalloc(C.byref(_shape(shape)), _ptrs(k_layers), _ptrs(v_layers), _addr(pool),
                                        int(pool_bytes), _stream(stream))


def kvpool_decode_into(pool, shape, layer_begin, layer_end, n_agents, k_dst, v_dst, stream=None):
    """k_dst/v_dst: n_agents * n_layers pointers, agent-major (a*L + l)."""
    return load().kvpool_decode_into(_addr(pool), C.byref(_shape(shape)), int(layer_begin), int(layer_end),
                                     int(n_agents), _ptrs(k_dst), _ptrs(v_dst), _stream(stream))


def kvpool_attend_workspace_bytes(shape, n_agents, n_q_heads):
    return int(load().kvpool_attend_workspace_bytes(C.byref(_shape(shape)), int(n_agents), int(n_q_heads)))


def kvpool_attend(pool, shape, layer, n_agents, n_q_heads, q, scale, out, lse, ws, ws_bytes, stream=None):
    return load().kvpool_attend(_addr(pool), C.byref(_shape(shape)), int(layer), int(n_agents), int(n_q_heads),
                                _addr(q), C.c_float(scale), _addr(out), _addr(lse), _addr(ws), int(ws_bytes),
                                _stream(stream))


def kvpool_attend_lora_workspace_bytes(shape, n_agents, n_q_heads, rank):
    return int(load().kvpool_attend_lora_workspace_bytes(C.byref(_shape(shape)), int(n_agents), int(n_q_heads),
                                                         int(rank)))


def kvpool_attend_lora(pool, shape, layer, n_agents, n_q_heads, q, scale, rank, v_lr, lora_b, out, lse, ws,
                       ws_bytes, stream=None):
    return load().kvpool_attend_lora(_addr(pool), C.byref(_shape(shape)), int(layer), int(n_agents),
                                     int(n_q_heads), _addr(q), C.c_float(scale), int(rank), _addr(v_lr),
                                     _addr(lora_b), _addr(out), _addr(lse), _addr(ws), int(ws_bytes),
                                     _stream(stream))


def kvpool_status(pool, stream=None):
    return load().kvpool_status(_addr(pool), _stream(stream))


def cachecard_bytes(shape, bits_host):
    b = bytes(bytearray(int(x) for x in bits_host))
    arr = (C.c_uint8 * max(1, len(b))).from_buffer_copy(b if b else b"\0")
    return int(load().cachecard_bytes(C.byref(_shape(shape)), arr))


def cachecard_pack(shape, model_id, pos_offset, bits_dev, k_layers, v_layers, card, card_bytes, stream=None):
    return load().cachecard_pack(C.byref(_shape(shape)), C.c_uint64(model_id), C.c_int64(pos_offset),
                                 _addr(bits_dev), _ptrs(k_layers), _ptrs(v_layers), _addr(card),
                                 int(card_bytes), _stream(stream))


def cachecard_read_header(card, out, stream=None):
    """Fills `out` (a CardHeader); returns the status."""
    return load().cachecard_read_header(_addr(card), C.byref(out), _stream(stream))


def cachecard_unpack(card, hdr, k_dst, v_dst, stream=None):
    return load().cachecard_unpack(_addr(card), C.byref(hdr), _ptrs(k_dst), _ptrs(v_dst), _stream(stream))


def cachecard_unpack_at(card, hdr, pos_dst, inv_freq, k_dst, v_dst, stream=None):
    """inv_freq: head_dim/2 host floats (any sequence; None passes NULL)."""
    if inv_freq is None:
        w = None
    else:
        vals = [float(x) for x in inv_freq]
        w = (C.c_float * max(1, len(vals)))(*vals)
    return load().cachecard_unpack_at(_addr(card), C.byref(hdr), C.c_int64(int(pos_dst)), w, _ptrs(k_dst),
                                      _ptrs(v_dst), _stream(stream))


def cachecard_status(card, stream=None):
    return load().cachecard_status(_addr(card), _stream(stream))


def _pages(c):
    return c if c.__class__ is PagesConfig else PagesConfig(*c)


_addressof = C.addressof


class _Types:
    """torch's types by the names used here (looked up with the first tensor)."""

    def __getattr__(self, name):
        import torch
        self.bf16, self.f32, self.i32, self.i64, self.u8 = (
            torch.bfloat16, torch.float32, torch.int32, torch.int64, torch.uint8)
        return self.__dict__[name]


_T = _Types()


def _strides(x):
    """A rows tensor's strides; one without elements may have any, and has those of a
    contiguous one here."""
    if x.numel():
        return x.stride()
    _, h, d = x.shape
    return h * d, d, 1


def rows(x, token_stride=None, head_stride=None):
    """kvp_rows of a [tokens][heads][head_dim] bf16 tensor (a strided view will
    do; its last dimension contiguous), or of an address with its strides."""
    if x is None or x.__class__ is Rows:
        return x
    if token_stride is not None:
        return Rows(_addr(x), token_stride, head_stride)
    t, h, e = _strides(x)
    if e != 1:
        raise ValueError("the last dimension of a rows tensor is contiguous, got strides %r" % ((t, h, e),))
    if x.dtype is not _T.bf16:
        raise ValueError("a rows tensor is bfloat16, got %s" % x.dtype)
    r = Rows(x.data_ptr(), t, h)
    r.shape = tuple(x.shape)
    return r


_pack_rows = struct.Struct("@Pqq").pack  # a kvp_rows as bytes, for one call


def _rows(x, tokens, heads, dim, name):
    """What the call takes for rows(x), of at least `tokens` tokens of `heads` heads of `dim`."""
    if x.__class__ is Rows:
        shape = x.shape
        if shape is not None:
            _rows_fit(shape, tokens, heads, dim, name)
        return _addressof(x)
    if x is None:
        return None
    shape, (t, h, e) = x.shape, _strides(x)
    if e != 1 or x.dtype is not _T.bf16:
        rows(x)  # raises
    _rows_fit(shape, tokens, heads, dim, name)
    return _pack_rows(x.data_ptr(), t, h)


def _rows_fit(shape, tokens, heads, dim, name):
    t, h, d = shape
    if t < tokens or h != heads or d != dim:
        raise ValueError("%s: a [%d][%d][%d] tensor is needed, got %r" % (name, tokens, heads, dim, (t, h, d)))


def _buf(x, dtype, least, name):
    """The address of a contiguous tensor of the type with at least `least`
    elements (or of bytes, as many as they take), of an address, or None."""
    if x is None:
        return None
    try:
        if x.dtype is dtype and x.numel() >= least and x.is_contiguous():
            return x.data_ptr()
    except AttributeError:
        return _addr(x)  # an integer, or a TypeError
    if x.dtype is _T.u8 and x.is_contiguous() and x.numel() >= least * dtype.itemsize:
        return x.data_ptr()
    raise ValueError("%s: a contiguous %s tensor of at least %d elements is needed, got %s %r with strides %r" % (
        name, dtype, least, x.dtype, tuple(x.shape), x.stride()))


def _bytes_buf(x, least, name):
    """The address of a contiguous tensor of at least `least` bytes, of an address, or None."""
    if x is None:
        return None
    try:
        if x.nbytes >= least and x.is_contiguous():
            return x.data_ptr()
    except AttributeError:
        return _addr(x)
    raise ValueError("%s: a contiguous tensor of at least %d bytes is needed, got %s %r with strides %r" % (
        name, least, x.dtype, tuple(x.shape), x.stride()))


def _ref(x):
    return None if x is None else _addressof(x)


def _floats(x, least=0):
    """A host float array as a ctypes array of at least `least` floats: one made
    earlier passes as it is."""
    if x is None:
        return None
    if not isinstance(x, C.Array):
        vals = [float(v) for v in x]
        x = (C.c_float * max(1, len(vals)))(*vals)
        n = len(vals)
    else:
        n = len(x)
    if n < least or x._type_ is not C.c_float:
        raise ValueError("inv_freq: %d floats are needed, got %d of %s" % (least, n, x._type_.__name__))
    return x


def kvpages_bytes(cfg):
    cfg = _pages(cfg)
    return int(load().kvpages_bytes(_ref(cfg)))


def kvpages_init(cfg, pages, pages_bytes, stream=None):
    cfg = _pages(cfg)
    return load().kvpages_init(_ref(cfg), _bytes_buf(pages, pages_bytes, "pages"), int(pages_bytes), _stream(stream))


def kvpages_append(pages, cfg, layer, n_tokens, n_q_heads, q, k, v, slots, positions, q_norm, k_norm, eps, rot_dim,
                   inv_freq, q_out, k_out, v_out, stream=None):
    """q, k, v: [tokens][heads][head_dim] tensors or Rows; inv_freq: rot_dim/2
    host floats (any sequence; a ctypes float array is passed as it is).

    ValueError for a tensor of another type, another shape (q, k, v), not
    contiguous or too small for the call; so with the calls below.  (A uint8
    tensor passes as memory for any output or input but q, k and v.)"""
    cfg, w = _pages(cfg), _floats(inv_freq, rot_dim // 2)
    h, d = cfg.n_kv_heads, cfg.head_dim
    q = _rows(q, n_tokens, n_q_heads, d, "q") if n_q_heads else None
    k, v = _rows(k, n_tokens, h, d, "k"), _rows(v, n_tokens, h, d, "v")
    return load().kvpages_append(_addr(pages), _ref(cfg), layer, n_tokens, n_q_heads, q, k, v,
                                 _buf(slots, _T.i64, n_tokens, "slots"), _buf(positions, _T.i64, n_tokens, "positions"),
                                 _buf(q_norm, _T.bf16, d, "q_norm"), _buf(k_norm, _T.bf16, d, "k_norm"), eps, rot_dim,
                                 _ref(w), _buf(q_out, _T.bf16, n_tokens * n_q_heads * d, "q_out"),
                                 _buf(k_out, _T.bf16, n_tokens * h * d, "k_out"),
                                 _buf(v_out, _T.bf16, n_tokens * h * d, "v_out"), _stream(stream))


def _axes(x, least):
    """A host array of axis numbers as a ctypes uint8 array of at least `least`: one
    made earlier passes as it is."""
    if x is None:
        return None
    if not isinstance(x, C.Array):
        vals = [int(v) for v in x]
        if vals and not 0 <= min(vals) <= max(vals) <= 255:
            raise ValueError("axes: numbers from 0 to n_axes - 1 are needed, got %r" % (vals,))
        x = (C.c_uint8 * max(1, len(vals)))(*vals)
        n = len(vals)
    else:
        n = len(x)
    if n < least or x._type_ is not C.c_uint8:
        raise ValueError("axes: %d numbers of 8 bits are needed, got %d of %s" % (least, n, x._type_.__name__))
    return x


def kvpages_append_axes(pages, cfg, layer, n_tokens, n_q_heads, q, k, v, slots, positions, n_axes, axes, q_norm, k_norm,
                        eps, rot_dim, inv_freq, q_out, k_out, v_out, stream=None):
    """positions: int64 [n_axes][n_tokens]; axes: rot_dim/2 host numbers (any
    sequence; a ctypes uint8 array is passed as it is); the rest as kvpages_append."""
    cfg, w, ax = _pages(cfg), _floats(inv_freq, rot_dim // 2), _axes(axes, rot_dim // 2)
    h, d = cfg.n_kv_heads, cfg.head_dim
    q = _rows(q, n_tokens, n_q_heads, d, "q") if n_q_heads else None
    k, v = _rows(k, n_tokens, h, d, "k"), _rows(v, n_tokens, h, d, "v")
    return load().kvpages_append_axes(_addr(pages), _ref(cfg), layer, n_tokens, n_q_heads,
                                      q, k, v, _buf(slots, _T.i64, n_tokens, "slots"),
                                      _buf(positions, _T.i64, n_axes * n_tokens, "positions"), n_axes, _ref(ax),
                                      _buf(q_norm, _T.bf16, d, "q_norm"), _buf(k_norm, _T.bf16, d, "k_norm"), eps, rot_dim,
                                      _ref(w), _buf(q_out, _T.bf16, n_tokens * n_q_heads * d, "q_out"),
                                      _buf(k_out, _T.bf16, n_tokens * h * d, "k_out"),
                                      _buf(v_out, _T.bf16, n_tokens * h * d, "v_out"), _stream(stream))


def kvpages_read(pages, cfg, layer, n_seqs, table, max_pages, lens, max_tokens, k_dst, v_dst, stream=None):
    cfg = _pages(cfg)
    n = n_seqs * cfg.n_kv_heads * max_tokens * cfg.head_dim
    return load().kvpages_read(_addr(pages), _ref(cfg), layer, n_seqs, _buf(table, _T.i32, n_seqs * max_pages, "table"),
                               max_pages, _buf(lens, _T.i32, n_seqs, "lens"), max_tokens, _buf(k_dst, _T.bf16, n, "k_dst"),
                               _buf(v_dst, _T.bf16, n, "v_dst"), _stream(stream))


def kvpages_attend_workspace_bytes(cfg, n_seqs, n_q_tokens, n_q_heads):
    cfg = _pages(cfg)
    return int(load().kvpages_attend_workspace_bytes(_ref(cfg), n_seqs, n_q_tokens, n_q_heads))


def kvpages_attend(pages, cfg, layer, n_seqs, n_q_tokens, n_q_heads, q, scale, table, max_pages, lens, base_out,
                   base_lse, out, lse, ws, ws_bytes, stream=None):
    cfg = _pages(cfg)
    n = n_seqs * n_q_tokens * n_q_heads
    nd = n * cfg.head_dim
    return load().kvpages_attend(_addr(pages), _ref(cfg), layer, n_seqs, n_q_tokens, n_q_heads, _buf(q, _T.bf16, nd, "q"),
                                 scale, _buf(table, _T.i32, n_seqs * max_pages, "table"), max_pages,
                                 _buf(lens, _T.i32, n_seqs, "lens"), _buf(base_out, _T.f32, nd, "base_out"),
                                 _buf(base_lse, _T.f32, n, "base_lse"), _buf(out, _T.bf16, nd, "out"),
                                 _buf(lse, _T.f32, n, "lse"), _bytes_buf(ws, ws_bytes, "ws"), ws_bytes, _stream(stream))


def kvpages_attend_window(pages, cfg, layer, n_seqs, n_q_tokens, n_q_heads, q, scale, window, sinks, table, max_pages, lens,
                          base_out, base_lse, out, lse, ws, ws_bytes, stream=None):
    cfg = _pages(cfg)
    n = n_seqs * n_q_tokens * n_q_heads
    nd = n * cfg.head_dim
    return load().kvpages_attend_window(
        _addr(pages), _ref(cfg), layer, n_seqs, n_q_tokens, n_q_heads, _buf(q, _T.bf16, nd, "q"), scale, window, sinks,
        _buf(table, _T.i32, n_seqs * max_pages, "table"), max_pages, _buf(lens, _T.i32, n_seqs, "lens"),
        _buf(base_out, _T.f32, nd, "base_out"), _buf(base_lse, _T.f32, n, "base_lse"), _buf(out, _T.bf16, nd, "out"),
        _buf(lse, _T.f32, n, "lse"), _bytes_buf(ws, ws_bytes, "ws"), ws_bytes, _stream(stream))


def kvpages_status(pages, stream=None):
    return load().kvpages_status(_addr(pages), _stream(stream))


def _prompt(s):
    return s if s.__class__ is PromptShape else PromptShape(*s)


def kvprompt_workspace_bytes(shape):
    shape = _prompt(shape)
    return int(load().kvprompt_workspace_bytes(_ref(shape)))


def kvprompt_attend(shape, q, k, v, q_first, k_first, k_lens, scale, window, sinks, base_out, base_lse, out, lse, error, ws,
                    ws_bytes, stream=None):
    """q, k, v: [tokens][heads][head_dim] tensors (strided views will do) or Rows;
    error: an int32 tensor of one element, or None.  ValueError for tensors that do not
    hold what the call reads or writes, as the page calls."""
    shape = _prompt(shape)
    b, n, t, nq, h, d = shape.n_seqs, shape.n_q_tokens, shape.n_k_tokens, shape.n_q_heads, shape.n_kv_heads, shape.head_dim
    q, k, v = _rows(q, n, nq, d, "q"), _rows(k, t, h, d, "k"), _rows(v, t, h, d, "v")
    return load().kvprompt_attend(_ref(shape), q, k, v, _buf(q_first, _T.i32, b + 1, "q_first"), _buf(k_first, _T.i32, b, "k_first"),
                                  _buf(k_lens, _T.i32, b, "k_lens"), scale, window, sinks,
                                  _buf(base_out, _T.f32, n * nq * d, "base_out"), _buf(base_lse, _T.f32, n * nq, "base_lse"),
                                  _buf(out, _T.bf16, n * nq * d, "out"), _buf(lse, _T.f32, n * nq, "lse"),
                                  _buf(error, _T.i32, 1, "error"), _bytes_buf(ws, ws_bytes, "ws"), ws_bytes, _stream(stream))


def kvprompt_status(error, stream=None):
    return load().kvprompt_status(_buf(error, _T.i32, 1, "error"), _stream(stream))


def kvp_strerror(status):
    return load().kvp_strerror(int(status)).decode()


def kvp_launch_count():
    return int(load().kvp_launch_count())


def kvp_bandwidth_probe(mode, dst, src, nbytes, stream=None):
    return load().kvp_bandwidth_probe(int(mode), _addr(dst), _addr(src), int(nbytes), _stream(stream))


def kvp_test_fail_next_encode(layer, spin_iters):
    return load().kvp_test_fail_next_encode(int(layer), int(spin_iters))


def kvp_test_limit_next_attend(polls):
    return load().kvp_test_limit_next_attend(int(polls))


def kvp_test_limit_next_unpack(polls):
    return load().kvp_test_limit_next_unpack(int(polls))


def kvp_test_limit_next_pages_attend(polls):
    return load().kvp_test_limit_next_pages_attend(int(polls))


def kvp_test_limit_next_pages_attend_lanes(polls, lanes):
    return load().kvp_test_limit_next_pages_attend_lanes(int(polls), int(lanes))


def kvp_test_limit_next_prompt(polls):
    return load().kvp_test_limit_next_prompt(int(polls))


class KVPError(RuntimeError):
    def __init__(self, status, what=""):
        self.status = status
        super().__init__("%s%s (%d)" % (what + ": " if what else "", kvp_strerror(status), status))


def check(status, what=""):
    """Raise KVPError for a non-zero status."""
    if status != KVP_OK:
        raise KVPError(status, what)
    return status
