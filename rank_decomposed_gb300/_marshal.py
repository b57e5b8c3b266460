"""The calls of csrc/lr_calls.c through ctypes: the same names, arguments, checks and errors.

Used where the extension is not there: a Python without its C headers at build
time, or another Python than the one that built it.  A call takes 8 to 13 us longer.
"""

from __future__ import annotations

import ctypes
import math
import operator

from . import LR_BF16, LR_F32, AttnDesc, ContextDesc, HeadMapDesc, KvCache, lib

_bf16 = _f32 = _i32 = None


def init(bf16, f32, i32, *addresses):
    """torch's dtypes; the functions' addresses are the library's, which ctypes has."""
    global _bf16, _f32, _i32
    _bf16, _f32, _i32 = bf16, f32, i32


class _Host:
    """The first tensor of a call that is not on the GPU."""

    def __init__(self):
        self.name = None

    def check(self, rows):
        if rows > 0 and self.name is not None:
            raise TypeError("%s must be on the GPU" % self.name)


class _Mat:
    __slots__ = ("p", "ld", "rows", "cols")

    def __init__(self, p=None, ld=0, rows=0, cols=0):
        self.p, self.ld, self.rows, self.cols = p, ld, rows, cols


def _int(v, name, bits=64):
    v = operator.index(v)
    if not -(1 << bits - 1) <= v < 1 << bits - 1:
        raise OverflowError("%s does not fit %d bits" % (name, bits))
    return v


def _address(t, name, host):
    if t is None:
        return None
    if t.is_cuda is not True and host.name is None:
        host.name = name
    return t.data_ptr() or None


def _typed(t, name, dtype):
    if t.dtype != dtype:
        raise TypeError("%s must be %s" % (name, dtype))


def _code(t):
    d = t.dtype
    if d != _bf16 and d != _f32:
        raise TypeError("a tensor of heads must be bfloat16 or float32")
    return (LR_BF16 if d == _bf16 else LR_F32), d


def _matrix(t, name, dtype, rows, cols, host):
    """A row-major matrix of a type; rows and cols < 0: any."""
    _typed(t, name, dtype)
    shape, stride = t.shape, t.stride()
    if len(shape) != 2 or (stride[1] != 1 and shape[1] > 1):
        raise ValueError("%s must be a row-major 2-D tensor" % name)
    if (rows >= 0 and shape[0] != rows) or (cols >= 0 and shape[1] != cols):
        raise ValueError("%s has another number of rows or columns than the call needs" % name)
    # one row's stride says nothing: it counts as at least the row's width
    ld = stride[0] if shape[0] > 1 or stride[0] >= shape[1] else (shape[1] + 7) // 8 * 8
    return _Mat(_address(t, name, host), ld, shape[0], shape[1])


def _table(t, name, dtype, dims, n, host):
    """Address and shape of a contiguous tensor of `dims` dimensions; None is NULL with sizes 0.  n < 0: any first size."""
    if t is None:
        return None, (0,) * dims
    _typed(t, name, dtype)
    if len(t.shape) != dims or not t.is_contiguous():
        raise TypeError("%s must be a contiguous %d-D tensor" % (name, dims))
    if n >= 0 and t.shape[0] != n:
        raise ValueError("%s has another number of entries than the call needs" % name)
    return _address(t, name, host), tuple(t.shape)


def _vector(t, name, n, host):
    return _table(t, name, _i32, 1, n, host)[0]


def _word(t, name, host):
    p, shape = _table(t, name, _i32, 1, -1, host)
    if t is not None and shape[0] < 1:
        raise ValueError("%s is empty" % name)
    return p


def _status(t, host):
    if t is None:
        return None
    _typed(t, "status", _i32)
    p = _address(t, "status", host)
    if p is None:
        raise ValueError("status is empty")
    return p


def _head_map(o, host):
    h = HeadMapDesc()
    h.norm = 1 if o.norm else 0
    h.eps = float(o.eps)
    h.head_dim, h.rot_dim, h.rot_style = (_int(getattr(o, x), x, 32) for x in ("head_dim", "rot_dim", "rot_style"))
    h.q_gain = _table(o.q_gain, "q_gain", _bf16, 1, h.head_dim, host)[0]
    h.k_gain = _table(o.k_gain, "k_gain", _bf16, 1, h.head_dim, host)[0]
    if h.rot_dim > 0:
        h.cos_sin, shape = _table(o.cos_sin, "cos_sin", _f32, 2, -1, host)
        if h.cos_sin is not None and shape[1] != h.rot_dim:
            raise ValueError("cos_sin must be [max_pos][rot_dim]")
        h.max_pos = shape[0]
    return h


def _kv_cache(o, host):
    k = _matrix(o.k_pool, "k_pool", _bf16, -1, -1, host)
    v = _matrix(o.v_pool, "v_pool", _bf16, k.rows, k.cols, host)
    heads, hd, br = (_int(getattr(o, x), x, 32) for x in ("n_kv_heads", "head_dim", "block_rows"))
    if k.ld != v.ld:
        raise ValueError("k_pool and v_pool must have one row stride")
    if k.cols < heads * hd:
        raise ValueError("the pools' rows are narrower than n_kv_heads * head_dim")
    if br <= 0 or k.rows % br:
        raise ValueError("the pools' rows must be whole pages of block_rows")
    return KvCache(k.p, v.p, k.ld, k.rows // br, br, heads, hd)


def _attn_desc(n_heads, cache, prefix_blocks, prefix_len, block_table, lengths, q_start, max_q, scale, host):
    d = AttnDesc()
    d.cache = _kv_cache(cache, host)
    d.n_heads, d.max_q = _int(n_heads, "n_heads", 32), _int(max_q, "max_q", 32)
    if scale is None:
        d.scale = 1.0 / math.sqrt(d.cache.head_dim) if d.cache.head_dim > 0 else 0.0
    else:
        d.scale = float(scale)
    if lengths is None or block_table is None:
        raise TypeError("lengths and block_table are needed")
    d.lengths, shape = _table(lengths, "lengths", _i32, 1, -1, host)
    n = shape[0]
    d.n_seq = _int(n, "the number of sequences", 32)
    d.block_table, shape = _table(block_table, "block_table", _i32, 2, n, host)
    d.blocks_per_seq = _int(shape[1], "blocks_per_seq", 32)
    d.prefix_blocks, shape = _table(prefix_blocks, "prefix_blocks", _i32, 1, -1, host)
    d.cap_prefix_blocks = _int(shape[0], "the number of prefix pages", 32)
    d.prefix_len = _word(prefix_len, "prefix_len", host)
    d.q_start = _vector(q_start, "q_start", n + 1, host)
    return d


def qk_norm_rope(q, k, pos, heads, q_out, k_out, status, n_active, stream):
    host = _Host()
    hm = _head_map(heads, host)
    first = q if q is not None else k
    if first is None or hm.head_dim <= 0:
        raise ValueError("qk_norm_rope: q or k and a positive head_dim are needed")
    code, dtype = _code(first)
    a, ao, b, bo, rows = _Mat(), _Mat(), _Mat(), _Mat(), -1
    if q is not None:
        a = _matrix(q, "q", dtype, -1, -1, host)
        ao = _matrix(q_out, "q_out", _bf16, a.rows, a.cols, host)
        rows = a.rows
    if k is not None:
        b = _matrix(k, "k", dtype, rows, -1, host)
        bo = _matrix(k_out, "k_out", _bf16, b.rows, b.cols, host)
        rows = b.rows
    if a.cols % hm.head_dim or b.cols % hm.head_dim:
        raise ValueError("qk_norm_rope: a width is not whole heads of head_dim")
    at, active, st = _vector(pos, "pos", rows, host), _word(n_active, "n_active", host), _status(status, host)
    host.check(rows)
    return lib.lr_qk_norm_rope(a.p, a.ld, a.cols // hm.head_dim, b.p, b.ld, b.cols // hm.head_dim, code, rows, at, active,
                               ctypes.byref(hm), ao.p, ao.ld, bo.p, bo.ld, st, stream)


def kv_append(k, v, pos, rows, heads, cache, status, q, q_out, n_active, stream):
    host = _Host()
    hm, c = _head_map(heads, host), _kv_cache(cache, host)
    code, dtype = _code(k)
    a = _matrix(k, "k", dtype, -1, c.n_kv_heads * c.head_dim, host)
    b = _matrix(v, "v", dtype, a.rows, a.cols, host)
    x, xo, nh = _Mat(), _Mat(), 0
    if q is not None:
        x = _matrix(q, "q", dtype, a.rows, -1, host)
        xo = _matrix(q_out, "q_out", _bf16, a.rows, x.cols, host)
        if hm.head_dim <= 0 or x.cols % hm.head_dim:
            raise ValueError("kv_append: q's width is not whole heads of head_dim")
        nh = x.cols // hm.head_dim
    at, to = _vector(pos, "pos", a.rows, host), _vector(rows, "rows", a.rows, host)
    active, st = _word(n_active, "n_active", host), _status(status, host)
    host.check(a.rows)
    return lib.lr_kv_append(a.p, a.ld, b.p, b.ld, x.p, x.ld, nh, code, a.rows, at, to, active, ctypes.byref(hm),
                            ctypes.byref(c), xo.p, xo.ld, st, stream)


def prefix_attention(q, n_heads, cache, prefix_blocks, prefix_len, block_table, lengths, out, workspace, status, q_start,
                     max_q, scale, stream):
    host = _Host()
    d = _attn_desc(n_heads, cache, prefix_blocks, prefix_len, block_table, lengths, q_start, max_q, scale, host)
    code, dtype = _code(out)
    a = _matrix(q, "q", _bf16, -1, d.n_heads * d.cache.head_dim, host)
    o = _matrix(out, "out", dtype, a.rows, a.cols, host)
    ws, size = _address(workspace, "workspace", host), 0 if workspace is None else workspace.nbytes
    st = _status(status, host)
    host.check(a.rows)
    return lib.lr_prefix_attention(a.p, a.ld, o.p, o.ld, code, a.rows, ctypes.byref(d), ws, size, st, stream)


def head_map(o):
    return bytes(_head_map(o, _Host()))


def kv_cache(o):
    return bytes(_kv_cache(o, _Host()))


def attn_desc(n_heads, cache, prefix_blocks, prefix_len, block_table, lengths, q_start, max_q, scale):
    return bytes(_attn_desc(n_heads, cache, prefix_blocks, prefix_len, block_table, lengths, q_start, max_q, scale, _Host()))


def context(c, M, n_heads, launch):
    host = _Host()
    d = ContextDesc()
    d.attn = _attn_desc(n_heads, c.cache, c.prefix_blocks, c.prefix_len, c.block_table, c.lengths, c.q_start, c.max_q,
                        c.scale, host)
    d.heads = _head_map(c.heads, host)
    d.pos, d.rows = _vector(c.pos, "pos", M, host), _vector(c.rows, "rows", M, host)
    d.n_active = _word(c.n_active, "n_active", host)
    if launch:
        host.check(M)
    return bytes(d)
