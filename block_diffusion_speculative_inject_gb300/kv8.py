"""The caller-owned 8-bit paged cache and rotary positions (include/dflash.h): argument checks and
marshalling around the library's kernels.

One round of a verify loop with blocks of `block` rows, with nothing read back to the host:

    plan = page_plan(ctx_len, n_new, block_table, free_list, n_free, max_rows)
    q, k = rope(rotary, plan["positions"], q, k)
    kv8_append(cache, k, v, plan["slot_map"])
    out = kv8_attention(cache, q, plan["cu_rows"], plan["new_len"], block_table, mask="causal", max_q=block)

qk_norm_rope does the per-head norms of q and k in the same pass. For long contexts, the blocks that a cheap score finds
are read alone:

    kv8_bounds(cache, bounds, block_table, ctx_len, plan["new_len"])          # after the append
    blocks = kv8_select(cache, bounds, q, plan["cu_rows"], plan["new_len"], block_table, n_select)
    out = kv8_attention(cache, q, ..., blocks=blocks)

A draft tree's rows are planned and appended alike, but their positions are the context's length plus their
depth, and the attention takes mask="tree" with ddtree_build's masks. The accepted path lies scattered among
them: kv8_compact moves its rows (ddtree_path's) to their place in all layers at once, after which page_plan with
n_path - rows gives the rest back. (Or drop them all, plan the path's rows and append these again from k and v.)

Calls run on the device of their tensors, on `stream` (default: that device's current stream), and
allocate outputs that are not given from torch's allocator. Arguments that do not fit raise
DFlashError before anything is launched. None of them records a gradient, so with grad mode on a floating-point
tensor that requires one is refused (rope's gradient is rope with transpose=True, qk_norm_rope's is
qk_norm_rope_backward, for a Function of the caller's), but by kv8_select, whose answer is whole numbers.
"""
import ctypes
import functools
import math

import torch

from . import _ffi

PAGE = 64
_MASKS = {"none": 0, "causal": 1, "tree": 2}
_SCALINGS = {"none": 0, "linear": 1, "yarn": 2}


_I4, _I8, _F4, _U1 = (torch.int32,), (torch.int64,), (torch.float32,), (torch.uint8,)
_S1 = (torch.int8,)
_E4M3 = (torch.float8_e4m3fn,)
_FLOATS = (torch.bfloat16, torch.float32)


def _error(msg, status=-1):
    from . import DFlashError
    return DFlashError(status, msg)


# A serving loop makes these calls many times a round: the checks build their messages only on failure.
def _tensor(name, t, dtypes, shape, contiguous=True):
    """The shape of t, a tensor of one of `dtypes` and of `shape` (None: any size)."""
    if isinstance(t, torch.Tensor) and t.dtype in dtypes and (not contiguous or t.is_contiguous()):
        have = t.shape
        if len(have) == len(shape):
            for n, w in zip(have, shape):
                if w is not None and n != w:
                    break
            else:
                return have
    if not isinstance(t, torch.Tensor):
        raise _error(f"{name} must be a tensor")
    if t.dtype not in dtypes:
        raise _error(f"{name} must be {' or '.join(str(d) for d in dtypes)}, not {t.dtype}")
    if contiguous and not t.is_contiguous():
        raise _error(f"{name} must be contiguous")
    raise _error(f"{name} must have the shape {tuple('any' if w is None else w for w in shape)}, not {tuple(t.shape)}")


def _row_stride(name, t, heads, hd):
    """Row stride of [rows, heads, hd] whose heads are contiguous."""
    least = heads * hd
    if t.is_contiguous():
        return least
    rows, by_head, by_dim = t.stride()
    if (by_dim != 1 and hd > 1) or (by_head != hd and heads > 1):
        raise _error(f"{name}: the heads of a row must be contiguous")
    if t.shape[0] <= 1:
        return least
    if rows < least:
        raise _error(f"{name}: rows must not overlap")
    return rows


def _aligned_rows(name, t, stride):
    """16-byte aligned rows, as the cache's calls want them."""
    if stride * t.element_size() % 16 or t.data_ptr() % 16:
        raise _error(f"{name}: rows must be 16-byte aligned")


def _device(first, *others):
    """The index of the GPU that holds all the tensors (None: an argument that was not given)."""
    i = first.get_device()
    for t in others:
        if t is not None and t.get_device() != i:
            raise _error(f"tensors on different devices: {first.device} and {t.device}")
    if i < 0:
        raise _error("tensors must be on a CUDA device")
    return i


def _no_gradient(name, *tensors):
    """Refuses a call whose result would silently have no history."""
    if torch.is_grad_enabled():
        for t in tensors:
            if t is not None and t.requires_grad:
                raise _error(f"{name} records no gradients: call it under torch.no_grad(), or detach its tensors")


def _ptr(t):
    return None if t is None else t.data_ptr()


def _on(dev, stream, body):
    """body(raw stream) with device `dev` current, and `stream` too if one is given (so that what body allocates
    belongs to it)."""
    if stream is not None:
        if stream.device.index != dev:
            raise _error(f"the stream is on {stream.device}, the tensors are on cuda:{dev}")
        with torch.cuda.stream(stream):
            return body(stream.cuda_stream)
    if torch.cuda.current_device() != dev:
        with torch.cuda.device(dev):
            return body(torch.cuda.current_stream(dev).cuda_stream)
    return body(torch._C._cuda_getCurrentRawStream(dev))     # current_stream().cuda_stream, 3 us cheaper


def _call(name, *args):
    st = getattr(_ffi.load(), name)(*args)
    if st != _ffi.OK:
        raise _error(f"{name} failed", st)


def _dt(t):
    return _ffi.BF16 if t.dtype is torch.bfloat16 else _ffi.F32


class _LaidOut:
    """Attributes can be set until `_sealed` is: the library is given what was laid out from them."""
    _sealed = False

    def __setattr__(self, name, value):
        if self._sealed:
            raise _error(f"{type(self).__name__}: {name} cannot be changed, make a new one")
        object.__setattr__(self, name, value)

    def __delattr__(self, name):
        raise _error(f"{type(self).__name__}: {name} cannot be taken away")


class KV8Cache(_LaidOut):
    """An 8-bit paged cache: k_pages [n_pages, kv heads, 64, head dim] and v_pages [n_pages, kv heads,
    head dim, 64] float8_e4m3fn, k_scale / v_scale [n_pages, kv heads] fp32, powers of two. The tensors are
    the caller's, and stay those of the cache; `KV8Cache.empty` allocates them."""

    def __init__(self, k_pages, v_pages, k_scale, v_scale):
        n, h, _, d = _tensor("k_pages", k_pages, _E4M3, (None, None, PAGE, None))
        _tensor("v_pages", v_pages, _E4M3, (n, h, d, PAGE))
        _tensor("k_scale", k_scale, _F4, (n, h))
        _tensor("v_scale", v_scale, _F4, (n, h))
        if d not in (64, 128):
            raise _error(f"head_dim must be 64 or 128, not {d}")
        if not (1 <= n <= 1 << 24 and 1 <= h <= 128):
            raise _error("n_pages must be in [1, 2^24] and kv heads in [1, 128]")
        self.k_pages, self.v_pages, self.k_scale, self.v_scale = k_pages, v_pages, k_scale, v_scale
        self.n_pages, self.n_kv_heads, self.head_dim = n, h, d
        self._c = _ffi.KV8Cache(n_pages=n, n_kv_heads=h, head_dim=d, k_pages=k_pages.data_ptr(),
                                v_pages=v_pages.data_ptr(), k_scale=k_scale.data_ptr(), v_scale=v_scale.data_ptr())
        self._ref = ctypes.byref(self._c)
        self._dev = k_pages.get_device() if len({t.device for t in self._tensors()}) == 1 else None
        self._sealed = True

    @classmethod
    def empty(cls, n_pages, n_kv_heads, head_dim, device="cuda"):
        """A cache whose pages hold nothing yet (their bytes are not initialised)."""
        e4 = dict(dtype=torch.float8_e4m3fn, device=device)
        f4 = dict(dtype=torch.float32, device=device)
        return cls(torch.empty((n_pages, n_kv_heads, PAGE, head_dim), **e4),
                   torch.empty((n_pages, n_kv_heads, head_dim, PAGE), **e4),
                   torch.ones((n_pages, n_kv_heads), **f4), torch.ones((n_pages, n_kv_heads), **f4))

    def _tensors(self):
        return self.k_pages, self.v_pages, self.k_scale, self.v_scale

    def _device(self, *others):
        """The GPU of the cache and the other tensors of a call."""
        dev = _device(*others)
        if dev != self._dev:
            raise _error(f"the cache's tensors are not all on cuda:{dev}")
        return dev


class KV8Layers(_LaidOut):
    """The caches of a model's layers (1 to 128, of one shape, on one GPU), checked and laid out once for kv8_compact; `caches`
    is the tuple of them."""

    def __init__(self, caches):
        self.caches = caches = tuple(caches)
        if not 1 <= len(caches) <= 128 or not all(isinstance(c, KV8Cache) for c in caches):
            raise _error("1 to 128 KV8Cache")
        c = caches[0]
        if any((x.n_pages, x.n_kv_heads, x.head_dim) != (c.n_pages, c.n_kv_heads, c.head_dim) for x in caches):
            raise _error("the caches must have one shape")
        for t in zip(*(x._tensors() for x in caches)):
            if len({x.data_ptr() for x in t}) != len(t):
                raise _error("a cache is given twice")
        self._array = (_ffi.KV8Cache * len(caches))(*(x._c for x in caches))
        self._dev = c._dev if all(x._dev == c._dev for x in caches) else None
        self._sealed = True


def page_plan(ctx_len, n_new, block_table, free_list, n_free, max_rows, stream=None):
    """Block tables and slot maps from request lengths (dflash_page_plan). ctx_len, n_new [n] int32;
    block_table [n, max_blocks] and free_list [n_pages] int32 are updated in place; n_free [1] int32.
    Returns a dict of new tensors: new_len [n], n_free [1], cu_rows [n + 1], refused [n], slot_map
    [max_rows] int64, positions [max_rows] int32."""
    n, = _tensor("ctx_len", ctx_len, _I4, (None,))
    _tensor("n_new", n_new, _I4, (n,))
    _, width = _tensor("block_table", block_table, _I4, (n, None))
    n_pages, = _tensor("free_list", free_list, _I4, (None,))
    _tensor("n_free", n_free, _I4, (1,))
    m = int(max_rows)
    if not 1 <= n <= 4096:
        raise _error(f"1 to 4096 requests, not {n}")
    if not (1 <= width <= 1 << 24 and 1 <= n_pages <= 1 << 24):
        raise _error("max_blocks and n_pages must be in [1, 2^24]")
    if not 0 <= m < 1 << 31:
        raise _error("max_rows must be in [0, 2^31)")
    dev = _device(ctx_len, n_new, block_table, free_list, n_free)

    def body(s):
        # one allocation for the int32 outputs
        buf = torch.empty((3 * n + 2 + m,), dtype=torch.int32, device=dev)
        slot = torch.empty((m,), dtype=torch.int64, device=dev)
        new_len, refused, cu, nf, pos = buf.split((n, n, n + 1, 1, m))
        at = buf.data_ptr()
        _call("dflash_page_plan", s, n, width, n_pages, m, ctx_len.data_ptr(), n_new.data_ptr(), block_table.data_ptr(),
              free_list.data_ptr(), n_free.data_ptr(), at, at + 4 * (3 * n + 1), at + 8 * n, at + 4 * n,
              slot.data_ptr(), at + 4 * (3 * n + 2))
        return dict(new_len=new_len, n_free=nf, cu_rows=cu, refused=refused, slot_map=slot, positions=pos)
    return _on(dev, stream, body)


class Rope:
    """Rotary frequencies (dflash_rope_init), made once for a model. scaling: "none", "linear" or "yarn"."""

    def __init__(self, head_dim, rot_dim=None, theta=1e6, interleaved=False, scaling="none", factor=1.0,
                 original_positions=1.0, beta_fast=32.0, beta_slow=1.0):
        rot_dim = head_dim if rot_dim is None else rot_dim
        if scaling not in _SCALINGS:
            raise _error(f"scaling must be one of {sorted(_SCALINGS)}")
        if not (2 <= rot_dim <= head_dim <= 256 and rot_dim % 2 == 0):
            raise _error("rot_dim must be even and at most head_dim, head_dim at most 256")
        self.head_dim = head_dim
        self._c = _ffi.RopeTable()
        p = _ffi.RopeParams(rot_dim=rot_dim, interleaved=int(bool(interleaved)), scaling=_SCALINGS[scaling],
                            theta=theta, factor=factor, original_positions=original_positions, beta_fast=beta_fast,
                            beta_slow=beta_slow)
        self._ref = ctypes.byref(self._c)
        _call("dflash_rope_init", ctypes.byref(p), self._ref)


def rope(table, positions, q, k=None, transpose=False, q_out=None, k_out=None, stream=None):
    """Rotates q [rows, heads, head_dim] and (unless None) k by positions [rows] int32 (dflash_rope_apply).
    Rows may be strided. q_out / k_out: new tensors if None; q / k themselves rotate in place.
    transpose: the transposed map, from gradients of the outputs to those of the inputs.
    Returns (q_out, k_out)."""
    hd = table.head_dim
    rows, nq, _ = _tensor("q", q, _FLOATS, (None, None, hd), False)
    dt = (q.dtype,)
    _tensor("positions", positions, _I4, (rows,))
    nk = ks = qos = kos = 0
    qs = _row_stride("q", q, nq, hd)
    if q_out is not None:
        _tensor("q_out", q_out, dt, (rows, nq, hd), False)
        qos = _row_stride("q_out", q_out, nq, hd)
    if k is not None:
        _, nk, _ = _tensor("k", k, dt, (rows, None, hd), False)
        ks = _row_stride("k", k, nk, hd)
        if k_out is not None:
            _tensor("k_out", k_out, dt, (rows, nk, hd), False)
            kos = _row_stride("k_out", k_out, nk, hd)
    elif k_out is not None:
        raise _error("k_out without k")
    _no_gradient("rope", q, k, q_out, k_out)
    dev = _device(q, k, positions, q_out, k_out)

    def body(s):
        qo, ko, qo_s, ko_s = q_out, k_out, qos, kos
        if qo is None:
            qo, qo_s = torch.empty((rows, nq, hd), dtype=q.dtype, device=dev), nq * hd
        if k is not None and ko is None:
            ko, ko_s = torch.empty((rows, nk, hd), dtype=q.dtype, device=dev), nk * hd
        _call("dflash_rope_apply", s, table._ref, rows, nq, nk, hd, _dt(q), positions.data_ptr(), 1 if transpose else 0,
              q.data_ptr(), qs, _ptr(k), ks, qo.data_ptr(), qo_s, _ptr(ko), ko_s)
        return qo, ko
    return _on(dev, stream, body)


def _norm_args(table, positions, q, k, q_weight, k_weight, eps):
    """(rows, heads of q, row stride of q, heads of k, row stride of k, eps), checked."""
    hd = table.head_dim
    rows, nq, _ = _tensor("q", q, _FLOATS, (None, None, hd), False)
    dt = (q.dtype,)
    _tensor("positions", positions, _I4, (rows,))
    _tensor("q_weight", q_weight, dt, (hd,))
    nk = ks = 0
    if (k is None) != (k_weight is None):
        raise _error("k and k_weight go together")
    if k is not None:
        _, nk, _ = _tensor("k", k, dt, (rows, None, hd), False)
        ks = _row_stride("k", k, nk, hd)
        _tensor("k_weight", k_weight, dt, (hd,))
    if nq < 1 or nq + nk > 1 << 20:
        raise _error("1 to 2^20 heads")
    eps = float(eps)
    if not 2.0 ** -150 < eps < 3.4028235e38:           # (positive and finite in fp32)
        raise _error("eps must be positive and finite")
    return rows, nq, _row_stride("q", q, nq, hd), nk, ks, eps


def _new_like(t):
    """A new contiguous tensor of t's shape, type and device."""
    return torch.empty_like(t) if t.is_contiguous() else torch.empty(t.shape, dtype=t.dtype, device=t.device)


def _like(name, t, ref, own):
    """Row stride of t, a tensor of ref's shape and type (None: 0). own: a tensor that t may be, with the same rows."""
    if t is None:
        return 0
    if ref is None:
        raise _error(f"{name} without k")
    rows, heads, hd = ref.shape
    if not isinstance(t, torch.Tensor) or t.dtype != ref.dtype or t.shape != ref.shape:
        _tensor(name, t, (ref.dtype,), ref.shape, False)
    stride = _row_stride(name, t, heads, hd)
    if own is not None and rows > 1 and t.data_ptr() == own.data_ptr() and stride != own.stride(0):
        raise _error(f"{name}: in place only with the same strides")
    return stride


def _not_over(name, t, **others):
    """Refuses an output `t` in the place of another tensor of the call."""
    if t is not None and t.numel():
        for other, x in others.items():
            if x is not None and x.data_ptr() == t.data_ptr():
                raise _error(f"{name} must not be {other}")


def qk_norm_rope(table, positions, q, k, q_weight, k_weight, eps=1e-6, q_out=None, k_out=None, stream=None):
    """Per-head RMSNorm and rotation in one pass (dflash_qk_norm_rope): every head of q [rows, heads, head_dim] and
    (unless None) k becomes the rotation of x / sqrt(mean(x^2) + eps) * weight by its row's position. q_weight, k_weight
    [head_dim] of q's type. Rows may be strided. q_out / k_out: new tensors if None; q / k themselves work in
    place, and no output may overlap anything else. Returns (q_out, k_out)."""
    rows, nq, qs, nk, ks, eps = _norm_args(table, positions, q, k, q_weight, k_weight, eps)
    hd = table.head_dim
    qos, kos = _like("q_out", q_out, q, q), _like("k_out", k_out, k, k)
    if q_out is not None or k_out is not None:
        _not_over("q_out", q_out, k=k, k_out=k_out)
        _not_over("k_out", k_out, q=q)
    _no_gradient("qk_norm_rope", q, k, q_weight, k_weight, q_out, k_out)
    dev = _device(q, k, positions, q_weight, k_weight, q_out, k_out)

    def body(s):
        qo, ko, qo_s, ko_s = q_out, k_out, qos, kos
        if qo is None:
            qo, qo_s = _new_like(q), nq * hd
        if k is not None and ko is None:
            ko, ko_s = _new_like(k), nk * hd
        _call("dflash_qk_norm_rope", s, table._ref, rows, nq, nk, hd, _dt(q), positions.data_ptr(), eps, q_weight.data_ptr(),
              _ptr(k_weight), q.data_ptr(), qs, _ptr(k), ks, qo.data_ptr(), qo_s, _ptr(ko), ko_s)
        return qo, ko
    return _on(dev, stream, body)


@functools.cache
def qk_norm_rope_workspace():
    """Bytes of workspace that qk_norm_rope_backward needs."""
    return _ffi.load().dflash_qk_norm_rope_workspace()


def qk_norm_rope_backward(table, positions, q, k, q_weight, k_weight, grad_q_out, grad_k_out, eps=1e-6, dq=None, dk=None,
                          workspace=None, stream=None):
    """The gradients of qk_norm_rope's q, k and weights from those of its outputs (dflash_qk_norm_rope_backward); q and
    k are its inputs as they were before it. dq / dk: new tensors if None; grad_q_out / grad_k_out themselves work in
    place, and no output may overlap anything else. workspace: a uint8 tensor of qk_norm_rope_workspace() bytes; allocated for the call if None.
    Returns (dq, dk, dq_weight, dk_weight), the last two [head_dim] fp32 (dk and dk_weight None without k)."""
    rows, nq, qs, nk, ks, eps = _norm_args(table, positions, q, k, q_weight, k_weight, eps)
    hd = table.head_dim
    if grad_q_out is None or (k is None) != (grad_k_out is None):
        raise _error("grad_q_out goes with q and grad_k_out with k")
    gqs, gks = _like("grad_q_out", grad_q_out, q, None), _like("grad_k_out", grad_k_out, k, None)
    dqs, dks = _like("dq", dq, q, grad_q_out), _like("dk", dk, k, grad_k_out)
    if dq is not None or dk is not None:               # (q and k are read for the weights' gradients)
        _not_over("dq", dq, q=q, k=k, grad_k_out=grad_k_out, dk=dk)
        _not_over("dk", dk, k=k, q=q, grad_q_out=grad_q_out)
    if workspace is not None:
        _tensor("workspace", workspace, _U1, (None,))
    _no_gradient("qk_norm_rope_backward", q, k, q_weight, k_weight, grad_q_out, grad_k_out, dq, dk)
    dev = _device(q, k, positions, q_weight, k_weight, grad_q_out, grad_k_out, dq, dk, workspace)

    def body(s):
        a, b, w = dq, dk, workspace
        a_s, b_s = dqs, dks
        if a is None:
            a, a_s = _new_like(q), nq * hd
        if k is not None and b is None:
            b, b_s = _new_like(k), nk * hd
        if w is None:
            w = torch.empty((qk_norm_rope_workspace(),), dtype=torch.uint8, device=dev)
        qw = torch.empty((hd,), dtype=torch.float32, device=dev)
        # (the library leaves dk_weight alone where k has no heads: a sum over nothing)
        kw = None if k is None else torch.empty_like(qw) if nk else torch.zeros_like(qw)
        x = _ffi.QKNormRopeGrad(rows, nq, nk, hd, _dt(q), eps, positions.data_ptr(), q_weight.data_ptr(), _ptr(k_weight),
                                q.data_ptr(), _ptr(k), grad_q_out.data_ptr(), _ptr(grad_k_out), qs, ks, gqs, gks, a.data_ptr(),
                                _ptr(b), a_s, b_s, qw.data_ptr(), _ptr(kw), w.data_ptr(), w.numel())
        _call("dflash_qk_norm_rope_backward", s, table._ref, ctypes.byref(x))
        return a, b, qw, kw
    return _on(dev, stream, body)


def kv8_append(cache, k, v, slot_map, stream=None):
    """Writes rows of k and v [rows, kv heads, head_dim] into the cache at slot_map [rows] int64, negative
    slots skipped (dflash_kv8_append). Rows may be strided."""
    heads, hd = cache.n_kv_heads, cache.head_dim
    rows, _, _ = _tensor("k", k, _FLOATS, (None, heads, hd), False)
    _tensor("v", v, (k.dtype,), (rows, heads, hd), False)
    _tensor("slot_map", slot_map, _I8, (rows,))
    ks, vs = _row_stride("k", k, heads, hd), _row_stride("v", v, heads, hd)
    _aligned_rows("k", k, ks)
    _aligned_rows("v", v, vs)
    _no_gradient("kv8_append", k, v)
    _on(cache._device(k, v, slot_map), stream,
        lambda s: _call("dflash_kv8_append", s, cache._ref, rows, _dt(k), k.data_ptr(), ks, v.data_ptr(), vs,
                        slot_map.data_ptr()))


def kv8_read(cache, slot_map, stream=None):
    """The cached values at slot_map [rows] int64 as fp32 (k, v) [rows, kv heads, head_dim]; zero where the slot
    is negative (dflash_kv8_read)."""
    rows, = _tensor("slot_map", slot_map, _I8, (None,))
    dev = cache._device(slot_map)

    def body(s):
        shape = (rows, cache.n_kv_heads, cache.head_dim)
        k = torch.empty(shape, dtype=torch.float32, device=dev)
        v = torch.empty(shape, dtype=torch.float32, device=dev)
        _call("dflash_kv8_read", s, cache._ref, rows, slot_map.data_ptr(), k.data_ptr(), v.data_ptr())
        return k, v
    return _on(dev, stream, body)


def kv8_attention(cache, q, cu_q, ctx_len, block_table, mask="causal", tree_mask=None, scale=None, max_q=None,
                  out=None, lse=None, want_lse=False, workspace=None, stream=None, blocks=None):
    """Attention of rows cu_q[b] .. cu_q[b + 1] of q [rows, heads, head_dim] over the first ctx_len[b] tokens of
    block_table[b] (dflash_kv8_attention). mask: "none", "causal", or "tree" with tree_mask [rows, words] int32
    (as ddtree_build's, flattened over its requests). scale: 1 / sqrt(head_dim) if None. max_q: the most rows
    of a request where the host knows it (default: q's rows), which steers the choice of kernel and nothing
    else; give it, for without it a batch of single tokens or short blocks goes to the kernel for many rows, which
    takes 1.1 to 3 times as long there. workspace: a uint8 tensor of kv8_workspace(...) bytes; allocated for the call if None.
    blocks: [n, kv heads, any] int32, the blocks of 64 tokens that each request and kv head reads, as kv8_select makes
    them (dflash_kv8_attention_blocks); everything if None. Of a list only the first entries count, as many as the context has
    blocks, so those that name a block come first; a block is to be listed once.
    Returns out [rows, heads, head_dim], or (out, lse [rows, heads] fp32) with want_lse."""
    a = _attn_args(cache, q, cu_q, ctx_len, block_table, mask, tree_mask, scale, max_q, out, lse)
    _no_gradient("kv8_attention", q, out, lse)
    if workspace is not None:
        _tensor("workspace", workspace, _U1, (None,))
    if blocks is not None:
        _, _, listed = _tensor("blocks", blocks, _I4, (a.n_req, cache.n_kv_heads, None))
        if not 1 <= listed <= 1 << 24:
            raise _error("blocks must list 1 to 2^24 for each request and kv head")
    dev = cache._device(q, cu_q, ctx_len, block_table, tree_mask, out, lse, workspace, blocks)

    def body(s):
        o, z, w = out, lse, workspace
        if o is None:
            o = torch.empty(q.shape, dtype=q.dtype, device=dev)
        if want_lse and z is None:
            z = torch.empty((a.rows, a.n_q_heads), dtype=torch.float32, device=dev)
        if w is None:
            w = torch.empty((_workspace_bytes(cache, a),), dtype=torch.uint8, device=dev)
        a.out, a.lse = o.data_ptr(), _ptr(z)
        a.workspace, a.workspace_bytes = w.data_ptr(), w.numel()
        if blocks is None:
            _call("dflash_kv8_attention", s, cache._ref, ctypes.byref(a))
        else:
            _call("dflash_kv8_attention_blocks", s, cache._ref, ctypes.byref(a), blocks.data_ptr(), listed)
        return (o, z) if want_lse else o
    return _on(dev, stream, body)


def kv8_bounds(cache, bounds, block_table, old_len, new_len, stream=None):
    """Makes the key bounds of every page that holds a token of [old_len[b], new_len[b]) of request b anew, from its rows
    below new_len[b] (dflash_kv8_bounds): after an append of those tokens, or from 0 for whole contexts. bounds
    [n_pages, kv heads, 2, head_dim] int8 is updated in place: the least and the largest key of each dim, rounded
    outwards to multiples of 4 k_scale."""
    _tensor("bounds", bounds, _S1, (cache.n_pages, cache.n_kv_heads, 2, cache.head_dim))
    if bounds.data_ptr() % 16:
        raise _error("bounds must be 16-byte aligned")
    n, width = _tensor("block_table", block_table, _I4, (None, None))
    _tensor("old_len", old_len, _I4, (n,))
    _tensor("new_len", new_len, _I4, (n,))
    if not 1 <= n <= 4096:
        raise _error(f"1 to 4096 requests, not {n}")
    if not 1 <= width <= 1 << 24:
        raise _error("max_blocks must be in [1, 2^24]")
    _on(cache._device(bounds, block_table, old_len, new_len), stream,
        lambda s: _call("dflash_kv8_bounds", s, cache._ref, bounds.data_ptr(), n, width, old_len.data_ptr(), new_len.data_ptr(),
                        block_table.data_ptr()))


def kv8_select(cache, bounds, q, cu_q, ctx_len, block_table, n_select, keep_first=1, keep_last=1, out=None, workspace=None,
               stream=None):
    """Chooses n_select blocks of 64 tokens of each request and kv head for kv8_attention(blocks=...)
    (dflash_kv8_select): the first keep_first, those of the request's own rows (the context's last) and keep_last before
    them, then by falling score, the largest product with a row of q that the key bounds allow (q rounded to 11 bits); ties
    go to the lowest index. Where the first two kinds are more than n_select, the lowest are kept and the last rows do not see
    themselves: keep_first + keep_last + (rows + 62) // 64 + 1 hold them all for a request of `rows` rows. Arguments as
    kv8_attention's. Returns blocks [n, kv heads, n_select] int32, rising, -1 after the last; out: a tensor for them.
    workspace: a uint8 tensor of kv8_select_workspace(...) bytes; allocated for the call if None."""
    a = _choice_args(cache, bounds, q, cu_q, ctx_len, block_table, n_select, keep_first, keep_last)
    shape = (a.n_req, cache.n_kv_heads, a.n_select)
    if out is not None:
        _tensor("out", out, _I4, shape)
    if workspace is not None:
        _tensor("workspace", workspace, _U1, (None,))
    dev = cache._device(bounds, q, cu_q, ctx_len, block_table, out, workspace)

    def body(s):
        o, w = out, workspace
        if o is None:
            o = torch.empty(shape, dtype=torch.int32, device=dev)
        if w is None:
            w = torch.empty((_choice_bytes(cache, a),), dtype=torch.uint8, device=dev)
        a.blocks, a.workspace, a.workspace_bytes = o.data_ptr(), w.data_ptr(), w.numel()
        _call("dflash_kv8_select", s, cache._ref, ctypes.byref(a))
        return o
    return _on(dev, stream, body)


def kv8_select_workspace(cache, bounds, q, cu_q, ctx_len, block_table, n_select, keep_first=1, keep_last=1):
    """Bytes of workspace that kv8_select needs for these arguments."""
    return _choice_bytes(cache, _choice_args(cache, bounds, q, cu_q, ctx_len, block_table, n_select, keep_first, keep_last))


def _choice_bytes(cache, a):
    n = _ffi.load().dflash_kv8_select_workspace(cache._ref, ctypes.byref(a))
    if n < 0:
        raise _error("arguments out of range")
    return n


def _choice_args(cache, bounds, q, cu_q, ctx_len, block_table, n_select, keep_first, keep_last):
    hd, nkv = cache.head_dim, cache.n_kv_heads
    rows, heads, _ = _tensor("q", q, _FLOATS, (None, None, hd), False)
    _tensor("bounds", bounds, _S1, (cache.n_pages, nkv, 2, hd))
    if bounds.data_ptr() % 16:
        raise _error("bounds must be 16-byte aligned")
    n, = _tensor("ctx_len", ctx_len, _I4, (None,))
    _tensor("cu_q", cu_q, _I4, (n + 1,))
    _, width = _tensor("block_table", block_table, _I4, (n, None))
    if not 1 <= n <= 4096:
        raise _error(f"1 to 4096 requests, not {n}")
    if not 1 <= width <= 1 << 24:
        raise _error("max_blocks must be in [1, 2^24]")
    if heads < 1 or heads % nkv or heads > 8 * nkv:
        raise _error(f"query heads must be a multiple of the {nkv} kv heads, at most 8 for each, not {heads}")
    k, first, last = int(n_select), int(keep_first), int(keep_last)
    if not (1 <= k <= 1 << 24 and n * nkv * k < 1 << 31):
        raise _error("n_select must be in [1, 2^24] and the list below 2^31 entries")
    if not (0 <= first <= 1 << 24 and 0 <= last <= 1 << 24):
        raise _error("keep_first and keep_last must be in [0, 2^24]")
    stride = _row_stride("q", q, heads, hd)
    _aligned_rows("q", q, stride)
    return _ffi.KV8Choice(n, rows, heads, width, k, first, last, _dt(q), q.data_ptr(), stride, cu_q.data_ptr(),
                          ctx_len.data_ptr(), block_table.data_ptr(), bounds.data_ptr())


def kv8_compact(caches, block_table, base_len, keep, n_keep, stream=None):
    """Moves token base_len[b] + keep[b, j] of request b to base_len[b] + j, for j < n_keep[b], in place in a cache or
    in all caches of a sequence at once (the layers of a model, up to 128, of one shape and with one block table; as KV8Layers
    they are checked once and not at every call), as if the rows were read and appended again (dflash_kv8_compact). base_len,
    n_keep [n] int32; keep [n, any] int32, rising from at least 0: after a draft tree the path of ddtree_path, with base_len
    the lengths before the tree."""
    if not isinstance(caches, KV8Layers):
        caches = KV8Layers([caches] if isinstance(caches, KV8Cache) else caches)
    n, width = _tensor("block_table", block_table, _I4, (None, None))
    _tensor("base_len", base_len, _I4, (n,))
    _, most = _tensor("keep", keep, _I4, (n, None))
    _tensor("n_keep", n_keep, _I4, (n,))
    if not 1 <= n <= 4096:
        raise _error(f"1 to 4096 requests, not {n}")
    if not (1 <= width <= 1 << 24 and 1 <= most <= 1 << 24):
        raise _error("max_blocks and keep's width must be in [1, 2^24]")
    dev = _device(block_table, base_len, keep, n_keep)
    if dev != caches._dev:
        raise _error(f"the caches' tensors are not all on cuda:{dev}")
    _on(dev, stream, lambda s: _call("dflash_kv8_compact", s, len(caches._array), caches._array, n, width, most,
                                     base_len.data_ptr(), keep.data_ptr(), n_keep.data_ptr(), block_table.data_ptr()))


def kv8_workspace(cache, q, cu_q, ctx_len, block_table, mask="causal", tree_mask=None, scale=None, max_q=None):
    """Bytes of workspace that kv8_attention needs for these arguments."""
    return _workspace_bytes(cache, _attn_args(cache, q, cu_q, ctx_len, block_table, mask, tree_mask, scale, max_q,
                                              None, None))


def _workspace_bytes(cache, a):
    n = _ffi.load().dflash_kv8_attention_workspace(cache._ref, ctypes.byref(a))
    if n < 0:
        raise _error("arguments out of range")
    return n


def _attn_args(cache, q, cu_q, ctx_len, block_table, mask, tree_mask, scale, max_q, out, lse):
    hd, nkv = cache.head_dim, cache.n_kv_heads
    rows, heads, _ = _tensor("q", q, _FLOATS, (None, None, hd), False)
    n, = _tensor("ctx_len", ctx_len, _I4, (None,))
    _tensor("cu_q", cu_q, _I4, (n + 1,))
    _, width = _tensor("block_table", block_table, _I4, (n, None))
    if not 1 <= n <= 4096:
        raise _error(f"1 to 4096 requests, not {n}")
    if not 1 <= width <= 1 << 24:
        raise _error("max_blocks must be in [1, 2^24]")
    if heads < 1 or heads % nkv or heads > 8 * nkv:
        raise _error(f"query heads must be a multiple of the {nkv} kv heads, at most 8 for each, not {heads}")
    if mask not in _MASKS:
        raise _error(f"mask must be one of {sorted(_MASKS)}")
    if (tree_mask is not None) != (mask == "tree"):
        raise _error("tree_mask goes with mask='tree'")
    words = 0
    if tree_mask is not None:
        _, words = _tensor("tree_mask", tree_mask, _I4, (rows, None))
        if words < 1:
            raise _error("tree_mask needs a word for each row")
    scale = hd ** -0.5 if scale is None else float(scale)
    if not (scale > 0 and math.isfinite(scale)):
        raise _error("scale must be positive and finite")
    if out is not None:
        _tensor("out", out, (q.dtype,), (rows, heads, hd))
        if out.data_ptr() % 16:
            raise _error("out must be 16-byte aligned")
    if lse is not None:
        _tensor("lse", lse, _F4, (rows, heads))
    max_q = rows if max_q is None else int(max_q)
    if not 0 <= max_q < 1 << 31:
        raise _error("max_q must be in [0, 2^31)")
    stride = _row_stride("q", q, heads, hd)
    _aligned_rows("q", q, stride)
    return _ffi.KV8Attn(n, rows, heads, width, max_q, _dt(q), _MASKS[mask], words, scale, q.data_ptr(), stride,
                        cu_q.data_ptr(), ctx_len.data_ptr(), block_table.data_ptr(), _ptr(tree_mask))
