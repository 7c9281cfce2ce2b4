"""The caller-owned 8-bit paged cache and rotary positions (include/dflash.h): argument checks and
marshalling around the library's kernels.

One round of a verify loop, with nothing read back to the host:

    plan = page_plan(ctx_len, n_new, block_table, free_list, n_free, max_rows)
    q, k = rope(rotary, plan["positions"], q, k)
    kv8_append(cache, k, v, plan["slot_map"])
    out = kv8_attention(cache, q, plan["cu_rows"], plan["new_len"], block_table, mask="causal")

Calls run on the device of their tensors, on `stream` (default: that device's current stream), and
allocate outputs that are not given from torch's allocator. Arguments that do not fit raise
DFlashError before anything is launched.
"""
import ctypes
import math

import torch

from . import _ffi

PAGE = 64
_MASKS = {"none": 0, "causal": 1, "tree": 2}
_SCALINGS = {"none": 0, "linear": 1, "yarn": 2}


def _error(msg):
    from . import DFlashError
    return DFlashError(-1, msg)


def _need(ok, msg):
    if not ok:
        raise _error(msg)


def _tensor(name, t, dtype, shape, contiguous=True):
    """t is a tensor of `dtype` (one or several) and `shape` (None: any size)."""
    _need(isinstance(t, torch.Tensor), f"{name} must be a tensor")
    dtypes = dtype if isinstance(dtype, tuple) else (dtype,)
    _need(t.dtype in dtypes, f"{name} must be {' or '.join(str(d) for d in dtypes)}, not {t.dtype}")
    _need(t.dim() == len(shape) and all(w is None or s == w for s, w in zip(t.shape, shape)),
          f"{name} must have the shape {tuple('any' if w is None else w for w in shape)}, not {tuple(t.shape)}")
    if contiguous:
        _need(t.is_contiguous(), f"{name} must be contiguous")


def _rows_of(name, t):
    """Row stride of [rows, heads, head_dim] whose heads are contiguous."""
    _need(t.shape[2] == 1 or t.stride(2) == 1, f"{name}: the last dimension must be contiguous")
    _need(t.shape[1] == 1 or t.stride(1) == t.shape[2], f"{name}: the heads of a row must be contiguous")
    least = t.shape[1] * t.shape[2]
    if t.shape[0] <= 1:
        return least
    _need(t.stride(0) >= least, f"{name}: rows must not overlap")
    return t.stride(0)


def _device(*tensors):
    devs = {t.device for t in tensors if t is not None}
    _need(len(devs) == 1, f"tensors on different devices: {sorted(str(d) for d in devs)}")
    dev = devs.pop()
    _need(dev.type == "cuda", "tensors must be on a CUDA device")
    return dev


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


class _On:
    """Makes a device current and gives the stream to launch on. Tensors allocated inside belong to it."""

    def __init__(self, dev, stream):
        self.dev, self.given = dev, stream

    def __enter__(self):
        self._d = torch.cuda.device(self.dev)
        self._d.__enter__()
        try:
            s = self.given if self.given is not None else torch.cuda.current_stream(self.dev)
            _need(s.device == self.dev, f"the stream is on {s.device}, the tensors are on {self.dev}")
            self._s = torch.cuda.stream(s) if self.given is not None else None
            if self._s is not None:
                self._s.__enter__()
        except BaseException:
            self._d.__exit__(None, None, None)
            raise
        return ctypes.c_void_p(s.cuda_stream)

    def __exit__(self, *exc):
        if self._s is not None:
            self._s.__exit__(*exc)
        self._d.__exit__(*exc)


def _call(name, *args):
    from . import DFlashError
    st = getattr(_ffi.load(), name)(*args)
    if st != _ffi.OK:
        raise DFlashError(st, f"{name} failed")


def _dt(t):
    return _ffi.BF16 if t.dtype == torch.bfloat16 else _ffi.F32


_FLOATS = (torch.bfloat16, torch.float32)


class KV8Cache:
    """An 8-bit paged cache: k_pages [n_pages, kv heads, 64, head dim] and v_pages [n_pages, kv heads,
    head dim, 64] float8_e4m3fn, k_scale / v_scale [n_pages, kv heads] fp32, powers of two. The tensors are
    the caller's; `KV8Cache.empty` allocates them."""

    def __init__(self, k_pages, v_pages, k_scale, v_scale):
        _tensor("k_pages", k_pages, torch.float8_e4m3fn, (None, None, PAGE, None))
        n, h, _, d = k_pages.shape
        _tensor("v_pages", v_pages, torch.float8_e4m3fn, (n, h, d, PAGE))
        _tensor("k_scale", k_scale, torch.float32, (n, h))
        _tensor("v_scale", v_scale, torch.float32, (n, h))
        _need(d in (64, 128), f"head_dim must be 64 or 128, not {d}")
        _need(1 <= n <= 1 << 24 and 1 <= h <= 128, "n_pages must be in [1, 2^24] and kv heads in [1, 128]")
        self.k_pages, self.v_pages, self.k_scale, self.v_scale = k_pages, v_pages, k_scale, v_scale
        self.n_pages, self.n_kv_heads, self.head_dim = n, h, d
        self._c = _ffi.KV8Cache(n_pages=n, n_kv_heads=h, head_dim=d, k_pages=k_pages.data_ptr(),
                                v_pages=v_pages.data_ptr(), k_scale=k_scale.data_ptr(), v_scale=v_scale.data_ptr())

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


def page_plan(ctx_len, n_new, block_table, free_list, n_free, max_rows, stream=None):
    """Block tables and slot maps from request lengths (dflash_page_plan). ctx_len, n_new [n] int32;
    block_table [n, max_blocks] and free_list [n_pages] int32 are updated in place; n_free [1] int32.
    Returns a dict of new tensors: new_len [n], n_free [1], cu_rows [n + 1], refused [n], slot_map
    [max_rows] int64, positions [max_rows] int32."""
    i4 = torch.int32
    _tensor("ctx_len", ctx_len, i4, (None,))
    n = ctx_len.shape[0]
    _tensor("n_new", n_new, i4, (n,))
    _tensor("block_table", block_table, i4, (n, None))
    _tensor("free_list", free_list, i4, (None,))
    _tensor("n_free", n_free, i4, (1,))
    _need(1 <= n <= 4096, f"1 to 4096 requests, not {n}")
    _need(1 <= block_table.shape[1] <= 1 << 24 and 1 <= free_list.shape[0] <= 1 << 24,
          "max_blocks and n_pages must be in [1, 2^24]")
    _need(0 <= int(max_rows) < 1 << 31, "max_rows must be in [0, 2^31)")
    with _On(_device(ctx_len, n_new, block_table, free_list, n_free), stream) as s:
        # one allocation for the int32 outputs
        m = int(max_rows)
        buf = torch.empty((3 * n + 2 + m,), dtype=i4, device=ctx_len.device)
        new_len, refused, cu, nf, pos = buf.split([n, n, n + 1, 1, m])
        slot = torch.empty((m,), dtype=torch.int64, device=ctx_len.device)
        _call("dflash_page_plan", s, n, block_table.shape[1], free_list.shape[0], m, _ptr(ctx_len), _ptr(n_new),
              _ptr(block_table), _ptr(free_list), _ptr(n_free), _ptr(new_len), _ptr(nf), _ptr(cu), _ptr(refused),
              _ptr(slot), _ptr(pos))
    return dict(new_len=new_len, n_free=nf, cu_rows=cu, refused=refused, slot_map=slot, positions=pos)


class Rope:
    """Rotary frequencies (dflash_rope_init), made once for a model. scaling: "none", "linear" or "yarn"."""

    def __init__(self, head_dim, rot_dim=None, theta=1e6, interleaved=False, scaling="none", factor=1.0,
                 original_positions=1.0, beta_fast=32.0, beta_slow=1.0):
        rot_dim = head_dim if rot_dim is None else rot_dim
        _need(scaling in _SCALINGS, f"scaling must be one of {sorted(_SCALINGS)}")
        _need(2 <= rot_dim <= head_dim <= 256 and rot_dim % 2 == 0,
              "rot_dim must be even and at most head_dim, head_dim at most 256")
        self.head_dim = head_dim
        self._c = _ffi.RopeTable()
        p = _ffi.RopeParams(rot_dim=rot_dim, interleaved=int(bool(interleaved)), scaling=_SCALINGS[scaling],
                            theta=theta, factor=factor, original_positions=original_positions, beta_fast=beta_fast,
                            beta_slow=beta_slow)
        _call("dflash_rope_init", ctypes.byref(p), ctypes.byref(self._c))


def rope(table, positions, q, k=None, transpose=False, q_out=None, k_out=None, stream=None):
    """Rotates q [rows, heads, head_dim] and (unless None) k by positions [rows] int32 (dflash_rope_apply).
    Rows may be strided. q_out / k_out: new tensors if None; q / k themselves rotate in place.
    transpose: the transposed map, from gradients of the outputs to those of the inputs.
    Returns (q_out, k_out)."""
    _tensor("q", q, _FLOATS, (None, None, table.head_dim), contiguous=False)
    rows = q.shape[0]
    _tensor("positions", positions, torch.int32, (rows,))
    if q_out is not None:
        _tensor("q_out", q_out, q.dtype, tuple(q.shape), contiguous=False)
    _need(k is not None or k_out is None, "k_out without k")
    if k is not None:
        _tensor("k", k, q.dtype, (rows, None, table.head_dim), contiguous=False)
        if k_out is not None:
            _tensor("k_out", k_out, q.dtype, tuple(k.shape), contiguous=False)
    strides = [0 if t is None else _rows_of(name, t) for name, t in
               (("q", q), ("k", k), ("q_out", q_out), ("k_out", k_out))]
    with _On(_device(q, k, positions, q_out, k_out), stream) as s:
        if q_out is None:
            q_out = torch.empty(q.shape, dtype=q.dtype, device=q.device)
            strides[2] = q.shape[1] * q.shape[2]
        if k is not None and k_out is None:
            k_out = torch.empty(k.shape, dtype=k.dtype, device=k.device)
            strides[3] = k.shape[1] * k.shape[2]
        _call("dflash_rope_apply", s, ctypes.byref(table._c), rows, q.shape[1], 0 if k is None else k.shape[1],
              table.head_dim, _dt(q), _ptr(positions), int(bool(transpose)), _ptr(q), strides[0], _ptr(k), strides[1],
              _ptr(q_out), strides[2], _ptr(k_out), strides[3])
    return q_out, k_out


def _aligned_rows(name, t, stride):
    """16-byte aligned rows, as the cache's calls want them."""
    v = 16 // t.element_size()
    _need(stride % v == 0 and t.data_ptr() % 16 == 0, f"{name}: rows must be 16-byte aligned")


def kv8_append(cache, k, v, slot_map, stream=None):
    """Writes rows of k and v [rows, kv heads, head_dim] into the cache at slot_map [rows] int64, negative
    slots skipped (dflash_kv8_append). Rows may be strided."""
    _tensor("k", k, _FLOATS, (None, cache.n_kv_heads, cache.head_dim), contiguous=False)
    _tensor("v", v, k.dtype, tuple(k.shape), contiguous=False)
    _tensor("slot_map", slot_map, torch.int64, (k.shape[0],))
    ks, vs = _rows_of("k", k), _rows_of("v", v)
    _aligned_rows("k", k, ks)
    _aligned_rows("v", v, vs)
    with _On(_device(k, v, slot_map, *cache._tensors()), stream) as s:
        _call("dflash_kv8_append", s, ctypes.byref(cache._c), k.shape[0], _dt(k), _ptr(k), ks, _ptr(v), vs,
              _ptr(slot_map))


def kv8_read(cache, slot_map, stream=None):
    """The cached values at slot_map [rows] int64 as fp32 (k, v) [rows, kv heads, head_dim]; zero where the slot
    is negative (dflash_kv8_read)."""
    _tensor("slot_map", slot_map, torch.int64, (None,))
    with _On(_device(slot_map, *cache._tensors()), stream) as s:
        shape = (slot_map.shape[0], cache.n_kv_heads, cache.head_dim)
        k = torch.empty(shape, dtype=torch.float32, device=slot_map.device)
        v = torch.empty(shape, dtype=torch.float32, device=slot_map.device)
        _call("dflash_kv8_read", s, ctypes.byref(cache._c), shape[0], _ptr(slot_map), _ptr(k), _ptr(v))
    return k, v


def kv8_attention(cache, q, cu_q, ctx_len, block_table, mask="causal", tree_mask=None, scale=None, max_q=None,
                  out=None, lse=None, want_lse=False, workspace=None, stream=None):
    """Attention of rows cu_q[b] .. cu_q[b + 1] of q [rows, heads, head_dim] over the first ctx_len[b] tokens of
    block_table[b] (dflash_kv8_attention). mask: "none", "causal", or "tree" with tree_mask [rows, words] int32
    (as ddtree_build's, flattened over its requests). scale: 1 / sqrt(head_dim) if None. max_q: the most rows
    of a request where the host knows it (default: q's rows), which steers the choice of kernel and nothing
    else. workspace: a uint8 tensor of kv8_workspace(...) bytes; allocated for the call if None.
    Returns out [rows, heads, head_dim], or (out, lse [rows, heads] fp32) with want_lse."""
    a = _attn_args(cache, q, cu_q, ctx_len, block_table, mask, tree_mask, scale, max_q, out, lse)
    if workspace is not None:
        _tensor("workspace", workspace, torch.uint8, (None,))
    dev = _device(q, cu_q, ctx_len, block_table, tree_mask, out, lse, workspace, *cache._tensors())
    with _On(dev, stream) as s:
        if out is None:
            out = torch.empty(q.shape, dtype=q.dtype, device=dev)
        if want_lse and lse is None:
            lse = torch.empty(q.shape[:2], dtype=torch.float32, device=dev)
        if workspace is None:
            workspace = torch.empty((_workspace_bytes(cache, a),), dtype=torch.uint8, device=dev)
        a.out, a.lse = out.data_ptr(), None if lse is None else lse.data_ptr()
        a.workspace, a.workspace_bytes = workspace.data_ptr(), workspace.numel()
        _call("dflash_kv8_attention", s, ctypes.byref(cache._c), ctypes.byref(a))
    return (out, lse) if want_lse else out


def kv8_workspace(cache, q, cu_q, ctx_len, block_table, mask="causal", tree_mask=None, scale=None, max_q=None):
    """Bytes of workspace that kv8_attention needs for these arguments."""
    return _workspace_bytes(cache, _attn_args(cache, q, cu_q, ctx_len, block_table, mask, tree_mask, scale, max_q,
                                              None, None))


def _workspace_bytes(cache, a):
    n = _ffi.load().dflash_kv8_attention_workspace(ctypes.byref(cache._c), ctypes.byref(a))
    _need(n >= 0, "arguments out of range")
    return n


def _attn_args(cache, q, cu_q, ctx_len, block_table, mask, tree_mask, scale, max_q, out, lse):
    i4 = torch.int32
    _tensor("q", q, _FLOATS, (None, None, cache.head_dim), contiguous=False)
    rows, heads, hd = q.shape
    _tensor("ctx_len", ctx_len, i4, (None,))
    n = ctx_len.shape[0]
    _tensor("cu_q", cu_q, i4, (n + 1,))
    _tensor("block_table", block_table, i4, (n, None))
    _need(1 <= n <= 4096, f"1 to 4096 requests, not {n}")
    _need(1 <= block_table.shape[1] <= 1 << 24, "max_blocks must be in [1, 2^24]")
    _need(heads >= 1 and heads % cache.n_kv_heads == 0 and heads // cache.n_kv_heads <= 8,
          f"query heads must be a multiple of the {cache.n_kv_heads} kv heads, at most 8 for each, not {heads}")
    _need(mask in _MASKS, f"mask must be one of {sorted(_MASKS)}")
    _need((tree_mask is not None) == (mask == "tree"), "tree_mask goes with mask='tree'")
    if tree_mask is not None:
        _tensor("tree_mask", tree_mask, i4, (rows, None))
        _need(tree_mask.shape[1] >= 1, "tree_mask needs a word for each row")
    scale = 1.0 / math.sqrt(hd) if scale is None else float(scale)
    _need(scale > 0 and math.isfinite(scale), "scale must be positive and finite")
    if out is not None:
        _tensor("out", out, q.dtype, tuple(q.shape))
        _need(out.data_ptr() % 16 == 0, "out must be 16-byte aligned")
    if lse is not None:
        _tensor("lse", lse, torch.float32, (rows, heads))
    max_q = rows if max_q is None else int(max_q)
    _need(0 <= max_q < 1 << 31, "max_q must be in [0, 2^31)")
    stride = _rows_of("q", q)
    _aligned_rows("q", q, stride)
    return _ffi.KV8Attn(n_req=n, rows=rows, n_q_heads=heads, max_blocks=block_table.shape[1], max_q=max_q,
                        dtype=_dt(q), mask=_MASKS[mask], tree_words=0 if tree_mask is None else tree_mask.shape[1],
                        scale=scale, q=q.data_ptr(), q_stride=stride, cu_q=cu_q.data_ptr(),
                        ctx_len=ctx_len.data_ptr(), block_table=block_table.data_ptr(),
                        tree_mask=None if tree_mask is None else tree_mask.data_ptr())
