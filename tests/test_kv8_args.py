"""Refusals of the 8-bit cache's calls, at the C entries and in the binding, before any CUDA call:
none of this needs a GPU. Then the host-made rotary table against its definition."""
import ctypes

import pytest
import torch

import kv8_reference as R


@pytest.fixture(scope="module")
def lib():
    import block_diffusion_speculative_inject_gb300 as pkg
    from block_diffusion_speculative_inject_gb300 import build as b
    b.build()
    return pkg.library()


A, B, C, D = 4096, 8192, 12288, 16384       # addresses that are never read: the calls fail before


def test_c_entries_are_exported(lib):
    for n in ("dflash_page_plan", "dflash_rope_init", "dflash_rope_apply", "dflash_kv8_append", "dflash_kv8_read",
              "dflash_kv8_attention", "dflash_kv8_attention_workspace"):
        assert hasattr(lib, n)


def _plan(lib, n=1, width=4, pages=8, rows=4, ins=(A, B, C, D, 20480), outs=(24576, 28672, 32768, 36864, 40960, 45056)):
    ctx, add, table, stack, nf = ins
    nl, nfo, cu, ref, slot, pos = outs
    return lib.dflash_page_plan(None, n, width, pages, rows, ctx, add, table, stack, nf, nl, nfo, cu, ref, slot, pos)


def test_page_plan_refusals(lib):
    for kw in (dict(n=0), dict(n=4097), dict(width=0), dict(width=(1 << 24) + 1), dict(pages=0), dict(rows=-1),
               dict(pages=(1 << 24) + 1)):
        assert _plan(lib, **kw) == -1
    ins, outs = (A, B, C, D, 20480), (24576, 28672, 32768, 36864, 40960, 45056)
    for i in range(5):
        assert _plan(lib, ins=ins[:i] + (None,) + ins[i + 1:]) == -1
        assert _plan(lib, ins=ins[:i] + (ins[i] + 2,) + ins[i + 1:]) == -1
        for j in range(6):                   # an output that is an input
            assert _plan(lib, outs=outs[:j] + (ins[i],) + outs[j + 1:]) == -1
    for j in range(6):
        assert _plan(lib, outs=outs[:j] + (None,) + outs[j + 1:]) == -1
    assert _plan(lib, outs=outs[:4] + (outs[4] + 4,) + outs[5:]) == -1       # slot_map on 4 bytes


def _params(**over):
    from block_diffusion_speculative_inject_gb300 import _ffi
    p = _ffi.RopeParams(rot_dim=64, interleaved=0, scaling=0, theta=1e4, factor=1.0, original_positions=4096,
                        beta_fast=32, beta_slow=1)
    for k, v in over.items():
        setattr(p, k, v)
    return p


@pytest.mark.parametrize("over", [
    dict(rot_dim=0), dict(rot_dim=63), dict(rot_dim=258), dict(interleaved=2), dict(scaling=3), dict(scaling=-1),
    dict(theta=1.0), dict(theta=float("nan")), dict(theta=float("inf")), dict(scaling=1, factor=0.5),
    dict(scaling=1, factor=float("nan")), dict(scaling=2, factor=4.0, original_positions=0.0),
    dict(scaling=2, factor=4.0, beta_fast=1.0), dict(scaling=2, factor=4.0, beta_slow=0.0)])
def test_rope_init_refusals(lib, over):
    from block_diffusion_speculative_inject_gb300 import _ffi
    t = _ffi.RopeTable()
    assert lib.dflash_rope_init(ctypes.byref(_params(**over)), ctypes.byref(t)) == -1


@pytest.mark.parametrize("rot,theta,kw", [(64, 1e4, {}), (128, 1e6, dict(scaling="linear", factor=2.5)), (2, 5e5, {}),
                                          (128, 1e6, dict(scaling="yarn", factor=4.0, original=32768.0)),
                                          (20, 1e4, dict(scaling="yarn", factor=8.0, original=4096.0)), (256, 1e4, {})])
def test_rope_table_matches_its_definition(lib, rot, theta, kw):
    """Each frequency is a double (relative 2^-52 after the exp and the divisions: four roundings), kept to 2^-64."""
    from block_diffusion_speculative_inject_gb300 import Rope
    args = {("original_positions" if k == "original" else k): v for k, v in kw.items()}
    t = Rope(256, rot_dim=rot, theta=theta, **args)._c
    freq, mag = R.rope_freq(rot, theta, **kw)
    for i, f in enumerate(freq):
        assert abs(t.turn[i] / 2.0 ** 64 - float(f)) <= float(f) * 2.0 ** -49 + 2.0 ** -64
    assert all(t.turn[i] == 0 for i in range(rot // 2, 128))
    assert abs(t.magnitude - mag) <= 2.0 ** -23 * mag


@pytest.mark.parametrize("rot,theta,kw", [
    (64, 1e4, {}), (128, 1e6, {}), (256, 5e5, {}), (2, 1.5, {}), (6, 3e38, {}), (128, 1e7, dict(scaling="linear", factor=3.7)),
    (128, 1e6, dict(scaling="yarn", factor=4.0, original=32768.0)), (20, 1e4, dict(scaling="yarn", factor=40.0, original=4096.0)),
    (64, 1e4, dict(scaling="yarn", factor=2.5, original=4.0)), (256, 1e6, dict(scaling="yarn", factor=1.0, original=131072.0))])
def test_rope_table_to_its_last_bit(lib, rot, theta, kw):
    """Turns per position to 60 digits, the ramp as a fraction of whole numbers: the table holds the nearest multiple of
    2^-64 (half a unit, and 2^-20 for what over 90 bits leave)."""
    import math
    from decimal import Decimal, getcontext

    import numpy as np

    from block_diffusion_speculative_inject_gb300 import Rope
    f32 = lambda x: Decimal(float(np.float32(x)))  # noqa: E731
    args = {("original_positions" if k == "original" else k): v for k, v in kw.items()}
    t = Rope(256, rot_dim=rot, theta=theta, **args)._c
    getcontext().prec = 60
    pi, lt = Decimal("3.14159265358979323846264338327950288419716939937510582097494"), f32(theta).ln()
    factor = f32(kw.get("factor", 1.0))
    if kw.get("scaling") == "yarn":
        dim = lambda b: rot * math.log(kw["original"] / (b * 2 * math.pi)) / (2 * math.log(theta))  # noqa: E731
        lo, hi = max(math.floor(dim(32.0)), 0), min(math.ceil(dim(1.0)), rot - 1)
    for i in range(rot // 2):
        f = (Decimal(-2 * i) * lt / rot).exp()
        if kw.get("scaling") == "linear":
            f /= factor
        if kw.get("scaling") == "yarn":
            g = Decimal(0) if i <= lo else Decimal(1) if i >= hi else Decimal(i - lo) / Decimal(hi - lo)
            f = f / factor * g + f * (1 - g)
        assert abs(Decimal(t.turn[i]) - f / (2 * pi) * 2 ** 64) <= Decimal(0.5) + Decimal(2) ** -20, i


def test_rope_apply_refusals(lib):
    from block_diffusion_speculative_inject_gb300 import _ffi
    t = _ffi.RopeTable()
    assert lib.dflash_rope_init(ctypes.byref(_params()), ctypes.byref(t)) == 0

    def call(rows=2, nq=2, nk=1, hd=64, dt=1, pos=A, tr=0, q=B, qs=128, k=C, ks=64, qo=D, qos=128, ko=20480, kos=64, tab=t):
        return lib.dflash_rope_apply(None, ctypes.byref(tab) if tab else None, rows, nq, nk, hd, dt, pos, tr, q, qs, k, ks,
                                     qo, qos, ko, kos)
    for kw in (dict(rows=-1), dict(nq=0), dict(nk=-1), dict(hd=32), dict(hd=258), dict(dt=2), dict(tr=2), dict(qs=127),
               dict(ks=63), dict(qos=127), dict(kos=63), dict(pos=None), dict(q=None), dict(qo=None), dict(ko=None),
               dict(q=B + 1), dict(ko=20481), dict(pos=A + 2), dict(tab=None), dict(qo=B, qos=256), dict(ko=C, kos=128),
               dict(nq=1 << 20, qs=1 << 30, qos=1 << 30)):
        assert call(**kw) == -1, kw
    assert call(rows=0) == 0


def _cache(**over):
    from block_diffusion_speculative_inject_gb300 import _ffi
    c = _ffi.KV8Cache(n_pages=4, n_kv_heads=2, head_dim=64, k_pages=A, v_pages=B, k_scale=C, v_scale=D)
    for k, v in over.items():
        setattr(c, k, v)
    return c


BAD_CACHES = [dict(n_pages=0), dict(n_pages=(1 << 24) + 1), dict(n_kv_heads=0), dict(n_kv_heads=129), dict(head_dim=96),
              dict(k_pages=None), dict(v_pages=B + 8), dict(k_scale=None), dict(v_scale=D + 2)]


def test_append_and_read_refusals(lib):
    def append(cache=None, rows=3, dt=1, k=20480, ks=128, v=24576, vs=128, slot=28672):
        return lib.dflash_kv8_append(None, ctypes.byref(cache or _cache()), rows, dt, k, ks, v, vs, slot)
    for over in BAD_CACHES:
        assert append(cache=_cache(**over)) == -1
        assert lib.dflash_kv8_read(None, ctypes.byref(_cache(**over)), 3, A, B, C) == -1
    for kw in (dict(rows=-1), dict(dt=2), dict(k=None), dict(v=None), dict(slot=None), dict(k=20488), dict(v=24584),
               dict(ks=120), dict(vs=132), dict(slot=28676)):
        assert append(**kw) == -1, kw
    assert append(rows=0) == 0
    assert lib.dflash_kv8_append(None, None, 0, 1, None, 128, None, 128, None) == -1
    c = ctypes.byref(_cache())
    assert lib.dflash_kv8_read(None, c, -1, A, B, C) == -1
    assert lib.dflash_kv8_read(None, c, 2, None, B, C) == -1
    assert lib.dflash_kv8_read(None, c, 0, None, None, None) == 0


def _attn(**over):
    from block_diffusion_speculative_inject_gb300 import _ffi
    a = _ffi.KV8Attn(n_req=2, rows=3, n_q_heads=4, max_blocks=4, max_q=2, dtype=1, mask=1, tree_words=0, scale=0.125,
                     q=A, q_stride=256, cu_q=B, ctx_len=C, block_table=D, tree_mask=None, out=20480, lse=None,
                     workspace=24576, workspace_bytes=1 << 40)
    for k, v in over.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("over", [
    dict(n_req=0), dict(n_req=4097), dict(rows=-1), dict(n_q_heads=3), dict(n_q_heads=0), dict(n_q_heads=18),
    dict(max_blocks=0), dict(max_blocks=(1 << 24) + 1), dict(max_q=-1), dict(dtype=3), dict(mask=3), dict(mask=-1),
    dict(mask=2), dict(mask=2, tree_words=1), dict(scale=0.0), dict(scale=float("nan")), dict(scale=float("inf")),
    dict(q=None), dict(q=A + 8), dict(q_stride=255), dict(q_stride=260), dict(cu_q=None), dict(ctx_len=None),
    dict(block_table=None), dict(out=None), dict(out=20488), dict(lse=24578), dict(workspace=None),
    dict(workspace=24576 + 16), dict(workspace_bytes=16)])
def test_attention_refusals(lib, over):
    a = _attn(**over)
    assert lib.dflash_kv8_attention(None, ctypes.byref(_cache()), ctypes.byref(a)) == -1


def test_attention_refuses_bad_caches_and_takes_no_rows(lib):
    for over in BAD_CACHES:
        assert lib.dflash_kv8_attention(None, ctypes.byref(_cache(**over)), ctypes.byref(_attn())) == -1
    assert lib.dflash_kv8_attention(None, None, ctypes.byref(_attn())) == -1
    assert lib.dflash_kv8_attention(None, ctypes.byref(_cache()), None) == -1
    assert lib.dflash_kv8_attention(None, ctypes.byref(_cache()), ctypes.byref(_attn(rows=0, q=None, out=None))) == 0
    assert lib.dflash_kv8_attention_workspace(ctypes.byref(_cache(k_pages=None)), ctypes.byref(_attn(q=None))) > 0
    assert lib.dflash_kv8_attention_workspace(ctypes.byref(_cache()), ctypes.byref(_attn(n_q_heads=3))) == -1


def test_binding_refusals():
    """What the binding refuses is refused on CPU tensors alike; the last check is that they are on a GPU."""
    import block_diffusion_speculative_inject_gb300 as pkg
    i4 = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    e4 = lambda *s: torch.zeros(s, dtype=torch.uint8).view(torch.float8_e4m3fn)  # noqa: E731
    f4, bf = torch.zeros, lambda *s: torch.zeros(s, dtype=torch.bfloat16)
    cache = pkg.KV8Cache(e4(4, 2, 64, 64), e4(4, 2, 64, 64), f4(4, 2), f4(4, 2))
    bad = lambda f, *a, **k: pytest.raises(pkg.DFlashError, f, *a, **k)  # noqa: E731
    bad(lambda: pkg.KV8Cache(e4(4, 2, 64, 96), e4(4, 2, 96, 64), f4(4, 2), f4(4, 2)))
    bad(lambda: pkg.KV8Cache(e4(4, 2, 64, 128), e4(4, 2, 64, 128), f4(4, 2), f4(4, 2)))       # V not transposed
    bad(lambda: pkg.KV8Cache(e4(4, 2, 64, 64).view(torch.uint8), e4(4, 2, 64, 64), f4(4, 2), f4(4, 2)))
    bad(lambda: pkg.KV8Cache(e4(4, 2, 64, 64), e4(4, 2, 64, 64), f4(4, 2), f4(4, 3)))
    plan = dict(ctx_len=i4(3), n_new=i4(3), block_table=i4(3, 4), free_list=i4(8), n_free=i4(1), max_rows=5)
    for k, v in (("ctx_len", i4(3).long()), ("n_new", i4(2)), ("block_table", i4(4, 3).t()), ("n_free", i4(2)),
                 ("max_rows", -1), ("free_list", i4(0))):
        bad(lambda: pkg.page_plan(**dict(plan, **{k: v})))
    r = pkg.Rope(64)
    for a in ((i4(2), bf(3, 2, 64)), (i4(3), bf(3, 2, 128)), (i4(3), bf(3, 2, 64).half()), (i4(3), bf(3, 2, 64), f4(3, 2, 64)),
              (i4(3), bf(3, 64, 2).transpose(1, 2)), (i4(3).float(), bf(3, 2, 64)), (i4(3), bf(1, 2, 64).expand(3, 2, 64))):
        bad(lambda: pkg.rope(r, *a))
    bad(lambda: pkg.Rope(64, rot_dim=66))
    bad(lambda: pkg.Rope(64, rot_dim=3))
    bad(lambda: pkg.Rope(64, scaling="cubic"))
    bad(lambda: pkg.Rope(64, scaling="linear", factor=0.5))
    s8 = lambda n: torch.zeros(n, dtype=torch.int64)  # noqa: E731
    for a in ((bf(3, 2, 64), bf(3, 2, 64), i4(3)), (bf(3, 2, 64), bf(3, 2, 64), s8(2)), (bf(3, 1, 64), bf(3, 1, 64), s8(3)),
              (bf(3, 2, 64), f4(3, 2, 64), s8(3)), (bf(3, 129)[:, 1:].unflatten(1, (2, 64)), bf(3, 2, 64), s8(3))):
        bad(lambda: pkg.kv8_append(cache, *a))
    bad(lambda: pkg.kv8_read(cache, i4(3)))
    att = dict(q=bf(5, 4, 64), cu_q=i4(3), ctx_len=i4(2), block_table=i4(2, 4))
    for k, v in (("q", bf(5, 3, 64)), ("q", bf(5, 18, 64)), ("q", bf(5, 4, 128)), ("cu_q", i4(2)), ("block_table", i4(3, 4)),
                 ("mask", "full"), ("mask", "tree"), ("tree_mask", i4(5, 1)), ("scale", 0.0), ("out", f4(5, 4, 64)),
                 ("lse", bf(5, 4)), ("max_q", -1), ("workspace", i4(9))):
        bad(lambda: pkg.kv8_attention(cache, **dict(att, **{k: v})))
    with pytest.raises(pkg.DFlashError, match="CUDA device"):
        pkg.kv8_attention(cache, **att)
    with pytest.raises(pkg.DFlashError, match="CUDA device"):
        pkg.page_plan(**plan)


def test_binding_refuses_to_lose_a_gradient():
    """A result without a history, or a cache written past autograd, is refused where gradients are recorded."""
    import block_diffusion_speculative_inject_gb300 as pkg
    i4 = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    e4 = lambda *s: torch.zeros(s, dtype=torch.uint8).view(torch.float8_e4m3fn)  # noqa: E731
    x = lambda grad: torch.zeros((3, 2, 64), requires_grad=grad)  # noqa: E731
    cache = pkg.KV8Cache(e4(4, 2, 64, 64), e4(4, 2, 64, 64), torch.zeros(4, 2), torch.zeros(4, 2))
    r, slots = pkg.Rope(64), torch.zeros(3, dtype=torch.int64)
    att = (i4(2), i4(1), i4(1, 4))
    calls = [lambda g: pkg.rope(r, i4(3), x(g)), lambda g: pkg.rope(r, i4(3), x(False), x(g)),
             lambda g: pkg.rope(r, i4(3), x(False), q_out=x(g)), lambda g: pkg.kv8_append(cache, x(g), x(False), slots),
             lambda g: pkg.kv8_append(cache, x(False), x(g), slots), lambda g: pkg.kv8_attention(cache, x(g), *att),
             lambda g: pkg.kv8_attention(cache, x(False), *att, out=x(g))]
    for call in calls:
        with pytest.raises(pkg.DFlashError, match="no gradients"):
            call(True)
        with torch.no_grad(), pytest.raises(pkg.DFlashError, match="CUDA device"):      # taken as far as a CPU tensor goes
            call(True)
        with pytest.raises(pkg.DFlashError, match="CUDA device"):
            call(False)
