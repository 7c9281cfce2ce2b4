"""Refusals of the calls for verify rounds over long contexts (per-head norms, key bounds, choice of blocks, attention over
them, moves of rows, accepted paths), at the C entries and in the binding, before any CUDA call: none of this needs a GPU."""
import ctypes

import pytest
import torch

from test_kv8_args import BAD_CACHES, _attn, _cache, _params, lib  # noqa: F401

A, B, C, D, E, F, G, H = (4096 * i for i in range(1, 9))     # addresses that are never read: the calls fail before


def test_c_entries_are_exported(lib):  # noqa: F811
    for n in ("dflash_qk_norm_rope", "dflash_qk_norm_rope_backward", "dflash_qk_norm_rope_workspace", "dflash_kv8_bounds",
              "dflash_kv8_select", "dflash_kv8_select_workspace", "dflash_kv8_attention_blocks", "dflash_kv8_compact",
              "dflash_ddtree_path"):
        assert hasattr(lib, n)


def _table(lib):  # noqa: F811
    from block_diffusion_speculative_inject_gb300 import _ffi
    t = _ffi.RopeTable()
    assert lib.dflash_rope_init(ctypes.byref(_params()), ctypes.byref(t)) == 0
    return t


def test_norm_refusals(lib):  # noqa: F811
    t = _table(lib)

    def call(rows=2, nq=2, nk=1, hd=64, dt=1, pos=A, eps=1e-6, qw=G, kw=H, q=B, qs=128, k=C, ks=64, qo=D, qos=128, ko=E, kos=64, tab=t):
        return lib.dflash_qk_norm_rope(None, ctypes.byref(tab) if tab else None, rows, nq, nk, hd, dt, pos, eps, qw, kw, q, qs,
                                       k, ks, qo, qos, ko, kos)
    for kw in (dict(rows=-1), dict(nq=0), dict(nk=-1), dict(hd=32), dict(hd=258), dict(dt=2), dict(eps=0.0), dict(eps=-1.0),
               dict(eps=float("nan")), dict(eps=float("inf")), dict(qs=127), dict(ks=63), dict(qos=127), dict(kos=63),
               dict(pos=None), dict(q=None), dict(qo=None), dict(ko=None), dict(qw=None), dict(kw=None), dict(qw=G + 1),
               dict(q=B + 1), dict(ko=E + 1), dict(pos=A + 2), dict(tab=None), dict(qo=B, qos=256), dict(ko=C, kos=128),
               dict(nq=1 << 20, qs=1 << 30, qos=1 << 30)):
        assert call(**kw) == -1, kw
    assert call(rows=0) == 0


def test_norm_gradient_refusals(lib):  # noqa: F811
    from block_diffusion_speculative_inject_gb300 import _ffi
    t, need = _table(lib), lib.dflash_qk_norm_rope_workspace()
    assert need > 0

    def call(tab=t, **over):
        a = _ffi.QKNormRopeGrad(2, 2, 1, 64, 1, 1e-6, A, G, H, B, C, D, E, 128, 64, 128, 64, F, F + 512, 128, 64, F + 1024, F + 2048,
                                4096 * 16, need)
        for k, v in over.items():
            setattr(a, k, v)
        return lib.dflash_qk_norm_rope_backward(None, ctypes.byref(tab) if tab else None, ctypes.byref(a))
    for kw in (dict(rows=-1), dict(n_q_heads=0), dict(n_k_heads=-1), dict(head_dim=62), dict(dtype=5), dict(eps=0.0),
               dict(positions=None), dict(q_weight=None), dict(k_weight=H + 1), dict(q=None), dict(grad_q_out=None),
               dict(grad_k_out=None), dict(q_stride=127), dict(grad_k_out_stride=63), dict(dq_stride=100), dict(dk=None),
               dict(dq=B), dict(dk=C), dict(dq=D, dq_stride=256), dict(dk=E, dk_stride=72), dict(dq_weight=None),
               dict(dk_weight=None), dict(dq_weight=F + 2), dict(workspace=None), dict(workspace=4096 * 16 + 8),
               dict(workspace_bytes=need - 1), dict(tab=None)):
        assert call(**kw) == -1, kw
    assert lib.dflash_qk_norm_rope_backward(None, ctypes.byref(t), None) == -1


def test_bounds_refusals(lib):  # noqa: F811
    def call(cache=None, bounds=E, n=2, width=4, old=F, new=G, table=H):
        return lib.dflash_kv8_bounds(None, ctypes.byref(cache or _cache()), bounds, n, width, old, new, table)
    for over in BAD_CACHES:
        assert call(cache=_cache(**over)) == -1
    for kw in (dict(n=0), dict(n=4097), dict(width=0), dict(width=(1 << 24) + 1), dict(bounds=None), dict(bounds=E + 8),
               dict(old=None), dict(new=None), dict(table=None), dict(old=F + 2), dict(new=G + 1), dict(table=H + 2)):
        assert call(**kw) == -1, kw
    assert lib.dflash_kv8_bounds(None, None, E, 2, 4, F, G, H) == -1


def _choice(**over):
    from block_diffusion_speculative_inject_gb300 import _ffi
    a = _ffi.KV8Choice(n_req=2, rows=3, n_q_heads=4, max_blocks=4, n_select=2, keep_first=1, keep_last=1, dtype=1, q=A, q_stride=256,
                       cu_q=B, ctx_len=C, block_table=D, bounds=E, blocks=F, workspace=G, workspace_bytes=1 << 40)
    for k, v in over.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("over", [
    dict(n_req=0), dict(n_req=4097), dict(rows=-1), dict(n_q_heads=3), dict(n_q_heads=0), dict(n_q_heads=18), dict(max_blocks=0),
    dict(max_blocks=(1 << 24) + 1), dict(n_select=0), dict(n_select=(1 << 24) + 1), dict(n_req=4096, n_select=1 << 18),
    dict(keep_first=-1), dict(keep_last=-1), dict(keep_first=(1 << 24) + 1), dict(dtype=3), dict(q=None), dict(q=A + 8),
    dict(q_stride=255), dict(q_stride=260), dict(cu_q=None), dict(ctx_len=None), dict(block_table=None), dict(bounds=None),
    dict(bounds=E + 8), dict(blocks=None), dict(blocks=F + 2), dict(workspace=None), dict(workspace=G + 16), dict(workspace_bytes=63)])
def test_select_refusals(lib, over):  # noqa: F811
    assert lib.dflash_kv8_select(None, ctypes.byref(_cache()), ctypes.byref(_choice(**over))) == -1


def test_select_workspace(lib):  # noqa: F811
    size = lambda cache, a: lib.dflash_kv8_select_workspace(ctypes.byref(cache), ctypes.byref(a))  # noqa: E731
    assert size(_cache(k_pages=None), _choice(q=None)) >= 2 * 2 * 4 * 4
    assert size(_cache(n_kv_heads=128), _choice(n_req=4096, n_q_heads=128, q_stride=8192, max_blocks=1 << 24)) >= 4096 * 128 * 4 << 24
    assert size(_cache(), _choice(n_q_heads=3)) == -1
    for over in BAD_CACHES[:5]:
        assert size(_cache(**over), _choice()) == -1
    for over in (dict(k_scale=None), dict(k_scale=C + 2)):
        assert lib.dflash_kv8_select(None, ctypes.byref(_cache(**over)), ctypes.byref(_choice())) == -1
    assert lib.dflash_kv8_select(None, None, ctypes.byref(_choice())) == -1
    assert lib.dflash_kv8_select(None, ctypes.byref(_cache()), None) == -1


def test_attention_blocks_refusals(lib):  # noqa: F811
    def call(blocks=H, n=3, **over):
        return lib.dflash_kv8_attention_blocks(None, ctypes.byref(_cache()), ctypes.byref(_attn(**over)), blocks, n)
    for kw in (dict(blocks=None), dict(blocks=H + 2), dict(n=0), dict(n=(1 << 24) + 1), dict(n_req=0), dict(q=None), dict(out=None),
               dict(workspace_bytes=16), dict(scale=0.0), dict(mask=2)):
        assert call(**kw) == -1, kw
    assert call(rows=0, q=None, out=None) == 0


def test_compact_refusals(lib):  # noqa: F811
    from block_diffusion_speculative_inject_gb300 import _ffi

    def call(caches=None, layers=None, n=2, width=4, most=3, base=E, keep=F, count=G, table=H):
        caches = caches or [_cache()]
        array = (_ffi.KV8Cache * len(caches))(*caches)
        return lib.dflash_kv8_compact(None, len(caches) if layers is None else layers, array, n, width, most, base, keep, count, table)
    for over in BAD_CACHES:
        assert call([_cache(**over)]) == -1
    far = dict(k_pages=1 << 20, v_pages=2 << 20, k_scale=3 << 20, v_scale=4 << 20)
    for over in (dict(far, n_pages=5), dict(far, n_kv_heads=1), dict(far, head_dim=128), dict(far, k_pages=A), dict(far, v_pages=B),
                 dict(far, k_scale=C), dict(far, v_scale=D), {}):
        assert call([_cache(), _cache(**over)]) == -1, over
    for kw in (dict(layers=0), dict(layers=129), dict(layers=-1), dict(n=0), dict(n=4097), dict(width=0), dict(width=(1 << 24) + 1),
               dict(most=0), dict(most=(1 << 24) + 1), dict(base=None), dict(keep=None), dict(count=None), dict(table=None),
               dict(base=E + 1), dict(keep=F + 2), dict(count=G + 2), dict(table=H + 2)):
        assert call(**kw) == -1, kw
    assert lib.dflash_kv8_compact(None, 1, None, 2, 4, 3, E, F, G, H) == -1


def test_path_refusals(lib):  # noqa: F811
    def call(n=1, depth=7, budget=8, ptrs=(A, B, C, D, E, F)):
        return lib.dflash_ddtree_path(None, n, depth, budget, *ptrs)
    for kw in (dict(n=-1), dict(depth=0), dict(depth=32), dict(budget=0), dict(budget=1025)):
        assert call(**kw) == -1, kw
    for i in range(6):
        p = [A, B, C, D, E, F]
        p[i] = None
        assert call(ptrs=p) == -1
    assert call(n=0, ptrs=[None] * 6) == 0


def _things():
    import block_diffusion_speculative_inject_gb300 as pkg
    i4 = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    e4 = lambda *s: torch.zeros(s, dtype=torch.uint8).view(torch.float8_e4m3fn)  # noqa: E731
    bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16)  # noqa: E731
    cache = lambda n=4: pkg.KV8Cache(e4(n, 2, 64, 64), e4(n, 2, 64, 64), torch.ones(n, 2), torch.ones(n, 2))  # noqa: E731
    return pkg, i4, e4, bf, cache


def test_binding_refusals():
    """What the binding refuses is refused on CPU tensors alike; the last check is that they are on a GPU."""
    pkg, i4, e4, bf, cache = _things()
    f4, s1 = torch.zeros, lambda *s: torch.zeros(s, dtype=torch.int8)  # noqa: E731

    def refuses(f, base, changes):
        for over in changes:
            with pytest.raises(pkg.DFlashError):
                f(**dict(base, **over))
        with pytest.raises(pkg.DFlashError, match="CUDA device"):
            f(**base)
    norm = dict(table=pkg.Rope(64), positions=i4(3), q=bf(3, 2, 64), k=bf(3, 1, 64), q_weight=bf(64), k_weight=bf(64))
    bad = [dict(positions=i4(2)), dict(positions=i4(3).long()), dict(q=bf(3, 2, 128)), dict(k=f4(3, 1, 64)), dict(k=None),
           dict(k_weight=None), dict(q_weight=bf(63)), dict(q_weight=f4(64)), dict(eps=0.0), dict(eps=float("nan")), dict(eps=1e-60),
           dict(q=bf(3, 0, 64)), dict(q=bf(3, 64, 2).transpose(1, 2))]
    refuses(pkg.qk_norm_rope, norm, bad + [dict(q_out=bf(3, 1, 64)), dict(k_out=f4(3, 1, 64)), dict(k=None, k_weight=None, k_out=bf(3, 1, 64))])
    wide = bf(3, 4, 64)
    refuses(pkg.qk_norm_rope, norm, [dict(q=wide[:, :2], q_out=wide.flatten()[:384].view(3, 2, 64))])
    grad = dict(norm, grad_q_out=bf(3, 2, 64), grad_k_out=bf(3, 1, 64))
    refuses(pkg.qk_norm_rope_backward, grad, bad + [dict(grad_q_out=None), dict(grad_k_out=None), dict(grad_q_out=f4(3, 2, 64)),
                                                    dict(dq=bf(2, 2, 64)), dict(dk=bf(3, 2, 64)), dict(workspace=i4(4))])
    q = bf(3, 2, 64)
    refuses(pkg.qk_norm_rope_backward, grad, [dict(q=q, dq=q)])
    bounds = dict(cache=cache(), bounds=s1(4, 2, 2, 64), block_table=i4(3, 5), old_len=i4(3), new_len=i4(3))
    refuses(pkg.kv8_bounds, bounds, [dict(bounds=s1(4, 2, 64)), dict(bounds=i4(4, 2, 2, 64)), dict(bounds=s1(5, 2, 2, 64)),
                                     dict(bounds=s1(4 * 256 + 8)[8:].view(4, 2, 2, 64)), dict(old_len=i4(2)), dict(new_len=i4(4)),
                                     dict(block_table=i4(5, 3).t()), dict(block_table=i4(3, 0))])
    choice = dict(cache=cache(), bounds=s1(4, 2, 2, 64), q=bf(5, 4, 64), cu_q=i4(4), ctx_len=i4(3), block_table=i4(3, 5), n_select=2)
    refuses(pkg.kv8_select, choice, [dict(n_select=0), dict(n_select=1 << 25), dict(keep_first=-1), dict(keep_last=-1), dict(q=bf(5, 3, 64)),
                                     dict(q=bf(5, 18, 64)), dict(q=bf(5, 4, 64).half()), dict(cu_q=i4(3)), dict(ctx_len=i4(2)),
                                     dict(bounds=s1(4, 2, 2, 128)), dict(out=i4(3, 2, 3)), dict(out=i4(3, 2, 2).long()),
                                     dict(workspace=i4(64)), dict(block_table=i4(2, 5))])
    att = dict(cache=cache(), q=bf(5, 4, 64), cu_q=i4(3), ctx_len=i4(2), block_table=i4(2, 4), blocks=i4(2, 2, 3))
    refuses(pkg.kv8_attention, att, [dict(blocks=i4(2, 3)), dict(blocks=i4(2, 1, 3)), dict(blocks=i4(3, 2, 3)), dict(blocks=i4(2, 2, 0)),
                                     dict(blocks=i4(2, 2, 3).long()), dict(blocks=i4(2, 3, 2).transpose(1, 2))])
    one = cache()
    move = dict(caches=[one, cache()], block_table=i4(2, 4), base_len=i4(2), keep=i4(2, 3), n_keep=i4(2))
    refuses(pkg.kv8_compact, move, [dict(caches=[]), dict(caches=[one, one]), dict(caches=[one, cache(5)]), dict(caches=[one, 3]),
                                    dict(caches=[cache() for _ in range(129)]), dict(base_len=i4(3)), dict(keep=i4(3, 3)), dict(keep=i4(2, 0)),
                                    dict(n_keep=i4(2).long()), dict(block_table=i4(4, 2).t())])
    refuses(pkg.kv8_compact, dict(move, caches=pkg.KV8Layers([one, cache()])), [])
    tree = dict(tok=i4(2, 8), parent=i4(2, 8), n_nodes=i4(2))
    path = dict(tree=tree, L=7, target_next=i4(2, 9))
    refuses(pkg.ddtree_path, path, [dict(L=0), dict(L=32), dict(target_next=i4(2, 8)), dict(target_next=i4(2, 9).long()),
                                    dict(tree=dict(tree, parent=i4(2, 7))), dict(tree=dict(tree, n_nodes=i4(3)))])


def test_binding_refuses_to_lose_a_gradient():
    pkg, i4, e4, bf, cache = _things()
    x = lambda heads, grad: torch.zeros((3, heads, 64), requires_grad=grad)  # noqa: E731
    w = lambda grad: torch.zeros(64, requires_grad=grad)  # noqa: E731
    t = pkg.Rope(64)

    def norm(f, *more):
        for i in range(4):
            for grad in (True, False):
                a = [x(2, i == 0 and grad), x(1, i == 1 and grad), w(i == 2 and grad), w(i == 3 and grad)]
                with pytest.raises(pkg.DFlashError, match="no gradients" if grad else "CUDA device"):
                    f(t, i4(3), *a, *more)
                with torch.no_grad(), pytest.raises(pkg.DFlashError, match="CUDA device"):
                    f(t, i4(3), *a, *more)
    norm(pkg.qk_norm_rope)
    norm(pkg.qk_norm_rope_backward, x(2, False), x(1, False))
    with pytest.raises(pkg.DFlashError, match="no gradients"):
        pkg.kv8_attention(cache(), x(2, True), i4(2), i4(1), i4(1, 4), blocks=i4(1, 2, 3))
    # the choice is whole numbers: a q that requires a gradient loses none
    with pytest.raises(pkg.DFlashError, match="CUDA device"):
        pkg.kv8_select(cache(), torch.zeros((4, 2, 2, 64), dtype=torch.int8), x(2, True), i4(2), i4(1), i4(1, 4), 2)


def test_layers_stay_as_they_were_laid_out(monkeypatch):
    """What kv8_compact hands to the library is the array that was checked: its caches can be neither added to nor replaced."""
    import block_diffusion_speculative_inject_gb300.kv8 as kv8
    pkg, i4, e4, bf, cache = _things()
    given = [cache(), cache()]
    layers = pkg.KV8Layers(given)
    seen = []
    monkeypatch.setattr(kv8, "_device", lambda *a: layers._dev)
    monkeypatch.setattr(kv8, "_on", lambda dev, stream, body: body(0))
    monkeypatch.setattr(kv8, "_call", lambda name, s, n, array, *a: seen.append((n, array)))
    move = (i4(2, 4), i4(2), i4(2, 3), i4(2))

    def laid_out():
        pkg.kv8_compact(layers, *move)
        n, array = seen.pop()
        assert n == len(array) == 2
        assert [c.k_pages for c in array] == [c.k_pages.data_ptr() for c in given[:2]]
    laid_out()
    given.append(cache())                              # (the caller's own list)
    laid_out()
    for change in (lambda: layers.caches.append(cache()), lambda: layers.caches.pop(), lambda: layers.caches.__setitem__(0, cache()),
                   lambda: setattr(layers, "caches", given), lambda: setattr(layers, "_array", None), lambda: delattr(layers, "caches")):
        with pytest.raises((AttributeError, pkg.DFlashError)):
            change()
        laid_out()


def test_caches_stay_as_they_were_laid_out():
    """A cache's tensors and sizes are what the library was given: another tensor in their place would leave the calls with
    the addresses of the old one, whose memory may be another's by then."""
    pkg, i4, e4, bf, cache = _things()
    c = cache()
    was = [t.data_ptr() for t in c._tensors()]
    for name in ("k_pages", "v_pages", "k_scale", "v_scale", "n_pages", "n_kv_heads", "head_dim"):
        with pytest.raises(pkg.DFlashError, match=name):
            setattr(c, name, getattr(cache(8), name))
        with pytest.raises(pkg.DFlashError, match=name):
            delattr(c, name)
    assert [t.data_ptr() for t in c._tensors()] == was == [c._c.k_pages, c._c.v_pages, c._c.k_scale, c._c.v_scale]
    assert c.n_pages == c._c.n_pages == 4


def test_norm_refuses_outputs_over_other_inputs(lib):  # noqa: F811
    """In place is the same tensor in and out. An output over another one that is still to be read, or two outputs over one
    another, would be a race: refused, at the C entries and in the binding, where the heads are as many."""
    from block_diffusion_speculative_inject_gb300 import _ffi
    t = _table(lib)

    def forward(qo, ko, q=B, k=C):
        return lib.dflash_qk_norm_rope(None, ctypes.byref(t), 2, 2, 2, 64, 1, A, 1e-6, G, H, q, 128, k, 128, qo, 128, ko, 128)
    for qo, ko in ((C, E), (C, C), (D, B), (C, B), (D, D)):
        assert forward(qo, ko) == -1
    p = [32768 + 4096 * i for i in range(11)]
    pos, qw, kw, q, k, gq, gk, dq, dk, dqw, dkw = p

    def backward(dq, dk):
        x = _ffi.QKNormRopeGrad(2, 2, 2, 64, 1, 1e-6, pos, qw, kw, q, k, gq, gk, 128, 128, 128, 128, dq, dk, 128, 128, dqw, dkw, A, 1 << 30)
        return lib.dflash_qk_norm_rope_backward(None, ctypes.byref(t), ctypes.byref(x))
    for a, b in ((k, dk), (gk, dk), (dk, dk), (dq, q), (dq, gq), (gk, gq), (q, dk), (dq, k)):
        assert backward(a, b) == -1
    pkg, i4, e4, bf, cache = _things()
    x = [bf(3, 2, 64) for _ in range(6)]
    norm = lambda **kw: pkg.qk_norm_rope(pkg.Rope(64), i4(3), x[0], x[1], bf(64), bf(64), **kw)  # noqa: E731
    grad = lambda **kw: pkg.qk_norm_rope_backward(pkg.Rope(64), i4(3), x[0], x[1], bf(64), bf(64), x[2], x[3], **kw)  # noqa: E731
    for f, over in ((norm, dict(q_out=x[1])), (norm, dict(k_out=x[0])), (norm, dict(q_out=x[4], k_out=x[4])), (grad, dict(dq=x[1])),
                    (grad, dict(dk=x[0])), (grad, dict(dq=x[3])), (grad, dict(dk=x[2])), (grad, dict(dq=x[4], dk=x[4]))):
        with pytest.raises(pkg.DFlashError, match="must not be"):
            f(**over)
    for f, over in ((norm, dict(q_out=x[0], k_out=x[1])), (grad, dict(dq=x[2], dk=x[3])), (grad, dict(dq=x[4], dk=x[5]))):
        with pytest.raises(pkg.DFlashError, match="CUDA device"):
            f(**over)
