"""Per-head norms with rotary positions and their gradient, key bounds, the choice of blocks, attention over them and the move
of kept rows on the GPU against 64-bit references (kv8_long_reference.py), alone and run together as a verify round over
long contexts runs them.

Tolerances (half steps: bf16 2^-8, fp32 2^-24, relative to the value; u = 2^-24 below):
  norm      r = 1 / sqrt(mean + eps): the sum of squares adds at most 16 values in a row and 5 times across lanes, all
            positive (21 u), the division, eps and the root round once each: (21 + 2) / 2 + 1 < 13 u. x r w adds 2 u:
            n is off by 15 u of itself, 9e-7. The rotation adds (|x| + |y|) magnitude 8e-7 for a pair (test_gpu_kv8.py),
            so the output is within S 1.7e-6, S = (|n_a| + |n_b|) magnitude (|n| where not turned), plus its rounding.
  gradient  n' = R^T y' within E = S 8e-7, S of y'. g = n' w: within G = E |w| + |g| u. The sum of g x (a product of two
            roundings, 16 in a row, 5 across) is within sum(G |x|) + 24 u sum |g x|; m = r mean(g x) is within
            M = r (sum(G |x|) + 24 u sum |g x|) / hd + 16 u |m| (r 13, the product and the division 3);
            x' = r (g - x r m) within r (G + |x r| M + |x r m| 16 u) + 18 u (|r g| + |r x r m|), plus its rounding.
            The weights' gradient: each term n' x r is within (E + 16 u |n'|) |x r|, and the sum of N of them in chains of at
            most c additions within c u sum |n' x r|.
  bounds, choice, moves: equal.
  attention over blocks: test_gpu_kv8.py's for attention.
"""
import math

import pytest
import torch

import kv8_long_reference as L
import kv8_reference as R
from test_gpu_kv8 import HALF, _attn_case, _cache_cpu, _cum, _i4, _same_cache, _to_gpu

pytestmark = pytest.mark.gpu

PAGE = 64
U = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _built():
    from block_diffusion_speculative_inject_gb300 import build
    build.build()


# ---------------------------------------------------------------- norms with rotary positions
NORM_SHAPES = [
    (1, 1, 0, 64, 64, False, "none"), (16, 32, 8, 128, 128, False, "none"), (37, 5, 3, 64, 32, True, "linear"),
    (9, 40, 8, 128, 64, False, "yarn"), (33, 3, 1, 256, 256, True, "none"), (5, 2, 2, 70, 20, False, "yarn"),
    (3, 1, 1, 2, 2, False, "none"), (7, 2, 1, 96, 96, False, "none"), (4, 3, 2, 255, 30, True, "linear"),
    (2, 300, 20, 64, 64, True, "none"), (130, 1, 1, 32, 16, False, "none"), (6, 7, 1, 80, 80, True, "yarn")]


def _norm_case(seed, rows, nq, nk, hd, rot, inter, scaling, dtype):
    from block_diffusion_speculative_inject_gb300 import Rope
    g = torch.Generator().manual_seed(seed)
    table = Rope(hd, rot_dim=rot, theta=1e5, interleaved=inter, scaling=scaling, factor=4.0, original_positions=4096.0)
    freq, mag = R.rope_freq(rot, 1e5, scaling, 4.0, 4096.0)
    pos = torch.randint(0, 200000, (rows,), generator=g, dtype=torch.int32)
    x = {}
    for name, heads in (("q", nq), ("k", nk)):
        size = torch.exp(2 * torch.randn((rows, heads, 1), generator=g))
        x[name] = (torch.randn((rows, heads, hd), generator=g) * size).to(dtype)
        x["d" + name] = torch.randn((rows, heads, hd), generator=g).to(dtype)
        x["w" + name] = torch.randn((hd,), generator=g).to(dtype)
    if rows > 2:
        x["q"][1, 0] = 0                                       # a head of zeros
        x["q"][2, 0] *= 1e-10 if dtype == torch.float32 else 1e-6
    return table, freq, mag, pos, x


def _check_norm(y, x, w, pos, rot, freq, mag, inter, eps):
    n, _ = L.norm(x.double(), w.double(), eps)
    want = R.rope(n, pos.tolist(), rot, freq, mag, inter)
    tol = L.size_of_pair(n, rot, inter, mag) * 1.7e-6 + want.abs() * HALF[y.dtype]
    assert bool(((y.cpu().double() - want).abs() <= tol).all())


def _check_grad(dx, dw, x, w, dy, pos, rot, freq, mag, inter, eps, chain):
    x, w, dy = x.double(), w.double(), dy.double()
    hd = x.shape[-1]
    _, r = L.norm(x, w, eps)
    dn = R.rope(dy, pos.tolist(), rot, freq, mag, inter, transpose=True)
    E = L.size_of_pair(dy, rot, inter, mag) * 8e-7
    g = dn * w
    G = E * w.abs() + g.abs() * U
    m = r * (g * x).sum(-1, keepdim=True) / hd
    want = r * (g - x * r * m)
    u = (x * r).abs()
    M = r * ((G * x.abs()).sum(-1, keepdim=True) + 24 * U * (g * x).abs().sum(-1, keepdim=True)) / hd + 16 * U * m.abs()
    tol = r * (G + u * M + u * m.abs() * 16 * U) + 18 * U * r * (g.abs() + u * m.abs()) + want.abs() * HALF[dx.dtype]
    assert bool(((dx.cpu().double() - want).abs() <= tol).all())
    t = (dn * x * r).abs()
    ww = (dn * x * r).sum((0, 1))
    wtol = ((E + 16 * U * dn.abs()) * u).sum((0, 1)) + chain * U * t.sum((0, 1))
    assert bool(((dw.cpu().double() - ww).abs() <= wtol).all())
    return want


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,nq,nk,hd,rot,inter,scaling", NORM_SHAPES)
def test_norm_and_gradient(dtype, rows, nq, nk, hd, rot, inter, scaling):
    from block_diffusion_speculative_inject_gb300 import qk_norm_rope, qk_norm_rope_backward
    table, freq, mag, pos, x = _norm_case(rows + hd, rows, nq, nk, hd, rot, inter, scaling, dtype)
    d = {n: t.cuda() for n, t in x.items()}
    eps = 1e-6
    k = (d["k"], d["wk"], d["dk"]) if nk else (None, None, None)
    q, kk = qk_norm_rope(table, pos.cuda(), d["q"], k[0], d["wq"], k[1], eps=eps)
    dq, dk, dqw, dkw = qk_norm_rope_backward(table, pos.cuda(), d["q"], k[0], d["wq"], k[1], d["dq"], k[2], eps=eps)
    args = (pos, rot, freq, mag, inter, eps)
    _check_norm(q, x["q"], x["wq"], *args)
    # a lane adds at most 8 terms for each head here, then 8 warps and 5 shuffles, 19 CTAs' sums and 5 shuffles
    chain = 8 * max(nq, nk) + 8 + 5 + 19 + 5
    _check_grad(dq, dqw, x["q"], x["wq"], x["dq"], *args, chain)
    if nk:
        _check_norm(kk, x["k"], x["wk"], *args)
        _check_grad(dk, dkw, x["k"], x["wk"], x["dk"], *args, chain)
    else:
        assert kk is None and dk is None and dkw is None


def test_norm_gradient_is_the_formulas_and_differences():
    """The kernel's gradients against autograd of the definition in 64 bits and against its central differences."""
    from block_diffusion_speculative_inject_gb300 import qk_norm_rope_backward
    table, freq, mag, pos, x = _norm_case(5, 4, 2, 1, 64, 48, True, "yarn", torch.float32)
    eps = 1e-5
    dq, dk, dqw, dkw = qk_norm_rope_backward(table, pos.cuda(), x["q"].cuda(), x["k"].cuda(), x["wq"].cuda(), x["wk"].cuda(),
                                             x["dq"].cuda(), x["dk"].cuda(), eps=eps)
    for name, dx, dw in (("q", dq, dqw), ("k", dk, dkw)):
        v, w = x[name].double().requires_grad_(), x["w" + name].double().requires_grad_()

        def loss(v, w):
            return (R.rope(L.norm(v, w, eps)[0], pos.tolist(), 48, freq, mag, True) * x["d" + name].double()).sum()
        loss(v, w).backward()
        want = _check_grad(dx, dw, x[name], x["w" + name], x["d" + name], pos, 48, freq, mag, True, eps, 8 * 2 + 37)
        assert float((want - v.grad).abs().max()) <= 1e-9 * float(v.grad.abs().max())
        for at in ((0, 0, 0), (3, 0, 63), (3, 0, 47)):
            h = 1e-6 * max(1.0, float(x[name][at].abs()))
            a, b = x[name].double(), x[name].double()
            a[at] += h
            b[at] -= h
            diff = float((loss(a, w) - loss(b, w)).detach()) / (2 * h)
            # the difference's own error: h^2 of the third derivative and 2^-52 |loss| / h
            assert abs(diff - float(dx[at])) <= 1e-4 * (float(dx.abs().max()) + abs(diff))
        a = x["w" + name].double()
        for i in (0, 47, 63):
            e = torch.zeros(64, dtype=torch.float64)
            e[i] = 1e-3
            diff = float(loss(x[name].double(), a + e) - loss(x[name].double(), a - e)) / 2e-3      # (linear in the weight)
            assert abs(diff - float(dw[i])) <= 1e-5 * (float(dw.abs().max()) + abs(diff))


@pytest.mark.parametrize("dtype,inter,shift,odd", [(torch.bfloat16, False, 0, 8), (torch.bfloat16, True, 1, 1), (torch.float32, False, 1, 1),
                                                   (torch.float32, True, 0, 4), (torch.bfloat16, False, 2, 2), (torch.float32, False, 2, 2)])
def test_norm_strided_in_place_and_the_same_bits(dtype, inter, shift, odd):
    """Rows of a fused projection at odd places (every width of access), in place, and with a workspace of the caller: the
    same bits as packed new ones where the accesses are alike, within the tolerance in any case; neighbours untouched."""
    from block_diffusion_speculative_inject_gb300 import qk_norm_rope, qk_norm_rope_backward, qk_norm_rope_workspace
    rows, nq, nk, hd = 11, 4, 2, 64
    table, freq, mag, pos, x = _norm_case(3, rows, nq, nk, hd, 32, inter, "none", dtype)
    eps = 1e-6
    width = (nq + nk) * hd + odd
    args = (pos, 32, freq, mag, inter, eps)

    def rows_of(a, b):
        buf = torch.full((rows, width + shift), 7.0, dtype=dtype)
        buf[:, shift:shift + nq * hd] = a.flatten(1)
        buf[:, shift + nq * hd:shift + (nq + nk) * hd] = b.flatten(1)
        buf = buf.cuda()
        return buf, buf[:, shift:shift + nq * hd].unflatten(1, (nq, hd)), buf[:, shift + nq * hd:shift + (nq + nk) * hd].unflatten(1, (nk, hd))
    w = [x[n].cuda() for n in ("wq", "wk")]
    buf, q, k = rows_of(x["q"], x["k"])
    gbuf, gq, gk = rows_of(x["dq"], x["dk"])
    qc, kc = q.contiguous(), k.contiguous()
    want = qk_norm_rope(table, pos.cuda(), qc, kc, *w, eps=eps)
    ws = torch.empty(qk_norm_rope_workspace(), dtype=torch.uint8, device="cuda")
    ws.fill_(255)
    grads = qk_norm_rope_backward(table, pos.cuda(), q, k, *w, gq, gk, eps=eps, dq=gq, dk=gk, workspace=ws)
    assert grads[0].data_ptr() == gq.data_ptr()
    _check_grad(gq, grads[2], x["q"], x["wq"], x["dq"], *args, 8 * 4 + 37)
    _check_grad(gk, grads[3], x["k"], x["wk"], x["dk"], *args, 8 * 4 + 37)
    qk_norm_rope(table, pos.cuda(), q, k, *w, eps=eps, q_out=q, k_out=k)
    _check_norm(q, x["q"], x["wq"], *args)
    _check_norm(k, x["k"], x["wk"], *args)
    if shift == 0 and odd % 8 == 0:
        assert torch.equal(q, want[0]) and torch.equal(k, want[1])
    for b in (buf, gbuf):
        assert bool((b[:, :shift] == 7).all()) and bool((b[:, shift + (nq + nk) * hd:] == 7).all())


def test_norm_many_rows_repeat_and_no_rows():
    """More tiles than CTAs; the same bits twice; no rows: the weights' gradients are zero."""
    from block_diffusion_speculative_inject_gb300 import Rope, qk_norm_rope, qk_norm_rope_backward
    g = torch.Generator(device="cuda").manual_seed(1)
    rows, nq, nk, hd = 9001, 4, 2, 64
    t = Rope(hd)
    pos = torch.arange(rows, dtype=torch.int32, device="cuda")
    q, gq = (torch.randn((rows, nq, hd), generator=g, device="cuda") for _ in range(2))
    k, gk = (torch.randn((rows, nk, hd), generator=g, device="cuda") for _ in range(2))
    w = torch.ones(hd, device="cuda")
    a = qk_norm_rope_backward(t, pos, q, k, w, w, gq, gk)
    b = qk_norm_rope_backward(t, pos, q, k, w, w, gq, gk)
    assert all(torch.equal(x, y) for x, y in zip(a, b))
    freq, mag = R.rope_freq(hd, 1e6)
    _check_grad(a[0], a[2], q.cpu(), w.cpu(), gq.cpu(), pos.cpu(), hd, freq, mag, False, 1e-6, 9001 * 4 // 608 + 60)
    _check_grad(a[1], a[3], k.cpu(), w.cpu(), gk.cpu(), pos.cpu(), hd, freq, mag, False, 1e-6, 9001 * 4 // 608 + 60)
    e = q[:0]
    out = qk_norm_rope(t, pos[:0], e, k[:0], w, w)
    assert out[0].shape == (0, nq, hd)
    z = qk_norm_rope_backward(t, pos[:0], e, k[:0], w, w, e, k[:0])
    assert bool((z[2] == 0).all()) and bool((z[3] == 0).all()) and z[0].shape == (0, nq, hd)


def test_norm_most_rows():
    """The largest number of rows, in place: a CTA's last rows are near 2^31."""
    from block_diffusion_speculative_inject_gb300 import Rope, qk_norm_rope
    rows = 2 ** 31 - 1
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 40 GB")
    g = torch.Generator().manual_seed(4)
    at = [0, 1, 255, 256, 2 ** 30 + 77, rows - 257, rows - 2, rows - 1]
    pos = torch.zeros(rows, dtype=torch.int32, device="cuda")
    q = torch.ones((rows, 1, 2), dtype=torch.bfloat16, device="cuda")
    x = torch.randn((len(at), 1, 2), generator=g).to(torch.bfloat16)
    p = torch.randint(0, 9999, (len(at),), generator=g, dtype=torch.int32)
    w = torch.randn(2, generator=g).to(torch.bfloat16)
    for i, r in enumerate(at):
        q[r], pos[r] = x[i].cuda(), int(p[i])
    qk_norm_rope(Rope(2), pos, q, None, w.cuda(), None, q_out=q)
    got = torch.stack([q[r] for r in at])
    _check_norm(got, x, w, p, 2, *R.rope_freq(2, 1e6), False, 1e-6)
    for start in range(2, rows, 1 << 28):              # position 0, all ones: the weights, to within one rounding
        part = q[start:start + (1 << 28), 0]
        same = (part == part[100]).all(1)
        assert int((~same).sum()) <= len(at)
    del q, pos, part, same
    torch.cuda.empty_cache()


def test_norm_inside_a_function_of_the_caller():
    """Autograd over both outputs through the caller's Function: the gradients are the backward call's, bit for bit."""
    from block_diffusion_speculative_inject_gb300 import Rope, qk_norm_rope, qk_norm_rope_backward
    t, pos = Rope(64, rot_dim=32), _i4([5, 0, 70000])

    class Norm(torch.autograd.Function):
        @staticmethod
        def forward(ctx, q, k, qw, kw):
            ctx.save_for_backward(q, k, qw, kw)
            return qk_norm_rope(t, pos, q, k, qw, kw)

        @staticmethod
        def backward(ctx, gq, gk):
            q, k, qw, kw = ctx.saved_tensors
            return qk_norm_rope_backward(t, pos, q, k, qw, kw, gq.contiguous(), gk.contiguous())

    g = torch.Generator().manual_seed(6)
    q, k = (torch.randn((3, h, 64), generator=g).cuda().requires_grad_() for h in (4, 2))
    qw, kw = (torch.randn(64, generator=g).cuda().requires_grad_() for _ in range(2))
    a, b = Norm.apply(q, k, qw, kw)
    (a.square().sum() + b.square().sum()).backward()
    with torch.no_grad():
        want = qk_norm_rope_backward(t, pos, q, k, qw, kw, 2 * a, 2 * b)
    for x, y in zip((q, k, qw, kw), want):
        assert torch.equal(x.grad, y)


def test_norm_loud_and_special_rows():
    """An infinity or NaN stays in its head; heads far from one another in size do not touch; positions of any sign."""
    from block_diffusion_speculative_inject_gb300 import Rope, qk_norm_rope, qk_norm_rope_backward
    t = Rope(64)
    pos = _i4([-3, 2 ** 31 - 1, -2 ** 31])
    g = torch.Generator().manual_seed(2)
    q = torch.randn((3, 4, 64), generator=g)
    q[0, 1] *= 1e15
    q[0, 2] *= 1e-15
    w = torch.ones(64)
    clean = qk_norm_rope(t, pos, q.cuda(), None, w.cuda(), None)[0]
    bad = q.clone()
    bad[1, 2, 5], bad[2, 0, 63] = math.nan, math.inf
    out = qk_norm_rope(t, pos, bad.cuda(), None, w.cuda(), None)[0]
    gone = torch.zeros((3, 4), dtype=torch.bool)
    gone[1, 2] = gone[2, 0] = True
    assert torch.equal(out.cpu()[~gone], clean.cpu()[~gone])
    assert bool(out.cpu()[1, 2].isnan().all()) and bool(out.cpu()[2, 0].isnan().any())
    _check_norm(clean, q, w, pos.cpu(), 64, *R.rope_freq(64, 1e6), False, 1e-6)
    d = qk_norm_rope_backward(t, pos, bad.cuda(), None, w.cuda(), None, q.cuda(), None)[0].cpu()
    assert bool(d[~gone].isfinite().all())


# ---------------------------------------------------------------- bounds
def _bounds_case(seed, old, new, nkv, hd, extra=3):
    g = torch.Generator().manual_seed(seed)
    blocks = [max(R.pages_of(max(a, b)), 0) for a, b in zip(old, new)]
    n_pages = sum(blocks) + extra
    c = _cache_cpu(seed, n_pages, nkv, hd)
    raw = c["k_pages"].view(torch.uint8)
    raw[torch.rand(raw.shape, generator=g) < 0.02] = 0x7F        # NaN of both signs, both zeros, the ends
    raw[torch.rand(raw.shape, generator=g) < 0.02] = 0xFF
    raw[torch.rand(raw.shape, generator=g) < 0.02] = 0x80
    raw[torch.rand(raw.shape, generator=g) < 0.005] = 0x7E
    raw[torch.rand(raw.shape, generator=g) < 0.005] = 0xFE
    table = torch.full((len(old), max(1, max(blocks)) + 1), -1, dtype=torch.int32)
    perm, at = torch.randperm(n_pages, generator=g), 0
    for b, k in enumerate(blocks):
        table[b, :k] = perm[at:at + k]
        at += k
    got = torch.randint(-128, 128, (n_pages, nkv, 2, hd), generator=g).to(torch.int8)
    return c, table, got


@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("nkv,old,new", [
    (1, [0], [1]), (2, [63, 64, 0], [64, 65, 0]), (8, [100, 5, 0, 128, 7], [116, 5, 64, 300, 3]), (3, [0, 70], [517, 71]),
    (1, [i % 130 for i in range(300)], [i % 130 + i % 3 for i in range(300)])])
def test_bounds(hd, nkv, old, new):
    from block_diffusion_speculative_inject_gb300 import kv8_bounds
    c, table, got = _bounds_case(nkv + hd, old, new, nkv, hd)
    c["k_pages"].view(torch.uint8)[int(table[0, 0]), 0, :, 3] = 0x7F           # a dim of nothing but NaN
    want = got.clone()
    L.bounds(c["k_pages"], old, new, table, want)
    out = got.cuda()
    for _ in range(2):
        kv8_bounds(_to_gpu(c), out, table.cuda(), _i4(old), _i4(new))
        assert torch.equal(out.cpu(), want)


def test_bounds_at_the_edges():
    """The most requests; lengths outside the table; pages outside the pool; pages that requests share."""
    from block_diffusion_speculative_inject_gb300 import kv8_bounds
    n = 4096
    c, _, got = _bounds_case(9, [0] * 40, [100] * 40, 1, 64)
    n_pages = got.shape[0]
    table = torch.stack([(torch.arange(2) + i) % n_pages for i in range(n)]).to(torch.int32)
    # every request that is touched sees whole pages, so that those who share one agree
    old = [(i * 7) % 90 for i in range(n)]
    new = [128 if i % 5 > 1 else x for i, x in enumerate(old)]
    old[5], new[5], old[6], new[6] = -5, 1 << 30, 1 << 30, -7
    table[7] = torch.tensor([-1, n_pages])
    old[7], new[7] = 0, 128
    want = got.clone()
    L.bounds(c["k_pages"], old, new, table, want)
    out = got.cuda()
    kv8_bounds(_to_gpu(c), out, table.cuda(), _i4(old), _i4(new))
    assert torch.equal(out.cpu(), want)


# ---------------------------------------------------------------- choice
def _choice_case(seed, ctx, n_q, nkv, hd, group, dtype, spread=1.5, pages=None):
    g = torch.Generator().manual_seed(seed)
    blocks = [R.pages_of(max(c, 0)) for c in ctx]
    n_pages = pages or sum(blocks) + 3
    width = max(1, max(blocks)) + 1
    table = torch.full((len(ctx), width), -1, dtype=torch.int32)
    perm, at = torch.randperm(n_pages, generator=g), 0
    for b, k in enumerate(blocks):
        table[b, :k] = perm[torch.arange(at, at + k) % n_pages]
        at += k
    mid = torch.randn((n_pages, nkv, hd), generator=g) * 30
    half = torch.rand((n_pages, nkv, hd), generator=g) * 30
    bound = torch.stack([(mid - half).floor(), (mid + half).ceil()], 2).clamp(-112, 112).to(torch.int8)
    scale = torch.exp2(torch.randint(-8, -3, (n_pages, nkv), generator=g).float())
    q = (torch.randn((sum(n_q), nkv * group, hd), generator=g) * spread).to(dtype)
    return table, bound, scale, q, _cum(n_q)


def _choose(table, bound, scale, q, cu, ctx, k, first, last, **kw):
    from block_diffusion_speculative_inject_gb300 import KV8Cache, kv8_select
    n_pages, nkv, _, hd = bound.shape
    e4 = dict(dtype=torch.float8_e4m3fn, device="cuda")
    cache = KV8Cache(torch.empty((n_pages, nkv, PAGE, hd), **e4), torch.empty((n_pages, nkv, hd, PAGE), **e4), scale.cuda(), scale.cuda())
    return kv8_select(cache, bound.cuda(), q.cuda(), _i4(cu), _i4(ctx), table.cuda(), k, keep_first=first, keep_last=last, **kw)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("hd,nkv,group", [(128, 2, 4), (64, 3, 1), (128, 1, 8), (64, 2, 5)])
@pytest.mark.parametrize("ctx,n_q,k,first,last", [
    ([1000], [1], 3, 1, 1), ([1, 64, 65, 700, 2000], [1, 1, 1, 1, 1], 5, 0, 0), ([500, 0, 900, 130], [16, 2, 0, 17], 4, 2, 1),
    ([3000, 1500], [20, 33], 10, 1, 3), ([64 * 70, 64 * 9 + 1], [1, 2], 9, 0, 0)])
def test_select(dtype, hd, nkv, group, ctx, n_q, k, first, last):
    table, bound, scale, q, cu = _choice_case(len(ctx) + hd + nkv, ctx, n_q, nkv, hd, group, dtype)
    want = L.select(q, cu, ctx, table, bound, scale, k, first, last)
    got = _choose(table, bound, scale, q, cu, ctx, k, first, last)
    assert torch.equal(got.cpu(), want)


@pytest.mark.parametrize("blocks,k", [(257, 100), (1025, 1024), (5000, 37), (20000, 4097), (70000, 3)])
def test_select_long_contexts_and_ties(blocks, k):
    """Contexts of many blocks over a small pool: the same page again and again, so that most scores tie."""
    ctx = [blocks * PAGE - 5, blocks // 2 * PAGE]
    table, bound, scale, q, cu = _choice_case(blocks, ctx, [1, 3], 2, 64, 2, torch.bfloat16, pages=41)
    want = torch.empty((2, 2, k), dtype=torch.int32)
    for b in range(2):                                 # as the reference, with every page scored once
        for h in range(2):
            one = torch.arange(41, dtype=torch.int32)[None]
            n = cu[b + 1] - cu[b]
            s = L.scores(q[cu[b]:cu[b + 1]], [0, n], [41 * PAGE], 0, h, one, bound, scale)
            own = (ctx[b] - n) // PAGE - 1
            pages = table[b].tolist()
            rank = sorted((0 if j < 1 or j >= own else 1, 0 if j < 1 or j >= own else -s[pages[j]], j)
                          for j in range(R.pages_of(ctx[b])))
            pick = sorted(j for _, _, j in rank[:k])
            want[b, h] = torch.tensor(pick + [-1] * (k - len(pick)), dtype=torch.int32)
    assert torch.equal(_choose(table, bound, scale, q, cu, ctx, k, 1, 1).cpu(), want)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_select_extremes(dtype):
    """Sums at 2^24, in which no bit may be lost; rows of zeros, tiny ones, infinities and NaN; more rows than one pass
    takes; pages outside the pool; more kept blocks than are asked for; rows that outnumber the context."""
    hd, nkv, group = 128, 1, 2
    ctx, n_q = [40 * PAGE], [1]
    table, bound, scale, q, cu = _choice_case(3, ctx, n_q, nkv, hd, group, dtype)
    scale.fill_(1.0)
    # blocks whose sums differ by one unit near the largest: all dims at the end, one of them a unit less
    bound[:] = torch.tensor([-112, 112], dtype=torch.int8)[:, None]
    q[:] = 1020.0
    q[0, 1] = -1020.0
    q[..., 5] = 1.0
    perm = table[0, :40].long()
    for j in range(40):
        bound[perm[j], 0, 1, 5] = 112 - (j * 17) % 40
        bound[perm[j], 0, 0, 5] = -112 + (j * 17) % 40
    want = L.select(q, cu, ctx, table, bound, scale, 7, 0, 0)
    assert torch.equal(_choose(table, bound, scale, q, cu, ctx, 7, 0, 0).cpu(), want)
    bound[:, :, 0], bound[:, :, 1] = -128, 127             # what no call makes: still whole numbers below 2^24
    for j in range(40):
        bound[perm[j], 0, 1, j] = 126
    assert torch.equal(_choose(table, bound, scale, q, cu, ctx, 7, 0, 0).cpu(), L.select(q, cu, ctx, table, bound, scale, 7, 0, 0))

    ctx, n_q = [2000, 900, 1200, 700, 1300, 50, 800], [1, 2, 3, 2, 100, 90, 1]
    table, bound, scale, q, cu = _choice_case(4, ctx, n_q, nkv, hd, group, dtype)
    q[0] = 0
    q[1:3] *= 2.0 ** -100
    q[3, 0, 7], q[4, 1, 0] = math.nan, -math.inf
    q[6:8] = math.inf
    table[1, 3], table[2, 5] = -1, 1 << 20
    for k, first, last in ((4, 0, 0), (3, 5, 2), (1, 0, 0), (2, 1 << 24, 1 << 24)):
        want = L.select(q, cu, ctx, table, bound, scale, k, first, last)
        assert torch.equal(_choose(table, bound, scale, q, cu, ctx, k, first, last).cpu(), want)


def test_select_strided_out_workspace_and_lengths():
    """Rows of a wider tensor, the caller's output and workspace (full of NaN), lengths outside the table, many requests."""
    from block_diffusion_speculative_inject_gb300 import KV8Cache, kv8_select, kv8_select_workspace
    n = 600
    ctx = [64 * (i % 9) + i % 64 for i in range(n)]
    table, bound, scale, q, cu = _choice_case(8, ctx, [i % 3 for i in range(n)], 2, 64, 2, torch.bfloat16)
    ctx[3], ctx[4] = -9, 1 << 30
    want = L.select(q, cu, ctx, table, bound, scale, 3, 1, 0)
    e4 = dict(dtype=torch.float8_e4m3fn, device="cuda")
    cache = KV8Cache(torch.empty((bound.shape[0], 2, PAGE, 64), **e4), torch.empty((bound.shape[0], 2, 64, PAGE), **e4), scale.cuda(), scale.cuda())
    wide = torch.zeros((q.shape[0], 6, 64), dtype=torch.bfloat16, device="cuda")
    wide[:, 1:5] = q.cuda()
    a = (cache, bound.cuda(), wide[:, 1:5], _i4(cu), _i4(ctx), table.cuda(), 3)
    ws = torch.full((kv8_select_workspace(*a, keep_last=0),), 255, dtype=torch.uint8, device="cuda")
    out = torch.full((n, 2, 3), 5, dtype=torch.int32, device="cuda")
    got = kv8_select(*a, keep_last=0, out=out, workspace=ws)
    assert got is out and torch.equal(out.cpu(), want)


# ---------------------------------------------------------------- attention over blocks
def _check_blocks(c, table, q, cu, ctx, blocks, mask, tree, dtype, max_q, gpu=None, **kw):
    from block_diffusion_speculative_inject_gb300 import kv8_attention
    gpu = gpu or _to_gpu(c)
    pad = 3
    rows, nq, hd = q.shape
    qg = torch.cat([q, torch.ones((pad, nq, hd), dtype=dtype)]).cuda()
    out = torch.full((rows + pad, nq, hd), 77.0, dtype=dtype, device="cuda")
    lse = torch.full((rows + pad, nq), 77.0, device="cuda")
    tg = torch.cat([tree, torch.zeros((pad, tree.shape[1]), dtype=torch.int32)]).cuda() if tree is not None else None
    kv8_attention(gpu, qg, _i4(cu), _i4(ctx), table.cuda(), mask=mask, tree_mask=tg, out=out, lse=lse, max_q=max_q,
                  blocks=blocks.cuda(), **kw)
    out, lse = out.cpu(), lse.cpu()
    assert bool((out[rows:] == 77).all()) and bool((lse[rows:] == 77).all())
    want, wl, absv, top = L.attention(c, q, cu, ctx, table, blocks, mask, tree)
    r = 2.0 ** -11 if dtype == torch.bfloat16 else 2.0 ** -20
    tol = want.abs() * HALF[dtype] + absv * (r + 2 * (top * 2.0 ** -19 + 2.0 ** -19)[..., None])
    err = (out[:rows].double() - want).abs()
    assert torch.equal(out[:rows].isnan(), want.isnan())
    assert bool(((err <= tol) | want.isnan()).all())
    fin = wl.isfinite()
    assert torch.equal(lse[:rows][~fin].nan_to_num(9.0), wl[~fin].float().nan_to_num(9.0))
    big = max([1] + list(ctx))
    ltol = (top * 2.0 ** -19 + wl.abs() * 2.0 ** -22 + (big + 32) * 2.0 ** -24)[fin]
    assert bool(((lse[:rows].double() - wl).abs()[fin] <= ltol).all())
    return out[:rows], lse[:rows]


def _lists(seed, ctx, nkv, k, own=0):
    """Rising lists of up to k of a request's blocks (the last `own` always), -1 after them."""
    g = torch.Generator().manual_seed(seed)
    out = torch.full((len(ctx), nkv, k), -1, dtype=torch.int32)
    for b, c in enumerate(ctx):
        p = R.pages_of(c)
        for h in range(nkv):
            last = list(range(max(0, p - min(own, k)), p))
            rest = torch.randperm(max(0, p - len(last)), generator=g)[:max(0, min(p, k) - len(last))].tolist()
            pick = sorted(rest + last)
            out[b, h, :len(pick)] = torch.tensor(pick, dtype=torch.int32)
    return out


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("hd,nkv,group,mask,rows,k", [
    (128, 2, 4, "causal", 1, 3), (64, 1, 8, "causal", 2, 2), (128, 2, 5, "causal", 16, 4), (64, 2, 8, "tree", 40, 5),
    (128, 1, 2, "none", 3, 1), (128, 2, 8, "tree", 5, 20), (64, 4, 1, "none", 150, 3), (128, 1, 7, "causal", 70, 6)])
def test_attention_blocks(dtype, hd, nkv, group, mask, rows, k):
    """Ragged contexts, lists shorter and longer than they are, NaN in every place that no row may read."""
    ctx = [0, 1, 63, 64, 65, 128, 129, 300, 517, 900]
    n_q = [min(rows, max(c, 1)) if mask != "none" else rows for c in ctx]
    n_q[4] = 0
    c, table, q, cu, tree = _attn_case(rows + hd, ctx, n_q, nkv, hd, nkv * group, mask, dtype)
    blocks = _lists(rows, ctx, nkv, k, own=rows // PAGE + 2 if mask != "none" else 0)
    _check_blocks(c, table, q, cu, ctx, blocks, mask, tree, dtype, max(n_q))


@pytest.mark.parametrize("dtype,n_q", [(torch.bfloat16, 1), (torch.bfloat16, 3), (torch.bfloat16, 40), (torch.float32, 2)])
def test_attention_blocks_out_of_range_entries_and_hidden_nan(dtype, n_q):
    """Entries past the context and below zero name nothing, also between others and in any order; a listed page outside the
    pool is not seen; the pages that are not listed hold NaN, and so do visible places that some rows see and others do not."""
    ctx = [600, 70, 700]
    c, table, q, cu, tree = _attn_case(7, ctx, [n_q] * 3, 2, 128, 8, "causal", dtype)
    blocks = torch.tensor([[[9, 3, -1, 0, 8, 10, 1 << 30, 2], [-5, 9, 5, 1, 0, 6, 4, 3]],
                           [[1, 0, -1, -1, -1, -1, -1, -1], [-1, 1, 0, 1, -1, -1, -1, -1]],
                           [[10, 4, 5, 6, 7, 8, 9, 3], [-1] * 8]], dtype=torch.int32)
    listed = {(b, int(j)) for b in range(3) for h in range(2) for j in blocks[b, h] if 0 <= int(j) < R.pages_of(ctx[b])}
    for b in range(3):
        for j in range(R.pages_of(ctx[b])):
            if (b, j) not in listed:
                c["k_pages"].view(torch.uint8)[int(table[b, j])] = 0x7F
                c["v_pages"].view(torch.uint8)[int(table[b, j])] = 0x7F
    table[2, 5] = -1
    table[2, 6] = 10 ** 6
    if n_q > 1:                                        # the last token's value is NaN in one dim: only the last row sees it
        p, o = int(table[0, 599 // PAGE]), 599 % PAGE
        c["v_pages"].view(torch.uint8)[p, 0, 17, o] = 0x7F
    _check_blocks(c, table, q, cu, ctx, blocks, "causal", tree, dtype, n_q)
    blocks[0, 0, 3:] = -1
    _check_blocks(c, table, q, cu, ctx, blocks, "causal", tree, dtype, n_q)


@pytest.mark.parametrize("n_q,dtype", [(1, torch.bfloat16), (2, torch.float32), (20, torch.bfloat16)])
def test_attention_blocks_split_items_and_whole_lists(n_q, dtype):
    """Long lists are cut between many workers; every block listed is the attention over the whole context."""
    from block_diffusion_speculative_inject_gb300 import kv8_attention
    ctx = [9000, 300]
    c, table, q, cu, tree = _attn_case(11, ctx, [n_q] * 2, 2, 64, 8, "causal", dtype)
    _check_blocks(c, table, q, cu, ctx, _lists(3, ctx, 2, 100, own=2), "causal", tree, dtype, n_q)
    whole = torch.full((2, 2, 150), -1, dtype=torch.int32)
    for b in range(2):
        whole[b, :, :R.pages_of(ctx[b])] = torch.arange(R.pages_of(ctx[b]), dtype=torch.int32)
    gpu = _to_gpu(c)
    out, lse = _check_blocks(c, table, q, cu, ctx, whole, "causal", tree, dtype, n_q, gpu=gpu)
    full, flse = kv8_attention(gpu, q.cuda(), _i4(cu), _i4(ctx), table.cuda(), max_q=n_q, want_lse=True)
    if n_q <= 2:                                       # (one tile of rows: cut in the same places)
        assert torch.equal(out, full.cpu()) and torch.equal(lse, flse.cpu())


@pytest.mark.parametrize("n_q", [1, 30])
def test_attention_blocks_many_requests(n_q):
    n = 70
    ctx = [1 + (i * 37) % 400 for i in range(n)]
    rows = [min(n_q, x) for x in ctx]
    c, table, q, cu, tree = _attn_case(13, ctx, rows, 1, 64, 4, "causal", torch.bfloat16)
    _check_blocks(c, table, q, cu, ctx, _lists(5, ctx, 1, 3, own=1), "causal", tree, torch.bfloat16, n_q)


# ---------------------------------------------------------------- moves
def _compact_case(seed, base, tree, counts, nkv, hd, layers=1, extra=2):
    g = torch.Generator().manual_seed(seed)
    n = len(base)
    blocks = [R.pages_of(b + tree) for b in base]
    n_pages = sum(blocks) + extra
    caches = [_cache_cpu(seed * 100 + i, n_pages, nkv, hd) for i in range(layers)]
    table = torch.full((n, max(blocks) + 1), -1, dtype=torch.int32)
    perm, at = torch.randperm(n_pages, generator=g), 0
    for b, k in enumerate(blocks):
        table[b, :k] = perm[at:at + k]
        at += k
    keep = torch.full((n, max(1, max(counts))), -1, dtype=torch.int32)
    for b, m in enumerate(counts):
        keep[b, :m] = torch.sort(torch.randperm(tree, generator=g)[:m]).values.to(torch.int32)
    return caches, table, keep


@pytest.mark.parametrize("hd,nkv", [(128, 2), (64, 3)])
@pytest.mark.parametrize("base,tree,counts", [
    ([0], 1, [1]), ([100], 65, [8]), ([63, 64, 0, 130], 40, [5, 0, 40, 1]), ([60, 1], 300, [10, 200]), ([5], 500, [430]),
    ([i * 13 for i in range(40)], 9, [i % 10 for i in range(40)])])
def test_compact(hd, nkv, base, tree, counts):
    from block_diffusion_speculative_inject_gb300 import kv8_compact
    caches, table, keep = _compact_case(hd + tree, base, tree, counts, nkv, hd)
    raw = caches[0]
    g = torch.Generator().manual_seed(1)
    for n in ("k_pages", "v_pages"):                   # NaN, both zeros, the smallest and the largest among them
        b = raw[n].view(torch.uint8)
        for byte in (0x7F, 0xFF, 0x80, 0x01, 0x7E):
            b[torch.rand(b.shape, generator=g) < 0.01] = byte
    for n in ("k_scale", "v_scale"):
        raw[n] = torch.exp2(torch.randint(-12, 9, raw[n].shape, generator=g).float())
    gpu = _to_gpu(raw)
    kv8_compact(gpu, table.cuda(), _i4(base), keep.cuda(), _i4(counts))
    L.compact(raw, table, base, keep, counts)
    _same_cache(gpu, raw)


def test_compact_layers_and_odd_arguments():
    """Several layers in one call equal each alone; entries outside the table or the pool, counts outside the list."""
    from block_diffusion_speculative_inject_gb300 import KV8Layers, kv8_compact
    base, counts = [70, 10, 200], [9, 12, 3]
    caches, table, keep = _compact_case(4, base, 30, counts, 2, 64, layers=5)
    gpus = [_to_gpu(c) for c in caches]
    kv8_compact(KV8Layers(gpus), table.cuda(), _i4(base), keep.cuda(), _i4(counts))
    for c, gpu in zip(caches, gpus):
        L.compact(c, table, base, keep, counts)
        _same_cache(gpu, c)
    caches, table, keep = _compact_case(6, base, 100, counts, 2, 64)
    keep[0, 3], keep[0, 8], keep[1, 0] = -4, 1 << 30, 2 ** 31 - 1
    table[0, 2] = -1
    table[2, 3] = 1 << 20
    base, counts = [70, 10, 200], [99, -3, 2]
    gpu = _to_gpu(caches[0])
    kv8_compact([gpu], table.cuda(), _i4(base), keep.cuda(), _i4(counts))
    L.compact(caches[0], table, base, keep, counts)
    _same_cache(gpu, caches[0])
    for b in ([1 << 30, -50, 320], [64 * table.shape[1] - 1] * 3):
        kv8_compact([gpu], table.cuda(), _i4(b), keep.cuda(), _i4([2, 0, 2]))
        L.compact(caches[0], table, b, keep, [2, 0, 2])
        _same_cache(gpu, caches[0])


def test_compact_scales_that_grow_and_values_beyond_fp32():
    """A page that keeps rows and takes louder ones grows its scale and rounds the kept rows anew; a page that begins with a
    moved row takes its scale from the moved rows alone; values past fp32 have no say."""
    from block_diffusion_speculative_inject_gb300 import kv8_compact
    caches, table, keep = _compact_case(8, [30, 64], 200, [4, 70], 1, 64)
    c = caches[0]
    for n in ("k_scale", "v_scale"):
        c[n].fill_(2.0 ** -6)
        c[n][int(table[0, 0])] = 2.0 ** -14
        c[n][int(table[0, 2])] = 2.0 ** 10
        c[n][int(table[1, 3])] = 2.0 ** 120
        c[n][int(table[1, 1])] = 2.0 ** -64
    keep[0, :4] = torch.tensor([0, 100, 110, 190], dtype=torch.int32)
    keep[1, :70] = torch.arange(130, 200, dtype=torch.int32)
    gpu = _to_gpu(c)
    kv8_compact(gpu, table.cuda(), _i4([30, 64]), keep.cuda(), _i4([4, 70]))
    L.compact(c, table, [30, 64], keep, [4, 70])
    _same_cache(gpu, c)


# ---------------------------------------------------------------- together
class _Long:
    """Two layers of a target over long contexts: a tree round with chosen blocks, then the accepted path in place."""

    def __init__(self, seed=0):
        from block_diffusion_speculative_inject_gb300 import KV8Cache, KV8Layers, Rope
        self.n, self.nkv, self.group, self.hd, self.pages, self.width, self.k = 3, 2, 4, 128, 60, 20, 5
        self.nq = self.nkv * self.group
        self.g = torch.Generator().manual_seed(seed)
        self.rope = Rope(self.hd, theta=1e4)
        self.caches = [KV8Cache.empty(self.pages, self.nkv, self.hd) for _ in range(2)]
        self.layers = KV8Layers(self.caches)
        for c in self.caches:
            c.k_pages.view(torch.uint8).fill_(0x7F), c.v_pages.view(torch.uint8).fill_(0x7F)
        self.ref = [{k: getattr(c, k).cpu().clone() for k in ("k_pages", "v_pages", "k_scale", "v_scale")} for c in self.caches]
        self.bounds = [torch.zeros((self.pages, self.nkv, 2, self.hd), dtype=torch.int8, device="cuda") for _ in range(2)]
        self.w = [torch.randn(self.hd, generator=self.g).to(torch.bfloat16).cuda() for _ in range(2)]
        self.len = _i4([0] * self.n)
        self.table = torch.full((self.n, self.width), -1, dtype=torch.int32, device="cuda")
        self.stack = torch.arange(self.pages, dtype=torch.int32, device="cuda")
        self.free = _i4([self.pages])

    def draw(self, rows):
        f = lambda h: torch.randn((rows, h, self.hd), generator=self.g).to(torch.bfloat16).cuda()  # noqa: E731
        return [(f(self.nq), f(self.nkv), f(self.nkv)) for _ in range(2)]

    def rows(self, add, total, x, positions=None, mask="causal", tree=None, max_q=1):
        """Plans the rows, appends them in both layers and attends over chosen blocks."""
        from block_diffusion_speculative_inject_gb300 import (kv8_append, kv8_attention, kv8_bounds, kv8_select, page_plan,
                                                              qk_norm_rope)
        p = page_plan(self.len, add, self.table, self.stack, self.free, total)
        out = []
        for i, (q, k, v) in enumerate(x):
            q, k = qk_norm_rope(self.rope, p["positions"] if positions is None else positions, q, k, *self.w)
            kv8_append(self.caches[i], k, v, p["slot_map"])
            kv8_bounds(self.caches[i], self.bounds[i], self.table, self.len, p["new_len"])
            blocks = kv8_select(self.caches[i], self.bounds[i], q, p["cu_rows"], p["new_len"], self.table, self.k)
            o = kv8_attention(self.caches[i], q, p["cu_rows"], p["new_len"], self.table, mask=mask, tree_mask=tree, max_q=max_q,
                              blocks=blocks)
            out.append((q, k, v, blocks, o))
        return p, out

    def check(self, p, out, mask="causal", tree=None):
        table = self.table.cpu()
        cu, ctx, slots = p["cu_rows"].tolist(), p["new_len"].tolist(), p["slot_map"].tolist()
        for i, (q, k, v, blocks, o) in enumerate(out):
            R.append(self.ref[i], k.cpu(), v.cpu(), slots)
            _same_cache(self.caches[i], self.ref[i])
            want = torch.zeros((self.pages, self.nkv, 2, self.hd), dtype=torch.int8)
            L.bounds(self.ref[i]["k_pages"], [0] * self.n, ctx, table, want)
            held = sorted(int(x) for b in range(self.n) for x in table[b, :R.pages_of(ctx[b])])
            assert torch.equal(self.bounds[i].cpu()[held], want[held])
            assert torch.equal(blocks.cpu(), L.select(q.cpu(), cu, ctx, table, want, self.ref[i]["k_scale"], self.k, 1, 1))
            exact, _, absv, top = L.attention(self.ref[i], q.cpu(), cu, ctx, table, blocks.cpu(), mask, tree)
            tol = exact.abs() * HALF[torch.bfloat16] + absv * (2.0 ** -11 + 2 * (top * 2.0 ** -19 + 2.0 ** -19))[..., None]
            assert bool(((o.cpu().double() - exact).abs() <= tol).all())

    def accept(self, p, path, n_path, rows):
        """The path to its place in both layers, the rest given back; bounds of what moved made anew."""
        from block_diffusion_speculative_inject_gb300 import kv8_bounds, kv8_compact, page_plan
        kv8_compact(self.layers, self.table, self.len, path, n_path)
        drop = page_plan(p["new_len"], n_path - rows, self.table, self.stack, p["n_free"], 0)
        for c, b in zip(self.caches, self.bounds):
            kv8_bounds(c, b, self.table, self.len, drop["new_len"])
        return drop


def _tree_of(lp, budget, depth):
    from block_diffusion_speculative_inject_gb300 import ddtree_build
    logp = -torch.sort(torch.rand((lp.n, depth, 4), generator=lp.g) * 3, dim=2).values
    tok = torch.arange(4, dtype=torch.int32).expand(lp.n, depth, 4).contiguous()
    return ddtree_build(tok.cuda(), logp.cuda(), budget)


@pytest.mark.parametrize("budget", [11, 70])
def test_tree_rounds_over_chosen_blocks(budget):
    """Prompts, then rounds of: a draft tree's rows normed, appended and attended over chosen blocks; the accepted path moved
    to its place in both layers (equal to the reference's), the rest given back; a single token over chosen blocks."""
    from block_diffusion_speculative_inject_gb300 import ddtree_path, ddtree_walk
    lp, depth = _Long(3), 7
    prompt = [700, 1, 300]
    p, out = lp.rows(_i4(prompt), sum(prompt), lp.draw(sum(prompt)), max_q=700)
    lp.check(p, out)
    lp.len, lp.free = p["new_len"], p["n_free"]
    for step in range(3):
        tree = _tree_of(lp, budget, depth)
        rows = budget + 1
        level = torch.cat([torch.zeros((lp.n, 1), dtype=torch.int32, device="cuda"), tree["depth"]], 1)
        positions = (lp.len[:, None] + level).reshape(-1).to(torch.int32)
        mask = tree["mask"].flatten(0, 1)
        p, out = lp.rows(_i4([rows] * lp.n), lp.n * rows, lp.draw(lp.n * rows), positions, "tree", mask, rows)
        lp.check(p, out, "tree", mask.cpu())
        target = torch.randint(0, 4, (lp.n, budget + 1), generator=lp.g, dtype=torch.int32).cuda()
        target[:, 0] = tree["tok"][:, step % 2]
        accept, tokens, _ = ddtree_walk(tree, depth, target)
        path, n_path = ddtree_path(tree, depth, target)
        assert torch.equal(n_path, accept + 1)
        for b in range(lp.n):
            at, n = 0, int(n_path[b])
            assert path[b, 0] == 0 and path[b, n:].tolist() == [-1] * (depth + 1 - n)
            for j, t in enumerate(tokens[b, :n - 1].tolist()):
                node = int(path[b, j + 1]) - 1
                assert int(tree["parent"][b, node]) == at - 1 and int(tree["tok"][b, node]) == t
                at = node + 1
        drop = lp.accept(p, path, n_path, rows)
        assert torch.equal(drop["new_len"], lp.len + n_path)
        for i in range(2):
            L.compact(lp.ref[i], lp.table.cpu(), lp.len.tolist(), path.cpu(), n_path.tolist())
            _same_cache(lp.caches[i], lp.ref[i])
        lp.len, lp.free = drop["new_len"], drop["n_free"]
        p, out = lp.rows(_i4([1] * lp.n), lp.n, lp.draw(lp.n))
        lp.check(p, out)
        lp.len, lp.free = p["new_len"], p["n_free"]
    held = [x for b in range(lp.n) for x in lp.table[b, :R.pages_of(int(lp.len[b]))].tolist()]
    assert sorted(held + lp.stack[:int(lp.free)].tolist()) == list(range(lp.pages))      # no page lost, none twice


def test_tree_round_in_a_graph():
    """A whole round captured once and replayed on new inputs equals the eager round, bit for bit."""
    from block_diffusion_speculative_inject_gb300 import ddtree_path
    budget, depth, rows = 20, 6, 21
    eager, captured = _Long(5), _Long(5)
    prompt = [500, 64, 200]
    for lp in (eager, captured):
        p, _ = lp.rows(_i4(prompt), sum(prompt), lp.draw(sum(prompt)), max_q=500)
        lp.len, lp.free = p["new_len"].clone(), p["n_free"].clone()
    tree = _tree_of(eager, budget, depth)
    level = torch.cat([torch.zeros((3, 1), dtype=torch.int32, device="cuda"), tree["depth"]], 1)
    mask = tree["mask"].flatten(0, 1)
    target = torch.randint(0, 4, (3, budget + 1), generator=eager.g, dtype=torch.int32).cuda()

    def round_(lp, x, add):
        positions = (lp.len[:, None] + level).reshape(-1).to(torch.int32)
        p, out = lp.rows(add, 3 * rows, x, positions, "tree", mask, rows)
        path, n_path = ddtree_path(tree, depth, target)
        return lp.accept(p, path, n_path, rows), [o[3:] for o in out]
    add = _i4([rows] * 3)
    x = eager.draw(3 * rows)
    held = [tuple(t.clone() for t in y) for y in x]

    def state(lp):
        return [t for c in lp.caches for t in c._tensors()] + lp.bounds + [lp.table, lp.stack]
    was = [t.clone() for t in state(captured)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        round_(captured, held, add)                     # warm up
    torch.cuda.current_stream().wait_stream(side)
    for t, w in zip(state(captured), was):
        t.view(torch.uint8).copy_(w.view(torch.uint8))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        drop, out = round_(captured, held, add)
    for step in range(3):
        for y, z in zip(held, x):
            for a, b in zip(y, z):
                a.copy_(b)
        graph.replay()
        de, oe = round_(eager, x, add)
        for (b1, o1), (b2, o2) in zip(out, oe):
            assert torch.equal(b1, b2) and torch.equal(o1, o2)
        assert torch.equal(drop["new_len"], de["new_len"])
        for s, t in zip(state(captured), state(eager)):
            assert torch.equal(s.view(torch.uint8), t.view(torch.uint8))
        captured.len.copy_(drop["new_len"])
        captured.free.copy_(drop["n_free"])
        eager.len, eager.free = de["new_len"], de["n_free"]
        x = eager.draw(3 * rows)


def test_two_calls_at_once_long():
    """Two streams with their own workspaces: each call equals itself alone, many times."""
    from block_diffusion_speculative_inject_gb300 import (Rope, kv8_attention, kv8_select, kv8_select_workspace, kv8_workspace,
                                                          qk_norm_rope_backward, qk_norm_rope_workspace)
    sets = []
    for seed in (1, 2):
        ctx = [6000, 900]
        c, table, q, cu, _ = _attn_case(seed, ctx, [3, 3], 2, 128, 8, "causal", torch.bfloat16)
        a = (_to_gpu(c), q.cuda(), _i4(cu), _i4(ctx), table.cuda())
        g = torch.Generator().manual_seed(seed)
        bound = torch.randint(-100, 100, (c["k_scale"].shape[0], 2, 2, 128), generator=g).to(torch.int8).cuda()
        sel = (a[0], bound, *a[1:], 9)
        x = (Rope(128), torch.arange(6, dtype=torch.int32, device="cuda"), q.cuda(), None, torch.ones(128, dtype=torch.bfloat16, device="cuda"),
             None, q.cuda(), None)
        ws = [torch.empty(n, dtype=torch.uint8, device="cuda") for n in
              (kv8_select_workspace(*sel), kv8_workspace(*a, max_q=3), qk_norm_rope_workspace())]
        blocks = kv8_select(*sel)
        sets.append((a, sel, x, ws, (blocks, kv8_attention(*a, max_q=3, blocks=blocks), qk_norm_rope_backward(*x)[2])))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    got = [[], []]
    for _ in range(10):
        for i, (a, sel, x, ws, _) in enumerate(sets):
            s = streams[i]
            b = kv8_select(*sel, workspace=ws[0], stream=s)
            got[i].append((b, kv8_attention(*a, max_q=3, blocks=b, workspace=ws[1], stream=s),
                           qk_norm_rope_backward(*x, workspace=ws[2], stream=s)[2]))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(x, y) for r in got[i] for x, y in zip(r, sets[i][4]))


# ---------------------------------------------------------------- further ends of the ranges
@pytest.mark.parametrize("rows", [0, 5])
def test_norm_gradient_of_no_key_heads(rows):
    """k of no heads: its weight's gradient is a sum over nothing, zeros, in memory that held something else."""
    from block_diffusion_speculative_inject_gb300 import Rope, qk_norm_rope, qk_norm_rope_backward
    g = torch.Generator().manual_seed(2)
    q, gq = (torch.randn((rows, 2, 64), generator=g).cuda() for _ in range(2))
    none, w, pos = torch.empty((rows, 0, 64), device="cuda"), torch.ones(64, device="cuda"), _i4(list(range(rows)))
    t = Rope(64)
    out = qk_norm_rope(t, pos, q, none, w, w)
    assert out[1].shape == (rows, 0, 64)
    want = qk_norm_rope_backward(t, pos, q, None, w, None, gq, None)
    for _ in range(4):
        held = [torch.full((64,), 7.0, device="cuda") for _ in range(64)]            # what the next ones are made of
        del held
        dq, dk, dqw, dkw = qk_norm_rope_backward(t, pos, q, none, w, w, gq, none)
        assert torch.equal(dq, want[0]) and torch.equal(dqw, want[2]) and dk.shape == (rows, 0, 64)
        assert bool((dkw == 0).all())


def test_attention_blocks_whole_lists_in_tiles():
    """Every block listed, in the kernel for many rows. With one tile of rows for a request and head, and without a causal mask,
    the line is cut in the same places as over the whole context, so the bits are its bits. Of several tiles of causal rows a
    listed item is as long for every tile, one over the whole context ends with its tile's last row, so the cuts differ."""
    from block_diffusion_speculative_inject_gb300 import kv8_attention
    for hd, group, n_q, mask, ctx in ((64, 4, [20, 20], "causal", [9000, 300]), (128, 8, [16, 9], "causal", [5000, 641]),
                                      (128, 2, [64, 3], "causal", [64, 4000]), (64, 4, [150, 90], "none", [3000, 1100]),
                                      (128, 8, [200, 40], "tree", [2000, 900]),
                                      (64, 4, [150, 90], "causal", [3000, 1100])):
        c, table, q, cu, tree = _attn_case(n_q[0] + hd, ctx, n_q, 2, hd, 2 * group, mask, torch.bfloat16)
        whole = torch.full((2, 2, 150), -1, dtype=torch.int32)
        for b in range(2):
            whole[b, :, :R.pages_of(ctx[b])] = torch.arange(R.pages_of(ctx[b]), dtype=torch.int32)
        gpu = _to_gpu(c)
        out, lse = _check_blocks(c, table, q, cu, ctx, whole, mask, tree, torch.bfloat16, max(n_q), gpu=gpu)
        full, flse = kv8_attention(gpu, q.cuda(), _i4(cu), _i4(ctx), table.cuda(), mask=mask, max_q=max(n_q), want_lse=True,
                                   tree_mask=None if tree is None else tree.cuda())
        if mask != "causal" or max(n_q) * group <= 128:
            assert torch.equal(out, full.cpu()) and torch.equal(lse, flse.cpu())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_norm_gradient_far_offsets(dtype):
    """Rows so far apart that the last ones lie past 2^31 elements of q, k, their gradients and the outputs, each with a
    stride of its own; the places between the rows stay as they are."""
    from block_diffusion_speculative_inject_gb300 import Rope, qk_norm_rope, qk_norm_rope_backward
    if torch.cuda.mem_get_info()[0] < 70 << 30:
        pytest.skip("needs 70 GB")
    rows, nq, nk, hd = 131, 3, 2, 64
    table, freq, mag, pos, x = _norm_case(9, rows, nq, nk, hd, 32, False, "yarn", dtype)
    eps = 1e-6

    def far(values, stride):
        assert (rows - 1) * stride > 2 ** 31
        buf = torch.empty(rows * stride, dtype=dtype, device="cuda")
        t = buf.view(rows, stride)
        edge = values.shape[1] * hd
        t[:, edge:edge + 8] = 5
        v = t[:, :edge].unflatten(1, (values.shape[1], hd))
        v.copy_(values)
        return t[:, edge:edge + 8], v

    step = (1 << 24) + (1 << 18)
    edges, t = {}, {}
    for i, name in enumerate(("q", "k", "dq", "dk")):
        edges[name], t[name] = far(x[name], step + 64 * i)
    w = [x[n].cuda() for n in ("wq", "wk")]
    qo, ko = qk_norm_rope(table, pos.cuda(), t["q"], t["k"], *w, eps=eps)
    args = (pos, 32, freq, mag, False, eps)
    _check_norm(qo, x["q"], x["wq"], *args)
    _check_norm(ko, x["k"], x["wk"], *args)
    # a lane adds at most 131 rows' terms of a head, as if one CTA held them all; then 8 warps, 5 shuffles, 19 CTAs' and 5 more
    chain = rows * max(nq, nk) + 8 + 5 + 19 + 5
    _, _, dqw, dkw = qk_norm_rope_backward(table, pos.cuda(), t["q"], t["k"], *w, t["dq"], t["dk"], eps=eps, dq=t["dq"], dk=t["dk"])
    _check_grad(t["dq"], dqw, x["q"], x["wq"], x["dq"], *args, chain)
    _check_grad(t["dk"], dkw, x["k"], x["wk"], x["dk"], *args, chain)
    assert torch.equal(t["q"].cpu(), x["q"]) and torch.equal(t["k"].cpu(), x["k"])
    assert all(bool((e == 5).all()) for e in edges.values())
    del t, edges
    torch.cuda.empty_cache()


def test_norm_gradient_long_sums():
    """Several hundred thousand rows of small heads: the weights' gradients are sums of a million terms, in chains of a CTA's
    share of the rows."""
    from block_diffusion_speculative_inject_gb300 import Rope, qk_norm_rope_backward
    rows, nq, nk, hd = 400003, 2, 1, 32
    g = torch.Generator(device="cuda").manual_seed(12)
    pos = torch.randint(0, 5000, (rows,), generator=g, dtype=torch.int32, device="cuda")
    # (terms that do not cancel: the products of a dim have a mean)
    q, k = (torch.randn((rows, h, hd), generator=g, device="cuda") + 0.5 for h in (nq, nk))
    gq, gk = (torch.randn((rows, h, hd), generator=g, device="cuda") + 0.25 for h in (nq, nk))
    w = torch.randn(hd, generator=g, device="cuda")
    dq, dk, dqw, dkw = qk_norm_rope_backward(Rope(hd, rot_dim=16), pos, q, k, w, w, gq, gk)
    freq, mag = R.rope_freq(16, 1e6)
    args = (pos.cpu(), 16, freq, mag, False, 1e-6)
    # 304 CTAs; a lane adds one head's terms of some of its CTA's rows, all of them at most; then warps, shuffles, CTAs
    chain = -(-rows // 304) * nq + 8 + 5 + 10 + 5
    _check_grad(dq, dqw, q.cpu(), w.cpu(), gq.cpu(), *args, chain)
    _check_grad(dk, dkw, k.cpu(), w.cpu(), gk.cpu(), *args, chain)


def test_compact_most_layers():
    """128 layers in one call, the most: each as alone."""
    from block_diffusion_speculative_inject_gb300 import KV8Layers, kv8_compact
    base, counts = [70, 3], [9, 6]
    caches, table, keep = _compact_case(21, base, 20, counts, 1, 64, layers=128)
    gpus = [_to_gpu(c) for c in caches]
    kv8_compact(KV8Layers(gpus), table.cuda(), _i4(base), keep.cuda(), _i4(counts))
    for c, gpu in zip(caches, gpus):
        L.compact(c, table, base, keep, counts)
        _same_cache(gpu, c)


@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("n_q,group", [(16, 8), (17, 8), (19, 7), (32, 8), (33, 8), (26, 5)])
def test_select_rows_about_a_round(hd, n_q, group):
    """As many rows as are staged at once (128), a few more, and two rounds of them, for one request and for ragged ones."""
    for ctx, n in (([2000], [n_q]), ([1500, 700, 900, 640], [n_q, 1, 0, n_q - 1])):
        table, bound, scale, q, cu = _choice_case(n_q + hd, ctx, n, 2, hd, group, torch.bfloat16)
        got = _choose(table, bound, scale, q, cu, ctx, 6, 1, 0).cpu()
        assert torch.equal(got, L.select(q, cu, ctx, table, bound, scale, 6, 1, 0))


def test_select_holds_a_requests_own_blocks():
    """keep_first + keep_last + (rows + 62) // 64 + 1 blocks hold all that are kept in any case, wherever the rows begin in a
    block; with one less there is a place where they do not fit, and the lowest stay."""
    first, last = 1, 2
    for rows in (1, 2, 63, 64, 65, 66, 129, 130):
        ctx = [64 * 12 + rows + o for o in (0, 1, 62, 63)]
        kept = [set(range(first)) | set(range((c - rows) // PAGE - last, R.pages_of(c))) for c in ctx]
        most = first + last + (rows + 62) // PAGE + 1
        assert max(len(x) for x in kept) == most
        table, bound, scale, q, cu = _choice_case(rows, ctx, [rows] * 4, 1, 64, 2, torch.bfloat16)
        for k in (most, most - 1):
            got = _choose(table, bound, scale, q, cu, ctx, k, first, last).cpu()
            for b in range(4):
                have = sorted(kept[b])[:k]
                assert set(have) <= set(got[b, 0].tolist()) and (len(kept[b]) <= k or got[b, 0].tolist() == have)
