"""The 8-bit paged cache on the GPU (page planning, rotary positions, quantised append, attention) against
64-bit references (kv8_reference.py), alone and run together as a verify loop runs them.

Tolerances (half steps: bf16 2^-8, f16 2^-11, fp32 2^-24, relative to the value):
  rope      one rounding of the output, plus (|x| + |y|) * magnitude * 8e-7 for fp32: the reduced angle
            (at most pi/4) is rounded once (2^-24 * 0.79 = 5e-8), sine and cosine are within 2 ulp (2.4e-7),
            and three fp32 roundings add 1.8e-7; times 2 for the two terms is under 1e-6.
  append    bytes and scales are equal: scaling by a power of two is exact and there is one rounding.
  attention per output: its own rounding, plus with A = sum p |v| (p the softmax weights) and
            D = max sum_d |q_d k_d| scale (and a part for small entries of q, see the reference):
            the weights' 11-bit (fp32: 22-bit) rounding r = 2^-11 (2^-20),
            and their error from the scores, 2 (D 2^-19 + 2^-19): fp32 sums over at most 128 terms in
            pieces that may truncate (16 2^-23 = 2^-19) and exp2's 2^-22 with its argument's rounding.
  lse       D 2^-19 + |lse| 2^-22 + (L + 32) 2^-24: a positive fp32 sum over at most L terms.
"""
import math

import pytest
import torch

import kv8_reference as R

pytestmark = pytest.mark.gpu

PAGE = 64
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


@pytest.fixture(scope="module", autouse=True)
def _built():
    from block_diffusion_speculative_inject_gb300 import build
    build.build()


def _i4(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _cum(v):
    out = [0]
    for x in v:
        out.append(out[-1] + x)
    return out


# ---------------------------------------------------------------- page planning
def _plan_inputs(seed, n, width, ctx_max, spare):
    g = torch.Generator().manual_seed(seed)
    ctx = torch.randint(0, ctx_max + 1, (n,), generator=g).tolist()
    used = sum(R.pages_of(c) for c in ctx)
    perm = torch.randperm(used + spare, generator=g).tolist()
    table, at = [], 0
    for c in ctx:
        k = R.pages_of(c)
        table.append(perm[at:at + k] + [-7] * (width - k))
        at += k
    return g, ctx, table, perm[at:], used + spare


@pytest.mark.parametrize("n,width,ctx_max,lo,hi,spare,max_rows", [
    (1, 1, 0, 0, 0, 1, 0), (1, 1, 64, 1, 1, 1, 1), (1, 40, 100, 2000, 2000, 50, 2000), (5, 6, 300, -64, 70, 20, 400),
    (33, 4, 200, -300, 100, 10, 900), (128, 30, 1536, 1, 8, 200, 1024), (700, 3, 150, -20, 20, 90, 5000),
    (4096, 2, 100, -5, 9, 500, 9000), (513, 9, 500, -600, 70, 0, 1 << 15), (32, 130, 0, 512, 8192, 4000, 140000),
    (1025, 5, 300, 1, 64, 300, 20000), (3, 1 << 12, 64, 60, 90, 9, 200)])
def test_page_plan(n, width, ctx_max, lo, hi, spare, max_rows):
    """Refusals (too few pages, rows or blocks), releases and grants at once; twice on the same inputs."""
    from block_diffusion_speculative_inject_gb300 import page_plan
    g, ctx, table, free, n_pages = _plan_inputs(n * 7 + hi, n, width, min(ctx_max, width * PAGE), spare)
    add = torch.randint(lo, hi + 1, (n,), generator=g).tolist()
    t_in, st = _i4(table), _i4(free + [-3] * (n_pages - len(free)))
    ctx_d, add_d, nf = _i4(ctx), _i4(add), _i4([len(free)])
    stack = list(free)
    want_t = [list(r) for r in table]
    new, cu, slot, pos, refused = R.plan(ctx, add, want_t, stack, max_rows)
    for _ in range(2):
        p = page_plan(ctx_d, add_d, t_in, st, nf, max_rows)
        assert p["new_len"].tolist() == new
        assert p["refused"].tolist() == refused
        assert p["cu_rows"].tolist() == cu
        assert p["n_free"].tolist() == [len(stack)]
        assert p["slot_map"].tolist() == slot + [-1] * (max_rows - len(slot))
        assert p["positions"].tolist() == pos + [0] * (max_rows - len(pos))
        assert t_in.tolist() == want_t
        assert st[:len(stack)].tolist() == stack
    gone = sum(max(0, R.pages_of(c) - R.pages_of(x)) for c, x in zip(ctx, new))
    assert st[len(free) + gone:].tolist() == [-3] * (n_pages - len(free) - gone)     # the rest of the stack stays


def test_page_plan_corrupt_lengths_stay_in_bounds():
    """Lengths and counts outside their range are read as the nearest end."""
    from block_diffusion_speculative_inject_gb300 import page_plan
    table = _i4([[0, 1], [2, 3], [4, 5]])
    p = page_plan(_i4([-5, 1 << 30, 64]), _i4([3, -(1 << 31), (1 << 31) - 1]), table, _i4([6, 7, 8, 9, 10, 11]), _i4([99]), 10)
    assert p["new_len"].tolist() == [3, 0, 64] and p["refused"].tolist() == [0, 0, 1]
    assert p["cu_rows"].tolist() == [0, 3, 3, 3]
    assert p["slot_map"].tolist()[:3] == [11 * 64, 11 * 64 + 1, 11 * 64 + 2]


def test_page_plan_gives_back_more_than_2_31_pages():
    """The table's width is the caller's, so the pages given back may be more than 2^31 (and than the stack holds):
    the first of them fill the stack, and the requests that grow take theirs from its top."""
    from block_diffusion_speculative_inject_gb300 import page_plan
    n, width, n_pages = 4096, (1 << 19) + 300, 100
    assert (n - 1) * width > 2 ** 31
    if torch.cuda.mem_get_info()[0] < 20 << 30:
        pytest.skip("needs 20 GB")
    table = torch.zeros((n, width), dtype=torch.int32, device="cuda")
    table[0, :200] = torch.arange(200, dtype=torch.int32)
    ctx, add = [width * PAGE] * (n - 1) + [0], [-width * PAGE] * (n - 1) + [130]
    stack = _i4([1000 + i for i in range(n_pages)])
    p = page_plan(_i4(ctx), _i4(add), table, stack, _i4([40]), 130)
    assert p["new_len"].tolist() == [0] * (n - 1) + [130] and int(p["refused"].sum()) == 0
    assert p["n_free"].tolist() == [97]
    assert stack.tolist() == [1000 + i for i in range(40)] + list(range(60))
    assert table[n - 1, :3].tolist() == [59, 58, 57] and int(table[n - 1, 3:].sum()) == 0
    assert p["slot_map"].tolist() == [(59 - i // PAGE) * PAGE + i % PAGE for i in range(130)]
    del table
    torch.cuda.empty_cache()


def test_page_plan_most_rows():
    """The largest max_rows: a thread's next row index passes 2^31 before the loop ends."""
    from block_diffusion_speculative_inject_gb300 import page_plan
    most = 2 ** 31 - 1
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 40 GB")
    p = page_plan(_i4([60, 0]), _i4([8, 3]), _i4([[4, -1], [-1, -1]]), _i4([0, 1, 2]), _i4([3]), most)
    assert p["cu_rows"].tolist() == [0, 8, 11] and p["refused"].tolist() == [0, 0]
    assert p["slot_map"].numel() == most and p["positions"].numel() == most
    assert p["slot_map"][:11].tolist() == [4 * 64 + i for i in range(60, 64)] + [2 * 64 + i for i in range(4)] + [64, 65, 66]
    assert p["positions"][:11].tolist() == list(range(60, 68)) + [0, 1, 2]
    for at in range(11, most, 1 << 28):
        assert bool((p["slot_map"][at:at + (1 << 28)] == -1).all()) and bool((p["positions"][at:at + (1 << 28)] == 0).all())
    del p
    torch.cuda.empty_cache()


# ---------------------------------------------------------------- rotary positions
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,nq,nk,hd,rot,inter,scaling", [
    (1, 1, 0, 64, 64, False, "none"), (3, 5, 2, 128, 128, False, "yarn"), (17, 40, 8, 128, 64, True, "linear"),
    (65, 3, 1, 64, 20, False, "none"), (9, 4, 4, 64, 20, True, "yarn"), (5, 2, 1, 96, 32, False, "none"),
    (4, 2, 2, 50, 50, True, "none"), (4, 1, 1, 50, 18, False, "linear"), (2, 1, 0, 256, 256, False, "none"),
    (700, 8, 2, 64, 64, True, "none"), (31, 1, 1, 7, 2, False, "none")])
def test_rope(dtype, rows, nq, nk, hd, rot, inter, scaling):
    from block_diffusion_speculative_inject_gb300 import Rope, rope
    g = torch.Generator().manual_seed(rows * 31 + hd)
    kw = dict(none={}, linear=dict(factor=2.5), yarn=dict(factor=4.0, original_positions=4096.0))[scaling]
    t = Rope(hd, rot_dim=rot, theta=1e4, interleaved=inter, scaling=scaling, **kw)
    rk = {("original" if k == "original_positions" else k): v for k, v in kw.items()}
    freq, mag = R.rope_freq(rot, 1e4, scaling, **rk)
    pos = torch.randint(0, 1 << 18, (rows,), generator=g, dtype=torch.int32)
    pos[0] = 0
    pos[-1] = (1 << 24) - 1
    q = torch.randn((rows, nq, hd), generator=g).to(dtype)
    k = torch.randn((rows, nk, hd), generator=g).to(dtype) if nk else None
    for transpose in (False, True):
        got = rope(t, pos.cuda(), q.cuda(), k.cuda() if nk else None, transpose=transpose)
        for x, y in ((q, got[0]), (k, got[1])):
            if x is None:
                assert y is None
                continue
            want = R.rope(x.double(), pos.tolist(), rot, freq, mag, inter, transpose)
            size = R.rope(x.double().abs(), [0] * rows, rot, freq, mag, inter) * 0 + x.double().abs().amax(-1, keepdim=True)
            tol = want.abs() * HALF[dtype] + 2 * size * mag * 8e-7
            tol[..., rot:] = 0
            assert bool(((y.cpu().double() - want).abs() <= tol).all())


def test_rope_far_and_negative_positions():
    """The last and first int32 positions. The frequencies are doubles good to 2^-51: their error times the
    position, 2 pi * 0.16 * 2^31 * 2^-51 = 1e-6, joins the tolerance."""
    from block_diffusion_speculative_inject_gb300 import Rope, rope
    freq, mag = R.rope_freq(128, 1e6)
    pos = torch.tensor([2 ** 31 - 1, 2 ** 31 - 2, -2 ** 31, -1, -77777, 123456789], dtype=torch.int32)
    x = torch.randn((6, 2, 128), generator=torch.Generator().manual_seed(1))
    got, _ = rope(Rope(128, theta=1e6), pos.cuda(), x.cuda())
    want = R.rope(x.double(), pos.tolist(), 128, freq, mag, False)
    assert bool(((got.cpu().double() - want).abs() <= 2 * x.double().abs().amax(-1, keepdim=True) * 1.8e-6).all())


@pytest.mark.parametrize("theta", [1e4, 1e6])
def test_rope_is_as_exact_far_away_as_near(theta):
    """One bound for positions near 0 and at both ends of int32. The phase is off by 2^31 * 2^-65 turns (4e-10 rad); the
    reduced angle (at most pi/4) is rounded to fp32 (pi/4 2^-24 = 4.7e-8), sine and cosine below 1 are within two units of
    2^-24 (1.2e-7), the second product is rounded once, and the output once."""
    from block_diffusion_speculative_inject_gb300 import Rope, rope
    freq, mag = R.rope_freq(128, theta)
    pos = [2 ** 31 - 1 - 7 ** i for i in range(11)] + [-2 ** 31 + 5 ** i for i in range(12)] + list(range(-9, 9))
    pos = torch.tensor(pos, dtype=torch.int32)
    x = torch.randn((len(pos), 4, 128), generator=torch.Generator().manual_seed(4))
    x[:, 2, :64], x[:, 3, 64:] = 0, 0
    got, _ = rope(Rope(128, theta=theta), pos.cuda(), x.cuda())
    want = R.rope(x.double(), pos.tolist(), 128, freq, mag, False)
    mine, other = x.double().abs(), x.double().abs().roll(64, -1)
    tol = (mine + other) * (4e-10 + 4.7e-8 + 1.2e-7) + torch.maximum(mine, other) * 2.0 ** -24 + want.abs() * 2.0 ** -24
    assert bool(((got.cpu().double() - want).abs() <= tol).all())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("shift", [0, 1])
def test_rope_strided_rows_in_place_and_out(dtype, inter, shift):
    """q and k as columns of one projection's output (shift: not 16-byte aligned), in place and into another buffer
    with its own stride; what lies between the rows stays."""
    from block_diffusion_speculative_inject_gb300 import Rope, rope
    rows, nq, nk, hd, rot = 11, 3, 2, 64, 32
    g = torch.Generator().manual_seed(5)
    pos = torch.randint(0, 9999, (rows,), generator=g, dtype=torch.int32).cuda()
    width = (nq + 2 * nk) * hd + 8
    buf = torch.randn((rows, width), generator=g).to(dtype).cuda()
    q = buf[:, shift:shift + nq * hd].unflatten(1, (nq, hd))
    k = buf[:, shift + nq * hd:shift + (nq + nk) * hd].unflatten(1, (nk, hd))
    t = Rope(hd, rot_dim=rot, interleaved=inter)
    want = rope(t, pos, q.contiguous(), k.contiguous())
    other = torch.full((rows, width + 24), 7.0, dtype=dtype, device="cuda")
    qo = other[:, 16:16 + nq * hd].unflatten(1, (nq, hd))
    rope(t, pos, q, k, q_out=qo)
    assert torch.equal(qo, want[0]) and bool((other[:, :16] == 7).all()) and bool((other[:, 16 + nq * hd:] == 7).all())
    before = buf.clone()
    rope(t, pos, q, k, q_out=q, k_out=k)
    assert torch.equal(q, want[0]) and torch.equal(k, want[1])
    assert torch.equal(buf[:, shift + (nq + nk) * hd:], before[:, shift + (nq + nk) * hd:])
    assert torch.equal(buf[:, :shift], before[:, :shift])


def test_rope_transpose_is_the_gradient():
    """<R x, y> = <x, R^T y> in fp32, and the transposed call against differences of the forward one
    (the map is linear, so the difference over any step is the derivative)."""
    from block_diffusion_speculative_inject_gb300 import Rope, rope
    g = torch.Generator().manual_seed(2)
    pos = torch.randint(0, 99999, (5,), generator=g, dtype=torch.int32).cuda()
    t = Rope(64, rot_dim=48, interleaved=True, scaling="yarn", factor=4.0, original_positions=2048.0)
    x, y = torch.randn((5, 2, 64), generator=g).cuda(), torch.randn((5, 2, 64), generator=g).cuda()
    fx, grad = rope(t, pos, x)[0].double(), rope(t, pos, y, transpose=True)[0].double()
    # fp32 outputs of size up to 1.14 |x|: each within 2e-6 of its value, summed over 640 terms
    assert abs(float((fx * y.double()).sum() - (x.double() * grad).sum())) < 2e-6 * 640
    for at in ((0, 0, 0), (4, 1, 47), (2, 0, 63), (3, 1, 20)):
        d = torch.zeros_like(x)
        d[at] = 1.0
        diff = rope(t, pos, x + d)[0].double() - fx
        assert abs(float((diff * y.double()).sum()) - float(grad[at])) < 1e-4      # 128 outputs, 2 * 4e-7 * |y| each


def test_rope_inside_a_function_of_the_caller():
    """Autograd over both outputs through the caller's Function: the gradients are the transposed calls', bit for bit."""
    from block_diffusion_speculative_inject_gb300 import Rope, rope
    t = Rope(64, rot_dim=32)
    pos = _i4([5, 0, 70000])

    class Turn(torch.autograd.Function):
        @staticmethod
        def forward(ctx, q, k):
            return rope(t, pos, q, k)

        @staticmethod
        def backward(ctx, gq, gk):
            return rope(t, pos, gq.contiguous(), gk.contiguous(), transpose=True)

    g = torch.Generator().manual_seed(6)
    q, k = (torch.randn((3, h, 64), generator=g).cuda().requires_grad_() for h in (4, 2))
    wq, wk = (torch.randn((3, h, 64), generator=g).cuda() for h in (4, 2))
    a, b = Turn.apply(q, k)
    ((a * wq).sum() + (b * wk).sum()).backward()
    want = rope(t, pos, wq, wk, transpose=True)
    assert torch.equal(q.grad, want[0]) and torch.equal(k.grad, want[1])


# ---------------------------------------------------------------- quantised append
def _cache_cpu(seed, n_pages, nkv, hd, poison=True):
    """A pool with finite random bytes in every page, scales 2^-8 .. 2^-4."""
    g = torch.Generator().manual_seed(seed)
    c = {}
    for name, shape in (("k_pages", (n_pages, nkv, PAGE, hd)), ("v_pages", (n_pages, nkv, hd, PAGE))):
        c[name] = (torch.randn(shape, generator=g) * 80).clamp(-448, 448).to(R.E4M3)
    for name in ("k_scale", "v_scale"):
        c[name] = torch.exp2(torch.randint(-8, -3, (n_pages, nkv), generator=g).float())
    return c


def _to_gpu(c):
    from block_diffusion_speculative_inject_gb300 import KV8Cache
    return KV8Cache(*(c[n].cuda().contiguous() for n in ("k_pages", "v_pages", "k_scale", "v_scale")))


def _same_cache(gpu, want):
    for n in ("k_scale", "v_scale"):
        assert torch.equal(getattr(gpu, n).cpu(), want[n]), n
    for n in ("k_pages", "v_pages"):
        a, b = getattr(gpu, n).cpu().float(), want[n].float()
        assert bool(((a == b) | (a.isnan() & b.isnan())).all()), n


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("nkv,spans", [
    (1, [(0, 0, 1)]), (2, [(3, 63, 1)]), (3, [(1, 17, 16), (2, 0, 64)]), (8, [(0, 1, 63), (5, 0, 30), (4, 40, 5)]),
    (1, [(i, i % 64, 1 + i % 3) for i in range(60)])])
def test_append(dtype, hd, nkv, spans):
    """Spans (page, first offset, rows) in one call: started and fresh pages, grown and unchanged scales; rows of
    sizes over forty powers of two; skipped rows between."""
    from block_diffusion_speculative_inject_gb300 import kv8_append
    n_pages = 64
    spans = [(p, o, min(n, PAGE - o)) for p, o, n in spans]
    slots = []
    for p, o, n in spans:
        slots += [p * PAGE + o + i for i in range(n)] + ([-1] if p % 2 else []) + ([n_pages * PAGE] if p % 3 == 2 else [])
    g = torch.Generator().manual_seed(len(slots) + hd)
    size = torch.exp2(torch.randint(-20, 21, (len(slots), nkv, 1), generator=g).float())
    k = (torch.randn((len(slots), nkv, hd), generator=g) * size).to(dtype)
    v = torch.randn((len(slots), nkv, hd), generator=g).to(dtype)
    want = _cache_cpu(9, n_pages, nkv, hd)
    gpu = _to_gpu(want)
    kv8_append(gpu, k.cuda(), v.cuda(), torch.tensor(slots, device="cuda"))
    R.append(want, k, v, slots)
    _same_cache(gpu, want)


def test_append_long_runs_and_windows():
    """A prompt over many windows of rows, starting in the middle of a page, then one row at a time."""
    from block_diffusion_speculative_inject_gb300 import kv8_append
    n_pages, nkv, hd = 130, 2, 64
    g = torch.Generator().manual_seed(3)
    order = torch.randperm(n_pages, generator=g).tolist()
    slots = [order[p // PAGE] * PAGE + p % PAGE for p in range(29, 29 + 8000)]
    k, v = (torch.randn((8000, nkv, hd), generator=g).bfloat16() for _ in range(2))
    want = _cache_cpu(1, n_pages, nkv, hd)
    gpu = _to_gpu(want)
    kv8_append(gpu, k.cuda(), v.cuda(), torch.tensor(slots, device="cuda"))
    R.append(want, k, v, slots)
    _same_cache(gpu, want)
    nxt = order[8029 // PAGE] * PAGE + 8029 % PAGE
    for i in range(4):
        x = (torch.randn((1, nkv, hd), generator=g) * 4.0 ** i).bfloat16()
        kv8_append(gpu, x.cuda(), x.cuda(), torch.tensor([nxt + i], device="cuda"))
        R.append(want, x, x, [nxt + i])
    _same_cache(gpu, want)


@pytest.mark.parametrize("hd,dtype", [(64, torch.bfloat16), (128, torch.float32)])
@pytest.mark.parametrize("gap", [0, 5, 70, 300])
def test_append_short_runs_in_wide_windows(hd, dtype, gap):
    """Runs of 1 to 5 rows, and whole pages with rows out of order, between stretches of skipped rows: windows that
    begin inside a run, inside a stretch, or hold none or many."""
    from block_diffusion_speculative_inject_gb300 import kv8_append
    n_pages, nkv = 400, 8
    g = torch.Generator().manual_seed(gap + hd)
    slots = []
    for p in torch.randperm(n_pages, generator=g).tolist():
        if len(slots) > 9000:
            break
        if p % 50 == 7:
            slots += [p * PAGE + o for o in torch.randint(0, PAGE, (90,), generator=g).tolist()]
        else:
            n, o = 1 + p % 5, int(torch.randint(0, PAGE - 5, (1,), generator=g))
            slots += [p * PAGE + o + i for i in range(n)]
        slots += [-1] * int(torch.randint(0, gap + 1, (1,), generator=g))
    k, v = (torch.randn((len(slots), nkv, hd), generator=g).to(dtype) for _ in range(2))
    want = _cache_cpu(2, n_pages, nkv, hd)
    gpu = _to_gpu(want)
    kv8_append(gpu, k.cuda(), v.cuda(), torch.tensor(slots, device="cuda"))
    R.append(want, k, v, slots)
    _same_cache(gpu, want)


def test_append_special_values():
    """Zeros (scale 2^-64), infinities (saturate, no say in the scale), NaN (kept), the largest and smallest
    fp32 values, amax on and just above a scale's edge; the last of two rows with one slot stays."""
    from block_diffusion_speculative_inject_gb300 import kv8_append, kv8_read
    n_pages, nkv, hd = 8, 1, 64
    k = torch.zeros((9, nkv, hd))
    k[1, 0, 3], k[1, 0, 4], k[1, 0, 5], k[1, 0, 6] = math.inf, -math.inf, math.nan, 1.0
    k[2, 0, 0], k[2, 0, 1] = 3.4e38, 1.0
    k[3, 0, 0] = 1e-42
    k[4, 0, 0] = 448.0
    k[5, 0, 0] = float(torch.nextafter(torch.tensor(448.0), torch.tensor(500.0)))
    k[6, 0, :] = torch.linspace(-5, 5, hd)
    k[7, 0, :] = 2.5
    k[8, 0, :] = 900.0
    slots = [0, 64, 128, 192, 256, 320, 384 + 5, 384 + 5, 384 + 6]
    want = _cache_cpu(4, n_pages, nkv, hd)
    gpu = _to_gpu(want)
    s = torch.tensor(slots, device="cuda")
    kv8_append(gpu, k.cuda(), (k * -1).cuda(), s)
    R.append(want, k, -k, slots)
    _same_cache(gpu, want)
    assert gpu.k_scale[0, 0] == 2.0 ** -64 and gpu.k_scale[4, 0] == 1.0 and gpu.k_scale[5, 0] == 2.0
    rk, rv = kv8_read(gpu, torch.tensor(slots + [-1, n_pages * PAGE], device="cuda"))
    assert rk[1, 0, 5].isnan() and rk[1, 0, 3] == 448 * gpu.k_scale[1, 0] and bool((rk[9:] == 0).all())
    for x, name in ((rk, "k"), (rv, "v")):
        pages = want["k_pages"] if name == "k" else want["v_pages"].transpose(2, 3)
        for r, sl in enumerate(slots):
            y = pages[sl // PAGE, 0, sl % PAGE].float() * want[name + "_scale"][sl // PAGE, 0]
            assert torch.equal(torch.nan_to_num(x[r, 0].cpu(), nan=-9), torch.nan_to_num(y, nan=-9))


def test_append_strided_rows_and_padding_tail():
    """k and v as columns of one buffer; a long tail of skipped rows; pages that are not named stay."""
    from block_diffusion_speculative_inject_gb300 import kv8_append
    nkv, hd, rows = 2, 64, 20000
    buf = torch.randn((rows, 5 * hd), generator=torch.Generator().manual_seed(8)).bfloat16()
    k, v = buf[:, :2 * hd].unflatten(1, (2, hd)), buf[:, 3 * hd:].unflatten(1, (2, hd))
    slots = [70 + i for i in range(50)] + [-1] * (rows - 50)
    want = _cache_cpu(2, 6, nkv, hd)
    gpu = _to_gpu(want)
    b = buf.cuda()
    kv8_append(gpu, b[:, :2 * hd].unflatten(1, (2, hd)), b[:, 3 * hd:].unflatten(1, (2, hd)), torch.tensor(slots, device="cuda"))
    R.append(want, k, v, slots)
    _same_cache(gpu, want)


# ---------------------------------------------------------------- attention
NAN_BYTE = 0x7F


def _attn_case(seed, ctx, n_q, nkv, hd, nq, mask, dtype, spread=1.5, extra=3):
    """Inputs with NaN in every place no row may read: unused pages, page tails, unused scales."""
    g = torch.Generator().manual_seed(seed)
    n = len(ctx)
    blocks = [R.pages_of(c) for c in ctx]
    n_pages = sum(blocks) + extra
    c = _cache_cpu(seed + 1, n_pages, nkv, hd)
    perm = torch.randperm(n_pages, generator=g).tolist()
    width = max(1, max(blocks)) + 1
    table = torch.full((n, width), -1, dtype=torch.int32)
    at = 0
    used = set()
    for b, k in enumerate(blocks):
        table[b, :k] = torch.tensor(perm[at:at + k], dtype=torch.int32)
        used |= set(perm[at:at + k])
        at += k
        if ctx[b] % PAGE:
            p, o = perm[at - 1], ctx[b] % PAGE
            c["k_pages"].view(torch.uint8)[p, :, o:] = NAN_BYTE
            c["v_pages"].view(torch.uint8)[p, :, :, o:] = NAN_BYTE
    for p in range(n_pages):
        if p not in used:
            c["k_pages"].view(torch.uint8)[p] = NAN_BYTE
            c["v_pages"].view(torch.uint8)[p] = NAN_BYTE
            c["k_scale"][p], c["v_scale"][p] = math.nan, math.nan
    rows = sum(n_q)
    q = (torch.randn((rows, nq, hd), generator=g) * spread).to(dtype)
    tree = None
    if mask == "tree":
        words = max(1, -(-max(n_q) // 32))
        tree = torch.randint(-2 ** 31, 2 ** 31, (rows, words), generator=g).to(torch.int32)
    return c, table, q, _cum(n_q), tree


def _check_attn(c, table, q, cu, ctx, mask, tree, dtype, scale=None, cache=None, max_q=None, **kw):
    from block_diffusion_speculative_inject_gb300 import kv8_attention
    gpu = cache or _to_gpu(c)
    pad = 3                                            # rows past the last request's stay as they were
    rows, nq, hd = q.shape
    qg = torch.cat([q, torch.ones((pad, nq, hd), dtype=dtype)]).cuda()
    out = torch.full((rows + pad, nq, hd), 77.0, dtype=dtype, device="cuda")
    lse = torch.full((rows + pad, nq), 77.0, device="cuda")
    tg = torch.cat([tree, torch.zeros((pad, tree.shape[1]), dtype=torch.int32)]).cuda() if tree is not None else None
    kv8_attention(gpu, qg, _i4(cu), _i4(ctx), table.cuda(), mask=mask, tree_mask=tg, scale=scale, out=out, lse=lse,
                  max_q=max_q, **kw)
    out, lse = out.cpu(), lse.cpu()
    assert bool((out[rows:] == 77).all()) and bool((lse[rows:] == 77).all())
    want, wl, absv, top = R.attention(c, q, cu, ctx, table, mask, tree, scale)
    r = 2.0 ** -11 if dtype == torch.bfloat16 else 2.0 ** -20
    delta = 2 * (top * 2.0 ** -19 + 2.0 ** -19)
    tol = want.abs() * HALF[dtype] + absv * (r + delta[..., None])
    err = (out[:rows].double() - want).abs()
    assert torch.equal(out[:rows].isnan(), want.isnan())
    bad = ~((err <= tol) | want.isnan())
    assert not bool(bad.any()), f"{int(bad.sum())} outputs off, worst {float((err / tol.clamp(min=1e-30))[bad].max()):.3g} x"
    fin = wl.isfinite()
    assert torch.equal(lse[:rows][~fin].nan_to_num(9.0), wl[~fin].float().nan_to_num(9.0))
    big = max([1] + list(ctx))
    ltol = (top * 2.0 ** -19 + wl.abs() * 2.0 ** -22 + (big + 32) * 2.0 ** -24)[fin]
    assert bool(((lse[:rows].double() - wl).abs()[fin] <= ltol).all())
    return out[:rows], lse[:rows]


RAGGED = [0, 1, 63, 64, 65, 127, 128, 129, 300, 517]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("hd,nkv,group", [(128, 2, 4), (64, 1, 1), (128, 1, 5), (64, 2, 8), (128, 1, 7)])
@pytest.mark.parametrize("mask", ["none", "causal", "tree"])
@pytest.mark.parametrize("rows", ["one", "block", "many"])
def test_attention(dtype, hd, nkv, group, mask, rows):
    """Ragged contexts and row counts (none for some requests, more rows than tokens for others)."""
    n_q = dict(one=[1] * 10, block=[1, 3, 0, 16, 2, 7, 16, 5, 16, 9], many=[40, 2, 70, 1, 0, 33, 150, 64, 31, 90])[rows]
    if rows == "many" and (dtype == torch.float32 or group in (1, 7)):
        n_q = [min(x, 37) for x in n_q]
    c, table, q, cu, tree = _attn_case(hd + group, RAGGED, n_q, nkv, hd, nkv * group, mask, dtype)
    _check_attn(c, table, q, cu, RAGGED, mask, tree, dtype, max_q=max(n_q))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("n_q", [[1], [16], [50]])
def test_attention_one_long_context(dtype, n_q):
    """One request whose context is split over many workers and merged."""
    ctx = [9001]
    c, table, q, cu, tree = _attn_case(77, ctx, n_q, 1, 128, 2, "causal", dtype)
    _check_attn(c, table, q, cu, ctx, "causal", tree, dtype, max_q=n_q[0])


@pytest.mark.parametrize("others", [0, 3, 40])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_attention_one_item_of_many_pieces(others, dtype):
    """A context of several hundred pages for one head beside empty and short ones: its pieces are kept few."""
    ctx = [(i * 29) % 70 for i in range(others // 2)] + [30011] + [(i * 31) % 90 for i in range(others - others // 2)]
    c, table, q, cu, tree = _attn_case(13 + others, ctx, [1] * len(ctx), 1, 64, 2, "causal", dtype)
    _check_attn(c, table, q, cu, ctx, "causal", tree, dtype, max_q=1)


@pytest.mark.parametrize("hd,n_q", [(64, 17), (128, 40), (128, 2)])
def test_attention_long_pieces(hd, n_q):
    """Several items and many tiles per worker: every ring wraps a few times within a piece."""
    ctx = [3000, 2600, 4100, 2049, 2048, 3333, 64, 2500]
    c, table, q, cu, tree = _attn_case(31, ctx, [n_q] * 8, 8, hd, 8, "causal", torch.bfloat16)
    _check_attn(c, table, q, cu, ctx, "causal", tree, torch.bfloat16, max_q=n_q)


@pytest.mark.parametrize("n_q", [1, 20])
def test_attention_many_requests(n_q):
    """More requests than workers, most of them short."""
    ctx = [(i * 37) % 200 for i in range(400)]
    c, table, q, cu, tree = _attn_case(5, ctx, [n_q if i % 5 else 0 for i in range(400)], 1, 64, 2, "none", torch.bfloat16)
    _check_attn(c, table, q, cu, ctx, "none", tree, torch.bfloat16, max_q=n_q)


@pytest.mark.parametrize("dtype,n_q", [(torch.bfloat16, 1), (torch.bfloat16, 6), (torch.bfloat16, 40), (torch.float32, 5)])
@pytest.mark.parametrize("n", [2, 9, 61, 170])
@pytest.mark.parametrize("mask", ["none", "causal"])
def test_attention_cuts_between_short_and_long_items(dtype, n_q, n, mask):
    """Items of one page among long ones: workers that get none of an item's pages, items that begin with the next one."""
    ctx = [1 + 61 * i % 130 if i % 7 else 700 + 64 * i for i in range(n)]
    c, table, q, cu, tree = _attn_case(n + n_q, ctx, [n_q - i % 2 for i in range(n)], 1, 64, 2, mask, dtype)
    _check_attn(c, table, q, cu, ctx, mask, tree, dtype, max_q=n_q)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("n_q", [3, 40])
def test_attention_nan_and_infinity_in_hidden_places(dtype, n_q):
    """Later rows' K and V hold NaN, and one row of q an infinity: rows that do not see them are untouched, a
    row that sees a NaN in one value dimension has NaN there alone, one that sees a NaN key is NaN."""
    from block_diffusion_speculative_inject_gb300 import kv8_attention
    ctx = [100 + n_q, 64 + n_q]
    c, table, q, cu, _ = _attn_case(3, ctx, [n_q, n_q], 1, 128, 4, "causal", dtype)
    for b in range(2):
        pv, pk = 100 + n_q - 2 if b == 0 else 64 + n_q - 1, ctx[b] - 1
        page, off = int(table[b, pv // PAGE]), pv % PAGE
        c["v_pages"].view(torch.uint8)[page, 0, 5, off] = NAN_BYTE
        page, off = int(table[b, pk // PAGE]), pk % PAGE
        c["k_pages"].view(torch.uint8)[page, 0, off, 9] = 0xFF
    q[cu[1]] = math.inf
    gpu = _to_gpu(c)
    out, lse = kv8_attention(gpu, q.cuda(), _i4(cu), _i4(ctx), table.cuda(), mask="causal", want_lse=True, max_q=n_q)
    out, lse = out.cpu(), lse.cpu()
    last = cu[1] - 1
    assert bool(out[:last - 1].isfinite().all()) and bool(lse[:last].isfinite().all())
    nan = out[last - 1].isnan()
    assert bool(nan[:, 5].all()) and int(nan.sum()) == nan.shape[0]
    assert bool(out[last].isnan().all()) and bool(lse[last].isnan().all())
    assert bool(out[cu[1]].isnan().all()) and bool(out[cu[1] + 1:-1].isfinite().all()) and bool(out[-1].isnan().all())


def test_attention_tree_bits_beyond_the_words_and_pages_out_of_range():
    """Rows past the mask's words are not seen; tokens on a page outside the pool are not seen."""
    ctx, n_q = [150, 90], [40, 5]
    c, table, q, cu, tree = _attn_case(6, ctx, n_q, 1, 64, 2, "tree", torch.bfloat16)
    table[0, 0], table[1, 1] = 1 << 20, -5
    _check_attn(c, table, q, cu, ctx, "tree", tree[:, :1].contiguous(), torch.bfloat16, max_q=40)
    _check_attn(c, table, q, cu, ctx, "none", None, torch.bfloat16, max_q=40)


@pytest.mark.parametrize("n_q", [2, 24])
def test_attention_rows_that_see_nothing(n_q):
    """A tree whose rows' bits are clear over a context of the rows alone, and an empty context."""
    ctx = [n_q, 0, 70]
    c, table, q, cu, tree = _attn_case(6, ctx, [n_q] * 3, 2, 64, 4, "tree", torch.bfloat16)
    tree[:n_q] = 0
    out, lse = _check_attn(c, table, q, cu, ctx, "tree", tree, torch.bfloat16, max_q=n_q)
    assert bool((out[:2 * n_q] == 0).all()) and bool((lse[:2 * n_q] == -math.inf).all())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("n_q", [1, 20])
def test_attention_scales_and_scores_of_very_different_size(dtype, n_q):
    """Page scales over 2^-64 .. 2^60, peaked and flat scores, one dominant token among thousands of small ones."""
    ctx = [1500, 400, 2000]
    c, table, q, cu, tree = _attn_case(12, ctx, [n_q] * 3, 1, 128, 4, "none", dtype)
    g = torch.Generator().manual_seed(1)
    fin = c["v_scale"].isfinite()
    c["v_scale"][fin] = torch.exp2(torch.randint(-64, 61, (int(fin.sum()),), generator=g).float())
    _check_attn(c, table, q, cu, ctx, "none", tree, dtype, max_q=n_q)
    c, table, q, cu, tree = _attn_case(13, ctx, [n_q] * 3, 1, 128, 4, "none", dtype, spread=30.0)
    _check_attn(c, table, q, cu, ctx, "none", tree, dtype, max_q=n_q)
    c, table, q, cu, tree = _attn_case(14, ctx, [n_q] * 3, 1, 128, 4, "none", dtype, spread=1e-3)
    for b in range(3):                                 # a token 14 nats above the rest
        p = int(table[b, 3])
        c["k_scale"][p], c["k_scale"][int(table[b, 0])] = 1.0, 1.0
        qm = q[cu[b]:cu[b] + 1, :1].float()
        c["k_pages"][p, 0, 7] = (qm[0, 0] / qm.norm() * 400).to(R.E4M3)
        q[cu[b]:cu[b + 1]] = (qm / qm.norm() * 0.4).to(dtype)
    _check_attn(c, table, q, cu, ctx, "none", tree, dtype, max_q=n_q)
    _check_attn(c, table, q, cu, ctx, "none", tree, dtype, scale=3.0, max_q=n_q)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("mask", ["none", "causal", "tree"])
@pytest.mark.parametrize("n_q,hint", [(3, 3), (3, 100), (40, 1), (40, 40)])
def test_attention_zero_and_tiny_queries_over_zero_keys(dtype, mask, n_q, hint):
    """Pages of zero keys have the smallest scale, 2^-64, and a row of zeros or of tiny entries a factor near 2^-110: their
    product is below fp32's range. Such rows weigh all that they see alike, in every kernel that the hint may choose,
    also on pages of which they see a part."""
    ctx = [100 + n_q, 64, n_q, 200]
    c, table, q, cu, tree = _attn_case(8, ctx, [n_q] * 4, 1, 128, 4, mask, dtype)
    for b in (0, 1, 2):                                # the last request's keys stay as they are
        for i in range(R.pages_of(ctx[b])):
            p, live = int(table[b, i]), min(PAGE, ctx[b] - i * PAGE)
            c["k_pages"].view(torch.uint8)[p, :, :live] = 0
            c["k_scale"][p] = 2.0 ** -64
    q[0::3] = 0
    q[1::3] = (q[1::3].float() * 2.0 ** -90).to(dtype)
    _check_attn(c, table, q, cu, ctx, mask, tree, dtype, max_q=hint)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("n_q", [1, 20])
def test_attention_value_scales_at_their_limit(dtype, n_q):
    """Pages whose V scales lie a factor 2^100 apart, in either order: the small ones' tokens keep their weight."""
    ctx = [1024, 333]
    for order in (0, 1):
        c, table, q, cu, tree = _attn_case(19 + order, ctx, [n_q, n_q], 1, 128, 4, "none", dtype, spread=0.5)
        for b in range(2):
            for i in range(R.pages_of(ctx[b])):
                c["v_scale"][int(table[b, i])] = 2.0 ** (36 if (i + order) % 4 == 0 else -64)
        _check_attn(c, table, q, cu, ctx, "none", tree, dtype, max_q=n_q)


@pytest.mark.parametrize("hint", [0, 1, 16, 17, 10 ** 6])
def test_attention_max_q_only_steers(hint):
    """Any max_q gives the rows of every request."""
    c, table, q, cu, tree = _attn_case(21, [200, 333], [1, 45], 2, 128, 8, "causal", torch.bfloat16)
    _check_attn(c, table, q, cu, [200, 333], "causal", tree, torch.bfloat16, max_q=hint)


def test_attention_strided_queries():
    """q as columns of a projection's output."""
    from block_diffusion_speculative_inject_gb300 import kv8_attention
    for n_q in (2, 30):
        c, table, q, cu, _ = _attn_case(4, [90, 140], [n_q, n_q], 2, 64, 4, "causal", torch.bfloat16)
        gpu = _to_gpu(c)
        args = (_i4(cu), _i4([90, 140]), table.cuda())
        want = kv8_attention(gpu, q.cuda(), *args, max_q=n_q)
        buf = torch.full((2 * n_q, 8 * 64 + 8), math.nan, dtype=torch.bfloat16, device="cuda")
        view = buf[:, 128:128 + 4 * 64].unflatten(1, (4, 64))
        view.copy_(q)
        assert torch.equal(kv8_attention(gpu, view, *args, max_q=n_q), want)


@pytest.mark.parametrize("n_q,hint", [(1, 1), (2, 64)])
def test_attention_most_requests(n_q, hint):
    """4096 requests, a fifth of them without rows, in both kernels."""
    ctx = [(i * 37) % 130 for i in range(4096)]
    c, table, q, cu, tree = _attn_case(15, ctx, [n_q if i % 5 else 0 for i in range(4096)], 1, 64, 1, "causal", torch.bfloat16)
    _check_attn(c, table, q, cu, ctx, "causal", tree, torch.bfloat16, max_q=hint)


@pytest.mark.parametrize("hint", [1, 3])
def test_attention_most_heads_and_blocks(hint):
    """128 kv heads of 8 query heads each; a block table of 2^24 entries."""
    from block_diffusion_speculative_inject_gb300 import kv8_attention
    ctx, n_q = [70, 130], [3, 1]
    c, table, q, cu, tree = _attn_case(16, ctx, n_q, 128, 64, 1024, "causal", torch.bfloat16, extra=0)
    _check_attn(c, table, q, cu, ctx, "causal", tree, torch.bfloat16, max_q=hint)
    gpu, q1 = _to_gpu(c), q[:3].cuda()
    wide = torch.full((1, 1 << 24), -1, dtype=torch.int32, device="cuda")
    wide[0, :table.shape[1]] = table[0].cuda()
    one = table[:1].cuda().contiguous()
    assert torch.equal(kv8_attention(gpu, q1, _i4([0, 3]), _i4([70]), wide, max_q=hint),
                       kv8_attention(gpu, q1, _i4([0, 3]), _i4([70]), one, max_q=hint))


def test_append_and_plan_at_their_limits():
    """128 kv heads; a table of 2^24 blocks and a stack of 2^24 pages; the largest and smallest slots."""
    from block_diffusion_speculative_inject_gb300 import kv8_append, page_plan
    n_pages, nkv, hd = 5, 128, 64
    g = torch.Generator().manual_seed(12)
    slots = [PAGE * 3 + 60 + i for i in range(4)] + [2 ** 63 - 1, -2 ** 63, n_pages * PAGE] + [PAGE + i for i in range(9)]
    k, v = (torch.randn((len(slots), nkv, hd), generator=g).bfloat16() for _ in range(2))
    want = _cache_cpu(5, n_pages, nkv, hd)
    gpu = _to_gpu(want)
    kv8_append(gpu, k.cuda(), v.cuda(), torch.tensor(slots, device="cuda"))
    R.append(want, k, v, slots)
    _same_cache(gpu, want)
    most = 1 << 24
    table = torch.full((1, most), -1, dtype=torch.int32, device="cuda")
    stack = torch.arange(most, dtype=torch.int32, device="cuda")
    full = page_plan(_i4([0]), _i4([most * PAGE]), table, stack, _i4([most]), 0)         # no room for the rows
    assert full["refused"].tolist() == [1] and full["n_free"].tolist() == [most]
    full = page_plan(_i4([0]), _i4([most * PAGE]), table, stack, _i4([most]), most * PAGE)
    assert full["refused"].tolist() == [0] and full["n_free"].tolist() == [0] and full["new_len"].tolist() == [most * PAGE]
    assert torch.equal(table[0], torch.arange(most - 1, -1, -1, dtype=torch.int32, device="cuda"))
    p = torch.arange(most * PAGE, dtype=torch.int32, device="cuda")
    assert torch.equal(full["positions"], p)
    assert torch.equal(full["slot_map"], (most - 1 - p.long() // PAGE) * PAGE + p % PAGE)
    del full, p
    back = page_plan(_i4([most * PAGE]), _i4([-2 ** 31]), table, stack.zero_(), _i4([0]), 0)
    assert back["n_free"].tolist() == [most] and torch.equal(stack, table[0])
    torch.cuda.empty_cache()


def test_far_pages_of_a_large_pool():
    """Pages whose bytes lie beyond 2^32: append, read and both attention kernels."""
    from block_diffusion_speculative_inject_gb300 import KV8Cache, kv8_append, kv8_attention, kv8_read
    n_pages, nkv, hd = 1_100_000, 1, 64
    cache = KV8Cache.empty(n_pages, nkv, hd)
    g = torch.Generator().manual_seed(1)
    pages = [n_pages - 1, 5, 1_048_577]
    slots = torch.tensor([pages[p // PAGE] * PAGE + p % PAGE for p in range(150)])
    k, v = (torch.randn((150, nkv, hd), generator=g).bfloat16() for _ in range(2))
    kv8_append(cache, k.cuda(), v.cuda(), slots.cuda())
    small = _cache_cpu(0, 3, nkv, hd)
    local = [p // PAGE * PAGE + p % PAGE for p in range(150)]
    R.append(small, k, v, local)
    rk, rv = kv8_read(cache, slots.cuda())
    idx = torch.tensor(local)
    assert torch.equal(rk.cpu()[:, 0], small["k_pages"].float()[idx // PAGE, 0, idx % PAGE] * small["k_scale"][idx // PAGE])
    for n_q in (1, 40):
        q = torch.randn((n_q, 2, hd), generator=g).bfloat16()
        got = kv8_attention(cache, q.cuda(), _i4([0, n_q]), _i4([150]), _i4([pages]), max_q=n_q)
        want, _, absv, top = R.attention(small, q, [0, n_q], [150], torch.tensor([[0, 1, 2]]), "causal")
        tol = want.abs() * 2.0 ** -8 + absv * (2.0 ** -11 + 2 * (top * 2.0 ** -19 + 2.0 ** -19))[..., None]
        assert bool(((got.cpu().double() - want).abs() <= tol).all())


# ---------------------------------------------------------------- together
class _Loop:
    """Verify rounds over an 8-bit cache, and the same rounds on the reference's cache."""

    def __init__(self, n, nkv, group, hd, n_pages, width, dtype, seed=0):
        from block_diffusion_speculative_inject_gb300 import KV8Cache, Rope
        self.n, self.nkv, self.nq, self.hd, self.dtype = n, nkv, nkv * group, hd, dtype
        self.g = torch.Generator().manual_seed(seed)
        self.rope = Rope(hd, theta=1e4)
        self.freq, self.mag = R.rope_freq(hd, 1e4)
        self.cache = KV8Cache.empty(n_pages, nkv, hd)
        self.ref = {k: getattr(self.cache, k).cpu().clone() for k in ("k_pages", "v_pages", "k_scale", "v_scale")}
        self.len = _i4([0] * n)
        self.table = torch.full((n, width), -1, dtype=torch.int32, device="cuda")
        self.stack = torch.arange(n_pages, dtype=torch.int32, device="cuda")
        self.free = _i4([n_pages])

    def draw(self, rows):
        f = lambda h: torch.randn((rows, h, self.hd), generator=self.g).to(self.dtype)  # noqa: E731
        return f(self.nq), f(self.nkv), f(self.nkv)

    def device_round(self, n_new, rows, q, k, v, max_q):
        from block_diffusion_speculative_inject_gb300 import kv8_append, kv8_attention, page_plan, rope
        p = page_plan(self.len, n_new, self.table, self.stack, self.free, rows)
        q, k = rope(self.rope, p["positions"], q, k)
        kv8_append(self.cache, k, v, p["slot_map"])
        out = kv8_attention(self.cache, q, p["cu_rows"], p["new_len"], self.table, mask="causal", max_q=max_q)
        return p, q, k, out

    def check_round(self, p, k, q, v, out):
        """The call's own rotated rows through the reference's cache and attention."""
        R.append(self.ref, k.cpu(), v, p["slot_map"].tolist())
        used = sorted({s // PAGE for s in p["slot_map"].tolist() if s >= 0})
        for name in ("k_pages", "v_pages"):
            a = getattr(self.cache, name).view(torch.uint8)[used].cpu()
            assert torch.equal(a, self.ref[name].view(torch.uint8)[used])
        cu, ctx = p["cu_rows"].tolist(), p["new_len"].tolist()
        want, _, absv, top = R.attention(self.ref, q.cpu(), cu, ctx, self.table.cpu(), "causal")
        r = 2.0 ** -11 if self.dtype == torch.bfloat16 else 2.0 ** -20
        tol = want.abs() * HALF[self.dtype] + absv * (r + 2 * (top * 2.0 ** -19 + 2.0 ** -19))[..., None]
        n = cu[-1]
        assert bool(((out.cpu().double()[:n] - want[:n]).abs() <= tol[:n]).all())


@pytest.mark.parametrize("dtype,group,hd", [(torch.bfloat16, 4, 128), (torch.float32, 2, 64)])
def test_verify_loop(dtype, group, hd):
    """Prompts, then rounds of a block of rows per request whose rejected part is dropped by the next plan;
    the accept lengths never leave the GPU."""
    from block_diffusion_speculative_inject_gb300 import page_plan
    n, blk = 5, 8
    lp = _Loop(n, 2, group, hd, 64, 8, dtype)
    prompt = [70, 1, 128, 33, 200]
    rows = sum(prompt)
    q, k, v = lp.draw(rows)
    p, qr, kr, out = lp.device_round(_i4(prompt), rows, q.cuda(), k.cuda(), v.cuda(), max(prompt))
    assert p["refused"].sum() == 0
    lp.check_round(p, kr, qr, v, out)
    lp.len, lp.free = p["new_len"], p["n_free"]
    for step in range(4):
        q, k, v = lp.draw(n * blk)
        p, qr, kr, out = lp.device_round(_i4([blk] * n), n * blk, q.cuda(), k.cuda(), v.cuda(), blk)
        lp.check_round(p, kr, qr, v, out)
        accept = torch.randint(0, blk, (n,), generator=lp.g, dtype=torch.int32).cuda()
        drop = page_plan(p["new_len"], accept + 1 - blk, lp.table, lp.stack, p["n_free"], 0)
        assert torch.equal(drop["new_len"], lp.len + accept + 1)
        held = sum(R.pages_of(x) for x in drop["new_len"].tolist())
        assert drop["n_free"].tolist() == [64 - held]
        lp.len, lp.free = drop["new_len"], drop["n_free"]
    got = [x for b in range(n) for x in lp.table[b, :R.pages_of(int(lp.len[b]))].tolist()]
    assert sorted(got + lp.stack[:int(lp.free)].tolist()) == list(range(64))      # no page lost, none twice


@pytest.mark.parametrize("budget", [11, 40])
def test_draft_tree_round(budget):
    """A round over draft trees: ddtree_build's masks go to the attention as they are (checked against the parents' chains),
    ddtree_walk accepts a path, and the path's rows, which lie scattered among the tree's, are appended anew after all of
    the tree's tokens were dropped."""
    from block_diffusion_speculative_inject_gb300 import (ddtree_build, ddtree_walk, kv8_append, kv8_attention, page_plan,
                                                          rope)
    n, L, kc, nkv, dtype = 3, 7, 4, 2, torch.bfloat16
    lp = _Loop(n, nkv, 4, 128, 40, 8, dtype, seed=3)
    prompt = [100, 1, 63]
    q, k, v = lp.draw(sum(prompt))
    p, qr, kr, out = lp.device_round(_i4(prompt), sum(prompt), q.cuda(), k.cuda(), v.cuda(), max(prompt))
    lp.check_round(p, kr, qr, v, out)
    lp.len, lp.free = p["new_len"], p["n_free"]

    logp = -torch.sort(torch.rand((n, L, kc), generator=lp.g) * 3, dim=2).values
    tok = torch.arange(kc, dtype=torch.int32).expand(n, L, kc).contiguous()
    tree = ddtree_build(tok.cuda(), logp.cuda(), budget)
    assert tree["n_nodes"].tolist() == [budget] * n
    rows = n * (budget + 1)
    q, k, v = lp.draw(rows)
    p = page_plan(lp.len, _i4([budget + 1] * n), lp.table, lp.stack, lp.free, rows)
    depth = torch.cat([torch.zeros((n, 1), dtype=torch.int32, device="cuda"), tree["depth"]], 1)
    positions = (lp.len[:, None] + depth).reshape(-1).to(torch.int32)
    qr, kr = rope(lp.rope, positions, q.cuda(), k.cuda())
    kv8_append(lp.cache, kr, v.cuda(), p["slot_map"])
    out = kv8_attention(lp.cache, qr, p["cu_rows"], p["new_len"], lp.table, mask="tree",
                        tree_mask=tree["mask"].flatten(0, 1), max_q=budget + 1)
    R.append(lp.ref, kr.cpu(), v, p["slot_map"].tolist())
    parent = tree["parent"].tolist()
    chain = torch.zeros((n, budget + 1, budget + 1), dtype=torch.bool)
    for b in range(n):
        for i in range(budget + 1):
            j = i
            while j > 0:
                chain[b, i, j] = True
                j = parent[b][j - 1] + 1
            chain[b, i, 0] = True
    bits = torch.zeros((n, budget + 1, 2), dtype=torch.int64)
    for j in range(budget + 1):
        bits[:, :, j // 32] |= chain[:, :, j].long() << (j % 32)
    bits = (bits - (bits >> 31 << 32)).to(torch.int32).flatten(0, 1)
    want, _, absv, top = R.attention(lp.ref, qr.cpu(), p["cu_rows"].tolist(), p["new_len"].tolist(), lp.table.cpu(), "tree", bits)
    tol = want.abs() * HALF[dtype] + absv * (2.0 ** -11 + 2 * (top * 2.0 ** -19 + 2.0 ** -19))[..., None]
    assert bool(((out.cpu().double() - want).abs() <= tol).all())

    target = torch.randint(0, kc, (n, budget + 1), generator=lp.g, dtype=torch.int32)
    target[:, 0] = tree["tok"][:, 0].cpu()
    accept, tokens, _ = ddtree_walk(tree, L, target.cuda())
    path = []                                          # rows of the accepted path, the root first
    for b in range(n):
        at = 0
        path.append(b * (budget + 1))
        for t in tokens[b, :int(accept[b])].tolist():
            at = next(i + 1 for i in range(budget) if parent[b][i] == at - 1 and int(tree["tok"][b, i]) == t)
            path.append(b * (budget + 1) + at)
    assert len(path) == int(accept.sum()) + n and int(accept.min()) >= 1
    drop = page_plan(p["new_len"], _i4([-budget - 1] * n), lp.table, lp.stack, p["n_free"], 0)
    assert torch.equal(drop["new_len"], lp.len)
    kept = page_plan(drop["new_len"], accept + 1, lp.table, lp.stack, drop["n_free"], rows)
    idx = torch.tensor(path)
    ka, va = (torch.cat([x, torch.zeros((rows - len(path),) + x.shape[1:], dtype=dtype)]) for x in (kr.cpu()[idx], v[idx]))
    kv8_append(lp.cache, ka.cuda(), va.cuda(), kept["slot_map"])
    R.append(lp.ref, ka, va, kept["slot_map"].tolist())
    assert torch.equal(kept["positions"][:len(path)].cpu(), positions.cpu()[idx])
    q, _, _ = lp.draw(n)
    cu, ctx = list(range(n + 1)), kept["new_len"].tolist()
    out = kv8_attention(lp.cache, q.cuda(), _i4(cu), kept["new_len"], lp.table, max_q=1)
    want, _, absv, top = R.attention(lp.ref, q, cu, ctx, lp.table.cpu(), "causal")
    tol = want.abs() * HALF[dtype] + absv * (2.0 ** -11 + 2 * (top * 2.0 ** -19 + 2.0 ** -19))[..., None]
    assert bool(((out.cpu().double() - want).abs() <= tol).all())


def test_round_in_a_graph_and_on_another_stream():
    """A whole round captured once and replayed on new inputs equals the eager round; two graphs with their own
    workspaces run at once on two streams."""
    n, blk = 3, 6
    eager, captured = (_Loop(n, 2, 4, 128, 32, 6, torch.bfloat16) for _ in range(2))
    q, k, v = (x.cuda() for x in eager.draw(n * blk))
    add = _i4([blk] * n)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        captured.device_round(add, n * blk, q, k, v, blk)        # warm up
    torch.cuda.current_stream().wait_stream(side)
    captured.len, captured.free = _i4([0] * n), _i4([32])
    captured.stack.copy_(torch.arange(32, dtype=torch.int32))
    graph = torch.cuda.CUDAGraph()
    sq, sk, sv = q.clone(), k.clone(), v.clone()
    with torch.cuda.graph(graph):
        p, _, _, out = captured.device_round(add, n * blk, sq, sk, sv, blk)
    for step in range(3):
        for s, x in ((sq, q), (sk, k), (sv, v)):
            s.copy_(x)
        graph.replay()
        pe, _, _, oe = eager.device_round(add, n * blk, q, k, v, blk)
        assert torch.equal(out, oe) and torch.equal(p["slot_map"], pe["slot_map"])
        captured.len.copy_(p["new_len"])
        captured.free.copy_(p["n_free"])
        eager.len, eager.free = pe["new_len"], pe["n_free"]
        q, k, v = (x.cuda() for x in eager.draw(n * blk))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_few_rows_after_kernels_that_fill_shared_memory(dtype):
    """Small few-row calls (no request is beyond the 32 that a warp sums up alone) between many-row ones, whose tiles of
    random bytes stay in shared memory: the abort word and the barriers are set before any warp looks at them."""
    from block_diffusion_speculative_inject_gb300 import kv8_attention
    c, table, q, cu, _ = _attn_case(41, [300, 70], [2, 2], 8, 128, 16, "causal", dtype)
    few = (_to_gpu(c), q.cuda(), _i4(cu), _i4([300, 70]), table.cuda())
    c, table, q, cu, _ = _attn_case(42, [900] * 4, [64] * 4, 8, 128, 16, "causal", torch.bfloat16)
    many = (_to_gpu(c), q.cuda(), _i4(cu), _i4([900] * 4), table.cuda())
    want = kv8_attention(*few, max_q=2)
    assert bool(want.isfinite().all())
    got = []
    for _ in range(100):
        kv8_attention(*many, max_q=64)
        got += [kv8_attention(*few, max_q=2) for _ in range(2)]
    assert all(torch.equal(x, want) for x in got)


@pytest.mark.parametrize("n_q", [1, 20])
def test_two_calls_at_once(n_q):
    """Two streams, their own workspaces, split contexts: each equals its call alone, bit for bit, many times."""
    from block_diffusion_speculative_inject_gb300 import kv8_attention, kv8_workspace
    sets = []
    for seed in (1, 2):
        c, table, q, cu, _ = _attn_case(seed, [6000, 900], [n_q, n_q], 2, 128, 8, "causal", torch.bfloat16)
        a = (_to_gpu(c), q.cuda(), _i4(cu), _i4([6000, 900]), table.cuda())
        ws = torch.empty(kv8_workspace(*a, max_q=n_q), dtype=torch.uint8, device="cuda")
        sets.append((a, ws, kv8_attention(*a, max_q=n_q)))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    got = [[], []]
    for _ in range(10):
        for i, (a, ws, _) in enumerate(sets):
            got[i].append(kv8_attention(*a, max_q=n_q, workspace=ws, stream=streams[i]))
    torch.cuda.synchronize()
    for i, (_, _, want) in enumerate(sets):
        assert all(torch.equal(x, want) for x in got[i])
