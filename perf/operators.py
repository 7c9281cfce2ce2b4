"""The operators of the 8-bit paged cache as measured workloads: block tables and slot maps from request
lengths, rotary positions, the quantised cache write, and attention over the cache.

`run` computes them in elementary torch operations, or, with `own` set, through the package's calls on the
same inputs. `exact` is their definition in 64 bits. Lengths follow from the case alone, values from the seed.

Cache layout (the package's): K pages [n_pages, kv heads, 64, head dim], V pages [n_pages, kv heads, head dim, 64]
in e4m3, one power-of-two scale per page and kv head for each of K and V.
"""
import math
import random

import torch

own = False

PAGE = 64
E4M3_MAX = 448.0
MIN_EXP = -64


def listed():
    return [
        # one decoding round of 128 requests (context 1024, 8 rows each): some finish, some roll back
        dict(name="plan_step_b128", op="plan", n=128, ctx_min=512, ctx_max=1536, add_min=1, add_max=8, drop=0.1, full=False),
        # admission of 32 ragged prompts at once: one slot for each of ~139 thousand rows
        dict(name="plan_prompts_b32", op="plan", n=32, ctx_min=0, ctx_max=0, add_min=512, add_max=8192, drop=0.0, full=False),
        # one request's verify block of 16 rows: the smallest call, latency only
        dict(name="rope_block_b1", op="rope", rows=16, nq=32, nkv=8, hd=128, rot=128, inter=False, scaling="none",
             factor=1.0, far=2048, dtype="bf16", transpose=False),
        # a long prompt's queries and keys with positions scaled for a context of 131072
        dict(name="rope_prompt_yarn", op="rope", rows=32768, nq=40, nkv=8, hd=128, rot=128, inter=False, scaling="yarn",
             factor=4.0, far=131072, dtype="bf16", transpose=False),
        # interleaved pairs on half of a small head, the gradient's direction, fp32, an odd number of rows
        dict(name="rope_partial_f32", op="rope", rows=5003, nq=12, nkv=4, hd=64, rot=32, inter=True, scaling="linear",
             factor=8.0, far=60000, dtype="f32", transpose=True),
        # the verify blocks of 8 requests appended in the middle of pages
        dict(name="append_block_b8", op="append", n=8, ctx_min=100, ctx_max=2000, add_min=16, add_max=16, nkv=8, hd=128,
             dtype="bf16"),
        # a chunk of 4096 prompt rows of each of 8 requests
        dict(name="append_prompt_b8", op="append", n=8, ctx_min=0, ctx_max=0, add_min=4096, add_max=4096, nkv=8, hd=128,
             dtype="bf16"),
        # a single request's single token at context 2048: latency
        dict(name="attn_token_b1", op="attn", n=1, ctx_min=2048, ctx_max=2048, q_min=1, q_max=1, nq=32, nkv=8, hd=128,
             mask="causal", dtype="bf16"),
        # a decoding batch with ragged contexts
        dict(name="attn_token_b64", op="attn", n=64, ctx_min=512, ctx_max=8192, q_min=1, q_max=1, nq=32, nkv=8, hd=128,
             mask="causal", dtype="bf16"),
        # verify blocks of 16 rows over long contexts
        dict(name="attn_block_32k_b8", op="attn", n=8, ctx_min=32768, ctx_max=32768, q_min=16, q_max=16, nq=40, nkv=8,
             hd=128, mask="causal", dtype="bf16"),
        # draft trees of 255 nodes and their root, ancestors only
        dict(name="attn_tree_256_b8", op="attn", n=8, ctx_min=1000, ctx_max=5000, q_min=256, q_max=256, nq=32, nkv=8,
             hd=128, mask="tree", dtype="bf16"),
        # small fp32 heads, ragged rows (none for some requests), every key of the context visible
        dict(name="attn_ragged_f32", op="attn", n=9, ctx_min=1, ctx_max=777, q_min=0, q_max=8, nq=4, nkv=2, hd=64,
             mask="none", dtype="f32"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["plan", "rope", "append", "attn", "attn", "attn"])
    if op == "plan":
        n = _log(rng, 1, 1024)
        if rng.random() < 0.5:
            c = _log(rng, 1, 4096)
            return dict(op=op, n=n, ctx_min=c // 2, ctx_max=c, add_min=0, add_max=rng.choice([1, 8, 16, 33]),
                        drop=rng.choice([0.0, 0.1, 0.5]), full=rng.random() < 0.3)
        a = _log(rng, 64, max(65, min(16384, 139000 // n)))
        return dict(op=op, n=n, ctx_min=0, ctx_max=rng.choice([0, 100]), add_min=a // 2, add_max=a, drop=0.0,
                    full=rng.random() < 0.2)
    hd = rng.choice([64, 128])
    nkv = rng.choice([1, 2, 4, 8])
    group = rng.choice([1, 2, 4, 5, 7, 8])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op == "rope":
        cost = 32768 * 48 * 128 * 2
        per = (nkv * group + nkv) * hd * (2 if dtype == "bf16" else 4)
        return dict(op=op, rows=_log(rng, 1, min(65536, cost // per)), nq=nkv * group, nkv=nkv, hd=hd,
                    rot=rng.choice([hd, hd, hd // 2, hd // 4, 20]), inter=rng.random() < 0.5,
                    scaling=rng.choice(["none", "linear", "yarn"]), factor=rng.choice([2.0, 4.0, 8.0, 2.5]),
                    far=_log(rng, 100, 1000000), dtype=dtype, transpose=rng.random() < 0.3)
    if op == "append":
        n = _log(rng, 1, 128)
        if rng.random() < 0.5:
            a = rng.choice([1, 2, 8, 16, 33])
            return dict(op=op, n=n, ctx_min=0, ctx_max=_log(rng, 1, 2000), add_min=rng.choice([0, a]), add_max=a,
                        nkv=nkv, hd=hd, dtype=dtype)
        a = _log(rng, 64, max(65, 16384 // n))
        return dict(op=op, n=n, ctx_min=0, ctx_max=rng.choice([0, 200]), add_min=a // 2, add_max=a, nkv=nkv, hd=hd,
                    dtype=dtype)
    q = rng.choice([1, 1, 2, 8, 16, 32, _log(rng, 33, 400)])
    most = 2.5e8 if dtype == "bf16" and q <= 32 else 4e9 / (group * q) / 64   # bytes of K and V the case may hold
    n = _log(rng, 1, 64 if q <= 32 else 8)
    top = max(1, min(65536, int(most / (n * nkv * hd * 2))))
    ctx = _log(rng, 1, top)
    return dict(op=op, n=n, ctx_min=rng.choice([ctx, ctx // 2, ctx // 8]), ctx_max=ctx,
                q_min=rng.choice([0, 1, q]) if n > 1 else q, q_max=q, nq=nkv * group, nkv=nkv, hd=hd,
                mask=rng.choice(["none", "causal", "causal", "tree"]), dtype=dtype)


# ---------------------------------------------------------------- sizes that follow from the case
def _ints(case, what, lo, hi):
    """n integers of [lo, hi] (the ends among them where n > 1), the same for every seed."""
    r = random.Random("%s/%d/%d/%d" % (what, case["n"], lo, hi))
    v = [r.randint(lo, hi) for _ in range(case["n"])]
    if case["n"] > 1:
        v[0], v[-1] = hi, lo
    return v


def _lens(case):
    """(context lengths before, rows added) of a plan or append case, or (context, query rows) of attention."""
    ctx = _ints(case, "ctx", case["ctx_min"], case["ctx_max"])
    if case["op"] == "attn":
        q = _ints(case, "q", case["q_min"], case["q_max"])
        if case["mask"] != "none":      # the rows are the context's last tokens
            ctx = [c + x for c, x in zip(ctx, q)]
        return ctx, q
    add = _ints(case, "add", case["add_min"], case["add_max"])
    if case["op"] == "plan" and case["drop"]:
        r = random.Random("drop/%d" % case["n"])
        for i in range(case["n"]):
            if r.random() < case["drop"]:
                add[i] = -ctx[i] if r.random() < 0.5 else -r.randint(0, 16)
    return ctx, add


def _pages(n):
    return -(-n // PAGE)


def work(case):
    op = case["op"]
    if op == "plan":
        ctx, add = _lens(case)
        rows = sum(a for a in add if a > 0)
        new = sum(max(0, _pages(c + a) - _pages(c)) for c, a in zip(ctx, add))
        return {"bytes": 5 * 4 * case["n"] + 8 * new + 12 * rows, "flops": 0}
    if op == "rope":
        e = case["rows"] * (case["nq"] + case["nkv"])
        size = 2 if case["dtype"] == "bf16" else 4
        return {"bytes": 2 * e * case["hd"] * size + 4 * case["rows"], "flops": 3 * e * case["rot"]}
    size = 2 if case["dtype"] == "bf16" else 4
    if op == "append":
        ctx, add = _lens(case)
        e = sum(add) * case["nkv"] * case["hd"] * 2
        return {"bytes": e * (size + 1) + 8 * sum(add), "flops": 3 * e}
    ctx, q = _lens(case)
    kv = sum(c for c, x in zip(ctx, q) if x) * case["nkv"] * case["hd"] * 2
    seen = sum(x * c - (x * (x - 1) // 2 if case["mask"] != "none" else 0) for c, x in zip(ctx, q))
    return {"bytes": kv + sum(q) * case["nq"] * (2 * case["hd"] * size + 4),
            "flops": 4 * seen * case["nq"] * case["hd"]}


# ---------------------------------------------------------------- inputs
def _dev():
    return "cuda" if torch.cuda.is_available() else "cpu"


def _gen(seed):
    return torch.Generator(device=_dev()).manual_seed(int(seed) * 1000003 + 17)


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device=_dev())


def _dtype(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def _cum(v):
    out = [0]
    for x in v:
        out.append(out[-1] + x)
    return out


def _tables(g, n_blocks, spare):
    """Block tables of a pool in use: the pages of the requests scattered over it (-1 past a request's last)."""
    total = sum(n_blocks)
    width = max(1, max(n_blocks))
    perm = torch.randperm(total + spare, generator=g, device=_dev()).to(torch.int32)
    table = torch.full((len(n_blocks), width), -1, dtype=torch.int32, device=_dev())
    have = torch.arange(width, device=_dev())[None] < _i32(n_blocks)[:, None]
    table[have] = perm[:total]
    return table, perm[total:].contiguous(), total + spare


def _cache(g, n_pages, nkv, hd):
    """A filled cache: e4m3 values of normal keys and values whose largest is near the type's, scales around 2^-6."""
    out = []
    for shape in ((n_pages, nkv, PAGE, hd), (n_pages, nkv, hd, PAGE)):
        pages = torch.empty(shape, dtype=torch.float8_e4m3fn, device=_dev())
        step = max(1, (1 << 26) // (nkv * PAGE * hd))
        for i in range(0, n_pages, step):
            x = torch.randn((min(step, n_pages - i),) + shape[1:], generator=g, device=_dev())
            pages[i:i + step] = (x * 90).clamp_(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
        e = torch.randint(-7, -5, (n_pages, nkv), generator=g, device=_dev())
        out += [pages, torch.exp2(e.float())]
    return out[0], out[2], out[1], out[3]


def _tree(g, q, rows, words):
    """Ancestor masks of one random tree for each request: row i sees itself and its parent's row's ancestors."""
    cu = _cum(q)
    cpu = torch.Generator().manual_seed(int(torch.randint(0, 1 << 30, (1,), generator=g, device=_dev())))
    mask = torch.zeros((rows, words * 32), dtype=torch.bool)
    for b, n in enumerate(q):
        u = torch.rand(n, generator=cpu).tolist()
        for i in range(n):
            r = cu[b] + i
            if i:
                mask[r] = mask[cu[b] + int(u[i] * i)]
            mask[r, i] = True
    w = (mask.view(rows, words, 32).long() << torch.arange(32)).sum(-1)
    return (w - ((w >> 31) << 32)).to(torch.int32).to(_dev())


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    s = dict(case)
    if op == "plan":
        ctx, add = _lens(case)
        blocks = [_pages(c) for c in ctx]
        most = max(1, max(_pages(max(c, c + a)) for c, a in zip(ctx, add)))
        new = sum(max(0, _pages(c + a) - _pages(c)) for c, a in zip(ctx, add))
        # a pool with room for every request, or (full) for about half of what they ask for
        spare = new // 2 if case["full"] else new + 64
        table, free, n_pages = _tables(g, blocks, spare)
        wide = torch.full((case["n"], most), -1, dtype=torch.int32, device=_dev())
        wide[:, :table.shape[1]] = table[:, :most]
        stack = torch.full((n_pages,), -1, dtype=torch.int32, device=_dev())
        stack[:spare] = free
        s.update(ctx_len=_i32(ctx), n_new=_i32(add), block_table=wide, free_list=stack, n_free=_i32([spare]),
                 max_rows=max(1, sum(a for a in add if a > 0)))
        return s
    dt = _dtype(case)
    if op == "rope":
        rows = case["rows"]
        # consecutive positions from a random start: a chunk of one sequence, or several requests' blocks
        start = torch.randint(0, max(1, case["far"] - rows), (-(-rows // 16),), generator=g, device=_dev())
        start = start[:1] if rows > 1024 else start
        pos = torch.arange(rows, device=_dev())
        pos = pos + start if rows > 1024 else start[pos // 16] + pos % 16
        s.update(q=torch.randn((rows, case["nq"], case["hd"]), generator=g, device=_dev()).to(dt),
                 k=torch.randn((rows, case["nkv"], case["hd"]), generator=g, device=_dev()).to(dt),
                 positions=pos.clamp_(max=case["far"] - 1).to(torch.int32))
        if own:     # the frequencies, set up once for a model
            from block_diffusion_speculative_inject_gb300 import Rope
            s["rope"] = Rope(case["hd"], rot_dim=case["rot"], theta=1e6, interleaved=case["inter"],
                             scaling=case["scaling"], factor=case["factor"], original_positions=32768)
        return s
    nkv, hd = case["nkv"], case["hd"]
    ctx, add = _lens(case)
    after = [c + a for c, a in zip(ctx, add)] if op == "append" else ctx
    table, _, n_pages = _tables(g, [_pages(c) for c in after], 8)
    kp, vp, ks, vs = _cache(g, n_pages, nkv, hd)
    s.update(k_pages=kp, v_pages=vp, k_scale=ks, v_scale=vs, block_table=table)
    if own:
        from block_diffusion_speculative_inject_gb300 import KV8Cache
        s["cache"] = KV8Cache(kp, vp, ks, vs)
    rows = sum(add)
    if op == "append":
        req = torch.repeat_interleave(torch.arange(case["n"], device=_dev()), _i32(add))
        pos = torch.arange(rows, device=_dev()) - _i32(_cum(add)[:-1]).long()[req] + _i32(ctx).long()[req]
        # keys have a few loud channels, and rows differ in size
        loud = torch.exp(0.7 * torch.randn((1, nkv, hd), generator=g, device=_dev()))
        size = torch.exp(0.3 * torch.randn((rows, 1, 1), generator=g, device=_dev()))
        s.update(slot_map=table[req, pos // PAGE].long() * PAGE + pos % PAGE,
                 k=(torch.randn((rows, nkv, hd), generator=g, device=_dev()) * loud * size).to(dt),
                 v=(torch.randn((rows, nkv, hd), generator=g, device=_dev()) * size).to(dt))
        return s
    s.update(q=(torch.randn((rows, case["nq"], hd), generator=g, device=_dev()) * 1.5).to(dt),
             cu_q=_i32(_cum(add)), ctx_len=_i32(ctx), tree_mask=None)
    if case["mask"] == "tree":
        s["tree_mask"] = _tree(g, add, rows, max(1, -(-max(add) // 32)))
    return s


# ---------------------------------------------------------------- one pass
def run(s):
    if own:
        return _run_own(s)
    return {"plan": _plain_plan, "rope": _plain_rope, "append": _plain_append, "attn": _plain_attn}[s["op"]](s)


def _run_own(s):
    import block_diffusion_speculative_inject_gb300 as pkg
    if s["op"] == "plan":
        p = pkg.page_plan(s["ctx_len"], s["n_new"], s["block_table"], s["free_list"], s["n_free"], s["max_rows"])
        return dict(p, block_table=s["block_table"])
    if s["op"] == "rope":
        q, k = pkg.rope(s["rope"], s["positions"], s["q"], s["k"], transpose=s["transpose"])
        return dict(q=q, k=k)
    if s["op"] == "append":
        pkg.kv8_append(s["cache"], s["k"], s["v"], s["slot_map"])
        return dict(k_pages=s["k_pages"], v_pages=s["v_pages"], k_scale=s["k_scale"], v_scale=s["v_scale"])
    out, lse = pkg.kv8_attention(s["cache"], s["q"], s["cu_q"], s["ctx_len"], s["block_table"], mask=s["mask"],
                                 tree_mask=s["tree_mask"], max_q=s["q_max"], want_lse=True)
    return dict(out=out, lse=lse)


def _plain_plan(s):
    ctx, add, table, stack = s["ctx_len"].long(), s["n_new"].long(), s["block_table"], s["free_list"]
    n, width = table.shape
    dev = table.device
    new = (ctx + add).clamp(min=0)
    old_p, new_p = (ctx + PAGE - 1) // PAGE, (new + PAGE - 1) // PAGE
    fits = new_p <= width
    gone = (old_p - new_p).clamp(min=0)
    need = torch.where(fits, (new_p - old_p).clamp(min=0), 0)
    rows = torch.where(fits, add.clamp(min=0), 0)
    n_free = s["n_free"].long()
    have = n_free + gone.sum()
    ok = fits & ((need == 0) | (need.cumsum(0) <= have)) & ((rows == 0) | (rows.cumsum(0) <= s["max_rows"]))
    need, rows = torch.where(ok, need, 0), torch.where(ok, rows, 0)
    new = torch.where(ok, new, ctx)
    # releases go on the stack in request order, from the first dropped page of each
    col = torch.arange(width, device=dev)[None]
    dropped = (col >= new_p[:, None]) & (col < old_p[:, None])
    back = (gone.cumsum(0) - gone)[:, None] + col - new_p[:, None] + n_free
    place = torch.where(dropped, back, stack.numel())
    stack = torch.cat([stack, stack.new_zeros(1)]).scatter(0, place.reshape(-1), table.reshape(-1))[:-1]
    s["free_list"].copy_(stack)
    # grants come off its top in request order
    given = (col >= old_p[:, None]) & (col < (old_p + need)[:, None])
    at = have - 1 - ((need.cumsum(0) - need)[:, None] + col - old_p[:, None])
    table.copy_(torch.where(given, stack[at.clamp(0, stack.numel() - 1)], table))
    cu = torch.cat([rows.new_zeros(1), rows.cumsum(0)])
    r = torch.arange(s["max_rows"], device=dev)
    live = r < cu[-1]
    req = torch.searchsorted(cu[1:], r, right=True).clamp(max=n - 1)
    pos = torch.where(live, ctx[req] + r - cu[req], 0)
    slot = torch.where(live, table[req, pos // PAGE].long() * PAGE + pos % PAGE, -1)
    return dict(new_len=new.int(), n_free=(have - need.sum()).int().reshape(1), cu_rows=cu.int(), slot_map=slot,
                positions=pos.int(), refused=(~ok).int(), block_table=table)


def _freq(case, dt, dev):
    """Angle per position of each rotated pair, and the factor of the rotated values."""
    rot = case["rot"]
    i = torch.arange(rot // 2, dtype=dt, device=dev)
    f = torch.exp(-2 * i / rot * math.log(1e6))
    if case["scaling"] == "none":
        return f, 1.0
    if case["scaling"] == "linear":
        return f / case["factor"], 1.0
    turn = lambda beta: rot * math.log(32768 / (beta * 2 * math.pi)) / (2 * math.log(1e6))  # noqa: E731
    low, high = max(math.floor(turn(32.0)), 0), min(math.ceil(turn(1.0)), rot - 1)
    ramp = ((i - low) / max(high - low, 0.001)).clamp(0, 1)
    return f / case["factor"] * ramp + f * (1 - ramp), 0.1 * math.log(case["factor"]) + 1


def _plain_rope(s):
    f, m = _freq(s, torch.float64, s["q"].device)      # far positions need 64-bit angles
    a = s["positions"].double()[:, None, None] * f
    cos, sin = (a.cos() * m).float(), (a.sin() * m).float()
    if s["transpose"]:
        sin = -sin
    out = {}
    h = s["rot"] // 2
    for name in ("q", "k"):
        x = s[name].float()
        part = x[..., :2 * h]
        u, v = (part[..., 0::2], part[..., 1::2]) if s["inter"] else (part[..., :h], part[..., h:])
        p, r = u * cos - v * sin, v * cos + u * sin
        both = torch.stack([p, r], -1).flatten(-2) if s["inter"] else torch.cat([p, r], -1)
        out[name] = torch.cat([both, x[..., 2 * h:]], -1).to(s[name].dtype)
    return out


def _plain_append(s):
    slot = s["slot_map"]
    slot = slot[slot >= 0]
    page, off = slot // PAGE, slot % PAGE
    n_pages = s["k_pages"].shape[0]
    dev = slot.device
    owned = torch.zeros((n_pages, PAGE), dtype=torch.bool, device=dev)
    owned[page, off] = True
    touched = owned.any(1)
    fresh = owned[:, 0]
    at = torch.arange(PAGE, device=dev)
    last = torch.where(owned, at, -1).amax(1)
    kept = ~owned & (at < last[:, None]) & ~fresh[:, None]
    for x, pages, scale, turned in ((s["k"], s["k_pages"], s["k_scale"], False), (s["v"], s["v_pages"], s["v_scale"], True)):
        x = x[s["slot_map"] >= 0].float()
        big = torch.where(x.isfinite(), x.abs(), 0).amax(-1)
        amax = torch.zeros_like(scale).scatter_reduce_(0, page[:, None].expand_as(big), big, "amax")
        m, e = torch.frexp(amax)                      # amax = m 2^e, 448 = 0.875 2^9
        e = torch.where(amax > 0, e - 9 + (m > 0.875), MIN_EXP).clamp(min=MIN_EXP)
        new = torch.ldexp(torch.ones_like(scale), e)
        new = torch.where(fresh[:, None], new, torch.maximum(new, scale))
        new = torch.where(touched[:, None], new, scale)
        old = pages.transpose(2, 3) if turned else pages          # [pages, heads, 64, hd]
        again = (old.float() * (scale / new)[..., None, None]).to(torch.float8_e4m3fn)
        raw = torch.where((kept & touched[:, None])[:, None, :, None], again.view(torch.uint8), old.view(torch.uint8))
        y = (x / new[page][..., None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
        raw[page, :, off] = y.view(torch.uint8)
        pages.view(torch.uint8).copy_(raw.transpose(2, 3) if turned else raw)
        scale.copy_(new)
    return dict(k_pages=s["k_pages"], v_pages=s["v_pages"], k_scale=s["k_scale"], v_scale=s["v_scale"])


def _seen(s, width):
    """[requests, most rows, width] visibility, and [requests, most rows] the rows' places."""
    cu, ctx = s["cu_q"].long(), s["ctx_len"].long()
    dev = cu.device
    n_q = cu[1:] - cu[:-1]
    t = torch.arange(max(1, s["q_max"]), device=dev)
    p = torch.arange(width, device=dev)
    row = (cu[:-1, None] + t).clamp(max=max(0, s["q"].shape[0] - 1))
    see = (p < ctx[:, None])[:, None, :].expand(-1, t.numel(), -1)
    if s["mask"] == "causal":
        see = see & (p <= (ctx - n_q)[:, None, None] + t[:, None])
    if s["mask"] == "tree":
        j = p - (ctx - n_q)[:, None]                               # index among the request's rows
        words = s["tree_mask"][row]                                # [n, t, words]
        at = j.clamp(0, 32 * words.shape[-1] - 1)[:, None, :].expand(-1, t.numel(), -1)
        bit = (words.long().gather(2, at // 32) >> (at % 32)) & 1
        see = see & ((j < 0)[:, None] | (bit == 1))
    return see, row, t[None] < n_q[:, None]


def _plain_attn(s):
    table = s["block_table"].long().clamp(min=0)
    n, width = table.shape[0], table.shape[1] * PAGE
    nq, nkv, hd = s["nq"], s["nkv"], s["hd"]
    k = s["k_pages"].view(torch.uint8)[table].view(torch.float8_e4m3fn).float() * s["k_scale"][table][..., None, None]
    k = k.transpose(1, 2).reshape(n, nkv, width, hd)
    v = s["v_pages"].view(torch.uint8)[table].view(torch.float8_e4m3fn).float() * s["v_scale"][table][..., None, None]
    v = v.permute(0, 2, 1, 4, 3).reshape(n, nkv, width, hd)
    see, row, live = _seen(s, width)
    v = torch.where(see.any(1)[:, None, :, None], v, 0)
    q = s["q"][row].float().view(n, -1, nkv, nq // nkv, hd).permute(0, 2, 3, 1, 4)      # [n, nkv, group, rows, hd]
    x = torch.matmul(q.flatten(2, 3), k.transpose(2, 3)).unflatten(2, (nq // nkv, -1)) / math.sqrt(hd)
    x = torch.where(see[:, None, None], x, -math.inf)
    top = x.amax(-1, keepdim=True)
    base = torch.where(top == -math.inf, 0, top)
    p = torch.exp(x - base)
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p.flatten(2, 3), v).unflatten(2, (nq // nkv, -1)) / torch.where(total == 0, 1, total)
    o, lse = o.permute(0, 3, 1, 2, 4).flatten(2, 3), (base + total.log())[..., 0].permute(0, 3, 1, 2).flatten(2, 3)
    return dict(out=o[live].to(s["q"].dtype), lse=lse[live])


# ---------------------------------------------------------------- the definitions in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    return {"plan": _exact_plan, "rope": _exact_rope, "append": _exact_append, "attn": _exact_attn}[case["op"]](s)


def _exact_plan(s):
    ctx, add = s["ctx_len"].tolist(), s["n_new"].tolist()
    table, stack = s["block_table"].tolist(), s["free_list"].tolist()[:int(s["n_free"])]
    width = len(table[0])
    for b, (c, a) in enumerate(zip(ctx, add)):
        stack += [table[b][i] for i in range(_pages(max(0, c + a)), _pages(c))]
    have, asked, asked_rows, rows = len(stack), 0, 0, 0
    new, cu, slot, pos, refused = [], [0], [], [], []
    for b, (c, a) in enumerate(zip(ctx, add)):
        to = max(0, c + a)
        bad = _pages(to) > width
        need = 0 if bad else max(0, _pages(to) - _pages(c))
        take = 0 if bad else max(0, a)
        asked, asked_rows = asked + need, asked_rows + take
        bad = bad or (need and asked > have) or (take and asked_rows > s["max_rows"])
        refused.append(int(bool(bad)))
        if bad:
            new.append(c)
        else:
            new.append(to)
            for i in range(_pages(c), _pages(c) + need):
                table[b][i] = stack.pop()
            for p in range(c, c + take):
                slot.append(table[b][p // PAGE] * PAGE + p % PAGE)
                pos.append(p)
            rows += take
        cu.append(rows)
    tail = s["max_rows"] - rows
    return dict(new_len=_i32(new), n_free=_i32([len(stack)]), cu_rows=_i32(cu),
                slot_map=torch.tensor(slot + [-1] * tail, dtype=torch.int64), positions=_i32(pos + [0] * tail),
                refused=_i32(refused), block_table=_i32(table))


def _exact_rope(s):
    rot, sign = s["rot"], -1.0 if s["transpose"] else 1.0
    f, m = _freq(s, torch.float64, "cpu")
    f = f.to(s["q"].device)
    turn = torch.polar(torch.full_like(f, m).expand(s["rows"], -1), sign * s["positions"].double()[:, None] * f)
    out = {}
    for name in ("q", "k"):
        x = s[name].double()
        y = x.clone()
        for i in range(rot // 2):
            a, b = (2 * i, 2 * i + 1) if s["inter"] else (i, i + rot // 2)
            z = torch.complex(x[..., a], x[..., b]) * turn[:, i, None]
            y[..., a], y[..., b] = z.real, z.imag
        out[name] = y
    return out


def _exact_append(s):
    # the stored bytes are a rounding to 8 bits that has no finer value; the scales are exact powers of two
    out = dict(k_pages=None, v_pages=None)
    rows = {}
    for r, slot in enumerate(s["slot_map"].tolist()):
        if slot >= 0:
            rows.setdefault(slot // PAGE, []).append((slot % PAGE, r))
    for name in ("k", "v"):
        scale = s[name + "_scale"].double()
        for page, at in rows.items():
            for h in range(s["nkv"]):
                big = float(s[name][at[0][1]:at[-1][1] + 1, h].double().abs().max())
                e = MIN_EXP
                while 448.0 * 2.0 ** e < big:
                    e += 1
                scale[page, h] = 2.0 ** e if at[0][0] == 0 else max(2.0 ** e, float(scale[page, h]))
        out[name + "_scale"] = scale
    return out


def _exact_attn(s):
    nq, nkv, hd = s["nq"], s["nkv"], s["hd"]
    cu, ctx = s["cu_q"].tolist(), s["ctx_len"].tolist()
    out = torch.zeros((cu[-1], nq, hd), dtype=torch.float64, device=s["q"].device)
    lse = torch.full((cu[-1], nq), -math.inf, dtype=torch.float64, device=s["q"].device)
    for b, length in enumerate(ctx):
        n = cu[b + 1] - cu[b]
        if not n or not length:
            continue
        ids = s["block_table"][b, :_pages(length)].long()
        see = torch.ones((n, length), dtype=torch.bool, device=ids.device)
        if s["mask"] == "causal":
            see = see.tril(length - n)
        elif s["mask"] == "tree":
            word = s["tree_mask"][cu[b]:cu[b + 1]].long()
            see[:, length - n:] = ((word[:, torch.arange(n) // 32] >> (torch.arange(n) % 32).to(ids.device)) & 1) == 1
        for h in range(nkv):
            k = s["k_pages"].view(torch.uint8)[ids, h].view(torch.float8_e4m3fn).double()
            k = (k * s["k_scale"][ids, h].double()[:, None, None]).reshape(-1, hd)[:length]
            v = s["v_pages"].view(torch.uint8)[ids, h].view(torch.float8_e4m3fn).double()
            v = (v * s["v_scale"][ids, h].double()[:, None, None]).transpose(1, 2).reshape(-1, hd)[:length]
            for i in range(h * nq // nkv, (h + 1) * nq // nkv):
                x = s["q"][cu[b]:cu[b + 1], i].double() @ k.T / math.sqrt(hd)
                x = x.masked_fill(~see, -math.inf)
                z = torch.logsumexp(x, 1)
                lse[cu[b]:cu[b + 1], i] = z
                out[cu[b]:cu[b + 1], i] = torch.exp(x - z.masked_fill(z == -math.inf, 0)[:, None]) @ v
    return dict(out=out, lse=lse)
