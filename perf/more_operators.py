"""A verify round over long contexts on the 8-bit paged cache as measured workloads: per-head norms with rotary
positions (and their gradient), key bounds of pages, the choice of pages by a cheap score, attention over the
chosen pages, and the move of an accepted path to its place.

`run` computes them in elementary torch operations, or, with `own` set, through the package's calls on the
same inputs. `exact` is their definition in 64 bits. Lengths follow from the case alone, values from the seed.

Cache layout (the package's): K pages [n_pages, kv heads, 64, head dim], V pages [n_pages, kv heads, head dim, 64]
in e4m3, one power-of-two scale per page and kv head for each of K and V. Key bounds: int8 [n_pages, kv heads, 2,
head dim], the least and the largest key of each dim, rounded outwards to multiples of 4 scale.
"""
import math
import random

import torch

own = False

PAGE = 64
E4M3_MAX = 448.0
MIN_EXP = -64
EPS = 1e-6


def listed():
    return [
        # one request's verify block of 16 rows: the smallest call, latency only
        dict(name="norm_block_b1", op="norm", rows=16, nq=32, nkv=8, hd=128, rot=128, inter=False, scaling="none",
             factor=1.0, far=2048, dtype="bf16", grad=False),
        # a long prompt's queries and keys with positions scaled for a context of 131072
        dict(name="norm_prompt_yarn", op="norm", rows=32768, nq=40, nkv=8, hd=128, rot=128, inter=False, scaling="yarn",
             factor=4.0, far=131072, dtype="bf16", grad=False),
        # the gradient of a training batch of 16384 positions
        dict(name="norm_grad", op="norm", rows=16384, nq=32, nkv=8, hd=128, rot=128, inter=False, scaling="none",
             factor=1.0, far=4096, dtype="bf16", grad=True),
        # the gradient in fp32 of small heads of which half is rotated, interleaved, an odd number of rows
        dict(name="norm_grad_partial_f32", op="norm", rows=5003, nq=12, nkv=4, hd=64, rot=32, inter=True,
             scaling="linear", factor=8.0, far=60000, dtype="f32", grad=True),
        # key bounds after the verify blocks of 8 requests were appended
        dict(name="bounds_block_b8", op="bounds", n=8, ctx_min=100, ctx_max=2000, add_min=16, add_max=16, nkv=8, hd=128),
        # key bounds of 8 whole prompts
        dict(name="bounds_prompt_b8", op="bounds", n=8, ctx_min=0, ctx_max=0, add_min=16384, add_max=32768, nkv=8, hd=128),
        # 16 of a single request's pages for its single token: latency
        dict(name="select_token_b1", op="select", n=1, ctx_min=8191, ctx_max=8191, q_min=1, q_max=1, nq=32, nkv=8, hd=128,
             n_select=16, first=1, last=1, dtype="bf16"),
        # 128 of up to 2049 pages for the verify blocks of 8 requests
        dict(name="select_block_b8", op="select", n=8, ctx_min=65536, ctx_max=131072, q_min=16, q_max=16, nq=40, nkv=8,
             hd=128, n_select=128, first=1, last=2, dtype="bf16"),
        # a decoding batch over 64 of 513 pages of each request
        dict(name="sparse_token_b16", op="sparse", n=16, ctx_min=32768, ctx_max=32768, q_min=1, q_max=1, nq=32, nkv=8,
             hd=128, n_select=64, mask="causal", dtype="bf16"),
        # verify blocks of 16 rows over 96 of about 500 pages
        dict(name="sparse_block_b8", op="sparse", n=8, ctx_min=16384, ctx_max=32768, q_min=16, q_max=16, nq=40, nkv=8,
             hd=128, n_select=96, mask="causal", dtype="bf16"),
        # one request's accepted path of 8 rows out of a tree of 65, one layer: latency
        dict(name="compact_path_b1", op="compact", layers=1, n=1, ctx_min=2048, ctx_max=2048, tree=65, keep_min=8,
             keep_max=8, nkv=8, hd=128),
        # 8 requests' paths out of trees of 256 rows in all of a target's 32 layers
        dict(name="compact_tree_b8", op="compact", layers=32, n=8, ctx_min=100, ctx_max=400, tree=256, keep_min=1,
             keep_max=16, nkv=8, hd=128),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "norm", "bounds", "select", "select", "sparse", "sparse", "compact"])
    hd = rng.choice([64, 128])
    nkv = rng.choice([1, 2, 4, 8])
    group = rng.choice([1, 2, 4, 5, 7, 8])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op == "norm":
        grad = rng.random() < 0.5
        cost = (16384 * 40 if grad else 32768 * 48) * 128 * 2
        per = (nkv * group + nkv) * hd * (2 if dtype == "bf16" else 4)
        return dict(op=op, rows=_log(rng, 1, min(65536, cost // per)), nq=nkv * group, nkv=nkv, hd=hd,
                    rot=rng.choice([hd, hd, hd // 2, hd // 4, 20]), inter=rng.random() < 0.5,
                    scaling=rng.choice(["none", "linear", "yarn"]), factor=rng.choice([2.0, 4.0, 8.0, 2.5]),
                    far=_log(rng, 100, 1000000), dtype=dtype, grad=grad)
    if op == "bounds":
        n = _log(rng, 1, 128)
        if rng.random() < 0.5:
            a = rng.choice([1, 2, 8, 16, 33])
            return dict(op=op, n=n, ctx_min=0, ctx_max=_log(rng, 1, 4000), add_min=rng.choice([0, a]), add_max=a,
                        nkv=nkv, hd=hd)
        a = _log(rng, 64, max(65, min(65536, 190000 // n)))
        return dict(op=op, n=n, ctx_min=0, ctx_max=rng.choice([0, 200]), add_min=a // 2, add_max=a, nkv=nkv, hd=hd)
    if op == "select":
        n = _log(rng, 1, 64)
        q = rng.choice([1, 1, 2, 8, 16, 33, 100])
        first, last = rng.choice([0, 1, 2]), rng.choice([0, 1, 3])
        least = first + last + q // PAGE + 2        # blocks that are kept in any case
        top = min(131072, 1000000 * 80 // max(16, n * q * group) // (nkv * hd // 64) * 8)
        ctx = _log(rng, 64 * (least + 4), max(64 * (least + 8), top))
        return dict(op=op, n=n, ctx_min=rng.choice([ctx, ctx // 2, ctx // 8]), ctx_max=ctx, q_min=rng.choice([1, q]), q_max=q,
                    nq=nkv * group, nkv=nkv, hd=hd, n_select=_log(rng, least, min(512, ctx // 64 - 2)), first=first,
                    last=last, dtype=dtype)
    if op == "sparse":
        q = rng.choice([1, 1, 2, 8, 16, 32, _log(rng, 33, 300)])
        n = _log(rng, 1, 64 if q <= 32 else 8)
        most = 1.2e8 if dtype == "bf16" and q <= 32 else 4e9 / (group * q) / 64     # bytes of K and V that the case may read
        n_select = _log(rng, q // PAGE + 2, max(q // PAGE + 3, min(256, int(most / (n * nkv * hd * 128)))))
        ctx = _log(rng, 16, max(65, min(65536, int(1.2e9 / (n * nkv * hd * 2)))))
        return dict(op=op, n=n, ctx_min=rng.choice([ctx, ctx // 2, ctx // 8]), ctx_max=ctx,
                    q_min=rng.choice([0, 1, q]) if n > 1 else q, q_max=q, nq=nkv * group, nkv=nkv, hd=hd,
                    n_select=n_select, mask=rng.choice(["none", "causal", "causal", "tree"]), dtype=dtype)
    n, tree = _log(rng, 1, 16), rng.choice([8, 16, 33, 65, 129, 257])
    top = min(tree, rng.choice([1, 5, 16, 32]))
    return dict(op=op, layers=rng.choice([1, 2, 5, 16]), n=n, ctx_min=rng.choice([0, 60, 100]), ctx_max=_log(rng, 101, 1000),
                tree=tree, keep_min=rng.choice([0, 1, top]), keep_max=top, nkv=nkv, hd=hd)


# ---------------------------------------------------------------- sizes that follow from the case
def _ints(case, what, lo, hi):
    """n integers of [lo, hi] (the ends among them where n > 1), the same for every seed."""
    r = random.Random("%s/%d/%d/%d" % (what, case["n"], lo, hi))
    v = [r.randint(lo, hi) for _ in range(case["n"])]
    if case["n"] > 1:
        v[0], v[-1] = hi, lo
    return v


def _lens(case):
    """(context lengths before, rows added) of a bounds case, (whole context, query rows) of the choice and the attention,
    (context before the tree, rows kept) of a move."""
    ctx = _ints(case, "ctx", case["ctx_min"], case["ctx_max"])
    if case["op"] == "bounds":
        return ctx, _ints(case, "add", case["add_min"], case["add_max"])
    if case["op"] == "compact":
        return ctx, _ints(case, "keep", case["keep_min"], case["keep_max"])
    q = _ints(case, "q", case["q_min"], case["q_max"])
    return [c + x for c, x in zip(ctx, q)], q


def _pages(n):
    return -(-n // PAGE)


def work(case):
    op = case["op"]
    size = 2 if case.get("dtype") == "bf16" else 4
    if op == "norm":
        e = case["rows"] * (case["nq"] + case["nkv"])
        if case["grad"]:
            return {"bytes": 3 * e * case["hd"] * size + 4 * case["rows"] + 2 * case["hd"] * (size + 4),
                    "flops": 9 * e * case["hd"] + 3 * e * case["rot"]}
        return {"bytes": 2 * e * case["hd"] * size + 4 * case["rows"] + 2 * case["hd"] * size,
                "flops": 4 * e * case["hd"] + 3 * e * case["rot"]}
    nkv, hd = case["nkv"], case["hd"]
    if op == "bounds":
        ctx, add = _lens(case)
        rows = sum(c + a - c // PAGE * PAGE for c, a in zip(ctx, add) if a)
        pages = sum(_pages(c + a) - c // PAGE for c, a in zip(ctx, add) if a)
        return {"bytes": rows * nkv * hd + pages * (2 * nkv * hd + 4) + 8 * case["n"], "flops": 2 * rows * nkv * hd}
    if op == "compact":
        _, keep = _lens(case)
        return {"bytes": case["layers"] * sum(keep) * nkv * hd * 4 + 4 * sum(keep), "flops": 0}
    ctx, q = _lens(case)
    if op == "select":
        pages = sum(_pages(c) for c, x in zip(ctx, q) if x)
        return {"bytes": pages * (nkv * (2 * hd + 4) + 4) + sum(q) * case["nq"] * hd * size + 4 * case["n"] * nkv * case["n_select"],
                "flops": 2 * hd * case["nq"] * sum(x * _pages(c) for c, x in zip(ctx, q))}
    have = [min(c, case["n_select"] * PAGE) for c in ctx]
    seen = sum(x * c - (x * (x - 1) // 2 if case["mask"] != "none" else 0) for c, x in zip(have, q))
    return {"bytes": sum(c for c, x in zip(have, q) if x) * nkv * hd * 2 + sum(q) * case["nq"] * (2 * hd * size + 4)
            + 4 * case["n"] * nkv * case["n_select"], "flops": 4 * seen * case["nq"] * hd}


# ---------------------------------------------------------------- inputs
def _dev():
    return "cuda" if torch.cuda.is_available() else "cpu"


def _gen(seed):
    return torch.Generator(device=_dev()).manual_seed(int(seed) * 1000003 + 29)


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
    return table, total + spare


def _pool(g, shape):
    """e4m3 values of normal keys or values whose largest is near the type's."""
    pages = torch.empty(shape, dtype=torch.float8_e4m3fn, device=_dev())
    step = max(1, (1 << 26) // (shape[1] * shape[2] * shape[3]))
    for i in range(0, shape[0], step):
        x = torch.randn((min(step, shape[0] - i),) + shape[1:], generator=g, device=_dev())
        pages[i:i + step] = (x * 90).clamp_(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
    return pages


def _scale(g, n_pages, nkv):
    return torch.exp2(torch.randint(-7, -5, (n_pages, nkv), generator=g, device=_dev()).float())


def _cache(g, n_pages, nkv, hd):
    return (_pool(g, (n_pages, nkv, PAGE, hd)), _pool(g, (n_pages, nkv, hd, PAGE)), _scale(g, n_pages, nkv),
            _scale(g, n_pages, nkv))


def _bounds(g, n_pages, nkv, hd):
    """Bounds of pages whose keys lie around a middle of their own in every dim."""
    mid = torch.randn((n_pages, nkv, hd), generator=g, device=_dev()) * 12 + torch.randn((1, nkv, hd), generator=g, device=_dev()) * 10
    half = torch.rand((n_pages, nkv, hd), generator=g, device=_dev()) * 30 + 10
    return torch.stack([(mid - half).floor(), (mid + half).ceil()], 2).clamp(-112, 112).to(torch.int8)


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


def _chosen(g, ctx, q, nkv, n_select):
    """Rising block lists [n, nkv, n_select]: the first block, those of the request's own rows, and others at random."""
    n, top = len(ctx), max(1, max(_pages(c) for c in ctx))
    u = torch.rand((n, nkv, max(top, n_select)), generator=g, device=_dev())
    j = torch.arange(u.shape[-1], device=_dev())
    blocks = _i32([_pages(c) for c in ctx])[:, None, None]
    mine = _i32([(c - x) // PAGE for c, x in zip(ctx, q)])[:, None, None]
    u = torch.where((j == 0) | (j >= mine), u + 2, u)
    u = torch.where(j < blocks, u, -1.0)
    val, at = u.topk(n_select, dim=-1)
    at = torch.where(val >= 0, at, 1 << 30).sort(-1).values
    return torch.where(at < 1 << 30, at, -1).to(torch.int32).contiguous()


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    s = dict(case)
    if op == "norm":
        rows, dt = case["rows"], _dtype(case)
        # consecutive positions from a random start: a chunk of one sequence, or several requests' blocks
        start = torch.randint(0, max(1, case["far"] - rows), (-(-rows // 16),), generator=g, device=_dev())
        start = start[:1] if rows > 1024 else start
        pos = torch.arange(rows, device=_dev())
        pos = pos + start if rows > 1024 else start[pos // 16] + pos % 16
        s["positions"] = pos.clamp_(max=case["far"] - 1).to(torch.int32)
        for x, heads in (("q", case["nq"]), ("k", case["nkv"])):
            # rows differ in size, as a projection's outputs do
            size = torch.exp(0.5 * torch.randn((rows, heads, 1), generator=g, device=_dev()))
            s[x] = (torch.randn((rows, heads, case["hd"]), generator=g, device=_dev()) * size).to(dt)
            s[x + "_weight"] = (1 + 0.3 * torch.randn((case["hd"],), generator=g, device=_dev())).to(dt)
            if case["grad"]:
                s["d" + x] = torch.randn((rows, heads, case["hd"]), generator=g, device=_dev()).to(dt)
        if own:     # the frequencies, set up once for a model
            from block_diffusion_speculative_inject_gb300 import Rope
            s["rope"] = Rope(case["hd"], rot_dim=case["rot"], theta=1e6, interleaved=case["inter"],
                             scaling=case["scaling"], factor=case["factor"], original_positions=32768)
        return s
    nkv, hd = case["nkv"], case["hd"]
    ctx, more = _lens(case)
    after = [c + a for c, a in zip(ctx, more)] if op == "bounds" else [c + case["tree"] for c in ctx] if op == "compact" else ctx
    table, n_pages = _tables(g, [_pages(c) for c in after], 8)
    s["block_table"] = table
    if op == "compact":     # the layers' pools are one tensor each
        layers = case["layers"]
        kp, vp, ks, vs = _cache(g, layers * n_pages, nkv, hd)
        pools = [x.unflatten(0, (layers, n_pages)) for x in (kp, vp, ks, vs)]
        width = max(1, case["keep_max"])
        cpu = random.Random(int(torch.randint(0, 1 << 30, (1,), generator=g, device=_dev())))
        paths = [sorted([0] + cpu.sample(range(1, case["tree"]), k - 1)) if k else [] for k in more]
        s.update(k_pages=pools[0], v_pages=pools[1], k_scale=pools[2], v_scale=pools[3], base_len=_i32(ctx),
                 n_keep=_i32(more), keep=_i32([p + [-1] * (width - len(p)) for p in paths]))
        if own:
            from block_diffusion_speculative_inject_gb300 import KV8Cache, KV8Layers
            s["layer_caches"] = KV8Layers(KV8Cache(*(x[i] for x in pools)) for i in range(layers))
        return s
    if op == "select":      # the pages themselves are not read
        kp = torch.empty((n_pages, nkv, PAGE, hd), dtype=torch.float8_e4m3fn, device=_dev())
        vp = torch.empty((n_pages, nkv, hd, PAGE), dtype=torch.float8_e4m3fn, device=_dev())
        ks, vs = _scale(g, n_pages, nkv), _scale(g, n_pages, nkv)
    else:
        kp, vp, ks, vs = _cache(g, n_pages, nkv, hd)
    s.update(k_pages=kp, v_pages=vp, k_scale=ks, v_scale=vs)
    if own:
        from block_diffusion_speculative_inject_gb300 import KV8Cache
        s["cache"] = KV8Cache(kp, vp, ks, vs)
    if op != "sparse":
        s["bounds"] = _bounds(g, n_pages, nkv, hd)
    if op == "bounds":
        s.update(old_len=_i32(ctx), new_len=_i32(after))
        return s
    rows, dt = sum(more), _dtype(case)
    s.update(q=(torch.randn((rows, case["nq"], hd), generator=g, device=_dev()) * 1.5).to(dt), cu_q=_i32(_cum(more)),
             ctx_len=_i32(ctx))
    if op == "sparse":
        s.update(blocks=_chosen(g, ctx, more, nkv, case["n_select"]), tree_mask=None)
        if case["mask"] == "tree":
            s["tree_mask"] = _tree(g, more, rows, max(1, -(-max(more) // 32)))
    return s


# ---------------------------------------------------------------- one pass
def run(s):
    if own:
        return _run_own(s)
    return {"norm": _plain_norm, "bounds": _plain_bounds, "select": _plain_select, "sparse": _plain_sparse,
            "compact": _plain_compact}[s["op"]](s)


def _run_own(s):
    import block_diffusion_speculative_inject_gb300 as pkg
    if s["op"] == "norm" and s["grad"]:
        dq, dk, dqw, dkw = pkg.qk_norm_rope_backward(s["rope"], s["positions"], s["q"], s["k"], s["q_weight"], s["k_weight"],
                                                     s["dq"], s["dk"], eps=EPS)
        return dict(dq=dq, dk=dk, dq_weight=dqw, dk_weight=dkw)
    if s["op"] == "norm":
        q, k = pkg.qk_norm_rope(s["rope"], s["positions"], s["q"], s["k"], s["q_weight"], s["k_weight"], eps=EPS)
        return dict(q=q, k=k)
    if s["op"] == "bounds":
        pkg.kv8_bounds(s["cache"], s["bounds"], s["block_table"], s["old_len"], s["new_len"])
        return dict(bounds=s["bounds"])
    if s["op"] == "select":
        return dict(blocks=pkg.kv8_select(s["cache"], s["bounds"], s["q"], s["cu_q"], s["ctx_len"], s["block_table"],
                                          s["n_select"], keep_first=s["first"], keep_last=s["last"]))
    if s["op"] == "sparse":
        out, lse = pkg.kv8_attention(s["cache"], s["q"], s["cu_q"], s["ctx_len"], s["block_table"], mask=s["mask"],
                                     tree_mask=s["tree_mask"], max_q=s["q_max"], blocks=s["blocks"], want_lse=True)
        return dict(out=out, lse=lse)
    pkg.kv8_compact(s["layer_caches"], s["block_table"], s["base_len"], s["keep"], s["n_keep"])
    return {x: s[x] for x in ("k_pages", "v_pages", "k_scale", "v_scale")}


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


def _turn(s, x, cos, sin):
    h = s["rot"] // 2
    part = x[..., :2 * h]
    u, v = (part[..., 0::2], part[..., 1::2]) if s["inter"] else (part[..., :h], part[..., h:])
    p, r = u * cos - v * sin, v * cos + u * sin
    both = torch.stack([p, r], -1).flatten(-2) if s["inter"] else torch.cat([p, r], -1)
    return torch.cat([both, x[..., 2 * h:]], -1)


def _plain_norm(s):
    f, m = _freq(s, torch.float64, s["q"].device)      # far positions need 64-bit angles
    a = s["positions"].double()[:, None, None] * f
    cos, sin = (a.cos() * m).float(), (a.sin() * m).float()
    out = {}
    for name in ("q", "k"):
        x, w = s[name].float(), s[name + "_weight"].float()
        r = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
        if not s["grad"]:
            out[name] = _turn(s, x * r * w, cos, sin).to(s[name].dtype)
            continue
        dn = _turn(s, s["d" + name].float(), cos, -sin)
        y = x * r
        grad = dn * w
        out["d" + name] = (r * (grad - y * (grad * y).mean(-1, keepdim=True))).to(s[name].dtype)
        out["d" + name + "_weight"] = (dn * y).sum((0, 1))
    return out


def _plain_bounds(s):
    old, new, table = s["old_len"].long(), s["new_len"].long(), s["block_table"]
    col = torch.arange(table.shape[1], device=table.device)
    touched = (col >= old[:, None] // PAGE) & (col < (new[:, None] + PAGE - 1) // PAGE) & (new > old)[:, None]
    req, blk = touched.nonzero(as_tuple=True)
    page = table[req, blk].long()
    x = s["k_pages"].view(torch.uint8)[page].view(torch.float8_e4m3fn).float() / 4
    there = (blk[:, None] * PAGE + torch.arange(PAGE, device=table.device) < new[req, None])[:, None, :, None]
    lo = torch.where(there, x, math.inf).amin(2).floor()
    hi = torch.where(there, x, -math.inf).amax(2).ceil()
    s["bounds"][page] = torch.stack([lo, hi], 2).to(torch.int8)
    return dict(bounds=s["bounds"])


def _rounded(q):
    """Each row as integers of at most 1024 and the power of two that they count."""
    top = q.abs().amax(-1, keepdim=True)
    e = torch.where(top > 0, torch.frexp(top).exponent, -100).clamp(min=-100) - 10
    return torch.ldexp(q, -e).round(), torch.ldexp(torch.ones_like(top), e)


def _plain_select(s):
    n, width = s["block_table"].shape
    nkv, group, k = s["nkv"], s["nq"] // s["nkv"], s["n_select"]
    cu, ctx = s["cu_q"].long(), s["ctx_len"].long()
    dev = ctx.device
    rows = cu[1:] - cu[:-1]
    page = s["block_table"].long().clamp(min=0)
    x, unit = _rounded(s["q"].float())
    t = torch.arange(s["q_max"], device=dev)
    at = (cu[:-1, None] + t).clamp(max=s["q"].shape[0] - 1)
    live = t < rows[:, None]
    x = x[at].view(n, -1, nkv, group, s["hd"]).permute(0, 2, 1, 3, 4).flatten(2, 3)          # [n, nkv, rows group, hd]
    unit = unit[at].view(n, -1, nkv, group).permute(0, 2, 1, 3).flatten(2, 3)
    live = live[:, None, :, None].expand(-1, nkv, -1, group).flatten(2, 3)
    score = torch.empty((n, nkv, width), device=dev)
    for b in range(0, width, 512):      # (whole numbers below 2^24: exact in 32 bits)
        both = s["bounds"][page[:, b:b + 512]].float()                                         # [n, blocks, nkv, 2, hd]
        lo, hi = both[..., 0, :].permute(0, 2, 3, 1), both[..., 1, :].permute(0, 2, 3, 1)
        y = torch.matmul(x.clamp(min=0), hi) + torch.matmul(x.clamp(max=0), lo)
        y = torch.where(live[..., None], y * unit[..., None], -math.inf).amax(2)
        score[..., b:b + 512] = y * (4 * s["k_scale"][page[:, b:b + 512]]).transpose(1, 2)
    j = torch.arange(width, device=dev)
    blocks = (ctx + PAGE - 1) // PAGE
    kept = (j < s["first"]) | (j >= ((ctx - rows) // PAGE - s["last"])[:, None])
    score = torch.where(kept[:, None], math.inf, score)
    score = torch.where((j < blocks[:, None])[:, None], score, -math.inf)
    order = score.sort(dim=-1, descending=True, stable=True).indices
    order = torch.cat([order, order.new_zeros((n, nkv, max(0, k - width)))], -1)[..., :k]
    taken = torch.arange(k, device=dev) < blocks[:, None, None]
    order = torch.where(taken, order, 1 << 30).sort(-1).values
    return dict(blocks=torch.where(order < 1 << 30, order, -1).int())


def _plain_sparse(s):
    nq, nkv, hd, n = s["nq"], s["nkv"], s["hd"], s["n"]
    cu, ctx, blk = s["cu_q"].long(), s["ctx_len"].long(), s["blocks"].long()
    dev = ctx.device
    rows = cu[1:] - cu[:-1]
    listed_ = blk >= 0
    blk = blk.clamp(min=0)
    page = s["block_table"].long()[torch.arange(n, device=dev)[:, None, None], blk].clamp(min=0)
    h = torch.arange(nkv, device=dev)[None, :, None]
    k = s["k_pages"].view(torch.uint8)[page, h].view(torch.float8_e4m3fn).float() * s["k_scale"][page, h][..., None, None]
    k = k.flatten(2, 3)                                                             # [n, nkv, tokens, hd]
    v = s["v_pages"].view(torch.uint8)[page, h].view(torch.float8_e4m3fn).float() * s["v_scale"][page, h][..., None, None]
    v = v.transpose(3, 4).flatten(2, 3)
    p = (blk[..., None] * PAGE + torch.arange(PAGE, device=dev)).flatten(2)          # positions [n, nkv, tokens]
    t = torch.arange(max(1, s["q_max"]), device=dev)
    row = (cu[:-1, None] + t).clamp(max=max(0, s["q"].shape[0] - 1))
    see = (listed_.repeat_interleave(PAGE, 2) & (p < ctx[:, None, None]))[:, :, None].expand(-1, -1, t.numel(), -1)
    first = (ctx - rows)[:, None, None, None]
    if s["mask"] == "causal":
        see = see & (p[:, :, None] <= first + t[:, None])
    if s["mask"] == "tree":
        j = p[:, :, None] - first                                                   # index among the request's rows
        words = s["tree_mask"][row].long()[:, None].expand(-1, nkv, -1, -1)
        at = j.clamp(0, 32 * words.shape[-1] - 1).expand(-1, -1, t.numel(), -1)
        see = see & ((j < 0) | ((words.gather(3, at // 32) >> (at % 32)) & 1 == 1))
    q = s["q"][row].float().view(n, -1, nkv, nq // nkv, hd).permute(0, 2, 3, 1, 4)      # [n, nkv, group, rows, hd]
    x = torch.matmul(q.flatten(2, 3), k.transpose(2, 3)).unflatten(2, (nq // nkv, -1)) / math.sqrt(hd)
    x = torch.where(see[:, :, None], x, -math.inf)
    top = x.amax(-1, keepdim=True)
    base = torch.where(top == -math.inf, 0, top)
    w = torch.exp(x - base)
    total = w.sum(-1, keepdim=True)
    o = torch.matmul(w.flatten(2, 3), v).unflatten(2, (nq // nkv, -1)) / torch.where(total == 0, 1, total)
    o, lse = o.permute(0, 3, 1, 2, 4).flatten(2, 3), (base + total.log())[..., 0].permute(0, 3, 1, 2).flatten(2, 3)
    live = t[None] < rows[:, None]
    return dict(out=o[live].to(s["q"].dtype), lse=lse[live])


def _plain_compact(s):
    """The kept rows' values, written again at their new places as rows appended there are; every layer's request is a
    request of its own in the pool of all layers."""
    layers, n_pages = s["k_scale"].shape[:2]
    shift = torch.arange(layers, device=s["keep"].device)[:, None] * n_pages
    table = (s["block_table"].long().clamp(min=0)[None] + shift[..., None]).flatten(0, 1)
    base, keep, n_keep = (x.long().repeat(layers, *[1] * (x.dim() - 1)) for x in (s["base_len"], s["keep"], s["n_keep"]))
    kb, vb = s["k_pages"].view(torch.uint8).flatten(0, 1), s["v_pages"].view(torch.uint8).flatten(0, 1)
    ks, vs = s["k_scale"].flatten(0, 1), s["v_scale"].flatten(0, 1)
    n, width = keep.shape
    dev = table.device
    req = torch.arange(n, device=dev)[:, None]
    last = table.shape[1] - 1
    src = base[:, None] + keep.clamp(min=0)
    src_page, src_off = table[req, (src // PAGE).clamp(max=last)], src % PAGE
    off = torch.arange(PAGE, device=dev)
    moved = []
    for raw, scale in ((kb[src_page, :, src_off], ks), (vb[src_page, :, :, src_off], vs)):
        moved.append(raw.view(torch.float8_e4m3fn).float() * scale[src_page][..., None])         # [n, width, nkv, hd]
    for i in range((width + PAGE - 2) // PAGE + 1):                                   # the i-th page that rows go to
        block = base // PAGE + i
        at = block[:, None] * PAGE + off - base[:, None]                              # row for each place of the page
        new, kept = (at >= 0) & (at < n_keep[:, None]), at < 0
        some = new.any(1)
        page = table[req[:, 0], block.clamp(max=last)]
        for x, pages, scale, turned in ((moved[0], kb, ks, False), (moved[1], vb, vs, True)):
            x = x[req, at.clamp(0, width - 1)]                                        # [n, 64, nkv, hd]
            big = torch.where(new[:, :, None, None] & x.isfinite(), x.abs(), 0).amax((1, 3))
            m, e = torch.frexp(big)
            e = torch.where(big > 0, e - 9 + (m > 0.875), MIN_EXP).clamp(min=MIN_EXP)
            to = torch.ldexp(torch.ones_like(big), e)
            was = scale[page]
            to = torch.where(new[:, :1], to, torch.maximum(to, was))
            old = pages[page]
            old = old.transpose(2, 3).contiguous() if turned else old                  # [n, nkv, 64, hd]
            again = old.view(torch.float8_e4m3fn).float() * (was / to)[..., None, None]
            y = (x / to[:, None, :, None]).clamp(-E4M3_MAX, E4M3_MAX).transpose(1, 2)
            pick = torch.where(new[:, None, :, None], y, again).to(torch.float8_e4m3fn).view(torch.uint8)
            pick = torch.where((new | kept)[:, None, :, None], pick, old)
            pick = pick.transpose(2, 3) if turned else pick
            pages[page[some]] = pick[some]
            scale[page[some]] = to[some]
    return {x: s[x] for x in ("k_pages", "v_pages", "k_scale", "v_scale")}


# ---------------------------------------------------------------- the definitions in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    return {"norm": _exact_norm, "bounds": _exact_bounds, "select": _exact_select, "sparse": _exact_sparse,
            "compact": _exact_compact}[case["op"]](s)


def _exact_norm(s):
    rot = s["rot"]
    f, m = _freq(s, torch.float64, "cpu")
    f = f.to(s["q"].device)
    turn = torch.polar(torch.full_like(f, m).expand(s["rows"], -1), s["positions"].double()[:, None] * f)
    places = [(2 * i, 2 * i + 1) if s["inter"] else (i, i + rot // 2) for i in range(rot // 2)]
    out = {}
    for name in ("q", "k"):
        x, w = s[name].double(), s[name + "_weight"].double()
        size = torch.sqrt(x.square().sum(-1, keepdim=True) / s["hd"] + EPS)
        unit = x / size
        y = unit * w if not s["grad"] else s["d" + name].double()
        z = y.clone()
        for i, (a, b) in enumerate(places):
            c = torch.complex(y[..., a], y[..., b]) * (turn[:, i, None].conj() if s["grad"] else turn[:, i, None])
            z[..., a], z[..., b] = c.real, c.imag
        if not s["grad"]:
            out[name] = z
            continue
        out["d" + name + "_weight"] = (z * unit).sum(0).sum(0)
        z = z * w
        out["d" + name] = (z - unit * (z * unit).sum(-1, keepdim=True) / s["hd"]) / size
    return out


def _exact_bounds(s):
    got = s["bounds"].clone()
    for b, (old, new) in enumerate(zip(s["old_len"].tolist(), s["new_len"].tolist())):
        if new <= old:
            continue
        for blk in range(old // PAGE, _pages(new)):
            page = int(s["block_table"][b, blk])
            x = s["k_pages"][page, :, :min(PAGE, new - blk * PAGE)].double()
            got[page, :, 0] = torch.floor(x.min(1).values / 4).to(torch.int8)
            got[page, :, 1] = torch.ceil(x.max(1).values / 4).to(torch.int8)
    return dict(bounds=got)


def _exact_select(s):
    group, k = s["nq"] // s["nkv"], s["n_select"]
    cu, ctx = s["cu_q"].tolist(), s["ctx_len"].tolist()
    out = []
    for b, length in enumerate(ctx):
        blocks, rows = _pages(length), cu[b + 1] - cu[b]
        page = s["block_table"][b, :blocks].long()
        for h in range(s["nkv"]):
            if not rows:
                out.append([-1] * k)
                continue
            lo, hi = s["bounds"][page, h, 0].double(), s["bounds"][page, h, 1].double()
            best = torch.full((blocks,), -math.inf, dtype=torch.float64, device=lo.device)
            for x in s["q"][cu[b]:cu[b + 1], h * group:(h + 1) * group].double().flatten(0, 1):
                top = float(x.abs().max())
                unit = 2.0 ** (max(math.frexp(top)[1] if top else -100, -100) - 10)
                whole = torch.round(x / unit)
                best = torch.maximum(best, torch.where(whole >= 0, hi, lo) @ whole * unit)
            best = best * 4 * s["k_scale"][page, h].double()
            rank = [(0 if j < s["first"] or j >= (length - rows) // PAGE - s["last"] else 1, -x, j) for j, x in enumerate(best.tolist())]
            pick = sorted(j for _, _, j in sorted(rank)[:k])
            out.append(pick + [-1] * (k - len(pick)))
    return dict(blocks=_i32(out).view(s["n"], s["nkv"], k))


def _exact_sparse(s):
    nq, nkv, hd = s["nq"], s["nkv"], s["hd"]
    cu, ctx = s["cu_q"].tolist(), s["ctx_len"].tolist()
    out = torch.zeros((cu[-1], nq, hd), dtype=torch.float64, device=s["q"].device)
    lse = torch.full((cu[-1], nq), -math.inf, dtype=torch.float64, device=s["q"].device)
    lists = s["blocks"].tolist()
    for b, length in enumerate(ctx):
        n = cu[b + 1] - cu[b]
        if not n or not length:
            continue
        for h in range(nkv):
            blk = [j for j in lists[b][h] if j >= 0]
            ids = s["block_table"][b].long()[blk]
            p = torch.cat([torch.arange(j * PAGE, j * PAGE + PAGE) for j in blk]).to(ids.device)
            i = torch.arange(n, device=ids.device)[:, None]
            see = (p < length)[None].expand(n, -1)
            if s["mask"] == "causal":
                see = see & (p <= length - n + i)
            elif s["mask"] == "tree":
                a = (p - (length - n)).clamp(0, n - 1)
                word = s["tree_mask"][cu[b]:cu[b + 1]].long()[:, a // 32]
                see = see & ((p < length - n) | (((word >> (a % 32)) & 1) == 1))
            k = s["k_pages"].view(torch.uint8)[ids, h].view(torch.float8_e4m3fn).double()
            k = (k * s["k_scale"][ids, h].double()[:, None, None]).reshape(-1, hd)
            v = s["v_pages"].view(torch.uint8)[ids, h].view(torch.float8_e4m3fn).double()
            v = (v * s["v_scale"][ids, h].double()[:, None, None]).transpose(1, 2).reshape(-1, hd)
            heads = slice(h * nq // nkv, (h + 1) * nq // nkv)
            x = s["q"][cu[b]:cu[b + 1], heads].double().transpose(0, 1) @ k.T / math.sqrt(hd)     # [group, n, tokens]
            x = x.masked_fill(~see, -math.inf)
            z = torch.logsumexp(x, 2)
            lse[cu[b]:cu[b + 1], heads] = z.T
            w = torch.exp(x - z.masked_fill(z == -math.inf, 0)[..., None])
            out[cu[b]:cu[b + 1], heads] = (w @ v).transpose(0, 1)
    return dict(out=out, lse=lse)


def _exact_compact(s):
    # the stored bytes are a rounding to 8 bits that has no finer value; the scales are exact powers of two
    base, count = s["base_len"].tolist(), s["n_keep"].tolist()
    keep, table = s["keep"].tolist(), s["block_table"].tolist()
    out = dict(k_pages=None, v_pages=None)
    for name, pages in (("k_scale", s["k_pages"]), ("v_scale", s["v_pages"].transpose(3, 4))):
        scale = s[name].double().cpu()
        out[name] = scale.clone()
        for b, c in enumerate(base):
            rows = {}
            for j in range(count[b]):
                rows.setdefault((c + j) // PAGE, []).append(c + keep[b][j])
            for blk, src in rows.items():
                big = torch.zeros(scale.shape[0], s["nkv"], dtype=torch.float64)
                for p in src:
                    page = table[b][p // PAGE]
                    big = torch.maximum(big, pages[:, page, :, p % PAGE].double().abs().amax(-1).cpu() * scale[:, page])
                to = table[b][blk]
                for layer, heads in enumerate(big.tolist()):
                    for h, y in enumerate(heads):
                        e = MIN_EXP
                        while 448.0 * 2.0 ** e < y:
                            e += 1
                        fresh = blk * PAGE >= c
                        out[name][layer, to, h] = 2.0 ** e if fresh else max(2.0 ** e, float(scale[layer, to, h]))
    return out
