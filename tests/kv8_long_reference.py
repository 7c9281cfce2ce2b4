"""Per-head norms with rotary positions, key bounds, the choice of blocks, attention over listed blocks and the move of kept
rows in 64 bits on the CPU, from their definitions."""
import math

import torch

import kv8_reference as R

PAGE, E4M3 = R.PAGE, R.E4M3


def pairs(rot, interleaved):
    a = slice(0, rot, 2) if interleaved else slice(0, rot // 2)
    b = slice(1, rot, 2) if interleaved else slice(rot // 2, rot)
    return a, b


def size_of_pair(y, rot, interleaved, magnitude):
    """|y_a| + |y_b| times the magnitude at both places of each rotated pair, |y| elsewhere."""
    out = y.abs().clone()
    a, b = pairs(rot, interleaved)
    both = (y[..., a].abs() + y[..., b].abs()) * magnitude
    out[..., a], out[..., b] = both, both
    return out


def norm(x, weight, eps):
    """(x r, r) of heads in float64."""
    r = 1 / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
    return x * r * weight, r


def bounds(pages, old, new, table, got):
    """pages [n_pages, heads, 64, hd] e4m3 and got [n_pages, heads, 2, hd] int8 on the CPU, got changed in place."""
    n_pages, width = pages.shape[0], table.shape[1]
    for b in range(table.shape[0]):
        lo, hi = (min(max(x, 0), width * PAGE) for x in (old[b], new[b]))
        if hi <= lo:
            continue
        for blk in range(lo // PAGE, R.pages_of(hi)):
            page = int(table[b, blk])
            if not 0 <= page < n_pages:
                continue
            x = pages[page, :, :min(PAGE, hi - blk * PAGE)].float().double()
            none = x.isnan().all(1)
            least = torch.where(x.isnan(), math.inf, x).amin(1)
            most = torch.where(x.isnan(), -math.inf, x).amax(1)
            got[page, :, 0] = torch.where(none, 0, torch.floor(least / 4)).to(torch.int8)
            got[page, :, 1] = torch.where(none, 0, torch.ceil(most / 4)).to(torch.int8)


def scores(q, cu, ctx, b, h, table, bound, k_scale):
    """The score of each block of request b for kv head h, as Python floats (exact)."""
    n_pages, nkv = k_scale.shape
    group = q.shape[1] // nkv
    length = min(max(ctx[b], 0), table.shape[1] * PAGE)
    rows = q[cu[b]:cu[b + 1], h * group:(h + 1) * group].double().flatten(0, 1)
    whole, unit = [], []
    for x in rows:
        if not bool(x.isfinite().all()):
            continue
        top = float(x.abs().max())
        e = max(math.frexp(top)[1] if top else -100, -100) - 10
        whole.append(torch.round(x * 2.0 ** -e).long())       # (to even)
        unit.append(2.0 ** e)
    out = []
    for blk in range(R.pages_of(length)):
        page = int(table[b, blk])
        if not 0 <= page < n_pages or not whole:
            out.append(-math.inf)
            continue
        lo, hi = bound[page, h].long()
        x = torch.stack(whole)
        s = torch.maximum(x * lo, x * hi).sum(1).double() * torch.tensor(unit, dtype=torch.float64)
        out.append(float(s.max()) * 4 * float(k_scale[page, h]))
    return out


def select(q, cu, ctx, table, bound, k_scale, k, first, last):
    nkv = k_scale.shape[1]
    out = []
    for b in range(table.shape[0]):
        n, length = cu[b + 1] - cu[b], min(max(ctx[b], 0), table.shape[1] * PAGE)
        for h in range(nkv):
            s = scores(q, cu, ctx, b, h, table, bound, k_scale) if n else []
            own = (length - n) // PAGE - last
            rank = sorted((0 if j < first or j >= own else 1, 0 if j < first or j >= own else -x, j) for j, x in enumerate(s))
            pick = sorted(j for _, _, j in rank[:k])
            out.append(pick + [-1] * (k - len(pick)))
    return torch.tensor(out, dtype=torch.int32).view(table.shape[0], nkv, k)


def attention(cache, q, cu, ctx, table, blocks, mask, tree=None, scale=None):
    """R.attention over the listed blocks: (out, lse, weight of |v|, D)."""
    rows, nq, hd = q.shape
    nkv = cache["k_scale"].shape[1]
    group = nq // nkv
    outs = [torch.zeros((rows, nq, hd), dtype=torch.float64), torch.full((rows, nq), -math.inf, dtype=torch.float64),
            torch.zeros((rows, nq, hd), dtype=torch.float64), torch.zeros((rows, nq), dtype=torch.float64)]
    for b in range(table.shape[0]):
        length = min(max(ctx[b], 0), table.shape[1] * PAGE)
        many = min(R.pages_of(length), blocks.shape[2])
        for h in range(nkv):
            # a table that names nothing but the listed blocks' pages, each at its place
            t = torch.full((1, table.shape[1]), -1, dtype=torch.int32)
            for j in blocks[b, h, :many].tolist():
                if 0 <= j < R.pages_of(length):
                    t[0, j] = table[b, j]
            one = {x: cache[x][:, h:h + 1] for x in cache}
            heads = slice(h * group, (h + 1) * group)
            part = slice(cu[b], cu[b + 1])
            got = R.attention(one, q[part, heads], [0, cu[b + 1] - cu[b]], [length], t, mask,
                              None if tree is None else tree[part], scale)
            for o, x in zip(outs, got):
                o[part, heads] = x
    return outs


def compact(cache, table, base, keep, count):
    """cache: dict of CPU tensors, changed in place: what R.append makes of the rows as read, page after page."""
    n_pages = cache["k_scale"].shape[0]
    width = table.shape[1]
    for b in range(table.shape[0]):
        start = min(max(base[b], 0), width * PAGE)
        k, v, slots = [], [], []
        for j in range(min(max(count[b], 0), keep.shape[1])):
            src, dst = start + int(keep[b, j]), start + j
            if int(keep[b, j]) < 0 or src >= width * PAGE or dst >= width * PAGE:
                continue
            sp, dp = int(table[b, src // PAGE]), int(table[b, dst // PAGE])
            if not (0 <= sp < n_pages and 0 <= dp < n_pages):
                continue
            k.append(cache["k_pages"][sp, :, src % PAGE].float() * cache["k_scale"][sp][:, None])
            v.append(cache["v_pages"][sp, :, :, src % PAGE].float() * cache["v_scale"][sp][:, None])
            slots.append(dp * PAGE + dst % PAGE)
        if slots:
            R.append(cache, torch.stack(k), torch.stack(v), slots)
