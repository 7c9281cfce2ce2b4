"""The 8-bit paged cache and rotary positions in 64 bits on the CPU, from their definitions."""
import math
from decimal import Decimal, getcontext

import numpy as np
import torch

PAGE = 64
E4M3 = torch.float8_e4m3fn


def pages_of(n):
    return -(-n // PAGE)


def plan(ctx, add, table, stack, max_rows):
    """Lists in, lists out; `table` and `stack` (the free pages only) are changed in place."""
    width = len(table[0])
    for b, (c, a) in enumerate(zip(ctx, add)):
        for i in range(pages_of(max(0, c + a)), pages_of(c)):
            stack.append(table[b][i])
    have, asked, asked_rows = len(stack), 0, 0
    new, cu, slot, pos, refused = [], [0], [], [], []
    for b, (c, a) in enumerate(zip(ctx, add)):
        to = max(0, c + a)
        bad = pages_of(to) > width
        need, rows = (0, 0) if bad else (max(0, pages_of(to) - pages_of(c)), max(0, a))
        asked, asked_rows = asked + need, asked_rows + rows
        bad = bad or (need > 0 and asked > have) or (rows > 0 and asked_rows > max_rows)
        refused.append(int(bad))
        new.append(c if bad else to)
        if not bad:
            for i in range(pages_of(c), pages_of(c) + need):
                table[b][i] = stack.pop()
            for p in range(c, c + rows):
                slot.append(table[b][p // PAGE] * PAGE + p % PAGE)
                pos.append(p)
        cu.append(len(slot))
    return new, cu, slot, pos, refused


def rope_freq(rot, theta, scaling="none", factor=1.0, original=1.0, fast=32.0, slow=1.0):
    """([rot / 2] Decimals: turns per position, magnitude) to 50 digits."""
    getcontext().prec = 50
    pi = Decimal("3.14159265358979323846264338327950288419716939937510")
    lt = Decimal(theta).ln()
    out = []
    dim = lambda b: rot * math.log(original / (b * 2 * math.pi)) / (2 * math.log(theta))  # noqa: E731
    if scaling == "yarn":
        lo, hi = max(math.floor(dim(fast)), 0), min(math.ceil(dim(slow)), rot - 1)
    for i in range(rot // 2):
        f = (Decimal(-2 * i) / rot * lt).exp()
        if scaling == "linear":
            f /= Decimal(factor)
        if scaling == "yarn":
            g = Decimal(min(max((i - lo) / max(hi - lo, 0.001), 0.0), 1.0))
            f = f / Decimal(factor) * g + f * (1 - g)
        out.append(f / (2 * pi))
    return out, (0.1 * math.log(factor) + 1 if scaling == "yarn" else 1.0)


def rope(x, positions, rot, freq, magnitude, interleaved, transpose=False):
    """x [rows, heads, hd] float64."""
    y = x.clone()
    ang = np.array([[float((int(p) * f) % 1) for f in freq] for p in positions]) * 2 * math.pi
    cos = torch.from_numpy(np.cos(ang) * magnitude)[:, None]
    sin = torch.from_numpy(np.sin(ang) * magnitude)[:, None] * (-1 if transpose else 1)
    a = slice(0, rot, 2) if interleaved else slice(0, rot // 2)
    b = slice(1, rot, 2) if interleaved else slice(rot // 2, rot)
    y[..., a] = x[..., a] * cos - x[..., b] * sin
    y[..., b] = x[..., b] * cos + x[..., a] * sin
    return y


def scale_exp(amax):
    e = -64
    while 448.0 * 2.0 ** e < amax:
        e += 1
    return e


def append(cache, k, v, slots):
    """cache: dict of CPU tensors k_pages, v_pages (e4m3), k_scale, v_scale, changed in place; k, v [rows, heads, hd]."""
    n_pages, heads = cache["k_scale"].shape
    runs = []
    for r, s in enumerate(slots):
        if 0 <= s < n_pages * PAGE:
            if not runs or runs[-1][0] != s // PAGE:
                runs.append((s // PAGE, {}))
            runs[-1][1][s % PAGE] = r
    for page, rows in runs:
        for x, name in ((k, "k"), (v, "v")):
            pages = cache[name + "_pages"] if name == "k" else cache["v_pages"].transpose(2, 3)
            for h in range(heads):
                new = x[list(rows.values()), h].double()
                fin = new[new.isfinite()].abs()
                s = 2.0 ** scale_exp(float(fin.max()) if fin.numel() else 0.0)
                old = float(cache[name + "_scale"][page, h])
                if 0 not in rows and old >= s:
                    s = old
                elif 0 not in rows:
                    for off in range(max(rows)):
                        if off not in rows:
                            was = pages[page, h, off].float()
                            pages[page, h, off] = (was * (old / s)).to(E4M3)
                cache[name + "_scale"][page, h] = s
                for off, r in rows.items():
                    pages[page, h, off] = (x[r, h].float() / s).clamp(-448, 448).to(E4M3)


def attention(cache, q, cu, ctx, table, mask, tree=None, scale=None):
    """(out, lse, weight of |v|, D) in float64; cache tensors on the CPU. D bounds the scores' terms: over a row's
    tokens the largest sum |q_d k_d| scale, plus a quarter of the largest |q| times sum |k_d| scale (what a q
    that is kept to 2^-21 of its row's largest entry, 2^-19 / 4, can be off by)."""
    rows, nq, hd = q.shape
    n_pages, nkv = cache["k_scale"].shape
    scale = 1 / math.sqrt(hd) if scale is None else scale
    out = torch.zeros((rows, nq, hd), dtype=torch.float64)
    lse = torch.full((rows, nq), -math.inf, dtype=torch.float64)
    absv = torch.zeros((rows, nq, hd), dtype=torch.float64)
    top = torch.zeros((rows, nq), dtype=torch.float64)
    q = q.double()
    for b, length in enumerate(ctx):
        n = cu[b + 1] - cu[b]
        length = min(length, table.shape[1] * PAGE)
        if not n or length <= 0:
            continue
        ids = table[b, :pages_of(length)].long()
        ok = ((ids >= 0) & (ids < n_pages)).repeat_interleave(PAGE)[:length]
        ids = ids.clamp(0, n_pages - 1)
        p, i = torch.arange(length), torch.arange(n)[:, None]
        see = ok[None].expand(n, -1)
        if mask == "causal":
            see = see & (p <= length - n + i)
        if mask == "tree":
            j = p - (length - n)
            w = tree[cu[b]:cu[b + 1]].long()
            bit = (w[:, (j.clamp(min=0) // 32).clamp(max=w.shape[1] - 1)] >> (j % 32)) & 1
            see = see & ((j < 0) | ((bit == 1) & (j < 32 * w.shape[1])))
        for h in range(nkv):
            k = cache["k_pages"].view(torch.uint8)[ids, h].view(E4M3).double() * cache["k_scale"][ids, h].double()[:, None, None]
            v = cache["v_pages"].view(torch.uint8)[ids, h].view(E4M3).double() * cache["v_scale"][ids, h].double()[:, None, None]
            k, v = k.reshape(-1, hd)[:length], v.transpose(1, 2).reshape(-1, hd)[:length]
            # a place is read for a row only if the row sees it
            for g in range(nq // nkv):
                hq = h * (nq // nkv) + g
                for r in range(n):
                    row, s = cu[b] + r, see[r]
                    if not bool(s.any()):
                        continue
                    if not bool(q[row, hq].isfinite().all()):
                        out[row, hq], lse[row, hq] = math.nan, math.nan
                        continue
                    x = (k[s] @ q[row, hq]) * scale
                    z = torch.logsumexp(x, 0)
                    w = torch.exp(x - z)
                    lse[row, hq] = z
                    out[row, hq] = w @ v[s]
                    absv[row, hq] = w @ v[s].abs()
                    top[row, hq] = ((k[s].abs() @ q[row, hq].abs()).max() + q[row, hq].abs().max() * k[s].abs().sum(1).max() / 4) * scale
    return out, lse, absv, top
