"""Plain 64-bit forms of a branching decode over the paged cache (a tree's
attention, keeping tokens, forking sequences) and of the norms of q and k, on
the CPU, for the tests of the kernels; nothing here is shared with the library.
"""
import math

import torch

import cache_ref as ref


# ------------------------------------------------------------------ norms
def norm(x, w, eps, offset, turn):
    """y of rows x [B, heads, N, d]; turn(x, back) rotates."""
    x = x.double()
    r = 1.0 / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
    f = 1.0 if w is None else w.double() + offset
    return turn(x * r * f, False)


def norm_backward(dy, x, w, eps, offset, turn):
    """(dx, dw) from the formula."""
    x, g = x.double(), turn(dy.double(), True)
    r = 1.0 / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
    f = 1.0 if w is None else w.double() + offset
    h, u = x * r, g * f
    return r * (u - h * (u * h).mean(-1, keepdim=True)), (g * h).sum((0, 1, 2))


# ------------------------------------------------------------------ tree
def random_tree(n, gen):
    """Parents of n drafted tokens, each one of the eight before it or none."""
    out = []
    for i in range(n):
        at = int(torch.randint(-1, 8, (1,), generator=gen))
        out.append(max(-1, i - 1 - at) if at >= 0 else -1)
    return out


def sees_of(parents):
    """bool [n, n]: row i sees drafted token j."""
    n = len(parents)
    sees = torch.zeros(n, n, dtype=torch.bool)
    for i, p in enumerate(parents):
        if p >= 0:
            sees[i] = sees[p]
        sees[i, i] = True
    return sees


def pack(sees, N):
    """int32 [N, words] of bool [n, n]."""
    words = -(-N // 32)
    out = torch.zeros(N, words, dtype=torch.int64)
    for i, j in sees.nonzero().tolist():
        out[i, j // 32] |= 1 << (j % 32)
    return torch.where(out >= 1 << 31, out - (1 << 32), out).to(torch.int32)


def attend_tree(q, k, v, table, lens, sees, scale):
    """(o, lse, slacks) as cache_ref.attend, sequence b's rows being its last
    len(sees[b]) tokens, which see the tokens before them and sees[b]."""
    B, H, N, d = q.shape
    q = q.double()
    Hkv = k.values.shape[1]
    o = torch.zeros(B, H, N, d, dtype=torch.float64)
    lse = torch.full((B, H, N), -math.inf, dtype=torch.float64)
    o_slack, l_slack = torch.zeros_like(o), torch.zeros(B, H, N, dtype=torch.float64)
    for b in range(B):
        n = len(sees[b])
        mask = torch.cat((torch.ones(n, lens[b] - n, dtype=torch.bool), sees[b][:, :n]), 1)
        some = mask.any(1)
        for h in range(H):
            if lens[b] == 0 or not some.any():
                continue
            K, V = (c.rows(table[b], lens[b], h // (H // Hkv)) for c in (k, v))
            # (what no row sees may be anything)
            seen = mask.any(0)
            K, V = torch.where(seen[:, None], K, 0.0), torch.where(seen[:, None], V, 0.0)
            x = q[b, h, :n]
            S = (x @ K.T * scale).masked_fill(~mask, -math.inf)
            L = torch.logsumexp(S, -1)
            P = torch.where(mask, torch.exp(S - L[:, None].nan_to_num(0.0, neginf=0.0)), 0.0)
            o[b, h, :n] = torch.where(some[:, None], P @ V, 0.0)
            lse[b, h, :n] = torch.where(some, L, -math.inf)
            # as in cache_ref.attend, for a whole head at a time
            see = mask.sum(1)
            size = torch.where(mask, x.abs() @ K.abs().T, 0.0).amax(1) * scale
            top = x.abs().amax(1)
            small = (x.abs() < top[:, None] * 2.0 ** -6).double()
            tail = top * 2.0 ** -17 * torch.where(mask, small @ K.abs().T, 0.0).amax(1) * scale
            big = torch.where(mask, S, 0.0).abs().amax(1)
            ds = size * d * 2.0 ** -23 + tail + 2.0 ** -20 * (1 + big)
            o_slack[b, h, :n] = (P @ V.abs()) * (2.0 ** -11 + 2 * ds + see * 2.0 ** -24)[:, None] \
                + (see * 2.0 ** -25 * 448 * float(v.scales.max()))[:, None]
            l_slack[b, h, :n] = torch.where(some, ds + see * 2.0 ** -24 + 2.0 ** -21 * (1 + lse[b, h, :n].abs()), 0.0)
    return o, lse, o_slack, l_slack


# ------------------------------------------------------------------ keep
def keep(held, table_row, base, kept):
    """Tokens base + kept[i] of a sequence become base + i, in place (a
    cache_ref.Paged with scales that are powers of two)."""
    page = held.values.shape[2]
    old, scales = held.values.clone(), held.scales.clone()
    end = base + len(kept)
    for number in range(base // page, -(-end // page)) if kept else ():
        toks = range(number * page, min(end, (number + 1) * page))
        srcs = [t if t < base else base + kept[t - base] for t in toks]
        at = [(int(table_row[t // page]), t % page) for t in srcs]
        p = int(table_row[number])
        for h in range(held.scales.shape[1]):
            top = max(float(scales[i, h]) for i, _ in at)
            for r, (i, row) in enumerate(at):
                held.values[p, h, r] = ref.to_e4m3(old[i, h, row] * (float(scales[i, h]) / top))
            held.scales[p, h] = top


# ------------------------------------------------------------------ fork
def fork(table, refs, parents, lens, reserve, page):
    """(new table, new refs, new lengths, copies [(source, page, rows)]) by the definition, one place at a time;
    pages that are out of range or lacking are -1."""
    B, W = len(table), len(table[0])
    pages = len(refs)
    free = [p for p, n in enumerate(refs) if n == 0]
    new, now, out, copies, seen = [], list(refs), [], [], set()
    for b in range(B):
        parent = parents[b] if -1 <= parents[b] < B else -1
        L = lens[parent] if parent >= 0 else 0
        L = L if 0 <= L <= W * page else 0
        want = max(L, min(reserve[b] if reserve else 0, W * page))
        row = [-1] * W
        for i in range(-(-want // page)):
            old = table[parent][i] if parent >= 0 else -1
            old = old if 0 <= old < pages else -1
            if i < L // page:
                row[i] = old
            elif old >= 0 and parent not in seen and refs[old] == 1:
                row[i] = old
            else:
                row[i] = free.pop(0) if free else -1
                if i == L // page and L % page and parent >= 0 and row[i] >= 0:
                    copies.append((old if old >= 0 else pages - 1, row[i], L % page))
            if row[i] >= 0:
                now[row[i]] += 1
        seen.add(parent)
        new.append(row)
        out.append(L)
    for row in table:
        for p in row:
            if 0 <= p < pages:
                now[p] -= 1
    return new, now, out, copies
