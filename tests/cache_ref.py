"""Plain 64-bit forms of the rotation, the 8-bit paged cache and attention over
it, on the CPU, for the tests of the kernels; nothing here is shared with the
library.

A `Paged` holds what a cache holds, as values; `append` and `attend` follow the
definitions in include/fa.h.
"""
import math

import torch

E4M3 = torch.tensor([(2.0 ** -9 * m if e == 0 else 2.0 ** (e - 7) * (1 + m / 8))
                     for e in range(16) for m in range(8)][:127], dtype=torch.float64)


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def to_e4m3(x):
    """Nearest e4m3 value, ties to the even code, 448 at most; NaN and infinities are NaN."""
    mid = (E4M3[1:] + E4M3[:-1]) / 2
    up = torch.searchsorted(mid, x.abs().nan_to_num(0.0, posinf=0.0).contiguous(), right=True)
    tie = (up > 0) & (x.abs() == mid[(up - 1).clamp(min=0)]) & (up % 2 == 1)
    y = E4M3[torch.where(tie, up - 1, up)]
    return torch.where(torch.isfinite(x), y * torch.sign(x), math.nan)


def codes_to_values(codes):
    return codes.cpu().view(torch.float8_e4m3fn).to(torch.float64)


def scale_of(amax):
    e = -100
    while amax > 448.0 * 2.0 ** e:
        e += 1
    return 2.0 ** e


def rotate(x, pos, freq, axis, interleaved, back=False):
    """x [B, heads, N, d], pos [axes, B, N] whole numbers."""
    x = x.double()
    P = len(freq)
    if P == 0:
        return x
    angle = torch.stack([pos[a].double() * f for a, f in zip(axis, freq)], -1)[:, None]
    c, s = torch.cos(angle), torch.sin(angle) * (-1 if back else 1)
    y = x.clone()
    one = slice(0, 2 * P, 2) if interleaved else slice(0, P)
    two = slice(1, 2 * P, 2) if interleaved else slice(P, 2 * P)
    y[..., one] = x[..., one] * c - x[..., two] * s
    y[..., two] = x[..., two] * c + x[..., one] * s
    return y


def rotate_slack(x, pairs, interleaved):
    """|x1| + |x2| of each rotated column (0 elsewhere): what an angle's error is multiplied by."""
    a = x.double().abs()
    out = torch.zeros_like(a)
    one = slice(0, 2 * pairs, 2) if interleaved else slice(0, pairs)
    two = slice(1, 2 * pairs, 2) if interleaved else slice(pairs, 2 * pairs)
    out[..., one] = out[..., two] = a[..., one] + a[..., two]
    return out


class Paged:
    """values [pages, Hkv, page, d] of the codes, scales [pages, Hkv]."""

    def __init__(self, codes, scales):
        self.values, self.scales = codes_to_values(codes), scales.double().cpu().clone()

    def append(self, x, start, table_row):
        """Rows x [Hkv, n, d] become tokens start .. start + n of one sequence."""
        page = self.values.shape[2]
        t, n = start, x.shape[1]
        while t < start + n:
            p, r = int(table_row[t // page]), t % page
            k = min(page - r, start + n - t)
            for h in range(x.shape[0]):
                rows = x[h, t - start:t - start + k]
                fine = rows[torch.isfinite(rows)]
                s = scale_of(float(fine.abs().max()) if fine.numel() else 0.0)
                if r:
                    was = float(self.scales[p, h])
                    s = max(s, was)
                    if s > was:
                        self.values[p, h, :r] = to_e4m3(self.values[p, h, :r] * (was / s))
                self.values[p, h, r:r + k] = to_e4m3(rows / s)
                self.scales[p, h] = s
            t += k

    def rows(self, table_row, n, h):
        """The first n tokens of a sequence, head h."""
        page = self.values.shape[2]
        ids = [int(i) for i in table_row[:-(-n // page)]]
        if not ids:
            return torch.zeros(0, self.values.shape[3], dtype=torch.float64)
        return torch.cat([self.values[i, h] * self.scales[i, h] for i in ids])[:n]


def attend(q, k, v, table, lens, new, causal, scale):
    """(o, lse, slack): q [B, H, Nq, d] on the CPU; slack: a bound of what the
    kernels' roundings can do to o before its own rounding, and of lse."""
    B, H, N, d = q.shape
    q = q.double()
    Hkv = k.values.shape[1]
    o = torch.zeros(B, H, N, d, dtype=torch.float64)
    lse = torch.full((B, H, N), -math.inf, dtype=torch.float64)
    o_slack, l_slack = torch.zeros_like(o), torch.zeros(B, H, N, dtype=torch.float64)
    for b in range(B):
        n = new[b]
        for h in range(H):
            K, V = (c.rows(table[b], lens[b], h // (H // Hkv)) for c in (k, v))
            for i in range(n):
                see = max(0, min(lens[b], lens[b] - n + i + 1)) if causal else lens[b]
                if see == 0:
                    continue
                x = q[b, h, i]
                S = (K[:see] @ x) * scale
                L = torch.logsumexp(S, 0)
                P = torch.exp(S - L)
                o[b, h, i], lse[b, h, i] = P @ V[:see], L
                # scores: products summed in fp32 (2^-23 a step, in any
                # order); exp2, the scaling and the running sums 2^-20
                # together.  q is exact as two (bf16, 8 bits) or three (f16, 11
                # bits) e4m3 values of 4 bits each where the last of them is a
                # multiple of e4m3's step 2^-9: the row's largest element is
                # brought to [2^7, 2^8), so for elements of at least 2, 2^-6 of
                # the largest or more; smaller ones are off by half a step,
                # 2^-10, at most, 2^-17 of the largest element
                size = float((K[:see].abs() @ x.abs()).max()) * scale
                top = float(x.abs().max())
                small = (x.abs() < top * 2.0 ** -6).double()
                tail = top * 2.0 ** -17 * float((K[:see].abs() @ small).max()) * scale
                ds = size * d * 2.0 ** -23 + tail + 2.0 ** -20 * (1 + float(S.abs().max()))
                # weights: half a step of f16, and 2^-25 of the largest for the small ones
                o_slack[b, h, i] = (P @ V[:see].abs()) * (2.0 ** -11 + 2 * ds + see * 2.0 ** -24) \
                    + see * 2.0 ** -25 * 448 * float(v.scales.max())
                l_slack[b, h, i] = ds + see * 2.0 ** -24 + 2.0 ** -21 * (1 + abs(float(L)))
    return o, lse, o_slack, l_slack


def make_cache(pages, Hkv, page, d, B, width, gen, lens=None, spread=1.0):
    """Random codes and power-of-two scales, and a table whose entries past a
    sequence's pages are out of range."""
    codes = [torch.randn(pages, Hkv, page, d, generator=gen).mul_(60).clamp_(-448, 448)
             .to(torch.float8_e4m3fn) for _ in range(2)]
    scales = [2.0 ** torch.randint(-8, -4, (pages, Hkv), generator=gen).float() * spread
              for _ in range(2)]
    order = torch.randperm(pages, generator=gen)
    table = torch.full((B, width), -7, dtype=torch.int32)
    at = 0
    for b in range(B):
        need = width if lens is None else -(-lens[b] // page)
        table[b, :need] = order[at:at + need].to(torch.int32)
        at += need
    return codes, scales, table
