"""The operators of a branching decode around the paged 8-bit cache, and the
norms of queries and keys; each in a plain form and through the library.

Definitions.  Norm: y = turn(x / sqrt(mean x^2 + eps) * (offset + w)) for every
row x of d elements (one token of one head), w one for all heads of q and one
for all of k; turn is the rotation by positions, pair p of a row by the angle
t * w_p, pairs being columns (p, p + P) or (2p, 2p + 1).  Backward: with g the
gradient turned back, h = x r, r = 1 / sqrt(mean x^2 + eps), u = g (offset + w):
dx = r (u - h mean(u h)), dw = sum over rows of g h.  Tree: query row i of a
sequence is drafted token i of its last n tokens; it sees every token before
those, and drafted token j where bit j of its mask is set.  Keep: of the last n
tokens of a sequence those numbered keep[0] < keep[1] < ... stay and move up to
the front of the n.  A page that takes moved tokens has the largest of the
scales that its tokens come with (its own, if one of them was in it), and codes
that come with a smaller one are rounded again for it; rows behind the kept ones
stay as they are.  Fork: sequence b goes on from sequence parents[b] (-1: it
ends).  Whole pages are shared; from the first page that is not full on, the
first of a parent's children keeps the pages that nobody else holds (count 1),
and every other place takes a page whose count was 0 before the call, in the
order of their numbers; tokens in a page that is not full are copied.  Counts of
holders follow; a sequence holds pages for its tokens and for those reserved.
"""
import math
import random

import torch

own = False


# ------------------------------------------------------------------ cases
def listed():
    return [
        # training, the repository's gqa8k layer: q and k of a projection's [B, N, H, d] layout
        {"name": "norm gqa8k", "op": "norm", "B": 2, "H": 32, "Hkv": 8, "N": 8192, "d": 128, "dtype": "bf16",
         "weights": "bf16", "offset": 0.0, "axes": 1, "interleaved": False, "rotated": 128, "backward": False},
        # its backward pass, with the weights' gradients
        {"name": "norm gqa8k backward", "op": "norm", "B": 2, "H": 32, "Hkv": 8, "N": 8192, "d": 128, "dtype": "bf16",
         "weights": "bf16", "offset": 0.0, "axes": 1, "interleaved": False, "rotated": 128, "backward": True},
        # training on video tokens: three axes, interleaved pairs, fp32 weights around one
        {"name": "norm video backward", "op": "norm", "B": 1, "H": 16, "Hkv": 16, "N": 4099, "d": 64, "dtype": "f16",
         "weights": "f32", "offset": 1.0, "axes": 3, "interleaved": True, "rotated": 64, "backward": True},
        # a verification step of a few tokens, part of each row rotated: the latency of a call
        {"name": "norm few tokens", "op": "norm", "B": 4, "H": 32, "Hkv": 8, "N": 5, "d": 128, "dtype": "bf16",
         "weights": "bf16", "offset": 0.0, "axes": 1, "interleaved": False, "rotated": 64, "backward": False},
        # drafts of one short conversation: the latency of a call
        {"name": "tree one", "op": "tree", "B": 1, "H": 32, "Hkv": 8, "n": 7, "L": 1000, "d": 128, "dtype": "bf16",
         "page": 64, "ragged": False},
        # the benchmark's decode batch with a tree of drafts for each sequence
        {"name": "tree batch", "op": "tree", "B": 8, "H": 32, "Hkv": 8, "n": 25, "L": 8192, "d": 128, "dtype": "bf16",
         "page": 64, "ragged": False},
        # small trees behind long documents of unlike lengths
        {"name": "tree long", "op": "tree", "B": 4, "H": 32, "Hkv": 8, "n": 6, "L": 131072, "d": 128, "dtype": "bf16",
         "page": 128, "ragged": True},
        # a wide search from a few prompts, the head256 head size, trees of unlike sizes
        {"name": "tree wide d256", "op": "tree", "B": 3, "H": 8, "Hkv": 4, "n": 333, "L": 16384, "d": 256,
         "dtype": "f16", "page": 32, "ragged": True},
        # after a verification step: the accepted branch of each sequence's drafts stays
        {"name": "keep drafts", "op": "keep", "B": 64, "Hkv": 8, "n": 25, "a": 6, "before": 1000, "d": 128, "page": 64},
        # long prompts thinned to half of their tokens
        {"name": "keep thinned", "op": "keep", "B": 2, "Hkv": 8, "n": 16384, "a": 8192, "before": 37, "d": 128,
         "page": 64},
        # a step of a beam search: 8 requests of 4 beams
        {"name": "fork beams", "op": "fork", "kind": "beams", "B": 32, "width": 4, "Hkv": 8, "L": 2000, "reserve": 1,
         "d": 128, "page": 64},
        # many samples of a few prompts begin
        {"name": "fork samples", "op": "fork", "kind": "samples", "B": 256, "width": 64, "Hkv": 8, "L": 4099,
         "reserve": 200, "d": 128, "page": 128},
    ]


def _spread(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["norm", "norm", "tree", "tree", "keep", "fork"])
    d = rng.choice([64, 128, 128, 256])
    Hkv = rng.choice([1, 2, 4, 8, 16])
    page = rng.choice([16, 32, 64, 64, 128, 256])
    H = Hkv * rng.choice([g for g in (1, 2, 3, 4, 7, 8, 16) if Hkv * g <= 32])
    dtype = rng.choice(["bf16", "bf16", "f16"])
    if op == "norm":
        tokens = _spread(rng, 1, min(16384, 2 * 8192 * 40 * 128 // ((H + Hkv) * d)))
        B = _spread(rng, 1, min(64, tokens))
        return {"op": op, "B": B, "H": H, "Hkv": Hkv, "N": max(1, tokens // B), "d": d, "dtype": dtype,
                "weights": rng.choice([dtype, "f32"]), "offset": rng.choice([0.0, 1.0]), "axes": rng.choice([1, 1, 2, 3]),
                "interleaved": rng.random() < 0.4, "rotated": rng.choice([d, d, d // 2, 0]),
                "backward": rng.random() < 0.5}
    if op == "tree":
        pairs = 333 * 26000 * 8 * 256 // (H * d)       # of a query and a key, for each head
        n = _spread(rng, 1, min(400, math.isqrt(pairs)))
        keys = _spread(rng, 64, min(320000 * 8 * 128 // (Hkv * d), max(64, pairs // n)))
        B = _spread(rng, 1, max(1, min(128, keys // max(64, n))))
        return {"op": op, "B": B, "H": H, "Hkv": Hkv, "n": n, "L": max(n, min(131072, keys // B)), "d": d,
                "dtype": dtype, "page": page, "ragged": rng.random() < 0.6}
    if op == "keep":
        rows = _spread(rng, 2, min(26000, 13000 * 8 * 128 // (Hkv * d)))
        B = _spread(rng, 1, min(128, rows // 2))
        n = rows // B
        return {"op": op, "B": B, "Hkv": Hkv, "n": n, "a": _spread(rng, 1, n), "before": _spread(rng, 1, 2000) - 1,
                "d": d, "page": page}
    width = rng.choice([2, 3, 4, 8, 16])
    size = 8 * 128 / (Hkv * d)
    B = width * _spread(rng, 1, max(1, min(256, int(80 * 128 * size) // page) // width))
    return {"op": op, "kind": rng.choice(["beams", "samples"]), "B": B, "width": width, "Hkv": Hkv,
            "L": _spread(rng, 1, max(1, min(8000, int(40000 * size) * width // B))),
            "reserve": _spread(rng, 1, page) - 1, "d": d, "page": page}


def _fractions(B):
    """A fixed uneven spread over (0, 1], the first sequence whole."""
    return [1.0 if b == 0 else (b * 0.6180339887498949) % 1.0 for b in range(B)]


def _lengths(case):
    """(tokens in the cache, the last ones among them) of each sequence."""
    f, B = _fractions(case["B"]), case["B"]
    if case["op"] == "fork":
        lens = [max(1, int(case["L"] * f[b // case["width"]])) for b in range(B)]
        return ([x if case["kind"] == "beams" or b % case["width"] == 0 else 0 for b, x in enumerate(lens)], None)
    if case["op"] == "keep":
        n = [max(1, int(case["n"] * (0.5 + x / 2))) for x in f]
        return [int(case["before"] * x) + k for x, k in zip(f, n)], n
    n = [max(1, int(case["n"] * (0.5 + x / 2))) if case["ragged"] else case["n"] for x in f]
    return [max(k, int(case["L"] * x)) if case["ragged"] else case["L"] for x, k in zip(f, n)], n


def _kept(case, n):
    """How many of the last n tokens of each sequence stay."""
    return [min(k, int(case["a"] * x + 0.999)) for x, k in zip(_fractions(case["B"]), n)]


def _parents(case):
    rng = random.Random(1009 * case["B"] + case["L"])
    out, w = [], case["width"]
    for b in range(case["B"]):
        first = b - b % w
        beams = min(w, case["B"] - first)
        out.append(first if case["kind"] == "samples" else -1 if rng.random() < 0.05 else first + rng.randrange(beams))
    return out


# ------------------------------------------------------------------ work
def work(case):
    B, Hkv, d = case["B"], case["Hkv"], case["d"]
    if case["op"] == "norm":
        tokens, heads = B * case["N"], case["H"] + Hkv
        return {"bytes": tokens * ((6 if case["backward"] else 4) * heads * d + 4 * case["axes"]),
                "flops": tokens * heads * ((10.0 if case["backward"] else 4.0) * d + 3.0 * case["rotated"])}
    lens, new = _lengths(case)
    if case["op"] == "tree":
        H, n = case["H"], case["n"]
        pairs = sum(k * (t - k) + k for t, k in zip(lens, new))          # the tokens before the drafts, and itself
        return {"bytes": sum(2 * t * Hkv * d + 8 * Hkv * -(-t // case["page"]) for t in lens)
                + B * H * n * (4 * d + 4) + B * n * 4 * -(-n // 32), "flops": 4.0 * H * d * pairs}
    if case["op"] == "keep":
        rows = sum(_kept(case, new))
        return {"bytes": rows * (4 * Hkv * d + 4), "flops": 2.0 * rows * Hkv * d}
    parents, page = _parents(case), case["page"]
    copies = sum(lens[p] % page for b, p in enumerate(parents) if p >= 0 and p in parents[:b])
    places = sum(-(-(lens[p] + case["reserve"]) // page) for p in parents if p >= 0)
    return {"bytes": 4 * Hkv * d * copies + 16 * places, "flops": 0.0}


# ------------------------------------------------------------------ inputs
_TYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}


def _quantise(x):
    """(codes, scales) of whole pages [..., rows, d]: powers of two that bring the largest to 448 at most."""
    mant, exp = torch.frexp(x.abs().amax((-1, -2)))
    s = torch.ldexp(torch.ones_like(mant), torch.where(mant <= 0.875, exp - 9, exp - 8).clamp(min=-100))
    return (x / s[..., None, None]).to(torch.float8_e4m3fn), s


def _cache(st, pages, g):
    case, dev = st["case"], "cuda"
    Hkv, page, d = case["Hkv"], case["page"], case["d"]
    for name, spread in (("k", 1.0), ("v", 0.7)):
        codes = torch.empty(pages, Hkv, page, d, dtype=torch.float8_e4m3fn, device=dev)
        scales = torch.empty(pages, Hkv, device=dev)
        step = max(1, (1 << 27) // (Hkv * page * d))
        for p in range(0, pages, step):
            x = torch.randn(min(step, pages - p), Hkv, page, d, generator=g, device=dev)
            # heads and pages of unlike size, as in a model
            x *= spread * torch.exp(0.5 * torch.randn(len(x), Hkv, 1, 1, generator=g, device=dev))
            codes[p:p + step], scales[p:p + step] = _quantise(x)
        st[name + "_codes"], st[name + "_scale"] = codes, scales


def _tree_bits(n, N, rng):
    """Masks of a random tree of n drafts in N rows: a node sees itself and what its parent sees."""
    sees = []
    for i in range(n):
        parent = rng.randrange(max(0, i - 8), i) if i > 0 and rng.random() < 0.95 else -1
        sees.append((sees[parent] if parent >= 0 else 0) | 1 << i)
    words = -(-N // 32)
    rows = [[x >> (32 * w) & 0xffffffff for w in range(words)] for x in sees] + [[0] * words] * (N - n)
    return [[w - (1 << 32) if w >> 31 else w for w in r] for r in rows]


def prepare(case, seed):
    dev = "cuda"
    g = torch.Generator(device=dev).manual_seed(seed)
    rng = random.Random(seed)
    B, Hkv, d = case["B"], case["Hkv"], case["d"]
    st = {"case": case}

    def ints(x):
        return torch.tensor(x, dtype=torch.int32).to(dev)

    if case["op"] == "norm":
        H, N, axes, dt = case["H"], case["N"], case["axes"], _TYPES[case["dtype"]]
        for name, heads in (("q", H), ("k", Hkv)):
            # a projection's output [B, N, heads, d], seen as [B, heads, N, d]; tokens of unlike size
            x = torch.randn(B, N, heads, d, generator=g, device=dev)
            x *= torch.exp(0.5 * torch.randn(B, N, 1, 1, generator=g, device=dev))
            st[name] = x.to(dt).transpose(1, 2)
            w = 1 - case["offset"] + 0.2 * torch.randn(d, generator=g, device=dev)
            st["w" + name] = w.to(_TYPES[case["weights"]])
            if case["backward"]:
                st["d" + name] = torch.randn(B, N, heads, d, generator=g, device=dev).to(dt).transpose(1, 2)
        pairs = case["rotated"] // 2
        st["inv_freq"] = [10000.0 ** (-i / pairs) for i in range(pairs)]
        st["axis"] = [i * axes // pairs for i in range(pairs)]
        t = torch.arange(N, device=dev)
        if axes > 1:      # rows of a grid of frames
            side = max(1, round(N ** (1 / 3)))
            t = torch.stack([t // (side * side), t // side % side, t % side][3 - axes:])
        t = t.reshape(axes, 1, N) + rng.randrange(100000)
        st["pos"] = t.expand(axes, B, N).to(torch.int32).contiguous()
        if own:
            from exact_io_aware_20_gb300 import binding
            st["rope"] = binding.Rope(st["inv_freq"], st["axis"], case["interleaved"]) if pairs else None
        return st

    lens, new = _lengths(case)
    page = case["page"]
    st["lens"] = ints(lens)
    need = [max(1, -(-t // page)) for t in lens]
    if case["op"] != "fork":
        pages, width = sum(need) + 3, max(need)
        order = torch.randperm(pages, generator=g, device=dev).tolist()
        table = [[order.pop() for _ in range(k)] + [-1] * (width - k) for k in need]
    else:
        parents = _parents(case)
        need = [-(-(x + case["reserve"]) // page) for x in lens]
        width = max(need) + 1
        own_pages = sum(need) + 2 * B * (case["reserve"] // page + 2)
        pages = own_pages + 5
        order = torch.randperm(pages, generator=g, device=dev).tolist()
        refs, table = [0] * pages, []
        for b in range(B):
            first = b - b % case["width"]
            full = lens[b] // page
            row = [table[first][i] if b > first and i < full else order.pop() for i in range(need[b] if lens[b] else 0)]
            table.append(row + [-1] * (width - len(row)))
            for p in row:
                refs[p] += 1
            if b == first and full:
                refs[row[0]] += 1          # a prefix that is also kept for others
        st["refs"], st["parents"] = ints(refs), ints(parents)
        st["reserve"] = ints([lens[p] + case["reserve"] if p >= 0 else 0 for p in parents])
    st["table"] = ints(table)
    _cache(st, pages, g)
    if case["op"] == "tree":
        n, H = case["n"], case["H"]
        st["q"] = torch.randn(B, n, H, d, generator=g, device=dev).to(_TYPES[case["dtype"]]).transpose(1, 2)
        st["mask"] = ints([_tree_bits(k, n, rng) for k in new])
        st["new"] = ints(new) if case["ragged"] else None
    if case["op"] == "keep":
        a = _kept(case, new)
        st["new"], st["kept"] = ints(new), ints(a)
        st["keep"] = ints([sorted(rng.sample(range(k), x)) + [-1] * (max(a) - x) for k, x in zip(new, a)])
    if own:
        from exact_io_aware_20_gb300 import binding
        st["cache"] = binding.Cache(st["k_codes"], st["v_codes"], st["k_scale"], st["v_scale"], st["table"])
    return st


# ------------------------------------------------------------------ the framework's calls
def _own(st):
    from exact_io_aware_20_gb300 import binding
    case = st["case"]
    if case["op"] == "norm":
        rest = (st["q"], st["k"], st["wq"], st["wk"], 1e-6, st["pos"] if st["rope"] else None, st["rope"], case["offset"])
        if case["backward"]:
            return binding.qk_norm_rope_backward(st["dq"], st["dk"], *rest)
        return binding.qk_norm_rope(*rest)
    if case["op"] == "tree":
        return binding.forward_cache_tree(st["q"], st["cache"], st["lens"], st["mask"], case["d"] ** -0.5,
                                          new_lens=st["new"])
    state = (st["k_codes"], st["v_codes"], st["k_scale"], st["v_scale"])
    if case["op"] == "keep":
        out = binding.cache_keep(st["cache"], st["lens"], case["n"], st["keep"], keep_lens=st["kept"], new_lens=st["new"])
        return (out,) + state
    out = binding.cache_fork(st["cache"], st["refs"], st["parents"], st["lens"], reserve_lens=st["reserve"])
    return (out, st["table"], st["refs"]) + state


# ------------------------------------------------------------------ plain forms
def _turn(st, x, back=False):
    """The rotation of x, in 32 bits; the angles in 64."""
    case = st["case"]
    P = case["rotated"] // 2
    if P == 0:
        return x
    w = torch.tensor(st["inv_freq"], dtype=torch.float64, device=x.device)
    axis = torch.tensor(st["axis"], device=x.device)
    angle = (st["pos"].double()[axis] * w[:, None, None]).permute(1, 2, 0)[:, None]     # [B, 1, N, P]
    c, s = angle.cos().float(), angle.sin().float()
    s = -s if back else s
    if case["interleaved"]:
        a, b = x[..., 0:2 * P:2], x[..., 1:2 * P:2]
        turned = torch.stack((a * c - b * s, b * c + a * s), -1).flatten(-2)
    else:
        a, b = x[..., :P], x[..., P:2 * P]
        turned = torch.cat((a * c - b * s, b * c + a * s), -1)
    return torch.cat((turned, x[..., 2 * P:]), -1)


def _norm(st):
    case = st["case"]
    out, sums = [], []
    for name in ("q", "k"):
        x, w = st[name].float(), st["w" + name].float() + case["offset"]
        r = 1.0 / torch.sqrt((x * x).mean(-1, keepdim=True) + 1e-6)
        if not case["backward"]:
            out.append(_turn(st, x * r * w).to(st[name].dtype))
            continue
        g = _turn(st, st["d" + name].float(), True)
        h = x * r
        u = g * w
        out.append((r * (u - h * (u * h).mean(-1, keepdim=True))).to(st[name].dtype))
        sums.append((g * h).sum((0, 1, 2), dtype=torch.float64).float())
    return tuple(out + sums)


def _tree(st):
    case, q = st["case"], st["q"]
    B, H, N, d = q.shape
    Hkv = case["Hkv"]
    lens = st["lens"].long()
    new = st["new"].long() if st["new"] is not None else torch.full_like(lens, N)
    phys = st["table"].long().clamp(min=0)
    T = phys.shape[1] * case["page"]
    tok = torch.arange(T, device=q.device)
    there = tok < lens[:, None]                                        # [B, T]

    def rows(name):
        x = st[name + "_codes"].view(torch.uint8)[phys].view(torch.float8_e4m3fn).float()
        x *= st[name + "_scale"][phys][..., None, None]
        return torch.where(there[:, None, :, None], x.transpose(1, 2).reshape(B, Hkv, T, d), 0.0)

    i = torch.arange(N, device=q.device)
    bits = (st["mask"][:, :, i // 32] >> (i % 32) & 1).bool()          # [B, N, N]: row i sees draft j
    draft = tok - (lens - new)[:, None]                                # [B, T]: the token's number among the drafts
    drafted = bits.gather(2, draft.clamp(0, N - 1)[:, None].expand(B, N, T))
    sees = there[:, None] & (i < new[:, None])[:, :, None] & ((draft < 0)[:, None] | drafted)
    S = q.float().reshape(B, Hkv, -1, d) @ rows("k").transpose(-1, -2)
    S = (S / math.sqrt(d)).reshape(B, H, N, T).masked_fill_(~sees[:, None], -math.inf)
    m = S.amax(-1, keepdim=True).clamp(min=-3e38)
    P = S.sub_(m).exp_()
    total = P.sum(-1, keepdim=True)
    O = (P.reshape(B, Hkv, -1, T) @ rows("v")).reshape(B, H, N, d) / total.clamp(min=1e-30)
    lse = torch.where(total > 0, m + total.log(), -math.inf)
    return O.to(q.dtype), lse[..., 0]


def _keep(st):
    case, page = st["case"], st["case"]["page"]
    lens, new, kept, keep = (st[k].long() for k in ("lens", "new", "kept", "keep"))
    K, table, dev = keep.shape[1], st["table"].long(), lens.device
    base = lens - new
    at = (base // page)[:, None] + torch.arange((K + page - 2) // page + 1, device=dev)     # [B, pages]
    used = (at <= (base + kept - 1)[:, None] // page) & (kept > 0)[:, None]
    to = table.gather(1, at.clamp(max=table.shape[1] - 1)).clamp(min=0)
    tok = at[..., None] * page + torch.arange(page, device=dev)        # [B, pages, page]
    i = tok - base[:, None, None]
    moved = (i >= 0) & (i < kept[:, None, None])
    src = torch.where(moved, base[:, None, None] + keep.gather(1, i.clamp(0, K - 1).flatten(1)).view_as(i), tok)
    src = src.clamp(0, table.shape[1] * page - 1)
    from_page = table.gather(1, (src // page).flatten(1)).view_as(src).clamp(min=0)
    put = moved | (i < 0)
    for name in ("k", "v"):
        codes, scales = st[name + "_codes"].view(torch.uint8), st[name + "_scale"]
        s = torch.where(put[..., None], scales[from_page], 0.0)        # [B, pages, page, Hkv]
        now = s.amax(2)                                                # [B, pages, Hkv]
        x = codes[from_page, :, src % page].view(torch.float8_e4m3fn).float()      # [B, pages, page, Hkv, d]
        x = (x * (s / now.clamp(min=1e-38)[:, :, None])[..., None]).to(torch.float8_e4m3fn).view(torch.uint8)
        x = torch.where(put[:, :, None, :, None], x.transpose(2, 3), codes[to])
        codes[to[used]] = x[used]
        scales[to[used]] = now[used]
    return (base + kept).int(), st["k_codes"], st["v_codes"], st["k_scale"], st["v_scale"]


def _fork(st):
    page, table, refs = st["case"]["page"], st["table"], st["refs"]
    parents, lens, reserve = st["parents"].long(), st["lens"].long(), st["reserve"].long()
    B, W = table.shape
    dev = table.device
    live = parents >= 0
    p = parents.clamp(min=0)
    L = torch.where(live, lens[p], 0)
    need = torch.where(live, (torch.maximum(L, reserve) + page - 1) // page, 0)
    b = torch.arange(B, device=dev)
    first = ~((parents[:, None] == parents) & (b[:, None] > b)).any(1)
    i = torch.arange(W, device=dev)
    old = torch.where(live[:, None], table[p].long(), -1)
    holders = refs.long()[old.clamp(min=0)]
    shared = i < (L // page)[:, None]
    place = i < need[:, None]
    stays = place & (shared | (first[:, None] & (old >= 0) & (holders == 1)))
    fresh = place & ~stays
    free = refs == 0
    rank = torch.where(free, free.long().cumsum(0) - 1, refs.shape[0])
    numbers = torch.full((refs.shape[0] + 1,), -1, dtype=torch.long, device=dev)
    numbers.scatter_(0, rank, torch.arange(refs.shape[0], device=dev))
    order = (fresh.flatten().long().cumsum(0) - 1).view_as(fresh).clamp(min=0)
    result = torch.where(stays, old, torch.where(fresh, numbers[order], -1))
    ones = torch.ones((), dtype=refs.dtype, device=dev)
    held = table.flatten()[table.flatten() >= 0].long()
    refs.index_add_(0, held, -ones.expand(len(held)))
    held = result.flatten()[result.flatten() >= 0]
    refs.index_add_(0, held, ones.expand(len(held)))
    # the tokens of pages that are not full
    copied = fresh & (i == (L // page)[:, None]) & (L % page > 0)[:, None]
    src, dst, rows = old[copied], result[copied], (L % page)[:, None].expand(B, W)[copied]
    takes = (torch.arange(page, device=dev) < rows[:, None])[:, None, :, None]
    for name in ("k", "v"):
        codes, scales = st[name + "_codes"].view(torch.uint8), st[name + "_scale"]
        codes[dst] = torch.where(takes, codes[src], codes[dst])
        scales[dst] = scales[src]
    table.copy_(result)
    return L.int(), table, refs, st["k_codes"], st["v_codes"], st["k_scale"], st["v_scale"]


def run(state):
    if own:
        return _own(state)
    return {"norm": _norm, "tree": _tree, "keep": _keep, "fork": _fork}[state["case"]["op"]](state)


# ------------------------------------------------------------------ in 64 bits
def _e4m3_values():
    """Code -> value: sign, 4 exponent bits (bias 7), 3 mantissa bits; 0x7f is NaN."""
    v = [(2.0 ** -6 * (m / 8) if e == 0 else 2.0 ** (e - 7) * (1 + m / 8)) for e in range(16) for m in range(8)]
    v[127] = math.nan
    return torch.tensor(v + [-x for x in v], dtype=torch.float64, device="cuda")


def _nearest_e4m3(x):
    v = _e4m3_values()[:127]
    mid = (v[1:] + v[:-1]) / 2
    up = torch.searchsorted(mid, x.abs().contiguous(), right=True)      # a tie goes up ...
    tie = (up > 0) & (x.abs() == mid[(up - 1).clamp(min=0)])
    up = torch.where(tie & (up % 2 == 1), up - 1, up)                   # ... unless the lower code is even
    return v[up] * torch.sign(x)


def _exact_norm(st):
    case = st["case"]
    P, d = case["rotated"] // 2, case["d"]
    cols = torch.arange(P, device="cuda")
    one, two = (2 * cols, 2 * cols + 1) if case["interleaved"] else (cols, cols + P)
    turn = None
    if P:
        pos = torch.stack([st["pos"][a].double() * w for a, w in zip(st["axis"], st["inv_freq"])], -1)   # [B, N, P]
        turn = torch.polar(torch.ones_like(pos), pos)
    out, sums = [], []
    for name in ("q", "k"):
        w = st["w" + name].double() + case["offset"]
        res = torch.empty(st[name].shape, dtype=torch.float64, device="cuda")
        dw = torch.zeros(d, dtype=torch.float64, device="cuda")
        for h in range(st[name].shape[1]):          # a head at a time
            x = st[name][:, h].double()             # [B, N, d]
            y = x / torch.linalg.vector_norm(torch.cat((x, torch.full_like(x[..., :1], math.sqrt(d * 1e-6))), -1),
                                             dim=-1, keepdim=True) * math.sqrt(d)
            r = 1.0 / torch.sqrt((x ** 2).sum(-1, keepdim=True) / d + 1e-6)
            if not case["backward"]:
                y = y * w
                if P:
                    z = torch.complex(y[..., one], y[..., two]) * turn
                    y[..., one], y[..., two] = z.real, z.imag
                res[:, h] = y
                continue
            g = st["d" + name][:, h].double()
            if P:
                z = torch.complex(g[..., one], g[..., two]) * turn.conj()
                g[..., one], g[..., two] = z.real, z.imag
            dw += torch.einsum("bnd,bnd->d", g, y)
            dot = torch.einsum("bnd,bnd,d->bn", g, x, w)
            res[:, h] = r * g * w - r ** 3 * x * dot[..., None] / d
        out.append(res)
        sums.append(dw)
    return tuple(out + sums) if case["backward"] else tuple(out)


def _exact_tree(st):
    case = st["case"]
    B, H, Hkv, d, page, N = (case[k] for k in ("B", "H", "Hkv", "d", "page", "n"))
    lens, new = _lengths(case)
    value = _e4m3_values()
    mask = st["mask"].tolist()
    O = torch.zeros(B, H, N, d, dtype=torch.float64, device="cuda")
    lse = torch.full((B, H, N), -math.inf, dtype=torch.float64, device="cuda")
    for b in range(B):
        ids = st["table"][b, :-(-lens[b] // page)].long()
        unseen = torch.zeros(new[b], lens[b], dtype=torch.bool)
        for i in range(new[b]):
            for j in range(new[b]):
                unseen[i, lens[b] - new[b] + j] = not (mask[b][i][j // 32] >> (j % 32)) & 1
        unseen = unseen.cuda()
        for h in range(Hkv):
            K, V = ((value[st[x + "_codes"][ids, h].view(torch.uint8).long()]
                     * st[x + "_scale"][ids, h].double()[:, None, None]).reshape(-1, d)[:lens[b]] for x in ("k", "v"))
            for head in range(h * (H // Hkv), (h + 1) * (H // Hkv)):
                S = st["q"][b, head, :new[b]].double() @ K.T / math.sqrt(d)
                S.masked_fill_(unseen, -math.inf)
                l = torch.logsumexp(S, -1)
                lse[b, head, :new[b]] = l
                O[b, head, :new[b]] = S.sub_(l[..., None]).exp_() @ V
    return O, lse


def _exact_keep(st):
    case, page = st["case"], st["case"]["page"]
    lens, new = _lengths(case)
    kept = _kept(case, new)
    table, keep = st["table"].tolist(), st["keep"].tolist()
    value = _e4m3_values()
    out = []
    for name in ("k", "v"):
        held, scale = value[st[name + "_codes"].view(torch.uint8).long()], st[name + "_scale"].double()
        held_now, scale_now = held.clone(), scale.clone()
        for b in range(case["B"]):
            base = lens[b] - new[b]
            end = base + kept[b]
            for number in range(base // page, -(-end // page)) if kept[b] else ():
                toks = range(number * page, min(end, (number + 1) * page))
                srcs = [t if t < base else base + keep[b][t - base] for t in toks]
                ids = torch.tensor([table[b][t // page] for t in srcs], device="cuda")
                rows = torch.tensor([t % page for t in srcs], device="cuda")
                s = scale[ids]                                         # [rows, Hkv]
                x, top = held[ids, :, rows], s.amax(0)
                p = table[b][number]
                held_now[p, :, :len(srcs)] = _nearest_e4m3(x * (s / top)[..., None]).transpose(0, 1)
                scale_now[p] = top
        out.append((held_now, scale_now))
    return (torch.tensor([t - n + a for t, n, a in zip(lens, new, kept)], dtype=torch.int32, device="cuda"),
            out[0][0], out[1][0], out[0][1], out[1][1])


def _exact_fork(st):
    page = st["case"]["page"]
    parents, lens, reserve, table, refs = (st[k].tolist() for k in ("parents", "lens", "reserve", "table", "refs"))
    free = [p for p, n in enumerate(refs) if n == 0]
    now, result, length, copies, taken = list(refs), [], [], [], set()
    for b, p in enumerate(parents):
        row, L = [-1] * len(table[b]), lens[p] if p >= 0 else 0
        for i in range(-(-max(L, reserve[b]) // page) if p >= 0 else 0):
            mine = p not in taken and table[p][i] >= 0 and refs[table[p][i]] == 1
            if i < L // page or mine:
                row[i] = table[p][i]
            else:
                row[i] = free.pop(0)
                if i == L // page and L % page:
                    copies.append((table[p][i], row[i], L % page))
            now[row[i]] += 1
        taken.add(p)
        result.append(row)
        length.append(L)
    for row in table:
        for page_held in row:
            if page_held >= 0:
                now[page_held] -= 1
    value = _e4m3_values()
    held = []
    for name in ("k", "v"):
        x, s = value[st[name + "_codes"].view(torch.uint8).long()], st[name + "_scale"].double()
        for src, dst, rows in copies:
            x[dst, :, :rows], s[dst] = x[src, :, :rows], s[src]
        held.append((x, s))

    def ints(v):
        return torch.tensor(v, dtype=torch.int32, device="cuda")

    return ints(length), ints(result), ints(now), held[0][0], held[1][0], held[0][1], held[1][1]


def exact(case, seed):
    global own
    was, own = own, False
    try:
        st = prepare(case, seed)
    finally:
        own = was
    return {"norm": _exact_norm, "tree": _exact_tree, "keep": _exact_keep, "fork": _exact_fork}[case["op"]](st)
