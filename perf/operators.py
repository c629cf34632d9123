"""The operators around the attention kernels: rotary positions on one or
several axes, appending to a paged 8-bit key/value cache, and attention over
that cache; each in a plain form and through the library.

Definitions.  Rotary: pair p of a row at position t (of the pair's axis) turns
by the angle t * w_p; the pairs are columns (p, p + P) of the first 2P columns,
or (2p, 2p + 1) when interleaved; the backward turns the other way.  Cache:
pages of `page` tokens, e4m3 codes with one scale for each (page, head), a
power of two: the smallest 2^e >= 2^-100 with max |x| <= 448 * 2^e over the
tokens being added to the page, but no smaller than the scale of tokens that
are in the page already, whose codes are rounded again when it grows.  The
table maps token t of sequence b to page table[b][t // page], row t % page;
seq_lens counts the new tokens too.  Attention: softmax(scale * q k^T) v over
a sequence's tokens; causal: row i of n new ones sees tokens <= len - n + i.
Rows behind a sequence's new tokens are O = 0, L = -inf, and their q is 0.
"""
import math

import torch

own = False
LIMIT = 448.0          # the largest e4m3 value
MIN_SCALE = 2.0 ** -100


# ------------------------------------------------------------------ cases
def listed():
    return [
        # training, the repository's gqa8k layer: q and k of a projection's [B, N, H, d] layout
        {"name": "rope gqa8k", "op": "rope", "B": 2, "H": 32, "Hkv": 8, "N": 8192, "d": 128, "dtype": "bf16",
         "axes": 1, "interleaved": False, "rotated": 128, "backward": False},
        # training on video tokens: gradients through three axes (time, height, width), interleaved pairs
        {"name": "rope video backward", "op": "rope", "B": 1, "H": 16, "Hkv": 16, "N": 4099, "d": 64, "dtype": "f16",
         "axes": 3, "interleaved": True, "rotated": 64, "backward": True},
        # a verification step of a few tokens, part of each row rotated: the latency of a call
        {"name": "rope few tokens", "op": "rope", "B": 4, "H": 32, "Hkv": 8, "N": 5, "d": 128, "dtype": "bf16",
         "axes": 1, "interleaved": False, "rotated": 64, "backward": False},
        # one token of each running sequence, while serving
        {"name": "append token", "op": "append", "B": 64, "H": 32, "Hkv": 8, "N": 1, "before": 1000, "d": 128,
         "dtype": "bf16", "page": 64, "axes": 1, "interleaved": False, "rotated": 128, "padded": False},
        # prompts, some with a cached prefix that ends inside a page
        {"name": "append prompts", "op": "append", "B": 4, "H": 32, "Hkv": 8, "N": 4099, "before": 300, "d": 128,
         "dtype": "bf16", "page": 64, "axes": 1, "interleaved": False, "rotated": 128, "padded": False},
        # a padded batch of image prompts, three axes, small pages
        {"name": "append padded images", "op": "append", "B": 6, "H": 16, "Hkv": 16, "N": 333, "before": 50, "d": 64,
         "dtype": "f16", "page": 16, "axes": 3, "interleaved": True, "rotated": 64, "padded": True},
        # one short conversation: the latency of a call
        {"name": "attend one", "op": "attend", "B": 1, "H": 32, "Hkv": 8, "Nq": 1, "L": 1000, "d": 128, "dtype": "bf16",
         "page": 64, "causal": True, "ragged": False},
        # the benchmark's decode batch, in this form of cache
        {"name": "attend batch", "op": "attend", "B": 8, "H": 32, "Hkv": 8, "Nq": 1, "L": 8192, "d": 128,
         "dtype": "bf16", "page": 64, "causal": True, "ragged": False},
        # long documents of unlike lengths
        {"name": "attend long", "op": "attend", "B": 4, "H": 32, "Hkv": 8, "Nq": 1, "L": 131072, "d": 128,
         "dtype": "bf16", "page": 128, "causal": True, "ragged": True},
        # a chunk of each prompt against what is cached of it
        {"name": "attend chunk", "op": "attend", "B": 2, "H": 32, "Hkv": 8, "Nq": 512, "L": 16384, "d": 128,
         "dtype": "bf16", "page": 64, "causal": True, "ragged": True},
        # a whole prompt at the repository's head256 sizes
        {"name": "attend prompt d256", "op": "attend", "B": 4, "H": 8, "Hkv": 8, "Nq": 4096, "L": 4096, "d": 256,
         "dtype": "f16", "page": 32, "causal": True, "ragged": False},
        # a whole serving step of a ragged batch: append one token of each sequence, attend
        {"name": "step", "op": "step", "B": 32, "H": 32, "Hkv": 8, "N": 1, "before": 4095, "d": 128, "dtype": "bf16",
         "page": 64, "axes": 1, "interleaved": False, "rotated": 128, "padded": False},
    ]


def _spread(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["rope", "append", "attend", "attend", "step"])
    d = rng.choice([64, 128, 128, 256])
    Hkv = rng.choice([1, 2, 4, 8, 16])
    H = Hkv * rng.choice([g for g in (1, 2, 3, 4, 7, 8, 16) if Hkv * g <= 32])
    c = {"op": op, "B": 1, "H": H, "Hkv": Hkv, "d": d, "dtype": rng.choice(["bf16", "bf16", "f16"])}
    rope = {"axes": rng.choice([1, 1, 2, 3]), "interleaved": rng.random() < 0.4,
            "rotated": rng.choice([d, d, d // 2])}
    page = rng.choice([16, 32, 64, 64, 128, 256])
    if op == "rope":
        tokens = _spread(rng, 1, min(16384, 2 * 8192 * 40 * 128 // ((H + Hkv) * d)))
        c["B"] = _spread(rng, 1, min(64, tokens))
        return {**c, "N": max(1, tokens // c["B"]), **rope, "backward": rng.random() < 0.5}
    if op == "append":
        tokens = _spread(rng, 1, min(16384, 4 * 4099 * 48 * 128 // ((H + 2 * Hkv) * d)))
        c["B"] = _spread(rng, 1, min(128, tokens))
        return {**c, "N": max(1, tokens // c["B"]), "before": _spread(rng, 1, 2000) - 1, "page": page, **rope,
                "padded": rng.random() < 0.5}
    if op == "step":
        keys = _spread(rng, 16, 32 * 4096 * 8 * 128 // (Hkv * d))
        c["B"] = _spread(rng, 1, min(128, keys // 16))
        N = rng.choice([1, 1, 1, 2, 5])
        return {**c, "N": N, "before": max(0, min(131072, keys // c["B"]) - N), "page": page, **rope, "padded": N > 1}
    kind = rng.random()
    pairs = 2 * 512 * 16384 * 32 * 128 // (H * d)      # of a query and a key, for each head
    Nq = 1 if kind < 0.45 else _spread(rng, 2, 16) if kind < 0.65 else _spread(rng, 17, min(4096, math.isqrt(pairs)))
    keys = _spread(rng, 64, min(4 * 131072 * 8 * 128 // (Hkv * d), max(64, pairs // Nq)))
    c["B"] = _spread(rng, 1, max(1, min(128, keys // max(64, Nq))))
    return {**c, "Nq": Nq, "L": max(Nq, min(131072, keys // c["B"])), "page": page,
            "causal": rng.random() < 0.8, "ragged": rng.random() < 0.6}


def _fractions(B):
    """A fixed uneven spread over (0, 1], the first sequence whole."""
    return [1.0 if b == 0 else (b * 0.6180339887498949) % 1.0 for b in range(B)]


def _lengths(case):
    """(tokens in the cache, the new ones among them) of each sequence."""
    B = case["B"]
    if case["op"] == "attend":
        n = [case["Nq"]] * B
        if not case["ragged"]:
            return [case["L"]] * B, n
        return [max(case["Nq"], int(case["L"] * f)) for f in _fractions(B)], n
    n = [max(1, int(case["N"] * f)) for f in _fractions(B)] if case["padded"] else [case["N"]] * B
    return [int(case["before"] * f) + k for f, k in zip(_fractions(B), n)], n


# ------------------------------------------------------------------ work
def _attend_work(case, lens, new, Nq, causal):
    H, Hkv, d = case["H"], case["Hkv"], case["d"]
    pairs = sum(n * t - (n * (n - 1) // 2 if causal else 0) for t, n in zip(lens, new))
    return {"bytes": sum(2 * t * Hkv * d + 8 * Hkv * -(-t // case["page"]) for t in lens)
            + case["B"] * H * Nq * (4 * d + 4), "flops": 4.0 * H * d * pairs}


def work(case):
    B, H, Hkv, d = (case[k] for k in ("B", "H", "Hkv", "d"))
    if case["op"] == "rope":
        return {"bytes": B * case["N"] * (4 * (H + Hkv) * d + 4 * case["axes"]),
                "flops": 3.0 * B * case["N"] * (H + Hkv) * case["rotated"]}
    lens, new = _lengths(case)
    if case["op"] == "attend":
        return _attend_work(case, lens, new, case["Nq"], case["causal"])
    # the new tokens' q, k and v read, q written, the codes and scales written
    tokens = sum(new)
    w = {"bytes": tokens * (4 * H * d + 4 * Hkv * d + 2 * Hkv * d + 4 * case["axes"])
         + 8 * Hkv * sum((t - 1) // case["page"] - (t - n) // case["page"] + 1 for t, n in zip(lens, new)),
         "flops": 3.0 * tokens * (H + Hkv) * case["rotated"]}
    if case["op"] == "append":
        return w
    a = _attend_work(case, lens, new, case["N"], True)
    return {k: w[k] + a[k] for k in w}


# ------------------------------------------------------------------ inputs
def _dtype(case):
    return torch.float16 if case["dtype"] == "f16" else torch.bfloat16


def _quantise(x):
    """(codes, scales) of whole pages [..., rows, d]."""
    amax = x.abs().amax((-1, -2))
    mant, exp = torch.frexp(amax)                      # amax = mant * 2^exp, mant in [1/2, 1)
    e = torch.where(mant <= 0.875, exp - 9, exp - 8)   # 448 = 0.875 * 2^9
    s = torch.ldexp(torch.ones_like(amax), e.clamp(min=-100))
    return (x / s[..., None, None]).to(torch.float8_e4m3fn), s


def prepare(case, seed):
    dev, dt = "cuda", _dtype(case)
    g = torch.Generator(device=dev).manual_seed(seed)
    B, H, Hkv, d, op = (case[k] for k in ("B", "H", "Hkv", "d", "op"))

    def projected(heads, N):   # a projection's output [B, N, heads, d], seen as [B, heads, N, d]
        return torch.randn(B, N, heads, d, generator=g, device=dev).to(dt).transpose(1, 2)

    st = {"case": case}
    N = case["Nq"] if op == "attend" else case["N"]
    st["q"] = projected(H, N)
    if op != "attend":
        st["k"], axes = projected(Hkv, N), case["axes"]
        pairs = case["rotated"] // 2
        st["inv_freq"] = [10000.0 ** (-i / pairs) for i in range(pairs)]
        st["axis"] = [i * axes // pairs for i in range(pairs)]
        start = int(torch.randint(0, 100000, (1,), generator=g, device=dev))
        t = torch.arange(N, device=dev)
        if axes > 1:      # rows of a grid of frames
            side = max(1, round(N ** (1 / 3)))
            t = torch.stack([t // (side * side), t // side % side, t % side][3 - axes:])
        st["pos"] = (t.reshape(axes, 1, N) + start).expand(axes, B, N).to(torch.int32).contiguous()
    if op != "rope":
        lens, new = _lengths(case)
        page = case["page"]
        need = [max(1, -(-t // page)) for t in lens]
        pages = sum(need) + 3
        order = torch.randperm(pages, generator=g, device=dev)
        table = torch.full((B, max(need)), -1, dtype=torch.int32)
        rows = torch.split(order[:sum(need)].to(torch.int32).cpu(), need)
        for b in range(B):
            table[b, :need[b]] = rows[b]
        st["table"] = table.to(dev)
        st["lens"] = torch.tensor(lens, dtype=torch.int32, device=dev)
        ragged = op != "attend" and case["padded"]
        st["new"] = torch.tensor(new, dtype=torch.int32, device=dev) if ragged else None
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
        if op != "attend":
            st["v"] = projected(Hkv, N)
    if own:
        from exact_io_aware_20_gb300 import binding
        if op != "attend":
            st["rope"] = binding.Rope(st["inv_freq"], st["axis"], case["interleaved"])
        if op != "rope":
            st["cache"] = binding.Cache(st["k_codes"], st["v_codes"], st["k_scale"], st["v_scale"], st["table"])
    return st


# ------------------------------------------------------------------ the framework's calls
def _own(st):
    from exact_io_aware_20_gb300 import binding
    case = st["case"]
    op = case["op"]
    if op == "rope":
        call = binding.rope_backward if case["backward"] else binding.rope
        return call(st["q"], st["k"], st["pos"], st["rope"])
    scale = 1.0 / math.sqrt(case["d"])
    if op == "attend":
        return binding.forward_cache(st["q"], st["cache"], st["lens"], case["causal"], scale)
    q = binding.cache_append(st["cache"], st["q"], st["k"], st["v"], st["lens"], new_lens=st["new"],
                             rope=st["rope"], positions=st["pos"])
    state = (st["k_codes"], st["v_codes"], st["k_scale"], st["v_scale"])
    if op == "append":
        return (q,) + state
    return binding.forward_cache(q, st["cache"], st["lens"], True, scale, new_lens=st["new"]) + state


# ------------------------------------------------------------------ plain forms
def _turn(st, x, back=False):
    """The rotation, in 32 bits; the angles in 64."""
    case = st["case"]
    P = case["rotated"] // 2
    w = torch.tensor(st["inv_freq"], dtype=torch.float64, device=x.device)
    axis = torch.tensor(st["axis"], device=x.device)
    angle = (st["pos"].double()[axis] * w[:, None, None]).permute(1, 2, 0)[:, None]     # [B, 1, N, P]
    c, s = angle.cos().float(), angle.sin().float()
    s = -s if back else s
    x = x.float()
    if case["interleaved"]:
        a, b = x[..., 0:2 * P:2], x[..., 1:2 * P:2]
        turned = torch.stack((a * c - b * s, b * c + a * s), -1).flatten(-2)
    else:
        a, b = x[..., :P], x[..., P:2 * P]
        turned = torch.cat((a * c - b * s, b * c + a * s), -1)
    return torch.cat((turned, x[..., 2 * P:]), -1)


def _store(st, name, x):
    """Adds the rows x [B, Hkv, N, d] (32 bits) to the cache's codes and scales of `name`, in place."""
    case, page = st["case"], st["case"]["page"]
    codes, scales = st[name + "_codes"].view(torch.uint8), st[name + "_scale"]
    B, Hkv, N, d = x.shape
    lens = st["lens"].long()
    new = st["new"].long() if st["new"] is not None else torch.full_like(lens, N)
    first = (lens - new) // page                                     # the window's first page of each sequence
    span = (N + page - 2) // page + 1
    at = first[:, None] + torch.arange(span, device=x.device)        # [B, span] page numbers
    used = at <= (lens[:, None] - 1) // page
    phys = st["table"].long().gather(1, at.clamp(max=st["table"].shape[1] - 1)).clamp(min=0)
    tok = at[..., None] * page + torch.arange(page, device=x.device)   # [B, span, page] token numbers
    row = tok - (lens - new)[:, None, None]                            # of x
    fresh = (row >= 0) & (row < new[:, None, None])
    fresh = fresh[:, :, None, :, None]
    take = row.clamp(0, N - 1).reshape(B, 1, span * page, 1).expand(B, Hkv, span * page, d)
    rows = x.gather(2, take).reshape(B, Hkv, span, page, d).transpose(1, 2)       # [B, span, Hkv, page, d]
    amax = torch.where(fresh, rows.abs(), 0.0).amax((-1, -2))
    mant, exp = torch.frexp(amax)
    s = torch.ldexp(torch.ones_like(amax), torch.where(mant <= 0.875, exp - 9, exp - 8).clamp(min=-100))
    kept = (row < 0)[:, :, None, :, None]                              # tokens that are there already
    was = torch.where(kept[..., 0].any(-1), scales[phys], MIN_SCALE)   # [B, span, Hkv]
    s = torch.maximum(s, was)
    old = codes[phys]                                                  # [B, span, Hkv, page, d]
    again = old.view(torch.float8_e4m3fn).float() * (was / s)[..., None, None]
    put = torch.where(fresh, rows / s[..., None, None], again).to(torch.float8_e4m3fn).view(torch.uint8)
    put = torch.where(fresh | kept, put, old)
    codes[phys[used]] = put[used]
    scales[phys[used]] = s[used]


def _attend(st, q, causal):
    case = st["case"]
    B, H, N, d = q.shape
    Hkv, W = case["Hkv"], st["table"].shape[1]
    lens = st["lens"].long()
    new = st["new"].long() if st.get("new") is not None else torch.full_like(lens, N)
    phys = st["table"].long().clamp(min=0)
    T = W * case["page"]
    tok = torch.arange(T, device=q.device)
    there = tok < lens[:, None]                                        # [B, T]

    def rows(name):
        x = st[name + "_codes"].view(torch.uint8)[phys].view(torch.float8_e4m3fn).float()
        x *= st[name + "_scale"][phys][..., None, None]
        return torch.where(there[:, None, :, None], x.transpose(1, 2).reshape(B, Hkv, T, d), 0.0)

    i = torch.arange(N, device=q.device)
    sees = there[:, None] & (i < new[:, None])[:, :, None]             # [B, N, T]
    if causal:
        sees = sees & (tok <= ((lens - new)[:, None] + i)[:, :, None])
    S = q.float().reshape(B, Hkv, -1, d) @ rows("k").transpose(-1, -2)
    S = (S / math.sqrt(d)).reshape(B, H, N, T).masked_fill_(~sees[:, None], -math.inf)
    m = S.amax(-1, keepdim=True).clamp(min=-3e38)
    P = S.sub_(m).exp_()
    total = P.sum(-1, keepdim=True)
    O = (P.reshape(B, Hkv, -1, T) @ rows("v")).reshape(B, H, N, d) / total.clamp(min=1e-30)
    lse = torch.where(total > 0, m + total.log(), -math.inf)
    return O.to(q.dtype), lse[..., 0]


def run(state):
    if own:
        return _own(state)
    case, st = state["case"], state
    op = case["op"]
    if op == "rope":
        return tuple(_turn(st, st[n], case["backward"]).to(st[n].dtype) for n in ("q", "k"))
    if op == "attend":
        return _attend(st, st["q"], case["causal"])
    q = _turn(st, st["q"]).to(st["q"].dtype)
    if st["new"] is not None:      # rows behind a sequence's new tokens
        q = torch.where((torch.arange(case["N"], device=q.device) < st["new"][:, None])[:, None, :, None], q, 0)
    _store(st, "k", _turn(st, st["k"]))
    _store(st, "v", st["v"].float())
    out = (st["k_codes"], st["v_codes"], st["k_scale"], st["v_scale"])
    return (q,) + out if op == "append" else _attend(st, q, True) + out


# ------------------------------------------------------------------ in 64 bits
def _e4m3_values(dev):
    """Code -> value: sign, 4 exponent bits (bias 7), 3 mantissa bits; 0x7f is NaN."""
    v = [(2.0 ** -6 * (m / 8) if e == 0 else 2.0 ** (e - 7) * (1 + m / 8)) for e in range(16) for m in range(8)]
    v[127] = math.nan
    return torch.tensor(v + [-x for x in v], dtype=torch.float64, device=dev)


def _nearest_e4m3(x):
    v = _e4m3_values(x.device)[:127]
    mid = (v[1:] + v[:-1]) / 2
    up = torch.searchsorted(mid, x.abs().contiguous(), right=True)      # a tie goes up ...
    tie = (up > 0) & (x.abs() == mid[(up - 1).clamp(min=0)])
    up = torch.where(tie & (up % 2 == 1), up - 1, up)                   # ... unless the lower code is even
    return v[up] * torch.sign(x)


def _exact_turn(st, x, back):
    case = st["case"]
    P = case["rotated"] // 2
    pos = torch.stack([st["pos"][a].double() * w for a, w in zip(st["axis"], st["inv_freq"])], -1)   # [B, N, P]
    turn = torch.polar(torch.ones_like(pos), -pos if back else pos)[:, None]
    x = x.double()
    y = x.clone()
    cols = torch.arange(P, device=x.device)
    one, two = (2 * cols, 2 * cols + 1) if case["interleaved"] else (cols, cols + P)
    z = torch.complex(x[..., one], x[..., two]) * turn
    y[..., one], y[..., two] = z.real, z.imag
    return y


def exact(case, seed):
    global own
    was, own = own, False
    try:
        st = prepare(case, seed)
    finally:
        own = was
    op = case["op"]
    if op == "rope":
        return tuple(_exact_turn(st, st[n], case["backward"]) for n in ("q", "k"))
    B, H, Hkv, d, page = (case[k] for k in ("B", "H", "Hkv", "d", "page"))
    lens, new = _lengths(case)
    table = st["table"].tolist()
    value = _e4m3_values("cuda")
    held, scale = {}, {}
    q = st["q"].double()
    for name in ("k", "v"):
        held[name], scale[name] = st[name + "_codes"], st[name + "_scale"].double()
    if op != "attend":
        q = _exact_turn(st, st["q"], False)
        fresh = {"k": _exact_turn(st, st["k"], False), "v": st["v"].double()}
        for name in ("k", "v"):
            # e4m3 codes as values: exact in 64 bits
            held[name] = value[held[name].view(torch.uint8).long()]
            for b in range(B):
                t = lens[b] - new[b]
                while t < lens[b]:
                    p, r = table[b][t // page], t % page
                    n = min(page - r, lens[b] - t)
                    i = t - (lens[b] - new[b])
                    rows = fresh[name][b, :, i:i + n]                       # [Hkv, n, d]
                    amax = rows.abs().amax((-1, -2))
                    e = torch.ceil(torch.log2(amax / LIMIT))
                    e = torch.where(amax > LIMIT * torch.exp2(e), e + 1, e)
                    e = torch.where(amax <= LIMIT * torch.exp2(e - 1), e - 1, e)
                    s = torch.exp2(e).clamp(min=MIN_SCALE)
                    if r:
                        s = torch.maximum(s, scale[name][p])
                        held[name][p, :, :r] = _nearest_e4m3(held[name][p, :, :r]
                                                             * (scale[name][p] / s)[:, None, None])
                    held[name][p, :, r:r + n] = _nearest_e4m3(rows / s[:, None, None])
                    scale[name][p] = s
                    t += n
    state = ()
    if op != "attend":
        state = (held["k"], held["v"], scale["k"], scale["v"])
    if op == "append":
        if case["padded"]:
            for b in range(B):
                q[b, :, new[b]:] = 0
        return (q,) + state
    if op == "step":
        q = q.to(_dtype(case)).double()     # the step hands q on in its own type
    N = q.shape[2]
    causal = op == "step" or case["causal"]
    O = torch.zeros(B, H, N, d, dtype=torch.float64, device="cuda")
    lse = torch.full((B, H, N), -math.inf, dtype=torch.float64, device="cuda")
    for b in range(B):
        ids = st["table"][b, :-(-lens[b] // page)].long()
        for h in range(Hkv):
            def of(name):
                x = held[name][ids, h]
                x = x if x.dtype == torch.float64 else value[x.view(torch.uint8).long()]
                return (x * scale[name][ids, h][:, None, None]).reshape(-1, d)[:lens[b]]
            K, V = of("k"), of("v")
            mine = slice(h * (H // Hkv), (h + 1) * (H // Hkv))
            S = q[b, mine, :new[b]] @ K.T / math.sqrt(d)
            if causal:
                i = torch.arange(new[b], device="cuda")[:, None] + lens[b] - new[b]
                S.masked_fill_(torch.arange(lens[b], device="cuda") > i, -math.inf)
            l = torch.logsumexp(S, -1)
            lse[b, mine, :new[b]] = l
            O[b, mine, :new[b]] = S.sub_(l[..., None]).exp_() @ V
    return (O, lse) + state
