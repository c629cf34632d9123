"""fa_qk_norm_rope and its backward against the formulas in 64 bits and against
differences: types, layouts, weights, extremes, in place, outputs beside others,
the same bits every time, streams and graphs."""
import math

import pytest
import torch

import branch_ref as branch
import cache_ref as ref
from exact_io_aware_20_gb300 import binding

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
T = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def dev(x):
    """To the device, with the strides that it has."""
    if x is None:
        return None
    y = torch.empty_strided(x.shape, x.stride(), dtype=x.dtype, device=DEV)
    return y.copy_(x)


def rotation(pos, freq, axis, pairs):
    def turn(x, back):
        return ref.rotate(x, pos, freq, axis, pairs, back)
    return turn


def spread(x, rotated, interleaved):
    """|x1| + |x2| of rotated columns, |x| of the others."""
    return torch.where(ref.rotate_slack(x, rotated, interleaved) > 0, ref.rotate_slack(x, rotated, interleaved),
                       x.double().abs())


def check_forward(got, x, w, eps, offset, turn, pairs, interleaved):
    """One rounding, and in fp32: r from a sum of up to 256 squares (13 steps one
    after another, 2^-24 each, halved by the root) and rsqrt (2^-22), the weight
    with its offset, three products and a sum (2^-24 each), the angle (2^-23),
    sine and cosine (2^-23): below 2^-20 of r (|x1 w1| + |x2 w2|)."""
    x, f = x.double(), 1.0 if w is None else w.double() + offset
    r = 1.0 / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
    want = branch.norm(x, w, eps, offset, turn)
    bound = ref.half_step(got.dtype) * want.abs() * 1.001 + 2.0 ** -25 \
        + 2.0 ** -20 * spread(x * r * f, pairs, interleaved)
    err = (got.cpu().double() - want).abs()
    assert (err <= bound).all(), float((err - bound).max())


def check_backward(got, dw, dy, x, w, eps, offset, turn, pairs, interleaved, terms):
    """As above: u and h are off by 2^-20 of their parts; the mean of their
    products adds 13 steps of 2^-24, its product with h one: 2^-19 of
    r (|u| + |h| mean |u h|) together.  The weights' sums: each term 2^-20, and
    `terms` of a thread one after another, 3 + 8 + 10 + 5 more of partial sums."""
    x, f = x.double(), 1.0 if w is None else w.double() + offset
    r = 1.0 / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
    want, want_dw = branch.norm_backward(dy, x, w, eps, offset, turn)
    g = spread(dy, pairs, interleaved)
    u, h = g * (f if w is None else f.abs()), (x * r).abs()
    bound = ref.half_step(got.dtype) * want.abs() * 1.001 + 2.0 ** -25 \
        + 2.0 ** -19 * r * (u + h * (u * h).mean(-1, keepdim=True))
    err = (got.cpu().double() - want).abs()
    assert (err <= bound).all(), float((err - bound).max())
    if w is not None:
        assert dw.dtype == torch.float32
        bound = (2.0 ** -20 + (terms + 26) * 2.0 ** -24) * (g * h).sum((0, 1, 2)) + 2.0 ** -140
        err = (dw.cpu().double() - want_dw).abs()
        assert (err <= bound).all(), float((err - bound).max())


def run(dtype, wtype, B, H, Hkv, N, d, interleaved, part, axes, offset, seed=0, size=1.0, eps=1e-6, given=True):
    g = torch.Generator().manual_seed(seed + B * N + d + axes)
    pairs = 0 if part == 0 else d // 2 // part if part < 8 else part       # (8 and more: how many)
    freq = [10000.0 ** (-i / max(1, pairs)) for i in range(pairs)]
    axis = [i * axes // max(1, pairs) for i in range(pairs)]
    table = binding.Rope(freq, axis, interleaved) if pairs else None
    if given:
        pos = torch.randint(-300000, 3000000, (axes, B, N), generator=g, dtype=torch.int32)
    else:
        pos = torch.arange(N, dtype=torch.int32).expand(axes, B, N)

    def layout(i, heads):
        x = torch.randn(B, N, heads, d, generator=g) if i else torch.randn(B, heads, N, d, generator=g)
        x = (x * size).to(T[dtype])
        return x.transpose(1, 2) if i else x

    q, k = layout(1, H), layout(0, Hkv) if Hkv else None
    dq, dk = layout(0, H), layout(1, Hkv) if Hkv else None
    if wtype is None:
        wq = wk = None
    else:
        wq, wk = ((1 - offset + 0.3 * torch.randn(d, generator=g)).to(T[wtype]) for _ in range(2))
        if not Hkv:
            wk = None
    turn = rotation(pos, freq, axis, interleaved)
    p = pos.to(DEV) if given else None
    rest = (dev(q), dev(k), dev(wq), dev(wk), eps, p, table, offset)
    qo, ko = binding.qk_norm_rope(*rest)
    dqi, dki, dwq, dwk = binding.qk_norm_rope_backward(dev(dq), dev(dk), *rest)
    binding.device_status()
    assert (dwq is None) == (wq is None) and (dwk is None) == (wk is None)
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    units = -(-B * N * (d // 16) // 256) * (H + Hkv)
    terms = -(-units // min(2 * sms, units)) + 1
    check_forward(qo, q, wq, eps, offset, turn, pairs, interleaved)
    check_backward(dqi, dwq, dq, q, wq, eps, offset, turn, pairs, interleaved, terms)
    if Hkv:
        check_forward(ko, k, wk, eps, offset, turn, pairs, interleaved)
        check_backward(dki, dwk, dk, k, wk, eps, offset, turn, pairs, interleaved, terms)
    else:
        assert ko is None and dki is None


@pytest.mark.parametrize("dtype,wtype", [("bf16", "bf16"), ("bf16", "f32"), ("f16", "f16"), ("f16", "f32")])
@pytest.mark.parametrize("B,H,Hkv,N,d", [(1, 1, 1, 1, 64), (2, 6, 2, 37, 128), (3, 5, 5, 130, 256), (1, 33, 1, 9, 64)])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("part", [0, 1, 2])
def test_matches_the_formulas(dtype, wtype, B, H, Hkv, N, d, interleaved, part):
    run(dtype, wtype, B, H, Hkv, N, d, interleaved, part, 1, 0.0)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("Hkv", [0, 4])
@pytest.mark.parametrize("wtype,offset", [(None, 0.0), ("f16", 1.0), ("f32", 1.0)])
def test_axes_offsets_and_no_weights(d, Hkv, wtype, offset):
    run("f16", wtype, 2, 12, Hkv, 45, d, True, 1, 3, offset)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("d,pairs", [(64, 8), (64, 24), (128, 40), (128, 56), (256, 16), (256, 72), (256, 120)])
def test_part_of_each_row_turned(interleaved, d, pairs):
    run("bf16", "bf16", 2, 6, 2, 21, d, interleaved, pairs, 1, 0.0)


@pytest.mark.parametrize("d", [64, 128, 256])
def test_many_rows_and_positions_by_default(d):
    run("bf16", "bf16", 2, 7, 3, 1500, d, False, 1, 1, 0.0, given=False)


@pytest.mark.parametrize("dtype,size,eps", [
    ("bf16", 2.0 ** 100, 1e-6), ("bf16", 2.0 ** 66, 1e-6), ("bf16", 2.0 ** -50, 2.0 ** -99), ("bf16", 2.0 ** -90, 1e-6),
    ("f16", 2.0 ** 13, 1e-6), ("f16", 2.0 ** -14, 1e-5), ("bf16", 1.0, 1e4)])
@pytest.mark.parametrize("d", [64, 256])
def test_sizes_far_from_one(dtype, size, eps, d):
    """Squares of bf16 leave fp32 at 2^64; gradients are as large as the inputs here."""
    g = torch.Generator().manual_seed(d)
    q = (torch.randn(1, 3, 9, d, generator=g) * size).to(T[dtype])
    dy = torch.randn(1, 3, 9, d, generator=g).to(T[dtype])
    w = torch.rand(d, generator=g).add(0.5).to(T[dtype])
    turn = rotation(torch.zeros(1, 1, 9), [], [], False)
    qo, _ = binding.qk_norm_rope(dev(q), None, dev(w), None, eps)
    dx, _, dw, _ = binding.qk_norm_rope_backward(dev(dy), None, dev(q), None, dev(w), None, eps)
    check_forward(qo, q, w, eps, 0.0, turn, 0, False)
    # bf16 gradients of rows far above one may be below its smallest normal number
    want, want_dw = branch.norm_backward(dy, q, w, eps, 0.0, turn)
    if want.abs().max() < 1e38 and want.abs().max() > 2.0 ** -120 and want.abs().max() < torch.finfo(T[dtype]).max:
        check_backward(dx, dw, dy, q, w, eps, 0.0, turn, 0, False, 3)


def test_zeros_infinities_and_nan_stay_in_their_rows():
    g = torch.Generator().manual_seed(3)
    q = torch.randn(1, 2, 8, 128, generator=g).bfloat16()
    q[0, 0, 1] = 0
    q[0, 0, 2, 5] = math.inf
    q[0, 1, 3, 100] = math.nan
    w = torch.ones(128).bfloat16()
    qo, _ = binding.qk_norm_rope(dev(q), None, dev(w), None, 1e-6)
    qo = qo.cpu().float()
    assert (qo[0, 0, 1] == 0).all()
    # 1 / sqrt(inf) = 0: the row's finite values become 0, the infinity NaN
    assert qo[0, 0, 2, 5].isnan() and (qo[0, 0, 2, :5] == 0).all() and (qo[0, 0, 2, 6:] == 0).all()
    assert qo[0, 1, 3].isnan().all()
    rest = torch.ones(1, 2, 8, dtype=torch.bool)
    rest[0, 0, 2] = rest[0, 1, 3] = False
    assert qo[rest].isfinite().all()
    dx, _, dw, _ = binding.qk_norm_rope_backward(dev(torch.ones_like(q)), None, dev(q), None, dev(w), None, 1e-6)
    assert dx.cpu()[rest].isfinite().all() and dw.isnan().any()


def test_against_differences():
    """The derivative along a random direction of sum(dy o y), by the 64-bit
    formula: its gradient, and the kernel's, which has the roundings that
    check_backward allows."""
    g = torch.Generator().manual_seed(4)
    B, H, N, d = 2, 3, 7, 64
    x, dy = (torch.randn(B, H, N, d, generator=g).half() for _ in range(2))
    w = torch.rand(d, generator=g).add(0.5).half()
    freq = [10000.0 ** (-i / 16) for i in range(16)]
    pos = torch.randint(0, 1000, (1, B, N), generator=g, dtype=torch.int32)
    turn = rotation(pos, freq, [0] * 16, False)
    vx, vw = torch.randn(x.shape, generator=g).double(), torch.randn(d, generator=g).double()

    def value(t):
        return float((branch.norm(x.double() + t * vx, w.double() + t * vw, 1e-3, 0.0, turn) * dy.double()).sum())

    t = 1e-5
    slope = (value(t) - value(-t)) / (2 * t)
    dx, dw = branch.norm_backward(dy, x, w, 1e-3, 0.0, turn)
    exact = float((dx * vx).sum() + (dw * vw).sum())
    assert abs(exact - slope) <= 1e-6 * abs(exact) + 1e-6
    got = binding.qk_norm_rope_backward(dev(dy), None, dev(x), None, dev(w), None, 1e-3, pos.to(DEV),
                                        binding.Rope(freq))
    mine = float((got[0].cpu().double() * vx).sum() + (got[2].cpu().double() * vw).sum())
    # half a step of f16 an element, fp32 in the sums
    bound = 2.0 ** -11 * 1.01 * float((dx * vx).abs().sum()) + 2.0 ** -18 * float((vx.abs() * 8).sum() + (vw.abs() * 99).sum())
    assert abs(mine - slope) <= bound


@pytest.mark.parametrize("d", [64, 128])
def test_in_place_and_beside_other_data(d):
    g = torch.Generator().manual_seed(5)
    B, H, Hkv, N = 2, 5, 2, 33
    # q and k of one packed projection, [B, N, H + Hkv and a gap, d]
    buf = torch.randn(B, N, H + Hkv + 1, d, generator=g).bfloat16().to(DEV)
    grads = torch.randn(B, N, H + Hkv + 1, d, generator=g).bfloat16().to(DEV)
    w = [torch.rand(d, generator=g).to(DEV) for _ in range(2)]
    table = binding.Rope([10000.0 ** (-i / 32) for i in range(32)])

    def views(x):
        return x[:, :, :H].transpose(1, 2), x[:, :, H:H + Hkv].transpose(1, 2)

    (q, k), (dq, dk) = views(buf), views(grads)
    want = binding.qk_norm_rope(q.contiguous(), k.contiguous(), *w, 1e-5, None, table)
    back = binding.qk_norm_rope_backward(dq.contiguous(), dk.contiguous(), q.contiguous(), k.contiguous(), *w, 1e-5,
                                         None, table)
    for which in range(3):
        x, y = buf.clone(), grads.clone()
        (q, k), (dq, dk) = views(x), views(y)
        if which == 0:
            got = binding.qk_norm_rope(q, k, *w, 1e-5, None, table, q_out=q, k_out=k)
            want_now = want
        else:
            to = (dq, dk) if which == 1 else (q, k)
            got = binding.qk_norm_rope_backward(dq, dk, q, k, *w, 1e-5, None, table, dq=to[0], dk=to[1])
            want_now = back
        for a, b in zip(got, want_now):
            assert torch.equal(a, b)
        assert torch.equal(x[:, :, -1], buf[:, :, -1]) and torch.equal(y[:, :, -1], grads[:, :, -1])


def test_the_same_bits_every_time_and_in_two_graphs():
    g = torch.Generator().manual_seed(6)
    B, H, Hkv, N, d = 3, 9, 3, 700, 128
    table = binding.Rope([10000.0 ** (-i / 64) for i in range(64)])
    runs = []
    for i in range(2):
        q, k, dq, dk = (torch.randn(B, h, N, d, generator=g).bfloat16().to(DEV) for h in (H, Hkv, H, Hkv))
        w = [torch.rand(d, generator=g).to(DEV) for _ in range(2)]
        args = (dq, dk, q, k, *w, 1e-6, None, table)
        want = binding.qk_norm_rope_backward(*args)
        ws = torch.full((binding.qk_norm_rope_bwd_workspace_size(B, H, Hkv, N, d),), 0xFF, dtype=torch.uint8, device=DEV)
        for x, y in zip(binding.qk_norm_rope_backward(*args, workspace=ws), want):
            assert torch.equal(x, y)
        s, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            out = binding.qk_norm_rope_backward(*args)
        runs.append((graph, s, out, want, args))
    torch.cuda.synchronize()
    for _ in range(10):
        for graph, s, *_rest in runs:
            with torch.cuda.stream(s):
                graph.replay()
    torch.cuda.synchronize()
    for _graph, _s, out, want, _args in runs:
        for x, y in zip(out, want):
            assert torch.equal(x, y)


def test_on_a_stream_of_its_own():
    g = torch.Generator().manual_seed(7)
    q = torch.randn(2, 4, 300, 128, generator=g).bfloat16().to(DEV)
    w = torch.rand(128, generator=g).to(DEV)
    want = binding.qk_norm_rope(q, None, w, None, 1e-6)[0]
    back = binding.qk_norm_rope_backward(q, None, q, None, w, None, 1e-6)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(20):
        x = q.clone()
        torch.cuda.current_stream().synchronize()
        got = binding.qk_norm_rope(x, None, w, None, 1e-6, stream=s)[0]
        got_back = binding.qk_norm_rope_backward(x, None, x, None, w, None, 1e-6, stream=s)
        del x
        torch.full_like(q, 7.0)
        s.synchronize()
        assert torch.equal(got, want) and all(torch.equal(a, b) for a, b in zip(got_back, back) if b is not None)


def test_refusals_of_the_binding():
    q = torch.zeros(1, 2, 3, 64, dtype=torch.bfloat16, device=DEV)
    w = torch.zeros(64, dtype=torch.bfloat16, device=DEV)
    for bad in ((q, None, w, w), (q, q[:, :, :2], w, w), (q, None, w[:32], None), (q, q, w, w[::2]),
                (q.transpose(2, 3), None, w, None), (q, q.half(), w, w)):
        with pytest.raises(ValueError):
            binding.qk_norm_rope(*bad, 1e-6)
    for bad in ((q, None, w.half(), None), (q, q, w, w.float())):
        with pytest.raises(TypeError):
            binding.qk_norm_rope(*bad, 1e-6)
    with pytest.raises(binding.FaError):
        binding.qk_norm_rope(q, None, w, None, 0.0)
    with pytest.raises(ValueError):
        binding.qk_norm_rope_backward(q, None, q, None, None, None, 1e-6, dq_weight=w.float())
    with pytest.raises(ValueError):
        binding.qk_norm_rope_backward(q, None, q, None, w, None, 1e-6, dq_weight=w)
