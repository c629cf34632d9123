"""fa_rope against the rotation in 64 bits: layouts, axes, pair orders, far and
negative positions, in place, and the backward against the formula and
differences."""
import math

import pytest
import torch

import cache_ref as ref
from exact_io_aware_20_gb300 import binding

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
T = {"bf16": torch.bfloat16, "f16": torch.float16}


def freqs(pairs, base=10000.0):
    return [base ** (-i / pairs) for i in range(pairs)]


def check(got, x, pos, freq, axis, interleaved, back):
    want = ref.rotate(x, pos, freq, axis, interleaved, back)
    # one rounding of the result; angles, sines and the sum in fp32: 2^-21 of
    # |x1| + |x2| (angle 2^-23, sine and cosine 2^-23, products and sum 2^-23);
    # results below f16's normal range round to 2^-25
    bound = ref.half_step(x.dtype) * want.abs() * 1.001 + 2.0 ** -25 \
        + 2.0 ** -21 * ref.rotate_slack(x, len(freq), interleaved)
    err = (got.cpu().double() - want).abs()
    assert (err <= bound).all(), float((err - bound).max())


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("B,H,Hkv,N,d", [(1, 1, 1, 1, 64), (2, 6, 2, 37, 128), (3, 5, 5, 130, 256),
                                         (1, 33, 1, 9, 64), (2, 32, 8, 257, 128)])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("part", [1, 2])
@pytest.mark.parametrize("axes", [1, 3])
def test_matches_the_rotation(dtype, B, H, Hkv, N, d, interleaved, part, axes):
    g = torch.Generator().manual_seed(B * N + d + axes)
    pairs = d // 2 // part
    freq, axis = freqs(pairs), [i * axes // pairs for i in range(pairs)]
    table = binding.Rope(freq, axis, interleaved)
    q = torch.randn(B, H, N, d, generator=g).to(T[dtype])
    k = torch.randn(B, N, Hkv, d, generator=g).to(T[dtype]).transpose(1, 2)   # a projection's layout
    pos = torch.randint(-300000, 3000000, (axes, B, N), generator=g, dtype=torch.int32)
    for back in (False, True):
        call = binding.rope_backward if back else binding.rope
        qo, ko = call(q.to(DEV), k.to(DEV), pos.to(DEV), table)
        check(qo, q, pos, freq, axis, interleaved, back)
        check(ko, k, pos, freq, axis, interleaved, back)


def test_far_positions_keep_their_angle():
    """At 2^31 - 1 an fp32 product of position and frequency is off by whole turns."""
    freq = freqs(32)
    table = binding.Rope(freq)
    q = torch.randn(1, 2, 4, 64, generator=torch.Generator().manual_seed(1)).half()
    pos = torch.tensor([[2 ** 31 - 1, -2 ** 31, 2 ** 30 + 1, 0]], dtype=torch.int32)
    qo, _ = binding.rope(q.to(DEV), None, pos.to(DEV), table)
    check(qo, q, pos[None], freq, [0] * 32, False, False)
    assert torch.equal(qo[:, :, 3].cpu(), q[:, :, 3])


def test_positions_shared_default_and_frequencies_beyond_a_turn():
    g = torch.Generator().manual_seed(3)
    q, k = (torch.randn(2, h, 19, 64, generator=g).bfloat16() for h in (4, 2))
    freq = [2 * math.pi * 3 + 0.25, -1.5] + freqs(6)
    table = binding.Rope(freq)
    rows = torch.arange(19, dtype=torch.int32)
    a = binding.rope(q.to(DEV), k.to(DEV), None, table)
    b = binding.rope(q.to(DEV), k.to(DEV), rows[None].to(DEV), table)
    c = binding.rope(q.to(DEV), k.to(DEV), rows.expand(2, 19).contiguous().to(DEV), table)
    for x in (b, c):
        assert torch.equal(a[0], x[0]) and torch.equal(a[1], x[1])
    check(a[0], q, rows.expand(1, 2, 19), freq, [0] * 8, False, False)


def test_in_place_views_and_rows_left_alone():
    """q and k inside one packed buffer, rotated in place: v stays as it is."""
    g = torch.Generator().manual_seed(4)
    qkv = torch.randn(2, 50, 3, 4, 128, generator=g).half().to(DEV)
    kept = qkv.clone()
    table = binding.Rope(freqs(64), interleaved=True)
    q, k = qkv[:, :, 0].transpose(1, 2), qkv[:, :, 1].transpose(1, 2)
    want = binding.rope(q, k, None, table)
    got = binding.rope(q, k, None, table, q_out=q, k_out=k)
    assert got[0] is q and torch.equal(q, want[0]) and torch.equal(k, want[1])
    assert torch.equal(qkv[:, :, 2], kept[:, :, 2])


def test_backward_against_differences():
    """<dq, u> is the slope of <rope(q), dq_out> along u (a linear map: exact up to rounding)."""
    g = torch.Generator().manual_seed(5)
    table = binding.Rope(freqs(32), [i % 3 for i in range(32)], True)
    pos = torch.randint(0, 5000, (3, 1, 33), generator=g, dtype=torch.int32).to(DEV)
    q, u, dout = (torch.randn(1, 4, 33, 128, generator=g).half().to(DEV) for _ in range(3))
    dq, _ = binding.rope_backward(dout, None, pos, table)
    up = binding.rope((q.float() + u.float()).half(), None, pos, table)[0].double()
    down = binding.rope((q.float() - u.float()).half(), None, pos, table)[0].double()
    slope = float(((up - down) / 2 * dout.double()).sum())
    size = float((u.double().abs() * dq.double().abs()).sum())
    # every value is rounded to f16 three times (inputs, outputs, dq), of size
    # up to |q| + |u| <= 3 |u| in the mean: 6 * 2^-11 of the sum of magnitudes
    assert abs(slope - float((u.double() * dq.double()).sum())) <= 6 * 2.0 ** -11 * 3 * size


def test_in_a_graph_and_on_a_stream():
    table = binding.Rope(freqs(64))
    q, k = (torch.randn(2, h, 64, 128, device=DEV).bfloat16() for h in (8, 2))
    pos = torch.arange(64, dtype=torch.int32, device=DEV)[None].clone()
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    on_stream = binding.rope(q, k, pos, table, stream=s)
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = binding.rope(q, k, pos, table)
    pos += 100
    graph.replay()
    later = binding.rope(q, k, pos, table)
    torch.cuda.synchronize()
    assert torch.equal(out[0], later[0]) and torch.equal(out[1], later[1])
    pos -= 100
    now = binding.rope(q, k, pos, table)
    assert torch.equal(on_stream[0], now[0]) and torch.equal(on_stream[1], now[1])
