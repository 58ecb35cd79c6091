"""Norm and rotation of query and key heads (moe_head_norm_rope) against the formula in 64 bits. Tolerances count roundings:
decode_ref.rope says which, and the result's own rounding to its type comes on top."""
import math

import numpy as np
import pytest
import torch

import decode_ref as R
import kv8_ref as K

pytestmark = pytest.mark.gpu

#: half an ulp, relative, and the least step (of subnormals), halved
HALF, LEAST = K.HALF_ULP, {"f32": 2.0 ** -150, "f16": 2.0 ** -25, "bf16": 2.0 ** -134}


@pytest.fixture(scope="module")
def m():
    import quantized_routed_expert_grouped_gb300 as mod
    mod.lib()
    return mod


def rows(g, N, H, D, dtype, layout="dense"):
    x = (torch.randn((N, H, D), generator=g) * torch.exp(torch.randn((N, H, 1), generator=g))).to(K.TYPES[dtype])
    if layout == "dense":
        return x.cuda()
    if layout == "fused":  # heads of one projection's rows
        buf = torch.full((N, H + 5, D), float("nan"), dtype=x.dtype, device="cuda")
        y = buf[:, 2:2 + H]
    elif layout == "odd":  # rows that no vector access may touch
        buf = torch.full((N, H, D + 1), float("nan"), dtype=x.dtype, device="cuda")
        y = buf[:, :, 1:]
    else:                  # heads before tokens
        buf = torch.empty((H, N, D), dtype=x.dtype, device="cuda")
        y = buf.transpose(0, 1)
    y.copy_(x)
    return y


def ints(v):
    return torch.tensor(list(v), dtype=torch.int32, device="cuda")


def check(got, x, positions, weight, rope, dtype, eps=1e-6):
    y, off = R.rope(x.double().cpu().numpy(), positions, None if weight is None else weight.double().cpu().numpy(),
                    [] if rope is None else rope.inv_freq, 1.0 if rope is None else float(np.float32(rope.factor)), 0 if rope is None else rope.start,
                    rope is not None and rope.interleaved, eps)
    bound = off + (np.abs(y) + off) * HALF[dtype] + LEAST[dtype]
    err = np.abs(got.double().cpu().numpy() - y)
    assert (err <= bound).all(), float((err / bound).max())


CASES = [
    # N, hq, hk, D, rot, start, interleaved
    (1, 1, 0, 16, 16, 0, False),
    (1, 16, 4, 128, 128, 0, False),
    (3, 5, 2, 128, 64, 0, True),
    (2, 3, 1, 128, 32, 96, False),
    (5, 7, 3, 80, 32, 48, True),
    (4, 9, 2, 96, 48, 24, False),
    (3, 33, 1, 64, 64, 0, True),
    (7, 12, 12, 112, 16, 8, False),
    (2, 4, 4, 256, 256, 0, False),
    (2, 70, 8, 256, 128, 64, True),
    (3, 6, 2, 32, 16, 16, False),
    (6, 2, 2, 48, 32, 0, True),
    (2, 17, 1, 240, 208, 32, False),
    (700, 24, 3, 64, 32, 16, False),  # several rounds a warp
]


@pytest.mark.parametrize("dtype", list(K.TYPES))
@pytest.mark.parametrize("case", range(len(CASES)))
def test_norm_and_rotation(m, case, dtype):
    N, hq, hk, D, rot, start, inter = CASES[case]
    g = torch.Generator().manual_seed(case)
    layout = ["dense", "fused", "odd", "heads"][case % 4]
    q, k = rows(g, N, hq, D, dtype, layout), rows(g, N, hk, D, dtype, ["odd", "dense", "fused"][case % 3]) if hk else None
    wdtype = ["f32", dtype, "f16", "bf16"][case % 4]
    qw, kw = (1 + 0.3 * torch.randn((2, D), generator=g)).to(K.TYPES[wdtype]).cuda()
    rope = m.Rope(rot, theta=10000.0, start=start, interleaved=inter, scaling={"kind": "yarn", "scale": 8.0, "original": 512} if case % 2 else None)
    pos = torch.randint(0, 100 if N > 100 else 200000, (N,), generator=g).tolist()
    for weights, r in (((qw, kw), rope), ((None, None), rope), ((qw, None), None), ((None, kw), rope)):
        if weights[1] is not None and k is None:
            weights = (weights[0], None)
        a, b = m.head_norm_rope(q, ints(pos), r, k=k, q_weight=weights[0], k_weight=weights[1])
        check(a, q, pos, weights[0], r, dtype)
        assert a.is_contiguous() and (b is None) == (k is None)
        if k is not None:
            check(b, k, pos, weights[1], r, dtype)
    # the same call gives the same bits, in place and into strided rows too
    a, b = m.head_norm_rope(q, ints(pos), rope, k=k, q_weight=qw, k_weight=kw)
    buf = torch.full((N, hq, D + 3), 7.0, dtype=q.dtype, device="cuda")
    a2, b2 = m.head_norm_rope(q, ints(pos), rope, k=k, q_weight=qw, k_weight=kw, q_out=buf[..., 1:D + 1], k_out=k)
    assert a2.data_ptr() == buf[..., 1:].data_ptr() and torch.equal(a2, a) and bool((buf[..., 0] == 7).all() and (buf[..., D + 1:] == 7).all())
    if k is not None:
        assert b2 is k and torch.equal(k, b)


@pytest.mark.parametrize("inter", [False, True])
def test_far_and_negative_positions(m, inter):
    """Angles are as exact at the ends of 32 bits as at the start, and a negative position turns back."""
    g = torch.Generator().manual_seed(1)
    pos = [0, 1, -1, 2 ** 31 - 1, -2 ** 31, 2 ** 30 + 7, 1048579, -77777]
    x = rows(g, len(pos), 3, 128, "f32")
    rope = m.Rope(128, theta=500000.0, interleaved=inter)
    y, _ = m.head_norm_rope(x, ints(pos), rope)
    check(y, x, pos, None, rope, "f32")
    assert torch.equal(y[0], x[0])
    back, _ = m.head_norm_rope(y[:4].contiguous(), ints([-p for p in pos[:4]]), rope)
    assert (back - x[:4]).abs().max() <= 2 ** -19 * x[:4].abs().max()  # two rotations of 10 half ulps of |a| + |b| each


def test_frequencies(m):
    """Frequencies that are given, of 32 bits, negative or zero; a factor."""
    g = torch.Generator().manual_seed(2)
    f = (10000.0 ** (-np.arange(0, 64, 2) / 64)).astype(np.float32)
    f[3], f[4] = 0.0, -f[4]
    rope = m.Rope(64, inv_freq=torch.from_numpy(f), factor=0.5)
    pos = [5, 1000, 33333]
    x = rows(g, 3, 4, 64, "f32")
    check(m.head_norm_rope(x, ints(pos), rope)[0], x, pos, None, rope, "f32")
    assert rope.factor == 0.5 and rope.inv_freq == [float(v) for v in f]


def test_values_at_the_ends(m):
    """Rows of zeros, infinities and NaN stay within their head, and without a norm within their pair."""
    x = torch.zeros((1, 6, 64), device="cuda")
    x[0, 1] = 1.0
    x[0, 2, 5] = float("inf")
    x[0, 3, 40] = float("nan")
    x[0, 4, 60] = float("-inf")
    x[0, 5] = 1e-30
    w = torch.ones(64, device="cuda")
    rope = m.Rope(32, start=0)
    y, _ = m.head_norm_rope(x, ints([3]), rope)
    bad = ~torch.isfinite(y[0])
    assert [sorted(bad[h].nonzero().flatten().tolist()) for h in range(6)] == [[], [], [5, 21], [40], [60], []]
    assert y[0, 4, 60] == float("-inf") and bool((y[0, 0] == 0).all())
    y, _ = m.head_norm_rope(x, ints([3]), rope, q_weight=w)
    assert bool((y[0, 0] == 0).all()) and bool(torch.isnan(y[0, 3]).all())
    check(y[:, [1, 5]], x[:, [1, 5]], [3], w, rope, "f32")


def test_norm_alone_and_empty(m):
    g = torch.Generator().manual_seed(3)
    x = rows(g, 5, 3, 64, "bf16")
    w = torch.ones(64, device="cuda")
    y, none = m.head_norm_rope(x, None, q_weight=w, eps=1e-3)
    check(y, x, [0] * 5, w, None, "bf16", 1e-3)
    assert none is None and torch.equal(m.head_norm_rope(x, None)[0], x)  # neither: a copy
    rope = m.Rope(64)
    y, k = m.head_norm_rope(x[:0], ints([]), rope, k=x[:0, :1])
    assert y.shape == (0, 3, 64) and k.shape == (0, 1, 64)


def test_stream_and_graph(m):
    """On another stream than the current one, and captured and replayed on new values."""
    g = torch.Generator().manual_seed(4)
    x, pos = rows(g, 9, 8, 128, "bf16"), ints(range(100, 109))
    w, rope = torch.ones(128, dtype=torch.bfloat16, device="cuda"), m.Rope(128)
    want, _ = m.head_norm_rope(x, pos, rope, q_weight=w)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got, _ = m.head_norm_rope(x, pos, rope, q_weight=w, stream=s)
    s.synchronize()
    assert torch.equal(got, want)
    xs, ps = torch.zeros_like(x), torch.zeros_like(pos)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, _ = m.head_norm_rope(xs, ps, rope, q_weight=w)
    xs.copy_(x)
    ps.copy_(pos)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    assert math.isfinite(float(out.float().sum()))
