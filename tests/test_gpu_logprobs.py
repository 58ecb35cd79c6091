"""Log probabilities of given tokens, the most likely tokens, entropy and log-sum-exp (moe_token_logprobs) against the formulas
in 64 bits. Tolerances count fp32 roundings (decode_ref.logprobs says which); token ids have to be equal."""
import numpy as np
import pytest
import torch

import decode_ref as R
import kv8_ref as K

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def m():
    import quantized_routed_expert_grouped_gb300 as mod
    mod.lib()
    return mod


def check(m, x, ids, top, scale=1.0):
    """x: device logits; ids: numpy [R, n]."""
    got = m.token_logprobs(x, torch.from_numpy(ids.astype(np.int32)).cuda(), top=top, scale=scale)
    lp, tl, ti, ent, lse = (None if t is None else t.cpu().numpy() for t in got)
    x64 = x.double().cpu().numpy()
    s = float(np.float32(scale))
    elp, etl, eti, eent, else_, off, eoff = R.logprobs(x64, ids, top, s, 4096)
    if top:
        assert np.array_equal(ti, eti)
    ulp = R.ULP

    def near(a, e, bound):
        some = ~np.isneginf(e)
        assert np.array_equal(np.isneginf(a), ~some)
        err, most = np.abs(a - np.where(some, e, 0))[some], np.broadcast_to(bound, e.shape)[some]
        assert (err <= most).all(), float((err / most).max())

    m_ = x64.max(1)
    m_ = np.where(np.isneginf(m_), 0, m_)
    ls = np.abs(np.where(np.isneginf(else_), 0, else_ - s * m_))
    # the difference, its product, the logarithm's own error and rounding (2), the last difference
    for a, e in ((lp, elp), (tl, etl)):
        if a is not None and a.size:
            near(a, e, off[:, None] + ulp * (3 * np.abs(np.where(np.isneginf(e), 0, e)) + 6 * ls[:, None] + 2))
    near(ent, eent, eoff + ulp * (4 * np.abs(eent) + 4 * ls + 2))
    near(lse, else_, off + ulp * (4 * ls + 2 * s * np.abs(m_) + 2))


def ids_for(rng, R, V, n):
    ids = rng.integers(0, V, (R, n))
    ids[rng.random((R, n)) < 0.2] = -1
    if R > 1:
        ids[1, 0] = V  # past the end
        ids[0, 0] = V - 1
    return ids


SIZES = [(1, 1), (3, 2), (2, 5), (5, 31), (4, 33), (3, 257), (2, 1000), (3, 4097), (2, 8191), (2, 8192), (3, 8193), (2, 16400), (5, 50001), (1, 131075),
         (40, 40000), (330, 9001), (700, 2500), (701, 33), (801, 1), (650, 700), (900, 2044)]


@pytest.mark.parametrize("dtype", list(K.TYPES))
@pytest.mark.parametrize("size", range(len(SIZES)))
def test_random(m, size, dtype):
    R_, V = SIZES[size]
    rng = np.random.default_rng(size)
    pad = [0, 1, 3, 8][size % 4]
    x = (2.5 * rng.standard_normal((R_, V + pad))).astype(np.float32)
    x[:, rng.integers(0, V)] += 8
    if size % 3 == 1:
        x[rng.random(x.shape) < 0.9] = -np.inf
    dev = torch.from_numpy(x).to(K.TYPES[dtype]).cuda()[:, :V]
    for top, n, scale in ((min(V, 20), 2, 1.0), (0, 1, 0.5), (min(V, 32), 1, 1 / 0.7), (1, 3, 1.0)):
        check(m, dev, ids_for(rng, R_, V, n), top, scale)
        if R_ * V > 1 << 20:
            break


@pytest.mark.parametrize("dtype", list(K.TYPES))
@pytest.mark.parametrize("V", [7, 260, 9000, 70001])
def test_hard_rows(m, V, dtype):
    """Rows whose order, masks or ties are hard on a selection: each by the same rules."""
    t = K.TYPES[dtype]
    low = torch.finfo(t).min
    rng = np.random.default_rng(V)
    i = np.arange(V)
    few = np.full(V, -np.inf)
    few[rng.integers(0, V, 3)] = 1.0
    lowest = np.full(V, low)
    lowest[[0, V // 2, V - 1]] = [1.0, 2.0, 1.0]
    zeros = np.where(rng.random(V) < 0.5, -0.0, 0.0)
    mixed = np.where(i % 3 == 0, -np.inf, low)
    rows = [np.full(V, -np.inf), np.full(V, 3.0), np.full(V, low), i * 10.0 / V, -i * 10.0 / V, few, lowest, zeros, mixed, np.round(rng.standard_normal(V)),
            np.where(i == V - 1, 0.0, -np.inf), np.where(i < V // 2, -np.inf, 5.0 * i / V), np.where(i % 8 == 7, 4.0, -4.0)]
    x = torch.from_numpy(np.stack(rows).astype(np.float64)).to(t).cuda()
    for top in (1, 5, min(V, 32)):
        check(m, x, ids_for(rng, len(rows), V, 2), top)
    if V < 9000:  # many short rows: by warps
        many = x.repeat(55, 1)
        got = [m.token_logprobs(many, top=t) for t in (1, 5)]
        for t, (_, tl, ti, ent, lse) in zip((1, 5), got):
            _, tl1, ti1, _, _ = m.token_logprobs(x, top=t)
            assert torch.equal(ti.view(55, *ti1.shape), ti1.expand(55, *ti1.shape)) and bool((ti >= 0).all())
            assert torch.allclose(tl.view(55, *tl1.shape), tl1.expand(55, *tl1.shape), rtol=1e-6, atol=1e-5)
        check(m, many[:len(rows) * 52], ids_for(rng, len(rows) * 52, V, 1), min(V, 24))
    # one row alone: by a cluster
    for r in range(len(rows)):
        check(m, x[r:r + 1], ids_for(rng, 1, V, 1), min(V, 32))


@pytest.mark.parametrize("dtype", list(K.TYPES))
@pytest.mark.parametrize("V", [40, 3000, 70001])
@pytest.mark.parametrize("more", [0, 700])
def test_not_finite(m, V, dtype, more):
    """A NaN or +inf makes a row's numbers NaN, but leaves the other rows and the order of what is a number."""
    x = (torch.zeros((4, V), device="cuda") + torch.arange(V, device="cuda") % 7).to(K.TYPES[dtype])
    x[1, 3] = float("nan")
    x[2, 5] = float("inf")
    x[3] = float("nan")
    ids = torch.tensor([[1], [-1], [2], [0]], dtype=torch.int32, device="cuda")
    if more and V < 9000:  # (many short rows are taken by warps)
        x, ids = torch.cat([x, x[:1].expand(more, V)]), torch.cat([ids, ids[:1].expand(more, 1)])
    lp, tl, ti, ent, lse = (t[:4] for t in m.token_logprobs(x.contiguous(), ids.contiguous(), top=3))
    assert torch.isfinite(lp[0]).all() and torch.isfinite(tl[0]).all() and torch.isfinite(ent[0]) and torch.isfinite(lse[0])
    for r in (1, 2, 3):
        assert torch.isnan(tl[r]).all() and torch.isnan(ent[r]) and torch.isnan(lse[r])
    assert float(lp[1]) == float("-inf") and torch.isnan(lp[2:]).all()
    assert ti.tolist() == [[6, 13, 20], [6, 13, 20], [5, 6, 13], [-1, -1, -1]]


@pytest.mark.parametrize("dtype", list(K.TYPES))
@pytest.mark.parametrize("V", [50, 9001, 70001])
def test_scales(m, V, dtype):
    """Scales near 0 and far above 1, small and large logits: where c x leaves fp32's range, or clamped logits would count, too."""
    rng = np.random.default_rng(V + 1)
    x = rng.standard_normal((5, V))
    x[1] *= 1e-3
    x[2] *= 1000
    x[3, rng.random(V) < 0.9] = -np.inf
    x[4] = np.where(rng.random(V) < 0.5, -np.inf, torch.finfo(K.TYPES[dtype]).min)
    dev = torch.from_numpy(x).to(K.TYPES[dtype]).cuda()
    for scale in (2.0 ** -100, 2.0 ** -30, 1e-3, 1.0, 30.0, 2.0 ** 20, 2.0 ** 100):
        some = dev[:3].repeat(210 if V == 50 else 1, 1)  # (many short rows are taken by warps)
        check(m, some, ids_for(rng, some.shape[0], V, 2), min(V, 9), scale)
        check(m, dev[3:4], ids_for(rng, 1, V, 2), 3, scale)
    check(m, dev[4:], ids_for(rng, 1, V, 2), 3, 0.5)


@pytest.mark.parametrize("dtype", list(K.TYPES))
@pytest.mark.parametrize("V", [50, 9001, 140001])
def test_mask_values(m, V, dtype):
    """Masks by large negative numbers, where most threads see nothing else, and rows with one far larger logit."""
    rng = np.random.default_rng(V + 2)
    for mask in (-1e4, -6e4, -1e9, -1e30, -3e38):
        x = rng.standard_normal((4, V))
        x[:3][rng.random((3, V)) < 0.999] = mask
        x[2] = mask
        x[3, V // 2] = -mask
        dev = torch.from_numpy(x).to(K.TYPES[dtype]).cuda()
        if dtype == "f16" and mask < -65504:
            dev = dev[:3]  # (-inf there, and the last row +inf)
        if V == 50:
            dev = dev.repeat(210, 1)  # (many short rows are taken by warps)
        for scale in (1.0, 0.1):
            check(m, dev, ids_for(rng, dev.shape[0], V, 2), 3, scale)
            check(m, dev[2:3], ids_for(rng, 1, V, 1), 2, scale)


@pytest.mark.parametrize("dtype", list(K.TYPES))
@pytest.mark.parametrize("size", [(620, 1030), (5, 1030), (620, 4100), (3, 4100), (610, 8200), (609, 12300), (2, 16390), (609, 24590)])
def test_row_sizes(m, size, dtype):
    """Rows about the sizes where their number of warps changes, for many and for few of them, at odd addresses."""
    R_, V = size
    rng = np.random.default_rng(V)
    x = torch.from_numpy(rng.standard_normal((R_, V + 3)).astype(np.float32)).to(K.TYPES[dtype]).cuda()[:, 1:V + 1]
    for v in (V, V - 7, V - 2):
        check(m, x[:, :v], ids_for(rng, R_, v, 2), 17)


@pytest.mark.parametrize("dtype", list(K.TYPES))
@pytest.mark.parametrize("size", [(700, 1000), (2, 1000), (700, 2040), (2, 2040), (620, 8000), (2, 16000)])
def test_best_in_few_places(m, size, dtype):
    """The large logits lie close together, in a pattern that few threads see: far more of them than `top` in some rows, far
    fewer in others, all equal in some."""
    R_, V = size
    W = 4 if dtype == "f32" else 8
    rng = np.random.default_rng(R_ + V)
    i = np.arange(V)
    x = np.full((R_, V), -10.0)
    for r in range(R_):
        period, width = [(32, 9), (64, 9), (128, 15), (32, 2), (128, 1), (1 << 30, 5)][r % 6]
        on = (i // W) % period < width
        x[r, on] = [rng.standard_normal(on.sum()), 2.0, np.round(rng.standard_normal(on.sum()))][r // 6 % 3]
        if r % 5 == 4:
            x[r, ~on] = -np.inf
    dev = torch.from_numpy(x).to(K.TYPES[dtype]).cuda()
    for top in (1, 20, 32):
        check(m, dev, ids_for(rng, R_, V, 1), top)


def test_many_ids_and_none(m):
    rng = np.random.default_rng(3)
    x = torch.from_numpy(rng.standard_normal((3, 901)).astype(np.float32)).cuda()
    check(m, x, ids_for(rng, 3, 901, 700), 4)
    a = m.token_logprobs(x)
    b = m.token_logprobs(x, top=4)
    assert a[0] is None and a[1] is None and a[2] is None and torch.equal(a[3], b[3]) and torch.equal(a[4], b[4])
    none = m.token_logprobs(x[:0], torch.zeros((0, 2), dtype=torch.int32, device="cuda"), top=2)
    assert [tuple(t.shape) for t in none] == [(0, 2), (0, 2), (0, 2), (0,), (0,)]


def test_same_bits(m):
    """Calls, streams and captured graphs give the same bits (the order of appended keys does not count)."""
    rng = np.random.default_rng(5)
    x = torch.from_numpy(np.round(4 * rng.standard_normal((6, 60000))).astype(np.float32)).cuda()
    ids = torch.from_numpy(rng.integers(0, 60000, (6, 2)).astype(np.int32)).cuda()
    want = m.token_logprobs(x, ids, top=32)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    runs = [m.token_logprobs(x, ids, top=32) for _ in range(20)] + [m.token_logprobs(x, ids, top=32, stream=s)]
    s.synchronize()
    buf = torch.zeros_like(x)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        runs.append(m.token_logprobs(buf, ids, top=32))
    buf.copy_(x)
    graph.replay()
    torch.cuda.synchronize()
    for got in runs:
        assert all(torch.equal(a, b) for a, b in zip(got, want))
