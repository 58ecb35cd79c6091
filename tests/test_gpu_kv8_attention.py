"""Attention over the 8-bit cache (moe_kv8_attention) against the formula in 64 bits.

Tolerance, from the kernel's roundings. A score is a sum of at most 256 products held in fp32 (each
product of a code with a 16-bit query, or with each of the two fp16 parts of an fp32 one, is exact;
the parts drop at most 2^-21 of the query): its error is at most ds = 2^-19 * scale * sum |q| |k|
plus 2^-20. That moves a weight by a factor e^(+-ds), so the quotient by 2 ds times the largest
|v|. 16-bit outputs hold their weights in fp16 (2^-11 each, at most that of the largest |v|); the
sums, rescalings and the exponential (2^-22) add less than 2^-17 of it; then the output rounds."""
import numpy as np
import pytest
import torch

import kv8_ref as R

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def m():
    import quantized_routed_expert_grouped_gb300 as mod
    mod.lib()
    return mod


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def make(seed, lens, T, hq, hkv, D, page, dtype, tree=False, scale=0.03, strided=False, q_scale=1.0):
    rng = np.random.default_rng(seed)
    table, n_pages = R.page_table(rng, lens, page)
    ref = R.Cache(R.random_pool(rng, n_pages, hkv, D, page, scale), table)
    # stale tokens after a sequence's end, and blocks after it, hold anything
    for b, n in enumerate(lens):
        last = -(-n // 32)
        for j in range(last, int((table[b] >= 0).sum()) * page // 32):
            ref.block(b, j)[:, :8] = 255  # NaN scales
    q = torch.from_numpy((q_scale * rng.standard_normal((len(lens), T, hq, D))).astype(np.float32)).to(R.TYPES[dtype])
    qd = q.cuda()
    if strided:
        buf = torch.full((len(lens), hq, T, D + 1), float("nan"), dtype=q.dtype, device="cuda")
        qd = buf[..., 1:].transpose(1, 2)
        qd.copy_(q)
    bits = rng.integers(0, 1 << min(T, 30), (len(lens), T)).astype(np.int32) if tree else None
    return ref, q.double().numpy(), qd, bits


def check(m, ref, q, qd, lens, dtype, window=0, tree=None, scale=None, workspace=None, stream=None):
    D = q.shape[3]
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    got, lse = m.kv8_attention(qd, dev(ref.pool), dev(ref.table), ints(lens), scale=scale, window=window,
                               tree=None if tree is None else dev(tree), with_lse=True, err=err,
                               workspace=workspace, stream=stream)
    torch.cuda.synchronize()
    assert int(err) == 0
    out, want_lse, reach, size = R.attention(q, ref, lens, D ** -0.5 if scale is None else scale, window, tree)
    ds = 2.0 ** -19 * size + 2.0 ** -20
    weights = 0.0 if dtype == "f32" else 2.0 ** -11
    tol = reach * (2 * ds[..., None] + weights + 2.0 ** -17) + 2 * R.HALF_ULP[dtype] * np.abs(out) + 2.0 ** -26
    far = np.abs(got.double().cpu().numpy() - out) / tol
    assert far.max() <= 1, far.max()
    empty = np.isneginf(want_lse)
    l = lse.double().cpu().numpy()
    assert np.array_equal(np.isneginf(l), empty)
    assert (np.abs(l[~empty] - want_lse[~empty]) <= (ds + 2.0 ** -18 * (1 + np.abs(want_lse)))[~empty]).all()
    assert (got[torch.from_numpy(empty).cuda()] == 0).all()
    return got, lse


SHAPES = [
    # lens, T, heads, kv heads, head dim, page
    ([1], 1, 1, 1, 32, 32),
    ([31, 32, 33, 0, 1], 1, 4, 2, 64, 32),
    ([700, 1, 95, 64], 4, 8, 2, 128, 64),
    ([2, 3, 130], 4, 6, 6, 96, 128),       # windows longer than their sequences
    ([513, 77], 3, 10, 2, 256, 32),
    ([300], 2, 17, 1, 128, 32),            # 34 rows on one key/value head
    ([260, 5], 9, 16, 2, 64, 64),          # 72 rows
    ([129], 32, 5, 1, 160, 64),            # the longest window, 160 rows
    ([1000, 999, 40], 4, 16, 1, 192, 64),
    ([66], 5, 3, 1, 224, 32),
    ([3000], 1, 2, 2, 128, 64),
]


@pytest.mark.parametrize("dtype", list(R.TYPES))
@pytest.mark.parametrize("shape", range(len(SHAPES)))
def test_attention(m, shape, dtype):
    lens, T, hq, hkv, D, page = SHAPES[shape]
    ref, q, qd, _ = make(shape, lens, T, hq, hkv, D, page, dtype, strided=shape % 2 == 1)
    check(m, ref, q, qd, lens, dtype)


@pytest.mark.parametrize("window", [1, 2, 31, 32, 33, 100, 100000])
@pytest.mark.parametrize("tree", [False, True])
def test_sliding_window(m, window, tree):
    lens, T = [200, 3, 64, 0, 33], 5
    ref, q, qd, bits = make(20 + window, lens, T, 6, 3, 64, 32, "f16", tree=tree)
    check(m, ref, q, qd, lens, "f16", window=window, tree=bits)


@pytest.mark.parametrize("T", [1, 2, 8, 31, 32])
def test_tree(m, T):
    """Random sets of the window's tokens, with rows that see none of it, or (short sequences) nothing."""
    lens = [T, T + 1, 150, 1, 64]
    ref, q, qd, bits = make(40 + T, lens, T, 4, 1, 128, 64, "f32", tree=True)
    bits[:, 0] = 0
    if T == 32:
        bits[:, 31] = -1  # the sign bit is window token 31
    check(m, ref, q, qd, lens, "f32", tree=bits)


@pytest.mark.parametrize("dtype", list(R.TYPES))
@pytest.mark.parametrize("what", ["peaked", "flat", "large_scales", "small_scales", "uneven_scales", "zero_values", "negative_scale", "wide_queries"])
def test_value_ranges(m, what, dtype):
    """Weights over many orders, value scales over most of the range, blocks of zeros."""
    lens, T, hq, hkv, D = [900, 33], 2, 4, 2, 64
    scale = {"large_scales": 1e30, "small_scales": 1e-25}.get(what, 0.03)
    q_scale = {"peaked": 30.0, "flat": 0.0, "large_scales": 1e-4, "small_scales": 1e4}.get(what, 1.0)
    if what == "wide_queries" and dtype != "f16":
        q_scale = 1e15
    ref, q, qd, _ = make(60, lens, T, hq, hkv, D, 32, dtype, scale=0.03, q_scale=q_scale)
    for b, n in enumerate(lens):
        for j in range(-(-n // 32)):
            s = ref.block(b, j)[:, 4:8].copy().view(np.float32)
            s *= np.float32(scale / 0.03)
            if what == "uneven_scales":
                s *= np.float32(10.0 ** ((7 * j) % 41 - 20))
            if what == "zero_values" and j % 3 == 0:
                s *= 0
            ref.block(b, j)[:, 4:8] = s.view(np.uint8)
    check_scale = {"negative_scale": -0.125, "wide_queries": 1e-15 if dtype != "f16" else None}.get(what)
    out, want_lse, reach, size = R.attention(q, ref, lens, D ** -0.5 if check_scale is None else check_scale)
    g, l = m.kv8_attention(qd, dev(ref.pool), dev(ref.table), ints(lens), scale=check_scale, with_lse=True)
    ds = 2.0 ** -19 * size + 2.0 ** -20
    weights = 0.0 if dtype == "f32" else 2.0 ** -11
    least = {"f32": 2.0 ** -120, "f16": 2.0 ** -24, "bf16": 2.0 ** -120}[dtype]
    tol = reach * (2 * ds[..., None] + weights + 2.0 ** -17) + 2 * R.HALF_ULP[dtype] * np.abs(out) + least
    got = g.double().cpu().numpy()
    most = float(torch.finfo(R.TYPES[dtype]).max)
    fits = np.abs(out) + tol < most  # what is past the type's range is its infinity, with its sign
    assert (np.abs(got - out)[fits] <= tol[fits]).all()
    past = np.abs(out) - tol > 1.001 * most
    assert (got[past] == np.sign(out[past]) * np.inf).all()
    assert (np.abs(l.double().cpu().numpy() - want_lse) <= ds + 2.0 ** -18 * (1 + np.abs(want_lse))).all()


def test_not_finite(m):
    """A NaN block makes the rows that see it NaN and no others; a NaN or infinite query its own row."""
    lens, T = [100, 64], 2
    ref, q, qd, _ = make(70, lens, T, 4, 2, 64, 32, "f32")
    ref.block(0, 1)[1, 4:8] = np.frombuffer(np.float32(np.nan).tobytes(), np.uint8)
    ref.block(1, 0)[0, 0:4] = np.frombuffer(np.float32(np.nan).tobytes(), np.uint8)
    qd[1, 1, 3, 5] = float("nan")
    qd[0, 0, 0, 9] = float("inf")
    got = m.kv8_attention(qd, dev(ref.pool), dev(ref.table), ints(lens))
    nan = got.isnan().all(-1).cpu().numpy()
    assert np.array_equal(nan, got.isnan().any(-1).cpu().numpy())
    want = np.zeros((2, T, 4), bool)
    want[0, :, 2:] = want[1, :, :2] = want[1, 1, 3] = want[0, 0, 0] = True
    assert np.array_equal(nan, want)
    # out of the sliding window, the block does not count
    got = m.kv8_attention(qd[:, :, 2:3].repeat(1, 1, 2, 1), dev(ref.pool), dev(ref.table), ints(lens), window=30)
    assert not got[0].isnan().any()


def test_workspace_is_ready_again(m):
    """Calls of several shapes, long and short, on one workspace give what a fresh one gives, bit for bit."""
    ws = m.kv8_attention_workspace(5, 4, 16, 1, 192)
    for rep in range(2):
        for lens, T, hq, hkv, D, page in [SHAPES[8], SHAPES[1], SHAPES[10], SHAPES[2]]:
            ref, q, qd, _ = make(80, lens, T, hq, hkv, D, page, "bf16")
            a, la = check(m, ref, q, qd, lens, "bf16", workspace=ws)
            b, lb = m.kv8_attention(qd, dev(ref.pool), dev(ref.table), ints(lens), with_lse=True)
            assert torch.equal(a, b) and torch.equal(la, lb)


def test_long_context_repeats(m):
    """A 200k-token context in a pool past 4 GiB, split over the whole device: right at sampled heads
    (constant keys make every weight equal, so the output is the mean of the values), the same bits
    on every run, on another stream, and from a replayed graph."""
    hkv, D, page, n = 4, 128, 128, 200003
    blocks = -(-n // 32)
    n_pages = max(-(-n // page) + 3, (1 << 32) // (hkv * (page // 32) * m.kv8_block_bytes(D)) + 2)
    pool = m.kv8_pool(n_pages, hkv, D, page)
    need = -(-n // page)
    table = torch.arange(n_pages - need, n_pages, dtype=torch.int32, device="cuda").flip(0).contiguous().view(1, -1)
    k = torch.ones((n, hkv, D), device="cuda")
    v = torch.randn((n, hkv, D), generator=torch.Generator("cuda").manual_seed(1), device="cuda") + 0.5
    cu, zero = ints([0, n]), ints([0])
    m.kv8_write(k, v, pool, table, cu, zero)
    kk, vv = m.kv8_read(pool, table, cu, zero, n, dtype=torch.float32)
    q = torch.randn((1, 2, 16, D), device="cuda")
    ws = m.kv8_attention_workspace(1, 2, 16, hkv, D)
    out, lse = m.kv8_attention(q, pool, table, ints([n]), workspace=ws, with_lse=True)
    for t in range(2):
        mean = vv[:n - 1 + t].double().mean(0).repeat_interleave(4, 0)
        assert (out[0, t].double() - mean).abs().max() <= 2.0 ** -15 * vv.abs().max()
    assert blocks > 6000
    for _ in range(3):
        o2, l2 = m.kv8_attention(q, pool, table, ints([n]), workspace=ws, with_lse=True)
        assert torch.equal(out, o2) and torch.equal(lse, l2)
    lens = ints([n])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    o3 = m.kv8_attention(q, pool, table, lens, workspace=ws, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(out, o3)
    g = torch.cuda.CUDAGraph()
    o4 = torch.empty_like(out)
    with torch.cuda.graph(g):
        m.kv8_attention(q, pool, table, lens, workspace=ws, out=o4)
    o4.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, o4)
    # the graph sees a new length on the device
    lens.fill_(64)
    g.replay()
    short = m.kv8_attention(q, pool, table, ints([64]), workspace=ws)
    assert torch.equal(short, o4)


@pytest.mark.parametrize("what", ["length", "past_table", "page"])
def test_bad_device_data(m, what):
    lens = [100, 50]
    ref, q, qd, _ = make(90, lens, 1, 4, 2, 64, 32, "f32")
    table = ref.table.copy()
    good, _ = m.kv8_attention(qd, dev(ref.pool), dev(table), ints(lens), with_lse=True)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    if what == "length":
        lens = [-3, 50]
    elif what == "past_table":
        lens = [129, 50]
    else:
        table[0, 1] = 1 << 20
    got, lse = m.kv8_attention(qd, dev(ref.pool), dev(table), ints(lens), with_lse=True, err=err)
    assert int(err) == (512 if what == "length" else 256)
    assert torch.equal(got[1], good[1])
    if what == "length":
        assert (got[0] == 0).all() and torch.isneginf(lse[0]).all()
    else:
        assert got[0].isfinite().all()
