"""Appending to the 8-bit cache with norm and rotation on the way (moe_kv8_append). Without a norm the fp32 keys are those of
moe_head_norm_rope, operation by operation, so the records must be moe_kv8_write's of these, bit for bit; with one, a key read
back is off by half a step and what decode_ref.rope bounds. Queries must be moe_head_norm_rope's, bit for bit."""
import numpy as np
import pytest
import torch

import decode_ref as D
import kv8_ref as K

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def m():
    import quantized_routed_expert_grouped_gb300 as mod
    mod.lib()
    return mod


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def ints(v):
    return torch.tensor([int(x) for x in v], dtype=torch.int32, device="cuda")


class Case:
    def __init__(self, seed, starts, counts, hq, hkv, d, page, dtype="f32", layout="fused"):
        rng = self.rng = np.random.default_rng(seed)
        table, n_pages = K.page_table(rng, [s + n for s, n in zip(starts, counts)], page)
        self.ref = K.Cache(K.random_pool(rng, n_pages, hkv, d, page), table)
        self.pool, self.table = dev(self.ref.pool), dev(table)
        self.starts, self.counts, self.cu = starts, counts, np.concatenate([[0], np.cumsum(counts)]).astype(int)
        self.N, self.d, self.dtype = int(self.cu[-1]), d, dtype
        self.err = ints([0])
        x = torch.from_numpy((rng.standard_normal((self.N, hq + 2 * hkv, d)) * np.exp(rng.uniform(-2, 2, (self.N, hq + 2 * hkv, 1)))).astype(np.float32))
        x = x.to(K.TYPES[dtype])
        if layout == "odd":  # rows that no vector access may touch
            buf = torch.full((self.N, hq + 2 * hkv, d + 1), float("nan"), dtype=x.dtype, device="cuda")[..., 1:]
            buf.copy_(x)
        elif layout == "heads":
            buf = torch.empty((hq + 2 * hkv, self.N, d), dtype=x.dtype, device="cuda").transpose(0, 1)
            buf.copy_(x)
        else:
            buf = x.cuda()
        self.q, self.k, self.v = buf[:, :hq] if hq else None, buf[:, hq:hq + hkv], buf[:, hq + hkv:]
        self.places = np.concatenate([np.arange(s, s + n) for s, n in zip(starts, counts)] or [np.zeros(0)]).astype(int)
        self.weights = [torch.from_numpy((1 + 0.3 * rng.standard_normal(d)).astype(np.float32)).cuda() for _ in range(2)]

    def append(self, m, pool=None, **kw):
        return m.kv8_append(self.k, self.v, self.pool if pool is None else pool, self.table, ints(self.cu), ints(self.starts), err=self.err, **kw)


SHAPES = [
    # starts, counts, hq, hkv, head dim, page, rot, start, interleaved
    ([0], [1], 4, 1, 32, 32, 32, 0, False),
    ([777], [1], 16, 4, 128, 64, 128, 0, False),
    ([0, 31, 32, 33], [1, 1, 1, 1], 2, 2, 64, 32, 32, 16, True),
    ([5, 0, 63, 30, 17], [4, 0, 4, 4, 3], 24, 4, 128, 64, 64, 64, False),
    ([0, 7], [200, 131], 0, 3, 96, 128, 96, 0, False),
    ([40], [95], 10, 2, 256, 32, 256, 0, True),
    ([3, 0, 0, 100] * 10, [2, 33, 0, 1] * 10, 3, 1, 64, 32, 16, 8, False),
    ([1, 64], [64, 32], 8, 8, 160, 64, 48, 24, True),
    ([9], [70], 6, 6, 224, 64, 208, 16, False),
    ([11, 2], [40, 3], 5, 5, 192, 32, 144, 0, False),
    ([1], [60], 3, 1, 32, 64, 16, 16, True),
    ([13, 0], [1500, 900], 40, 5, 64, 64, 64, 0, False),   # many blocks: several heads a CTA, the last fewer
    ([0, 50], [4100, 6001], 0, 9, 32, 64, 32, 0, True),
]


@pytest.mark.parametrize("dtype", list(K.TYPES))
@pytest.mark.parametrize("shape", range(len(SHAPES)))
def test_rotation(m, shape, dtype):
    starts, counts, hq, hkv, d, page, rot, start, inter = SHAPES[shape]
    c = Case(shape, starts, counts, hq, hkv, d, page, dtype, ["fused", "odd", "heads"][shape % 3])
    rope = m.Rope(rot, theta=10000.0, start=start, interleaved=inter, factor=1.25)
    for positions in (None, ints(c.rng.integers(-5, 100000, c.N))):
        p = ints(c.places) if positions is None else positions
        want, got = c.pool.clone(), c.pool.clone()
        k32, _ = m.head_norm_rope(c.k.float(), p, rope)
        m.kv8_write(k32, c.v.float(), want, c.table, ints(c.cu), ints(c.starts), err=c.err)
        q = c.append(m, got, rope=rope, q=c.q, positions=positions)
        assert int(c.err) == 0 and torch.equal(got, want)
        if hq:
            assert torch.equal(q, m.head_norm_rope(c.q, p, rope)[0])
        else:
            assert q is None
    # neither norm nor rotation: moe_kv8_write
    want, got = c.pool.clone(), c.pool.clone()
    m.kv8_write(c.k, c.v, want, c.table, ints(c.cu), ints(c.starts), err=c.err)
    q = c.append(m, got, q=c.q)
    assert int(c.err) == 0 and torch.equal(got, want) and (q is None or torch.equal(q, c.q))


@pytest.mark.parametrize("dtype", list(K.TYPES))
@pytest.mark.parametrize("shape", range(len(SHAPES)))
def test_norm_and_rotation(m, shape, dtype):
    starts, counts, hq, hkv, d, page, rot, start, inter = SHAPES[shape]
    c = Case(100 + shape, starts, counts, hq, hkv, d, page, dtype, ["odd", "heads", "fused"][shape % 3])
    rope = m.Rope(rot, theta=10000.0, start=start, interleaved=inter)
    qw, kw = (w.to(K.TYPES[["f32", "bf16", "f16"][shape % 3]]) for w in c.weights)
    q = c.append(m, rope=rope, q=c.q, q_weight=qw, k_weight=kw)
    assert int(c.err) == 0
    if hq:
        assert torch.equal(q, m.head_norm_rope(c.q, ints(c.places), rope, q_weight=qw)[0])
    few = c.N <= 1000
    rows = range(c.N) if few else range(0, c.N, 37)  # (the angles of the reference are slow)
    y, off = D.rope(c.k.double().cpu().numpy()[rows], c.places[rows], kw.double().cpu().numpy(), rope.inv_freq, 1.0, start, inter)
    got, v = K.Cache(c.pool.cpu().numpy(), c.ref.table), c.v.float().cpu().numpy()
    at = dict(zip(rows, range(len(rows))))
    for b, (s, n) in enumerate(zip(c.starts, c.counts)):
        if not n:
            continue
        c.ref.write(b, s, (np.zeros((n, hkv, d), np.float32), v[c.cu[b]:c.cu[b] + n]))  # values: bit for bit
        for j in range(s // 32, (s + n + 31) // 32):
            t0, t1 = max(0, s - 32 * j), min(32, s + n - 32 * j)
            first = c.cu[b] + 32 * j + t0 - s
            for h in range(hkv):
                gc, gs = got.codes(b, j, h, 1)
                ec, es = c.ref.codes(b, j, h, 1)
                assert gs == es and np.array_equal(gc[:t1], ec[:t1])
                gc, gs = got.codes(b, j, h, 0)
                for t in range(t0, t1):
                    if first + t - t0 in at:
                        i = at[first + t - t0]
                        step = gs * (0.5 + 127 * 3 * D.ULP)
                        assert (np.abs(gc[t] * float(gs) - y[i, h]) <= step + off[i, h]).all()
                if few:
                    i = slice(at[first], at[first] + t1 - t0)
                    most = np.abs(y[i, h]).max()
                    # the scale: the largest key's, or the kept tokens'
                    new = most / 127
                    assert gs >= new * (1 - 2 * D.ULP) - off[i, h].max() / 127
                    if not t0:
                        assert gs <= new * (1 + 2 * D.ULP) + off[i, h].max() / 127


def test_kept_tokens(m):
    """Tokens that a block holds before the new ones are kept under the larger scale, as moe_kv8_write keeps them."""
    c = Case(31, [5, 45], [30, 2], 0, 3, 128, 64)
    before = K.Cache(c.ref.pool.copy(), c.ref.table)
    c.k.mul_(20)  # wider than what the blocks hold
    c.append(m, rope=m.Rope(128), k_weight=c.weights[1] * 50)
    got = K.Cache(c.pool.cpu().numpy(), c.ref.table)
    for b, (s, j) in enumerate(((5, 0), (45, 1))):
        for h in range(3):
            for w in range(2):
                old, a = before.codes(b, j, h, w)
                new, e = got.codes(b, j, h, w)
                kept = np.rint(old[:s % 32].astype(np.float32) * (a / e))
                assert e >= a and np.array_equal(new[:s % 32], kept)
                assert w == 1 or e > a
    assert int(c.err) == 0


@pytest.mark.parametrize("what", ["page_low", "past_table", "start", "cu"])
def test_bad_device_data(m, what):
    """Bad pages and ranges are skipped and reported; the other sequence is written, its queries too."""
    c = Case(14, [0, 3], [40, 40], 2, 1, 32, 32)
    rope = m.Rope(32)
    before, good = c.pool.clone(), c.pool.clone()
    table, starts, cu = c.table.clone(), list(c.starts), list(c.cu)
    m.kv8_write(m.head_norm_rope(c.k, ints(c.places), rope)[0], c.v, good, table, ints(cu), ints(starts))
    if what == "page_low":
        table[0] = -1
    elif what == "past_table":
        starts[0] = 32 * table.shape[1]
    elif what == "start":
        starts[0] = -1
    else:
        cu[0] = -5
    q = torch.full_like(c.q, 5.0)
    m.kv8_append(c.k, c.v, c.pool, table, ints(cu), ints(starts), rope, q=c.q, q_out=q, err=c.err)
    assert int(c.err) == (256 if what in ("page_low", "past_table") else 512)
    first = [int(p) for p in c.ref.table[0] if p >= 0]
    for p in range(c.pool.shape[0]):
        assert torch.equal(c.pool[p], (before if p in first else good)[p])
    want = m.head_norm_rope(c.q, ints(c.places), rope)[0]
    assert torch.equal(q[40:], want[40:])
    if what in ("start", "cu"):
        assert bool((q[:40] == 5).all())


def test_rows_behind_the_last_sequence(m):
    """Rows past cu_tokens' last value belong to no sequence: their queries are left as they were."""
    c = Case(15, [3, 9], [20, 13], 4, 2, 64, 64)
    rope, cu = m.Rope(64), [0, 20, 27]
    q, want = torch.full_like(c.q, 5.0), c.pool.clone()
    m.kv8_append(c.k, c.v, c.pool, c.table, ints(cu), ints(c.starts), rope, q=c.q, q_out=q, err=c.err)
    m.kv8_write(m.head_norm_rope(c.k, ints(c.places), rope)[0][:27], c.v[:27], want, c.table, ints(cu), ints(c.starts))
    assert int(c.err) == 0 and torch.equal(c.pool, want)
    assert torch.equal(q[:27], m.head_norm_rope(c.q, ints(c.places), rope)[0][:27]) and bool((q[27:] == 5).all())


def test_not_finite_and_zero(m):
    """A head that holds a NaN makes its blocks of keys NaN, no other; zeros stay zeros."""
    c = Case(16, [0], [64], 0, 3, 64, 64)
    c.k[:, 0] = 0
    c.k[40, 1, 7] = float("nan")
    c.append(m, rope=m.Rope(64), k_weight=c.weights[0])
    k, v = m.kv8_read(c.pool, c.table, ints([0, 64]), ints([0]), 64, dtype=torch.float32)
    assert bool((k[:, 0] == 0).all()) and bool(torch.isfinite(k[:32]).all()) and bool(torch.isnan(k[32:, 1]).all())
    assert bool(torch.isfinite(k[32:, 2]).all()) and bool(torch.isfinite(v).all())


@pytest.mark.parametrize("dtype", list(K.TYPES))
@pytest.mark.parametrize("shape", [([5, 64], [500, 470], 600, 2, 32), ([31, 0, 62], [9, 6, 11], 7, 1, 256), ([0, 30, 7], [40, 3, 70], 9, 3, 192),
                                   ([3, 9], [1500, 1100], 33, 1, 160), ([1] * 5, [5, 4, 6, 5, 4], 3, 2, 224)])
def test_query_parts(m, shape, dtype):
    """Queries by few and by many CTAs, a block's tokens by one, two and four, heads that leave part of a warp's round."""
    starts, counts, hq, hkv, d = shape
    c = Case(21, starts, counts, hq, hkv, d, 64, dtype)
    rope = m.Rope(16, start=d - 16)
    want = c.pool.clone()
    q = c.append(m, rope=rope, q=c.q, q_weight=c.weights[0], k_weight=c.weights[1], q_out=torch.full_like(c.q, 5.0))
    c.append(m, want, rope=rope, k_weight=c.weights[1])
    assert int(c.err) == 0 and torch.equal(c.pool, want)
    assert torch.equal(q, m.head_norm_rope(c.q, ints(c.places), rope, q_weight=c.weights[0])[0])


@pytest.mark.parametrize("dtype", list(K.TYPES))
def test_norm_without_eps(m, dtype):
    """eps 0: the places of a block that hold no new token do not count; a key of zeros is 0 / 0, and makes its block NaN."""
    c = Case(19, [3, 40], [7, 2], 2, 2, 96, 32, dtype)
    rope = m.Rope(32, start=16)
    q = c.append(m, rope=rope, q=c.q, q_weight=c.weights[0], k_weight=c.weights[1], eps=0.0)
    assert int(c.err) == 0 and bool(torch.isfinite(q).all())
    y, off = D.rope(c.k.double().cpu().numpy(), c.places, c.weights[1].double().cpu().numpy(), rope.inv_freq, 1.0, 16, False, 0.0)
    k, v = m.kv8_read(c.pool, c.table, ints(c.cu), ints(c.starts), c.N, dtype=torch.float32)
    got = K.Cache(c.pool.cpu().numpy(), c.ref.table)
    for b, j in ((0, 0), (1, 1)):
        rows = slice(c.cu[b], c.cu[b + 1])
        for h in range(2):
            step = got.codes(b, j, h, 0)[1] * (0.5 + 127 * 3 * D.ULP)
            assert (np.abs(k[rows, h].cpu().numpy() - y[rows, h]) <= step + off[rows, h]).all()
    c.k[8, 1] = 0
    c.append(m, rope=rope, k_weight=c.weights[1], eps=0.0)
    k, _ = m.kv8_read(c.pool, c.table, ints(c.cu), ints(c.starts), c.N, dtype=torch.float32)
    assert bool(torch.isnan(k[7:, 1]).all()) and bool(torch.isfinite(k[:, 0]).all()) and bool(torch.isfinite(k[:7]).all())


def test_empty(m):
    c = Case(17, [5], [0], 2, 2, 64, 64)
    before = c.pool.clone()
    q = c.append(m, rope=m.Rope(64), q=c.q)
    assert q.shape == (0, 2, 64) and torch.equal(c.pool, before) and int(c.err) == 0


def test_in_place_stream_and_graph(m):
    """Queries in place; another stream; a captured call replayed on new rows and places."""
    c = Case(18, [9, 0], [33, 4], 8, 2, 128, 64, "bf16")
    rope, kw = m.Rope(128), dict(q_weight=c.weights[0].bfloat16(), k_weight=c.weights[1].bfloat16())
    pools = [c.pool.clone() for _ in range(4)]
    want = c.append(m, pools[0], rope=rope, q=c.q, **kw)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = c.append(m, pools[1], rope=rope, q=c.q, stream=s, **kw)
    s.synchronize()
    assert torch.equal(got, want) and torch.equal(pools[1], pools[0])
    buf, start, cu = torch.zeros_like(c.q), ints([0, 0]), ints(c.cu)
    k, v = torch.zeros_like(c.k), torch.zeros_like(c.v)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = m.kv8_append(k, v, pools[2], c.table, cu, start, rope, q=buf, **kw)
    pools[2].copy_(c.pool)
    for a, b in ((buf, c.q), (k, c.k), (v, c.v), (start, ints(c.starts))):
        a.copy_(b)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want) and torch.equal(pools[2], pools[0])
    q = c.q
    again = c.append(m, pools[3], rope=rope, q=q, q_out=q, **kw)
    assert again is q and torch.equal(q, want) and torch.equal(pools[3], pools[0])


def test_offsets_past_32_bits(m):
    """A pool of more than 4 GiB, and rows more than 2^31 elements apart from their first."""
    hkv, d, page = 2, 256, 128
    n_pages = (1 << 32) // (hkv * 4 * m.kv8_block_bytes(d)) + 4
    pool = torch.empty((n_pages, hkv, page // 32, m.kv8_block_bytes(d)), dtype=torch.uint8, device="cuda")
    g = torch.Generator("cuda").manual_seed(1)
    n, apart = 130, (1 << 31) // 120
    far = torch.empty(n * apart + 4 * hkv * d, dtype=torch.bfloat16, device="cuda")
    rows = far.as_strided((n, 3 * hkv, d), (apart, d, 1))
    rows.copy_(torch.randn((n, 3 * hkv, d), generator=g, device="cuda"))
    table, rope = ints([n_pages - 1, n_pages - 2]).view(1, 2), m.Rope(256)
    q = m.kv8_append(rows[:, hkv:2 * hkv], rows[:, 2 * hkv:], pool, table, ints([0, n]), ints([0]), rope, q=rows[:, :hkv])
    near = rows.contiguous()
    small = m.kv8_pool(2, hkv, d, page)
    want = m.kv8_append(near[:, hkv:2 * hkv], near[:, 2 * hkv:], small, ints([1, 0]).view(1, 2), ints([0, n]), ints([0]), rope, q=near[:, :hkv])
    assert torch.equal(q, want)
    for a, b in zip(m.kv8_read(pool, table, ints([0, n]), ints([0]), n), m.kv8_read(small, ints([1, 0]).view(1, 2), ints([0, n]), ints([0]), n)):
        assert torch.equal(a, b)
