"""moe_kv8_attention at the ends of its ranges, against the formula in 64 bits."""
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


def scaled_blocks(rng, scores, powers, D, hkv):
    """A cache of one sequence whose block j's tokens all score scores[j] (in powers of two, 0 or below, for a query
    of one in dim 0) and whose values have the scale 2^powers[j] times 1 to 2; a page a block."""
    n = len(scores)
    ref = R.Cache(R.random_pool(rng, n, hkv, D, 32), np.arange(n, dtype=np.int32)[None])
    for j, (s, e) in enumerate(zip(scores, powers)):
        rec = ref.block(0, j)
        rec[:, 16:16 + 32 * D] = 128
        rec[:, ref.at[0][:, 0]] = 28  # -100
        rec[:, :4] = np.full((hkv, 1), -s * np.log(2) / 100, np.float32).view(np.uint8)
        rec[:, 4:8] = (2.0 ** e * rng.uniform(1, 1.9, (hkv, 1))).astype(np.float32).view(np.uint8)
    return ref


def blocks_of(what):
    if what == "seen":    # as found: infinity in the first, NaN in the second where one warp met both
        return [[(0, -90), (-120, 30)], [(0, -100), (-150, 20)], [(-150, 20), (0, -100)], [(0, -7), (-126, 119)], [(-30, 119), (0, -90)]]
    if what == "past":    # the weight itself is far below fp32's range, its share of the output is not
        return [[(0, -100), (-205, 105)], [(-205, 105), (0, -100)], [(0, -60), (-170, 110)], [(-190, 95), (-10, -85)]]
    return []


@pytest.mark.parametrize("dtype", list(R.TYPES))
@pytest.mark.parametrize("rows", [1, 20])
@pytest.mark.parametrize("many", [False, True])
@pytest.mark.parametrize("what", ["seen", "past", "drawn"])
def test_scales_far_apart(m, what, many, rows, dtype):
    """Blocks whose value scales lie up to 2^210 apart, with scores that make up for it, in every order. Sequences
    of up to 12 blocks: many of them, so that a warp takes several blocks of one, or one alone, in parts.

    Tolerance, as in test_gpu_kv8_attention.py but for each token's share: (2 ds + 2^-11 for 16-bit outputs, + 2^-17) of
    sum p |v| / sum p, and what fp16 does not hold of a weight, 2^-34 of the largest p * scale, at codes up to 127 and a scale of
    up to 1.9 times its power of two. ds = 2^-19 of the score, plus 2^-20."""
    rng = np.random.default_rng(["seen", "past", "drawn"].index(what))
    D, hkv = 32, 8
    cases = blocks_of(what)
    if what == "drawn":
        cases = [[(-(e + 105) + rng.uniform(-5, 0), e) for e in rng.integers(-105, 112, 3)] for _ in range(6)]
        cases = [[(min(s, 0.0), int(e)) for s, e in c] for c in cases]
    if dtype == "f16":    # what its range holds of the outputs: the block of the largest score has values near 1
        cases = [[(s, e + up) for s, e in c] for c in cases for up in [-max(c)[1] - 4] if max(e for _, e in c) + up < 120]
        cases.append([(0, -3), (-118, 117)])
    lens, T, G = ([317] * 57 if many else [317]), rows, 1
    for c in cases:
        kinds = [c[int(rng.integers(len(c)))] for _ in range(10)]
        kinds[:len(c)] = c
        ref = scaled_blocks(rng, [s for s, _ in kinds], [e for _, e in kinds], D, hkv)
        q = torch.zeros((len(lens), T, hkv * G, D), dtype=R.TYPES[dtype], device="cuda")
        q[..., 0] = 1
        pool, table = dev(ref.pool), dev(np.repeat(ref.table, len(lens), 0))
        got, lse = m.kv8_attention(q, pool, table, ints(lens), scale=1.0, with_lse=True)
        got, lse = got.double().cpu().numpy(), lse.double().cpu().numpy()
        k, v = (x.astype(np.float64) for x in ref.read(0, 0, 317))
        s = k[:, :, 0].T  # [heads, tokens]: the query is one in dim 0
        power = np.repeat([e for _, e in kinds], 32)[:317]
        for t in range(T):
            n = 317 - T + t + 1
            p = np.exp(s[:, :n] - s[:, :n].max(1, keepdims=True))
            total = p.sum(1, keepdims=True)
            out = np.einsum("hn,nhd->hd", p, v[:n]) / total
            size = np.einsum("hn,nhd->hd", p * (2 * (2.0 ** -19 * np.abs(s[:, :n]) + 2.0 ** -20) + (0 if dtype == "f32" else 2.0 ** -11) + 2.0 ** -17),
                             np.abs(v[:n])) / total
            lost = n * 2.0 ** -34 * 254 * (p * 2.0 ** power[:n]).max(1, keepdims=True) / total
            least = 2.0 ** -25 if dtype == "f16" else 2.0 ** -134
            tol = size + lost + 2 * R.HALF_ULP[dtype] * np.abs(out) + least
            fits = np.abs(out) + tol < float(torch.finfo(R.TYPES[dtype]).max)
            assert fits.all()
            assert (np.abs(got[:, t] - out) <= tol).all(), (c, t)
            want = s[:, :n].max(1) + np.log(total[:, 0])
            assert (np.abs(lse[:, t] - want) <= 2.0 ** -17 * (1 + np.abs(want))).all()


@pytest.mark.parametrize("T,tree", [(1, False), (3, False), (3, True)])
def test_last_positions(m, T, tree):
    """Lengths up to 2^31 - 1, over two pages of 2^20 tokens that the table names by turns."""
    rng = np.random.default_rng(30)
    D, page = 32, 1 << 20
    pool = m.kv8_pool(2, 1, D, page)
    part = R.random_pool(rng, 2, 1, D, 128)
    pool[:, :, -4:] = dev(part)      # the ends of the pages are the only blocks that a short window reaches
    ref = R.Cache(part, np.array([[0, 1]], np.int32))
    table = ints([0, 1] * 1024).view(1, 2048)
    q = torch.randn((1, T, 3, D), device="cuda")
    bits = ints([[1, 3, 5]]) if tree else None
    for n in [(1 << 31) - 1, (1 << 31) - 30, (1 << 31) - 33]:
        # of the window's last 128 positions: those of page 1's last four blocks
        end = 256 - ((1 << 31) - n)
        for window in (1, 40, 90):
            got = m.kv8_attention(q, pool, table, ints([n]), window=window, tree=bits)
            want, _, reach, size = R.attention(q.double().cpu().numpy(), ref, [end], D ** -0.5, window, None if bits is None else bits.cpu().numpy())
            tol = reach * (2 * (2.0 ** -19 * size + 2.0 ** -20)[..., None] + 2.0 ** -17) + 2.0 ** -23 * np.abs(want) + 2.0 ** -26
            assert (np.abs(got.double().cpu().numpy() - want) <= tol).all(), (n, window)
    # and written there
    start, n = (1 << 31) - 49, 48
    x = torch.randn((2, n, 1, D), device="cuda")
    err = ints([0])
    m.kv8_write(x[0], x[1], pool, table, ints([0, n]), ints([start]), err=err)
    k, v = m.kv8_read(pool, table, ints([0, n]), ints([start]), n, dtype=torch.float32, err=err)
    assert int(err) == 0
    old = ref.block(0, 6).copy()
    ref.write(0, 256 - 49, [a.cpu().numpy() for a in x])
    want = ref.read(0, 256 - 49, 255)
    assert np.array_equal(k.cpu().numpy(), want[0]) and np.array_equal(v.cpu().numpy(), want[1])
    assert not np.array_equal(old, ref.block(0, 6))


@pytest.mark.parametrize("dtype", list(R.TYPES))
@pytest.mark.parametrize("T,window", [(2, 1), (8, 3), (8, 40), (13, 33), (32, 5), (32, 64), (9, 0), (9, 1000)])
def test_tree_depths(m, T, window, dtype):
    """With depths, each draft token sees under a sliding window what decoding its path token by token would: the last
    `window` tokens of context, ancestors and itself. Tolerance as in test_gpu_kv8_attention.py."""
    rng = np.random.default_rng(40 + T + window)
    lens, hq, hkv, D = [T, T + 1, 70, 200, T + 31], 6, 2, 64
    table, n_pages = R.page_table(rng, lens, 32)
    ref = R.Cache(R.random_pool(rng, n_pages, hkv, D, 32), table)
    q = torch.from_numpy(rng.standard_normal((len(lens), T, hq, D)).astype(np.float32)).to(R.TYPES[dtype])
    paths, bits, depth = [], [], []
    for _ in lens:
        path = [[0]]
        for t in range(1, T):  # a child of an earlier token, or another first token
            parent = int(rng.integers(-1, t))
            path.append((path[parent] if parent >= 0 else []) + [t])
        paths.append(path)
        bits.append([sum(1 << w for w in p) - (1 << 32 if 31 in p else 0) for p in path])
        depth.append([len(p) - 1 for p in path])
    err = ints([0])
    got = m.kv8_attention(q.cuda(), dev(ref.pool), dev(table), ints(lens), window=window, tree=ints(bits), depth=ints(depth), err=err)
    got, q = got.double().cpu().numpy(), q.double().numpy()
    assert int(err) == 0
    for b, n in enumerate(lens):
        k, v = (x.astype(np.float64) for x in ref.read(b, 0, n))
        for t, path in enumerate(paths[b]):
            see = (list(range(n - T)) + [n - T + w for w in path])[-window:]
            for h in range(hq):
                kk, vv = k[see, h // 3], v[see, h // 3]
                s = kk @ q[b, t, h] * D ** -0.5
                e = np.exp(s - s.max())
                out, ds = e @ vv / e.sum(), 2.0 ** -19 * (np.abs(kk) @ np.abs(q[b, t, h])).max() * D ** -0.5 + 2.0 ** -20
                tol = np.abs(vv).max() * (2 * ds + (0 if dtype == "f32" else 2.0 ** -11) + 2.0 ** -17) + 2 * R.HALF_ULP[dtype] * np.abs(out) + 2.0 ** -26
                assert (np.abs(got[b, t, h] - out) <= tol).all(), (b, t, h)


def test_tree_depths_refused(m):
    rng = np.random.default_rng(50)
    ref = R.Cache(R.random_pool(rng, 3, 1, 64, 64), np.array([[0, 1]], np.int32))
    q, pool, table, lens = torch.randn((1, 3, 2, 64), device="cuda"), dev(ref.pool), dev(ref.table), ints([100])
    tree = ints([[1, 3, 5]])
    with pytest.raises(m.MoeError):
        m.kv8_attention(q, pool, table, lens, window=9, depth=ints([[0, 1, 1]]))
    with pytest.raises(m.MoeError):
        m.kv8_attention(q, pool, table, lens, window=9, tree=tree, depth=ints([0, 1]))
    # a depth that no token has at its index counts as the nearest
    got = m.kv8_attention(q, pool, table, lens, window=2, tree=tree, depth=ints([[5, -1, 3]]))
    assert torch.equal(got, m.kv8_attention(q, pool, table, lens, window=2, tree=tree, depth=ints([[0, 0, 2]])))
    # every token a child of the one before: the window's own positions
    tree = ints([[1, 3, 7]])
    got = m.kv8_attention(q, pool, table, lens, window=2, tree=tree, depth=ints([[0, 1, 2]]))
    assert torch.equal(got, m.kv8_attention(q, pool, table, lens, window=2, tree=tree))
    # and with the widest window there is, in a sequence shorter than the queries
    for n in (2, 100):
        got = m.kv8_attention(q, pool, table, ints([n]), window=(1 << 31) - 1, tree=tree, depth=ints([[0, 1, 1]]))
        assert torch.equal(got, m.kv8_attention(q, pool, table, ints([n]), tree=tree))


@pytest.mark.parametrize("rows", [1, 20])
def test_copy_that_does_not_arrive(m, rows):
    """The abort path: no stage's barrier completes. Every wait gives up, the call ends with MOE_ERR_TIMEOUT, and the
    next call, on the same workspace, is right."""
    import ctypes
    rng = np.random.default_rng(60)
    lens, D = [400, 90], 256
    table, n_pages = R.page_table(rng, lens, 64)
    ref = R.Cache(R.random_pool(rng, n_pages, 1, D, 64), table)
    pool, table, lens = dev(ref.pool), dev(table), ints(lens)
    q = torch.randn((2, rows, 1, D), device="cuda")
    want = m.kv8_attention(q, pool, table, lens)
    out, ws, err = torch.zeros_like(q), m.kv8_attention_workspace(2, rows, 1, 1, D), ints([0])
    cache = m.KV8CacheC(pool=pool.data_ptr(), n_pages=n_pages, n_kv_heads=1, head_dim=D, page_tokens=64, page_table=table.data_ptr(),
                        table_stride=table.shape[1], max_pages=table.shape[1], n_seqs=2)
    call = m.KV8AttentionC(cache=cache, q=q.data_ptr(), type=0, T=rows, n_heads=1, q_seq_stride=rows * D, q_token_stride=D, q_head_stride=D,
                           lens=lens.data_ptr(), scale=D ** -0.5, out=out.data_ptr(), workspace=ws.data_ptr(), workspace_bytes=ws.numel(),
                           err=err.data_ptr(), flags=m.F_TEST_EXPIRE)
    stream = ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    assert m.lib().moe_kv8_attention(ctypes.byref(call), stream) == 0
    torch.cuda.synchronize()
    assert int(err) == 64
    err.zero_()
    call.flags = 0
    assert m.lib().moe_kv8_attention(ctypes.byref(call), stream) == 0
    assert torch.equal(out, want) and int(err) == 0


@pytest.mark.parametrize("dtype,queries,keys", [("bf16", 104, -104), ("f32", 104, -104), ("f32", -95, 95), ("bf16", -95, 95), ("f16", 104, -104), ("f16", -95, 95),
                                                ("f32", -110, 112), ("bf16", 115, -105)])
def test_query_ranges(m, dtype, queries, keys):
    """scale * max |q| at the ends of its range, with keys that bring the scores back to size (16-bit queries of fp16 by
    the scale alone). Tolerance as in test_gpu_kv8_attention.py."""
    rng = np.random.default_rng(70)
    lens, T, D = [700, 33], 3, 64
    table, n_pages = R.page_table(rng, lens, 32)
    pool = R.random_pool(rng, n_pages, 2, D, 32)
    s = pool[..., :4].copy().view(np.float32) * np.float32(2.0 ** keys)
    pool[..., :4] = s.view(np.uint8)
    ref = R.Cache(pool, table)
    q = rng.standard_normal((2, T, 4, D)).astype(np.float32)
    q /= np.abs(q).max(-1, keepdims=True)  # at most one
    part = 0 if dtype == "f16" else queries + 8 if queries > 0 else queries - 5  # of the power, in the queries; the rest in the scale
    q = torch.from_numpy(q * np.float32(2.0 ** part)).to(R.TYPES[dtype])
    scale = 2.0 ** (queries - part)
    got, lse = m.kv8_attention(q.cuda(), dev(ref.pool), dev(table), ints(lens), scale=scale, with_lse=True)
    out, want, reach, size = R.attention(q.double().numpy(), ref, lens, scale)
    ds = 2.0 ** -19 * size + 2.0 ** -20
    tol = reach * (2 * ds[..., None] + (0 if dtype == "f32" else 2.0 ** -11) + 2.0 ** -17) + 2 * R.HALF_ULP[dtype] * np.abs(out) + 2.0 ** -26
    assert (np.abs(got.double().cpu().numpy() - out) <= tol).all()
    assert (np.abs(lse.double().cpu().numpy() - want) <= ds + 2.0 ** -18 * (1 + np.abs(want))).all()
