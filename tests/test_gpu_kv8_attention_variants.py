"""moe_kv8_attention where a warp takes many blocks, a CTA several sequences and a call more rows than one tile:
each of the kernels that the host's rules choose between, against the formula in 64 bits (on the GPU, from the
records' definition). Sequences share pages, which they only read.

Tolerance as in test_gpu_kv8_attention.py: a score is off by at most ds = 2^-19 * scale * sum |q| |k| + 2^-20, the output by
2 ds, 2^-11 for weights held in fp16, and 2^-17, of the largest |v|. What a warp sums over more than a few blocks adds its
roundings: four additions of weights a block and two products' sums of 16 (2^-23 each, as they may truncate), less than
2^-21 a block."""
import math

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


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def dense(pool):
    """Every page's keys and values in 64 bits, [pages * page tokens, heads, D]."""
    n, hkv, nb, rec = pool.shape
    D = (rec - 16) // 64
    scale = pool[..., :8].contiguous().view(torch.float32).double()
    out = []
    for w, at in enumerate((R.k_index(D), R.v_index(D))):
        x = pool[..., torch.from_numpy(at).cuda().view(-1)].double().view(n, hkv, nb, 32, D) - 128
        out.append((x * scale[..., w, None, None]).permute(0, 2, 3, 1, 4).reshape(n * nb * 32, hkv, D))
    return out


def attention64(q, k, v, n, scale, window, tree):
    """One sequence: q [T, hq, D] and its n positions' k, v [.., hkv, D] -> out, lse, and max |v|, max scale * sum |q| |k| per row."""
    T, hq, D = q.shape
    hkv = k.shape[1]
    qg = q.view(T, hkv, hq // hkv, D)
    j = torch.arange(n, device="cuda")
    p = n - T + torch.arange(T, device="cuda")[:, None]
    if tree is None:
        see = j <= p
    else:
        w = j - (n - T)
        see = (w < 0) | (tree[:, None].long() >> w.clamp(0, 31) & 1).bool()
    see = see & (p >= 0)
    if window:
        see = see & (j > p - window)
    see = see[:, None, None]
    s = (torch.einsum("thgd,nhd->thgn", qg, k) * scale).masked_fill(~see, -math.inf)
    size = (torch.einsum("thgd,nhd->thgn", qg.abs(), k.abs()) * abs(scale)).masked_fill(~see, 0).amax(-1)
    top = s.amax(-1, keepdim=True)
    e = (s - top.masked_fill(top == -math.inf, 0)).exp()
    total = e.sum(-1)
    out = torch.einsum("thgn,nhd->thgd", e, v) / total.masked_fill(total == 0, 1)[..., None]
    lse = top[..., 0] + total.log()
    reach = v.abs().amax(-1).T[None, :, None].masked_fill(~see, 0).amax(-1).expand(size.shape)
    return out.reshape(T, hq, D), lse.reshape(T, hq), reach.reshape(T, hq, 1), size.reshape(T, hq)


def run(m, seed, dtype, lens, T, hq, hkv, D, page=64, width=0, window=0, tree=False, blocks=64):
    """blocks: at most so many blocks a warp."""
    g = torch.Generator("cuda").manual_seed(seed)
    rng = np.random.default_rng(seed)
    need = -(-max(max(lens), 1) // page)
    n_pages = need + 5
    pool = torch.randint(1, 256, (n_pages, hkv, page // 32, 64 * D + 16), dtype=torch.uint8, generator=g, device="cuda")
    # scales that move the running maxima, keys' and values' on their own
    s = 0.05 * torch.exp(0.7 * torch.randn((n_pages, hkv, page // 32, 2), generator=g, device="cuda"))
    pool[..., :8] = s.view(torch.uint8).view(n_pages, hkv, page // 32, 8)
    table = np.full((len(lens), max(need, width)), -1, np.int32)
    for b, n in enumerate(lens):
        c = -(-n // page)
        table[b, :c] = rng.permutation(n_pages)[:c]
    q = torch.randn((len(lens), T, hq, D), generator=g, device="cuda").to(R.TYPES[dtype])
    bits = ints(rng.integers(0, 1 << T, (len(lens), T)).tolist()) if tree else None
    err = ints([0])
    got, lse = m.kv8_attention(q, pool, torch.from_numpy(table).cuda(), ints(lens), window=window, tree=bits, with_lse=True, err=err)
    again = m.kv8_attention(q, pool, torch.from_numpy(table).cuda(), ints(lens), window=window, tree=bits)
    assert int(err) == 0 and torch.equal(got, again)
    k, v = dense(pool)
    for b, n in enumerate(lens):
        if n == 0:
            assert (got[b] == 0).all() and torch.isneginf(lse[b]).all()
            continue
        rows = (torch.from_numpy(table[b, :-(-n // page)]).cuda().long()[:, None] * page + torch.arange(page, device="cuda")).view(-1)[:n]
        out, want, reach, size = attention64(q[b].double(), k[rows], v[rows], n, D ** -0.5, window, None if bits is None else bits[b])
        ds = 2.0 ** -19 * size + 2.0 ** -20
        sums = 2.0 ** -17 + 2.0 ** -21 * blocks
        tol = reach * (2 * ds[..., None] + (0 if dtype == "f32" else 2.0 ** -11) + sums) + 2 * R.HALF_ULP[dtype] * out.abs() + 2.0 ** -26
        far = (got[b].double() - out).abs() / tol
        assert float(far.max()) <= 1, (b, n, float(far.max()))
        empty = torch.isneginf(want)
        assert torch.equal(torch.isneginf(lse[b]), empty) and (got[b][empty] == 0).all()
        assert ((lse[b].double() - want).abs() <= ds + sums * (1 + want.abs()))[~empty].all()


def ragged(n, top, seed):
    """n lengths up to top, over their logarithm, some 0 and one `top`."""
    rng = np.random.default_rng(seed)
    v = np.exp(rng.uniform(0, np.log(top), n)).astype(int)
    v[rng.integers(0, n, n // 10)] = 0
    v[n // 2] = top
    return v.tolist()


@pytest.mark.parametrize("dtype", list(R.TYPES))
@pytest.mark.parametrize("window,tree", [(0, False), (0, True), (400, False), (33, True)])
def test_several_sequences_a_cta(m, dtype, window, tree):
    """More segments than CTAs: ranges of equal cost that begin and end within sequences; more than 32 sequences."""
    run(m, 1 + window, dtype, ragged(120, 1500, 3), 3, 16, 8, 64, window=window, tree=tree)


@pytest.mark.parametrize("dtype", list(R.TYPES))
@pytest.mark.parametrize("lens", ["short", "long", "one_long"])
def test_many_sequences_few_segments(m, lens, dtype):
    """More than 32 sequences of one key/value head: left whole, or cut into even parts."""
    v = {"short": ragged(70, 1400, 4), "long": ragged(45, 9000, 5), "one_long": [40] * 50 + [30000]}[lens]
    run(m, 20, dtype, v, 2, 4, 1, 96, page=32)


@pytest.mark.parametrize("dtype", list(R.TYPES))
@pytest.mark.parametrize("D", [32, 128, 160, 256])
def test_two_warps_a_ring(m, D, dtype):
    """17 to 32 rows, sequences longer than a ring: both warps release a stage before it is filled again."""
    lens = [1660 - 29 * (i % 11) for i in range(57)]
    run(m, 30 + D, dtype, lens, 4, 40, 8, D)


@pytest.mark.parametrize("dtype", list(R.TYPES))
@pytest.mark.parametrize("D", [64, 192])
def test_passes_over_rows(m, D, dtype):
    """More rows than one pass takes, over several blocks a warp."""
    run(m, 40 + D, dtype, [1500, 0, 1, 700, 1213] * 4, 7, 40, 2, D, page=128)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("D", [32, 64, 96, 128])
@pytest.mark.parametrize("rows", [20, 32, 40, 130])
def test_two_tiles_a_warp(m, rows, D, dtype):
    """Page tables of 24,576 blocks or more: two row tiles a warp, one or two warps a ring, one pass or more; few
    sequences under wide tables, and as many segments as there are CTAs."""
    T = 5 if rows % 5 == 0 else 4
    run(m, 50 + rows, dtype, [900, 77, 0, 1333], T, rows // T * 2, 2, D, width=4 * 400, window=0 if rows % 3 else 700, tree=rows == 40)
    run(m, 60 + rows, dtype, ragged(60, 1664, 6)[:59] + [1664], T, rows // T * 8, 8, D)


@pytest.mark.parametrize("rows", [20, 48])
def test_weights_in_one_part(m, rows):
    """fp16, more than 16 rows, page tables of 4096 blocks or more (and fewer than 24,576)."""
    run(m, 70, "f16", [1000, 64, 2200], 4, rows // 4 * 2, 2, 128, width=600)


@pytest.mark.parametrize("dtype", list(R.TYPES))
@pytest.mark.parametrize("D", [64, 96, 256])
def test_joining_many_rows(m, D, dtype):
    """More than 768 rows in parts: joined by a warp each."""
    run(m, 80 + D, dtype, [3000, 1, 0, 450, 1999, 33, 777, 2048], 4, 32, 8, D)


@pytest.mark.parametrize("dtype", list(R.TYPES))
@pytest.mark.parametrize("D,n,T,hq,hkv", [(128, 131077, 4, 16, 4), (96, 100003, 1, 7, 1), (256, 130001, 2, 8, 1), (64, 200001, 5, 4, 1), (192, 60001, 2, 32, 2)])
def test_long_context(m, D, n, T, hq, hkv, dtype):
    """One sequence over the whole device, each warp several blocks, up to the most parts; keys drawn at random, so
    that the parts' maxima differ."""
    run(m, 90, dtype, [n], T, hq, hkv, D, page=128)


def test_wide_table_same_result(m):
    """A page table wider than its sequences need changes what a call is cut into, and its error, but not beyond the bound."""
    for width in (0, 40, 5000):
        for dtype in R.TYPES:
            run(m, 95, dtype, [777], 1, 16, 4, 128, width=width)
            run(m, 96, dtype, [200, 3000], 4, 16, 2, 64, width=width)
