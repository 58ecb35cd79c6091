"""The paged 8-bit cache (moe_kv8_write, moe_kv8_read) against its definition, bit for bit: every
step is one fp32 operation, so codes, scales and read-back values must be the reference's."""
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
    return torch.tensor(list(v), dtype=torch.int32, device="cuda")


class Case:
    def __init__(self, seed, starts, counts, hkv, D, page, extra=0):
        rng = self.rng = np.random.default_rng(seed)
        self.starts, self.counts = starts, counts
        table, n_pages = R.page_table(rng, [s + n + extra for s, n in zip(starts, counts)], page)
        self.ref = R.Cache(R.random_pool(rng, n_pages, hkv, D, page), table)
        self.pool, self.table = dev(self.ref.pool), dev(table)
        self.cu = np.concatenate([[0], np.cumsum(counts)])
        self.N, self.hkv, self.D = int(self.cu[-1]), hkv, D
        self.err = torch.zeros(1, dtype=torch.int32, device="cuda")

    def rows(self, dtype, layout="dense"):
        """k, v on the device (strided as `layout` says) and their fp32 values."""
        x = torch.from_numpy(self.rng.standard_normal((2, self.N, self.hkv, self.D)).astype(np.float32)
                             * np.exp(self.rng.uniform(-3, 3, (2, self.N, 1, 1))).astype(np.float32)).to(R.TYPES[dtype])
        if layout == "dense":
            k, v = x[0].cuda(), x[1].cuda()
        elif layout == "fused":  # slices of one projection's rows
            buf = torch.full((self.N, 5 * self.hkv, self.D), float("nan"), dtype=x.dtype, device="cuda")
            k, v = buf[:, 2 * self.hkv:3 * self.hkv], buf[:, 3 * self.hkv:4 * self.hkv]
        elif layout == "odd":    # rows that no vector load may touch
            buf = torch.full((2, self.N, self.hkv, self.D + 1), float("nan"), dtype=x.dtype, device="cuda")
            k, v = buf[0, :, :, 1:], buf[1, :, :, 1:]
        else:                    # heads before tokens
            buf = torch.empty((2, self.hkv, self.N, self.D), dtype=x.dtype, device="cuda")
            k, v = buf[0].transpose(0, 1), buf[1].transpose(0, 1)
        if layout != "dense":
            k.copy_(x[0])
            v.copy_(x[1])
        return k, v, [a.float().numpy() for a in x]

    def expect(self, xs):
        for b, (s, n) in enumerate(zip(self.starts, self.counts)):
            self.ref.write(b, s, [x[self.cu[b]:self.cu[b] + n] for x in xs])

    def same(self):
        """Every position that the sequences hold, codes and scales, is the reference's."""
        got = R.Cache(self.pool.cpu().numpy(), self.ref.table)
        for b, (s, n) in enumerate(zip(self.starts, self.counts)):
            for j in range((s + n + 31) // 32):
                t1 = min(32, s + n - 32 * j)
                for h in range(self.hkv):
                    for w in range(2):
                        c, a = got.codes(b, j, h, w)
                        e, r = self.ref.codes(b, j, h, w)
                        assert np.array_equal(np.float32(a).view(np.uint32), np.float32(r).view(np.uint32)) or \
                            (np.isnan(a) and np.isnan(r)), (b, j, h, w, a, r)
                        assert np.array_equal(c[:t1], e[:t1]), (b, j, h, w)
        assert int(self.err) == 0


SHAPES = [
    # starts, counts, kv heads, head dim, page
    ([0], [1], 1, 32, 32),
    ([0, 31, 32, 33], [1, 1, 1, 1], 2, 64, 32),
    ([5, 0, 63, 30, 17], [4, 0, 4, 4, 3], 4, 128, 64),
    ([0, 7], [200, 131], 3, 96, 128),
    ([40], [95], 2, 256, 32),
    ([3, 0, 0, 100] * 10, [2, 33, 0, 1] * 10, 1, 64, 32),
    ([1, 64], [64, 32], 8, 160, 64),
]


@pytest.mark.parametrize("dtype", list(R.TYPES))
@pytest.mark.parametrize("shape", range(len(SHAPES)))
def test_write_and_read(m, shape, dtype):
    c = Case(shape, *SHAPES[shape])
    k, v, xs = c.rows(dtype, ["dense", "fused", "odd", "heads"][shape % 4])
    c.expect(xs)
    m.kv8_write(k, v, c.pool, c.table, ints(c.cu), ints(c.starts), err=c.err)
    c.same()
    # the whole sequences back, in each type
    whole = [s + n for s, n in zip(c.starts, c.counts)]
    cu = np.concatenate([[0], np.cumsum(whole)])
    ref = [c.ref.read(b, 0, n) for b, n in enumerate(whole)]
    for out in R.TYPES.values():
        got = m.kv8_read(c.pool, c.table, ints(cu), ints([0] * len(whole)), int(cu[-1]), dtype=out, err=c.err)
        for w in range(2):
            want = torch.from_numpy(np.concatenate([r[w] for r in ref])).to(out)
            assert torch.equal(got[w].cpu(), want)
    # a range, into strided rows
    p0 = [min(3, n) for n in whole]
    cu = np.concatenate([[0], np.cumsum([n - p for n, p in zip(whole, p0)])])
    buf = torch.full((int(cu[-1]), c.hkv, 2, c.D + 3), 7.0, dtype=torch.float32, device="cuda")
    m.kv8_read(c.pool, c.table, ints(cu), ints(p0), int(cu[-1]), k=buf[:, :, 0, 1:c.D + 1], v=buf[:, :, 1, :c.D], err=c.err)
    want = [np.concatenate([r[w][p:] for r, p in zip(ref, p0)]) for w in range(2)]
    got = buf.cpu().numpy()
    assert np.array_equal(got[:, :, 0, 1:c.D + 1], want[0]) and np.array_equal(got[:, :, 1, :c.D], want[1])
    assert (got[:, :, 0, 0] == 7).all() and (got[:, :, 0, c.D + 1:] == 7).all() and (got[:, :, 1, c.D:] == 7).all()
    assert int(c.err) == 0


def test_write_one_by_one_and_again(m):
    """Tokens appended one and two at a time over a block edge, each step against the reference; a
    repeated write leaves the same bytes; a rejected draft is written over."""
    c = Case(11, [30], [1], 2, 64, 32, extra=12)
    pos = 30
    for n in [1, 1, 2, 1, 4]:
        c.starts, c.counts, c.cu, c.N = [pos], [n], np.array([0, n]), n
        k, v, xs = c.rows("bf16")
        c.expect(xs)
        for _ in range(2):
            m.kv8_write(k, v, c.pool, c.table, ints(c.cu), ints(c.starts), err=c.err)
            c.same()
        pos += n
    c.starts, c.counts, c.cu, c.N = [pos - 3], [2], np.array([0, 2]), 2
    k, v, xs = c.rows("bf16")
    c.expect(xs)
    m.kv8_write(k, v, c.pool, c.table, ints(c.cu), ints(c.starts), err=c.err)
    c.same()


@pytest.mark.parametrize("what", ["zero", "tiny", "huge", "inf", "nan", "zero_after", "nan_kept", "negative_zero"])
def test_write_values(m, what):
    """Blocks of zeros, below and above the range, and not finite; keys and values on their own."""
    c = Case(12, [5], [40], 2, 32, 32)
    k, v, xs = c.rows("f32")
    if what == "zero":
        k.zero_()
    elif what == "tiny":
        k.mul_(2.0 ** -103)
        v.mul_(2.0 ** -95)
    elif what == "huge":
        k.copy_(torch.where(k.abs() > 1, 3.3e38, -1e38))
    elif what == "inf":
        v[3, 1, 7] = -float("inf")
    elif what == "nan":
        k[30, 0, 0] = float("nan")
    elif what == "zero_after":
        k[:27].zero_()
        v[:27].fill_(1e-35)
    elif what == "nan_kept":
        c.ref.block(0, 0)[1, :4] = np.frombuffer(np.float32(np.nan).tobytes(), np.uint8)
        c.pool.copy_(dev(c.ref.pool))
    else:
        k.fill_(-0.0)
    c.expect([k.cpu().numpy(), v.cpu().numpy()])
    m.kv8_write(k, v, c.pool, c.table, ints(c.cu), ints(c.starts), err=c.err)
    c.same()
    got = m.kv8_read(c.pool, c.table, ints([0, 45]), ints([0]), 45, dtype=torch.float32)
    for w in range(2):
        assert np.array_equal(got[w].cpu().numpy(), c.ref.read(0, 0, 45)[w], equal_nan=True)


def test_untouched(m):
    """Blocks that the call does not reach keep their bytes."""
    c = Case(13, [32, 10], [20, 0], 2, 64, 64)
    before = c.pool.clone()
    k, v, xs = c.rows("f16")
    m.kv8_write(k, v, c.pool, c.table, ints(c.cu), ints(c.starts), err=c.err)
    changed = (c.pool != before).flatten(3).any(-1).nonzero().tolist()
    page = int(c.ref.table[0, 0])
    assert sorted(map(tuple, changed)) == [(page, 0, 1), (page, 1, 1)]


@pytest.mark.parametrize("what", ["page_low", "page_high", "past_table", "start", "cu"])
def test_bad_device_data(m, what):
    """Bad pages and ranges are skipped and reported; the other sequence is written."""
    c = Case(14, [0, 3], [40, 40], 1, 32, 32)
    k, v, xs = c.rows("f32")
    before = c.pool.clone()
    table, starts, cu = c.table.clone(), list(c.starts), list(c.cu)
    if what == "page_low":
        table[0] = -1
    elif what == "page_high":
        table[0] = c.pool.shape[0]
    elif what == "past_table":
        starts[0] = 32 * table.shape[1]
    elif what == "start":
        starts[0] = -1
    else:
        cu[0] = -5
    m.kv8_write(k, v, c.pool, table, ints(cu), ints(starts), err=c.err)
    bits = int(c.err)
    assert bits == (256 if what in ("page_low", "page_high", "past_table") else 512)
    c.ref.write(1, 3, [x[40:] for x in xs])
    c.err.zero_()
    c.starts[0] = c.counts[0] = 0
    c.same()
    own = {int(p) for p in c.ref.table[0] if p >= 0}
    for p in own:
        assert torch.equal(c.pool[p], before[p])
    out = torch.full((2, 80, 1, 32), 5.0, device="cuda")
    m.kv8_read(c.pool, table, ints(cu), ints(starts), 80, k=out[0], v=out[1], err=c.err)
    assert int(c.err) == bits and (out[:, :40] == 5).all() and not (out[:, 40:] == 5).all()


def test_offsets_past_32_bits(m):
    """A pool of more than 4 GiB: records in its last pages."""
    hkv, D, page = 2, 256, 128
    n_pages = (1 << 32) // (hkv * 4 * m.kv8_block_bytes(D)) + 4
    pool = torch.empty((n_pages, hkv, page // 32, m.kv8_block_bytes(D)), dtype=torch.uint8, device="cuda")
    rng = np.random.default_rng(15)
    x = torch.from_numpy(rng.standard_normal((2, 130, hkv, D)).astype(np.float32)).cuda()
    table = ints([n_pages - 1, n_pages - 2]).view(1, 2)
    m.kv8_write(x[0], x[1], pool, table, ints([0, 130]), ints([0]))
    ref = R.Cache(R.random_pool(rng, 2, hkv, D, page), np.array([[1, 0]], np.int32))
    ref.write(0, 0, [a.cpu().numpy() for a in x])
    got = m.kv8_read(pool, table, ints([0, 130]), ints([0]), 130, dtype=torch.float32)
    for w in range(2):
        assert np.array_equal(got[w].cpu().numpy(), ref.read(0, 0, 130)[w])


def test_other_stream(m):
    c = Case(16, [9], [300], 4, 128, 64)
    k, v, xs = c.rows("bf16")
    c.expect(xs)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    m.kv8_write(k, v, c.pool, c.table, ints(c.cu), ints(c.starts), err=c.err, stream=s)
    got = m.kv8_read(c.pool, c.table, ints([0, 309]), ints([0]), 309, dtype=torch.float32, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    c.same()
    assert np.array_equal(got[1].cpu().numpy(), c.ref.read(0, 0, 309)[1])
