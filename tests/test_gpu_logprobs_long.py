"""Log probabilities of rows above 48 KB, whose CTA goes through several spans of them: signs where one token has all of the
probability, rows that are hard on the picking of the best keys in spans after the first, many rows (a CTA each) and few (several each).
Values against the formulas in 64 bits, as in test_gpu_logprobs.py."""
import numpy as np
import pytest
import torch

import kv8_ref as K
from test_gpu_logprobs import check, ids_for

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def m():
    import quantized_routed_expert_grouped_gb300 as mod
    mod.lib()
    return mod


@pytest.mark.parametrize("dtype", list(K.TYPES))
@pytest.mark.parametrize("V", [300, 20001, 70001])
@pytest.mark.parametrize("R_", [40, 320])
def test_signs(m, R_, V, dtype):
    """Where one token has nearly all of the probability, its log is at most 0, and the entropy at least 0."""
    rng = np.random.default_rng(V)
    at = rng.integers(0, V, R_)
    best = 7.3 + 0.37 * np.arange(R_) % 9 - 4
    x = best[:, None] - 30 - 10 * rng.random((R_, V))
    x[np.arange(R_), at] = best
    x[::3] = np.where(x[::3] < best[::3, None] - 1, -60000.0, x[::3])
    x[1::6] = np.where(x[1::6] < best[1::6, None] - 1, -np.inf, x[1::6])
    dev = torch.from_numpy(x).to(K.TYPES[dtype]).cuda()
    ids = torch.from_numpy(at.astype(np.int32)).cuda().view(-1, 1)
    for scale in (1.0, 1 / 0.7, 3.0, 1000.0):
        lp, tl, ti, ent, _ = m.token_logprobs(dev, ids, top=3, scale=scale)
        assert torch.equal(ti[:, :1], ids)
        assert bool((lp <= 0).all() and (tl <= 0).all() and (ent >= 0).all()), (float(lp.max()), float(tl.max()), float(ent.min()))
        check(m, dev[:12], at[:12, None], 3, scale)


def batch(x, dtype, copies, aligned):
    """`copies` copies of rows x on the device, all at a 16-byte boundary (then equal rows give equal bits) or one behind another."""
    x = torch.from_numpy(x).to(K.TYPES[dtype]).cuda()
    V = x.shape[1]
    out = torch.zeros((copies * len(x), -(-V // 8) * 8 if aligned else V), dtype=x.dtype, device="cuda")[:, :V]
    return out.copy_(x.repeat(copies, 1))


def check_first(m, dev, ids, top, n):
    """check() of the first n rows as a call with all rows gives them."""
    class All:
        @staticmethod
        def token_logprobs(x, some, top, scale):
            return [t[:n] for t in m.token_logprobs(dev, torch.from_numpy(ids.astype(np.int32)).cuda(), top=top, scale=scale)]
    check(All, dev[:n], ids[:n], top)


@pytest.mark.parametrize("dtype", list(K.TYPES))
@pytest.mark.parametrize("V", [70001, 131075])
def test_hard_rows_in_number(m, V, dtype):
    """Rows whose order, masks or ties are hard on a selection, so many that each is one CTA's, over several spans; rows with a NaN or an
    infinity among them."""
    low = torch.finfo(K.TYPES[dtype]).min
    rng = np.random.default_rng(V)
    i = np.arange(V)
    few = np.full(V, -np.inf)
    few[rng.integers(0, V, 3)] = 1.0
    lowest = np.full(V, low)
    lowest[[0, V // 2, V - 1]] = [1.0, 2.0, 1.0]
    late = np.full(V, low)
    late[-40000:] = np.round(rng.standard_normal(40000))
    rows = [np.full(V, -np.inf), np.full(V, 3.0), np.full(V, low), i * 10.0 / V, -i * 10.0 / V, few, lowest, np.where(rng.random(V) < 0.5, -0.0, 0.0),
            np.where(i % 3 == 0, -np.inf, low), np.round(rng.standard_normal(V)), np.where(i == V - 1, 0.0, -np.inf), np.where(i < V // 2, -np.inf, 5.0 * i / V), late,
            np.where(i % 8 == 7, 4.0, -4.0), np.where(rng.random(V) < 1e-4, rng.standard_normal(V), -1e4), np.where(rng.random(V) < 0.999, low, rng.standard_normal(V))]
    n = len(rows)
    x = np.stack(rows)
    for aligned, tops in ((True, (1, 5, 32)), (False, (20,))):
        dev = batch(x, dtype, 20, aligned)
        bad = [0, 4, 9, 12]  # (of the third copy)
        dev[2 * n + bad[0], V // 3] = float("nan")
        dev[2 * n + bad[1], V - 1] = float("inf")
        dev[2 * n + bad[2]] = float("nan")
        dev[2 * n + bad[3], :1000] = float("nan")
        ids = ids_for(rng, 20 * n, V, 2)
        for top in tops:
            check_first(m, dev, ids, top, n)
            _, tl, ti, ent, lse = m.token_logprobs(dev, torch.from_numpy(ids.astype(np.int32)).cuda(), top=top)
            for r in bad:
                assert torch.isnan(tl[2 * n + r]).all() and torch.isnan(ent[2 * n + r]) and torch.isnan(lse[2 * n + r])
            assert bool((ti[2 * n + bad[2]] == -1).all()) and int(ti[2 * n + bad[1], 0]) == V - 1 and V // 3 not in ti[2 * n + bad[0]].tolist()
            assert torch.equal(ti[2 * n + bad[3]], ti[bad[3]])  # (its first places hold the lowest value)
            same = [r for r in range(n) if r not in bad]
            for c in range(1, 20):
                some = same if c == 2 else list(range(n))
                for t in (tl, ti, ent, lse):
                    a, b = t[:n][some], t[c * n:(c + 1) * n][some]
                    assert torch.equal(a, b) if aligned or t is ti else torch.allclose(a, b, rtol=1e-5, atol=1e-5), c


@pytest.mark.parametrize("dtype", list(K.TYPES))
@pytest.mark.parametrize("R_", [1, 320])
@pytest.mark.parametrize("top", [1, 20, 32])
def test_threads_above_the_bar(m, top, R_, dtype):
    """In every span (8 vectors of each of a CTA's 256 threads) so many threads hold a logit above all of the spans before: as many as
    wait for a look together, one more, and all; rising, equal among themselves, and level with the span before."""
    W = 4 if dtype == "f32" else 8
    span, V = 256 * 8 * W, 131075
    rng = np.random.default_rng(top)
    rows = []
    for threads in (20, 33, 40, 50, 63, 64, 65, 100, 256):
        for kind in ("rise", "ties", "level"):
            row = -20 + rng.random(V)
            for s, first in enumerate(range(0, V, span)):
                t = rng.permutation(256)[:threads]
                at = first + ((rng.integers(0, 8, threads) * 256 + t) * W + rng.integers(0, W, threads))
                at = at[at < V]
                row[at] = {"rise": s + rng.random(len(at)), "ties": s, "level": s // 3}[kind]
            rows.append(row)
    x = np.stack(rows)
    n = len(rows)
    if R_ == 1:
        for r in range(n):
            check(m, batch(x[r:r + 1], dtype, 1, True), ids_for(rng, 1, V, 1), top)
    else:
        dev = batch(x, dtype, -(-R_ // n), True)
        check_first(m, dev, ids_for(rng, dev.shape[0], V, 1), top, n)


def test_unaligned_rows_in_number(m):
    """Rows one behind another at every alignment, their best tokens among the first and last few, which no vector holds."""
    for dtype in K.TYPES:
        R_, V = 311, 131075
        rng = np.random.default_rng(R_)
        x = rng.standard_normal((R_, V)).astype(np.float32)
        x[:, :8] += 3 * rng.random((R_, 8)).astype(np.float32)
        x[:, -8:] += 6 * rng.random((R_, 8)).astype(np.float32)
        dev = torch.from_numpy(x).to(K.TYPES[dtype]).cuda()
        check_first(m, dev, ids_for(rng, R_, V, 1), 20, 17)
