"""How far the cache's requantising moves a value, on the plain write that the kernel equals bit for bit (no GPU)."""
import numpy as np
import pytest

import kv8_ref as R


def appended(x, step, D):
    """Blocks of 32 tokens [n, 32, D] written `step` tokens at a time: what is read back, and each token's sum of the
    scales that its block had from its own write on."""
    n = x.shape[0]
    c = R.Cache(np.zeros((1, n, 1, 64 * D + 16), np.uint8), np.zeros((1, 1), np.int32))
    had = np.zeros((n, 32))
    scale = np.zeros(n)
    for t in range(0, 32, step):
        rows = np.ascontiguousarray(x[:, t:t + step].transpose(1, 0, 2))  # a block of x is a head of the cache
        c.write(0, t, (rows, rows))
        new = np.array([c.codes(0, 0, h, 0)[1] for h in range(n)], np.float64)
        had[:, :t] += np.where(new > scale, new, 0)[:, None]
        had[:, t:t + step] = new[:, None]
        scale = new
    return c.read(0, 0, 32)[0].transpose(1, 0, 2).astype(np.float64), had, scale


@pytest.mark.parametrize("step", [1, 4])
@pytest.mark.parametrize("what", ["normal", "growing", "doubling"])
def test_requantised_values(what, step):
    """A value is off by at most half a step of each scale that its block has had since it was written (and the fp32
    roundings of a scale, a ratio and a code, 2^-20 of the value); normal values end below 0.5 steps of the last scale rms."""
    rng = np.random.default_rng(["normal", "growing", "doubling"].index(what))
    x = rng.standard_normal((40, 32, 64)) if what == "normal" else rng.uniform(-1, 1, (40, 32, 64))
    x *= {"normal": 1.0, "growing": 1.02, "doubling": 2.0}[what] ** np.arange(32)[None, :, None]
    x = x.astype(np.float32)
    v, had, scale = appended(x, step, 64)
    far = np.abs(v - x)
    assert (far <= had[..., None] / 2 + 2.0 ** -20 * np.abs(x) + 2.0 ** -20 * scale[:, None, None]).all()
    assert (far <= 16 * (1 + 2.0 ** -20) * scale[:, None, None]).all()
    if what == "normal":
        assert np.sqrt((far ** 2).mean()) <= 0.5 * np.sqrt((scale ** 2).mean())


def test_rejected_outlier():
    """A rejected draft's large value costs its block's kept tokens, and those written over it, the resolution that the grown
    scale leaves; a block that is written from its first token on starts anew."""
    rng = np.random.default_rng(5)
    D = 32
    c = R.Cache(np.zeros((2, 1, 1, 64 * D + 16), np.uint8), np.array([[0, 1]], np.int32))
    row = lambda n, size=1.0: tuple(2 * [(size * rng.uniform(-1, 1, (n, 1, D))).astype(np.float32)])  # noqa: E731
    x = row(10)
    c.write(0, 0, x)
    c.write(0, 10, row(4, 100.0))
    large = c.codes(0, 0, 0, 0)[1]
    y = row(4)
    c.write(0, 10, y)
    assert c.codes(0, 0, 0, 0)[1] == large > 0.7 * 100 / 127
    assert np.abs(c.read(0, 10, 14)[0] - y[0]).max() <= 0.501 * large
    assert np.abs(c.read(0, 0, 10)[0] - x[0]).max() <= 0.51 * large + 0.51 / 127
    z = row(14)
    c.write(0, 0, z)
    assert c.codes(0, 0, 0, 0)[1] <= 1 / 127
