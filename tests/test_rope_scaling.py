"""The frequencies of a Rope with a scaling for long contexts, against the scalings' definitions written apart from the
package's code, pair by pair."""
import math

import pytest

from test_kv8_abi import m  # noqa: F401


def powers(rot, theta):
    return [theta ** (-2.0 * i / rot) for i in range(rot // 2)]


def turns(f, original):
    """How many times a pair turns over the original length."""
    return original * f / (2 * math.pi)


def test_yarn_of_given_frequencies(m):  # noqa: F811
    """Given frequencies get the scaling that the theta whose powers they are gives them; without that theta, or where they are
    not its powers, there is no line between the pairs that turn often and seldom, and the call is refused."""
    yarn = {"kind": "yarn", "scale": 16, "original": 8192}
    for rot, theta in ((128, 500000.0), (64, 10000.0), (32, 1e6)):
        f = powers(rot, theta)
        want = m.Rope(rot, theta=theta, scaling=yarn, device="cpu")
        got = m.Rope(rot, theta=theta, inv_freq=f, scaling=yarn, device="cpu")
        assert got.inv_freq == want.inv_freq and got.factor == want.factor
        rounded = [x * (1 + 2.0 ** -8 * (-1) ** i) for i, x in enumerate(f)]  # as bf16 has them, at most
        got = m.Rope(rot, theta=theta, inv_freq=rounded, scaling=yarn, device="cpu")
        assert all(math.isclose(x / r, y / p) for x, r, y, p in zip(got.inv_freq, rounded, want.inv_freq, f))
        for kw in (dict(), dict(theta=2 * theta), dict(theta=1.0), dict(theta=0.0), dict(theta=math.nan)):
            with pytest.raises(m.MoeError):
                m.Rope(rot, inv_freq=f, scaling=yarn, device="cpu", **kw)
        with pytest.raises(m.MoeError):
            m.Rope(rot, theta=theta, inv_freq=[-x for x in f], scaling=yarn, device="cpu")
    # without a line there is nothing to find: no theta is needed, and none is looked at
    f = powers(64, 500000.0)
    for kw in (dict(), dict(theta=7.0)):
        assert m.Rope(64, inv_freq=f, device="cpu", **kw).inv_freq == f
        assert m.Rope(64, inv_freq=f, scaling={"kind": "linear", "scale": 4}, device="cpu", **kw).inv_freq == [x / 4 for x in f]
    bands = {"kind": "bands", "scale": 8, "original": 8192}
    assert m.Rope(64, inv_freq=f, scaling=bands, device="cpu").inv_freq == m.Rope(64, theta=500000.0, scaling=bands, device="cpu").inv_freq
    assert m.Rope(64, device="cpu").inv_freq == powers(64, 10000.0)


def test_yarn_refusals(m):  # noqa: F811
    """Bounds in the wrong order have no line between them, and below a scale of 1 the factor is less than 1, at last negative."""
    for kw in (dict(fast=1.0, slow=32.0), dict(fast=1.0), dict(slow=32.0), dict(fast=4.0, slow=4.0), dict(scale=0.5), dict(scale=1e-5)):
        with pytest.raises(m.MoeError):
            m.Rope(64, scaling={"kind": "yarn", "scale": 4, "original": 4096, **kw}, device="cpu")
    one = m.Rope(64, scaling={"kind": "yarn", "scale": 1, "original": 4096}, device="cpu")
    assert one.factor == 1.0 and all(math.isclose(a, b) for a, b in zip(one.inv_freq, powers(64, 10000.0)))
    short = m.Rope(64, scaling={"kind": "linear", "scale": 0.5}, device="cpu")
    assert short.inv_freq == [2 * x for x in powers(64, 10000.0)] and short.factor == 1.0


def yarn_share(i, rot, theta, original, fast, slow):
    """How much of pair i's frequency is divided: none up to the last whole pair (pair 0 at least) before the place where pairs turn
    `fast` times, all from the first whole one behind the place where they turn `slow` times, a line in i between."""
    def place(r):  # a real index, by halving (pairs turn less and less)
        lo, hi = -10.0 * rot, 10.0 * rot
        for _ in range(200):
            mid = (lo + hi) / 2
            lo, hi = (mid, hi) if turns(theta ** (-2 * mid / rot), original) > r else (lo, mid)
        return lo
    first, last = max(0, math.floor(place(fast))), math.ceil(place(slow))
    return 1.0 if i >= last else 0.0 if i <= first else (i - first) / (last - first)


@pytest.mark.parametrize("rot,theta,original,fast,slow,scale", [
    (64, 10000.0, 4096, 32.0, 1.0, 4.0), (128, 500000.0, 8192, 32.0, 1.0, 16.0), (128, 1e6, 32768, 32.0, 1.0, 4.0), (32, 10000.0, 100, 32.0, 1.0, 2.0),
    (96, 150000.0, 4096, 32.0, 1.0, 32.0), (64, 10000.0, 1 << 20, 32.0, 1.0, 8.0), (16, 100.0, 2048, 8.0, 2.0, 40.0), (64, 10000.0, 7, 32.0, 1.0, 2.0),
    # shorter than a turn of the first pair: all pairs turn less than `slow` times
    (64, 10000.0, 6, 32.0, 1.0, 2.0), (64, 10000.0, 1, 2.0, 1.0, 4.0), (64, 10000.0, 2, 2.0, 1.0, 1.0)])
def test_yarn_line(m, rot, theta, original, fast, slow, scale):  # noqa: F811
    got = m.Rope(rot, theta=theta, scaling={"kind": "yarn", "scale": scale, "original": original, "fast": fast, "slow": slow}, device="cpu")
    assert math.isclose(got.factor, 0.1 * math.log(scale) + 1)
    for i, (f, y) in enumerate(zip(powers(rot, theta), got.inv_freq)):
        share = yarn_share(i, rot, theta, original, fast, slow)
        assert math.isclose(y, f * (1 - share) + f / scale * share, rel_tol=1e-9), i
        if turns(f, original) < slow * (1 - 1e-9) * theta ** (-2 / rot):  # (a pair further: the ends are moved outward)
            assert math.isclose(y, f / scale)


def test_bands_line(m):  # noqa: F811
    """A line in the number of turns, of pairs that turn either way."""
    f = powers(64, 10000.0)
    f = [-x if i % 3 == 1 else x for i, x in enumerate(f)]
    got = m.Rope(64, inv_freq=f, scaling={"kind": "bands", "scale": 8, "original": 1024, "low": 1, "high": 4}, device="cpu")
    for x, y in zip(f, got.inv_freq):
        keep = min(max((abs(turns(x, 1024)) - 1) / 3, 0), 1)
        assert math.isclose(y, x * keep + x / 8 * (1 - keep)), x


def test_numbers_out_of_range(m):  # noqa: F811
    """Numbers that give no frequency or no factor, or are none, are argument errors."""
    far, yarn = {"kind": "linear", "scale": 1e-320}, {"kind": "yarn", "scale": 4, "original": 4096}
    bad = [dict(factor=math.nan), dict(factor=math.inf), dict(factor=1e39), dict(factor="x"), dict(theta=1e-320), dict(theta="x"), dict(theta=math.nan), dict(theta=10 ** 400),
           dict(scaling=far), dict(scaling={"kind": "linear", "scale": "4"}), dict(scaling={"kind": "linear", "scale": 10 ** 400}), dict(scaling={**yarn, "original": math.inf}),
           dict(scaling={**yarn, "fast": math.inf}), dict(scaling={**yarn, "fast": math.nan}), dict(scaling={**yarn, "original": 10 ** 400}), dict(scaling={**yarn, "slow": 1e-320}),
           dict(scaling={**yarn, "original": "4096"}), dict(scaling={**yarn, "scale": None}), dict(scaling="linear"), dict(inv_freq=[10 ** 400] * 32), dict(inv_freq=["x"] * 32),
           dict(inv_freq=5), dict(rot=64.0), dict(rot="64"), dict(start=8.0), dict(start=None)]
    for kw in bad:
        with pytest.raises(m.MoeError):
            m.Rope(**{"rot": 64, "device": "cpu", **kw})
            pytest.fail(f"not refused: {kw}")
    assert m.Rope(64, factor=-2, theta=1e-300, device="cpu").factor == -2.0
