"""What the head norm, append and log probability calls refuse on the host, without a GPU (nothing is launched when an argument
error is returned), and the frequencies that a Rope holds."""
import ctypes
import fractions
import math
import struct

import pytest
import torch

from test_kv8_abi import ALIGN, BAD_CACHE, CAP, NULL, OK, SHAPE, TYPE, cache, m  # noqa: F401


def rope(m, **kw):  # noqa: F811
    return m.RopeC(**{**dict(turns=16, rot=64, start=0, interleaved=0, factor=1.0), **kw})


def heads(m, **kw):  # noqa: F811
    return m.HeadsC(**{**dict(x=16, out=16, weight=16, x_token_stride=1024, x_head_stride=128, out_token_stride=1024, out_head_stride=128, n_heads=8), **kw})


BAD_ROPE = [(dict(rot=0), SHAPE), (dict(rot=-16), SHAPE), (dict(rot=24), SHAPE), (dict(rot=144), SHAPE), (dict(start=-8), SHAPE), (dict(start=4), SHAPE),
            (dict(start=72), SHAPE), (dict(start=2 ** 31 - 8), SHAPE), (dict(turns=20), ALIGN)]
BAD_HEADS = [(dict(n_heads=-1), SHAPE), (dict(n_heads=65536), CAP), (dict(x=None), NULL), (dict(out=None), NULL), (dict(x=17), ALIGN), (dict(out=17), ALIGN), (dict(weight=24), ALIGN)]


def test_head_norm_refusals(m):  # noqa: F811
    def call(**kw):
        f = dict(q=heads(m), k=heads(m, n_heads=2), rope=rope(m), positions=16, n_tokens=4, type=2, w_type=0, head_dim=128, eps=1e-6)
        return m.lib().moe_head_norm_rope(ctypes.byref(m.HeadNormCallC(**{**f, **kw})), None)
    assert m.lib().moe_head_norm_rope(None, None) == NULL
    for kw, rc in BAD_HEADS:
        assert call(q=heads(m, **kw)) == rc and call(k=heads(m, **kw)) == rc, kw
    for kw, rc in BAD_ROPE:
        assert call(rope=rope(m, **kw)) == rc, kw
    for d in (0, 8, 40, 272, -16):
        assert call(head_dim=d) == SHAPE
    assert call(n_tokens=-1) == SHAPE and call(n_tokens=1 << 31) == SHAPE
    assert call(n_tokens=1 << 28) == CAP and call(q=heads(m, n_heads=2 ** 31 - 1), n_tokens=2) == CAP
    assert call(type=3) == TYPE and call(w_type=-1) == TYPE
    assert call(positions=None) == NULL and call(positions=18) == ALIGN
    # nothing to do: nothing launched, and unused fields are not looked at
    assert call(n_tokens=0, q=heads(m, x=None, out=None), positions=None) == OK
    assert call(q=heads(m, n_heads=0, x=17), k=heads(m, n_heads=0, weight=3), w_type=9) == OK
    assert call(rope=rope(m, turns=None, rot=3), n_tokens=0) == OK


def test_append_refusals(m):  # noqa: F811
    def call(c=None, **kw):
        f = dict(cache=c or cache(m), rows=m.KV8RowsC(k=16, v=16, type=0, n_tokens=8, k_token_stride=256, k_head_stride=128, v_token_stride=256, v_head_stride=128),
                 q=heads(m), rope=rope(m), k_weight=16, cu_tokens=16, start=16, positions=16, w_type=0, eps=1e-6, err=16)
        for k in list(kw):
            if k in ("k", "v", "type", "n_tokens"):
                setattr(f["rows"], k, kw.pop(k))
        return m.lib().moe_kv8_append(ctypes.byref(m.KV8AppendC(**{**f, **kw})), None)
    assert m.lib().moe_kv8_append(None, None) == NULL
    for kw, rc in BAD_CACHE:
        assert call(cache(m, **kw)) == rc, kw
    for kw, rc in BAD_HEADS:
        assert call(q=heads(m, **kw)) == rc, kw
    for kw, rc in BAD_ROPE:
        assert call(rope=rope(m, **kw)) == rc, kw
    for name in ("k", "v", "cu_tokens", "start"):
        assert call(**{name: None}) == NULL, name
    assert call(type=3) == TYPE and call(w_type=7) == TYPE and call(w_type=7, q=heads(m, weight=None)) == TYPE
    assert call(n_tokens=-1) == SHAPE and call(n_tokens=1 << 31) == SHAPE
    assert call(k=18) == ALIGN and call(k_weight=8) == ALIGN
    for name in ("cu_tokens", "start", "positions", "err"):
        assert call(**{name: 18}) == ALIGN, name
    assert call(n_tokens=2 ** 31 - 1, q=heads(m, n_heads=64)) == CAP and call(q=heads(m, n_heads=1 << 30)) == CAP
    assert call(n_tokens=0, k=None, v=None, q=heads(m, x=None, out=None), k_weight=None, w_type=9, rope=rope(m, turns=None)) == TYPE  # (q's weight)
    assert call(n_tokens=0, k=None, v=None, q=heads(m, x=None, out=None, weight=None), k_weight=None, w_type=9, rope=rope(m, turns=None)) == OK


def test_logprobs_refusals(m):  # noqa: F811
    def call(**kw):
        f = dict(logits=16, row_stride=100, type=0, rows=3, vocab=100, n_ids=2, top=5, scale=1.0, ids=16, logprobs=16, top_logprobs=16, top_ids=16, entropy=16, lse=16)
        return m.lib().moe_token_logprobs(ctypes.byref(m.LogprobsCallC(**{**f, **kw})), None)
    assert m.lib().moe_token_logprobs(None, None) == NULL
    assert call(type=3) == TYPE
    for kw in (dict(rows=-1), dict(vocab=0), dict(vocab=-5), dict(n_ids=-1), dict(top=-1), dict(top=33), dict(top=5, vocab=4), dict(row_stride=99), dict(scale=0.0),
               dict(scale=-1.0), dict(scale=math.inf), dict(scale=math.nan), dict(scale=2.0 ** -101), dict(scale=2.0 ** 101)):
        assert call(**kw) == SHAPE, kw
    assert call(rows=1 << 28) == CAP and call(rows=1 << 20, n_ids=1 << 11) == CAP
    for name in ("logits", "ids", "logprobs", "top_logprobs", "top_ids"):
        assert call(**{name: None}) == NULL, name
    for name in ("logits", "ids", "logprobs", "top_logprobs", "top_ids", "entropy", "lse"):
        assert call(**{name: 18}) == ALIGN, name
    assert call(type=1, logits=17) == ALIGN
    assert call(rows=0, logits=None) == OK


def test_binding_refusals(m, monkeypatch):  # noqa: F811
    """Tensors of the wrong kind never reach the library."""
    monkeypatch.setattr(m, "_device", lambda t: -1)
    monkeypatch.setattr(m, "_ptr", lambda t, dev: t.data_ptr())
    monkeypatch.setattr(m, "_launch", lambda *a: pytest.fail("launched"))
    r = m.Rope(64, device="cpu")
    other = m.Rope(64, device="cpu")
    other._device = 1
    q, pos, w = torch.zeros((3, 4, 64)), torch.zeros(3, dtype=torch.int32), torch.ones(64)
    pool, table = m.kv8_pool(2, 2, 64, 32, device="cpu"), torch.zeros((1, 2), dtype=torch.int32)
    k, cu, start = torch.zeros((3, 2, 64)), torch.tensor([0, 3], dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
    app = lambda *a, **kw: m.kv8_append(*(a or (k, k)), pool, table, cu, start, **kw)  # noqa: E731
    x, ids = torch.zeros((2, 50)), torch.zeros((2, 1), dtype=torch.int32)
    bad = [
        lambda: m.head_norm_rope(q[0], pos, r), lambda: m.head_norm_rope(q, None, r), lambda: m.head_norm_rope(q, pos.long(), r), lambda: m.head_norm_rope(q, pos[:2], r),
        lambda: m.head_norm_rope(q, pos, other), lambda: m.head_norm_rope(q.transpose(1, 2), pos, r), lambda: m.head_norm_rope(q[..., :48].contiguous(), pos, r),
        lambda: m.head_norm_rope(q, pos, r, k=q[:2]), lambda: m.head_norm_rope(q, pos, r, k=q.half()), lambda: m.head_norm_rope(q, pos, r, q_weight=w[:32]),
        lambda: m.head_norm_rope(q, pos, r, k=q, q_weight=w, k_weight=w.half()), lambda: m.head_norm_rope(q, pos, r, q_out=q.half()),
        lambda: m.head_norm_rope(q, pos, r, q_out=q[:2]), lambda: m.head_norm_rope(q.double(), pos, r), lambda: m.head_norm_rope(q, pos, r, eps="1"),
        lambda: app(k[:, :1], k), lambda: app(k, k[:2]), lambda: app(k, k.half()), lambda: app(q=q[:2]), lambda: app(q=q.half()), lambda: app(k_weight=w[:1]),
        lambda: app(rope=other), lambda: app(positions=pos.long()), lambda: app(q=q, q_out=torch.zeros((3, 4, 64)).half()),
        lambda: app(rope=m.Rope(64, start=64, device="cpu")),
        lambda: m.token_logprobs(x[0]), lambda: m.token_logprobs(x.t()), lambda: m.token_logprobs(x, ids.long()), lambda: m.token_logprobs(x, ids[:1]),
        lambda: m.token_logprobs(x, ids[:, 0]), lambda: m.token_logprobs(x, top=33), lambda: m.token_logprobs(x, top=-1), lambda: m.token_logprobs(x.double()),
        lambda: m.token_logprobs(x, scale=None), lambda: m.token_logprobs(x, scale=10 ** 400),
    ]
    for i, f in enumerate(bad):
        with pytest.raises(m.MoeError):
            f()
            pytest.fail(f"not refused: {i}")


def test_two_descriptions_agree(m):  # noqa: F811
    """The binding packs the calls' structures by format; the ctypes structures say the same, field by field."""
    kinds = {ctypes.c_void_p: "P", ctypes.c_int32: "i", ctypes.c_int64: "q", ctypes.c_float: "f"}

    def flat(s, base=0):
        for name, t in s._fields_:
            at = base + getattr(s, name).offset
            if isinstance(t, type) and issubclass(t, ctypes.Structure):
                yield from flat(t, at)
            else:
                yield at, kinds[t]
    for s, pack in ((m.HeadNormCallC, m._pack_heads), (m.KV8AppendC, m._pack_append), (m.LogprobsCallC, m._pack_logprobs)):
        fields = list(flat(s))
        packed = pack(*range(1, len(fields) + 1))
        assert ctypes.sizeof(s) - 8 < len(packed) <= ctypes.sizeof(s)
        for v, (at, kind) in enumerate(fields, 1):
            assert struct.unpack_from("@" + kind, packed, at)[0] == v


def test_empty_batches(m, monkeypatch):  # noqa: F811
    monkeypatch.setattr(m, "_device", lambda t: -1)
    monkeypatch.setattr(m, "_ptr", lambda t, dev: t.data_ptr())
    monkeypatch.setattr(m, "_current_device", lambda: -1)
    monkeypatch.setattr(m, "_raw_stream", lambda dev: 0)
    pool, table = m.kv8_pool(2, 2, 64, 32, device="cpu"), torch.zeros((0, 3), dtype=torch.int32)
    none = torch.zeros(0, dtype=torch.int32)
    x = torch.zeros((0, 2, 64))
    assert m.kv8_append(x, x, pool, table, torch.zeros(1, dtype=torch.int32), none) is None
    assert m.kv8_append(x, x, pool, table, torch.zeros(1, dtype=torch.int32), none, q=torch.zeros((0, 6, 64))).shape == (0, 6, 64)
    q, k = m.head_norm_rope(x, none, k=x)
    assert q.shape == k.shape == (0, 2, 64)
    out = m.token_logprobs(torch.zeros((0, 9)), torch.zeros((0, 2), dtype=torch.int32), top=4)
    assert [tuple(t.shape) for t in out] == [(0, 2), (0, 4), (0, 4), (0,), (0,)]


def test_rope_frequencies(m):  # noqa: F811
    """theta's powers, their scalings, and the fractions of a turn that the kernels take."""
    r = m.Rope(64, theta=1e6, device="cpu")
    assert r.inv_freq == [1e6 ** (-i / 32) for i in range(32)] and r.factor == 1.0 and r.turns.shape == (32,) and r.turns.dtype == torch.int64
    two_pi = 2 * fractions.Fraction("3.14159265358979323846264338327950288")
    for f, t in zip(r.inv_freq, r.turns.tolist()):
        assert abs(fractions.Fraction(t % 2 ** 64, 2 ** 64) - fractions.Fraction(f) / two_pi) <= fractions.Fraction(1, 2 ** 65)
    f = m.Rope(16, inv_freq=[0, -1, 1, 2, 3, 4, 5, 7], device="cpu")  # (7 radians are more than a turn, -1 the other way)
    turns = [t % 2 ** 64 / 2 ** 64 for t in f.turns.tolist()]
    assert turns[0] == 0 and abs(turns[1] + turns[2] - 1) < 1e-15 and abs(turns[7] - (7 / (2 * math.pi) - 1)) < 1e-15
    lin = m.Rope(64, theta=1e6, scaling={"kind": "linear", "scale": 4}, device="cpu")
    assert lin.inv_freq == [x / 4 for x in r.inv_freq] and lin.factor == 1.0
    yarn = m.Rope(64, theta=1e6, scaling={"kind": "yarn", "scale": 4, "original": 4096}, device="cpu")
    turn = [4096 * x / (2 * math.pi) for x in r.inv_freq]
    assert yarn.factor == 0.1 * math.log(4) + 1
    for x, y, t in zip(r.inv_freq, yarn.inv_freq, turn):
        assert x / 4 <= y * (1 + 1e-12) and y <= x
        # a line whose ends lie outside both counts: as much as a pair further
        if t > 32 * 1e6 ** (1 / 32):
            assert y == x
        if t < 1e6 ** (-1 / 32):
            assert math.isclose(y, x / 4)
    assert any(x / 4 < y < x for x, y in zip(r.inv_freq, yarn.inv_freq))
    bands = m.Rope(64, theta=1e6, scaling={"kind": "bands", "scale": 8, "original": 8192, "low": 1, "high": 4}, device="cpu")
    for x, y in zip(r.inv_freq, bands.inv_freq):
        t = 8192 * x / (2 * math.pi)
        assert math.isclose(y, x if t >= 4 else x / 8 if t <= 1 else x * ((t - 1) / 3 + (1 - (t - 1) / 3) / 8))
    assert m.Rope(64, scaling={"kind": "yarn", "scale": 4, "original": 4096}, factor=1, device="cpu").factor == 1.0


def test_rope_refusals(m):  # noqa: F811
    bad = [dict(rot=0), dict(rot=24), dict(rot=-16), dict(rot=64, start=4), dict(rot=64, start=-8), dict(rot=64, theta=0), dict(rot=64, theta=math.inf),
           dict(rot=64, inv_freq=[1.0] * 31), dict(rot=32, inv_freq=[math.nan] * 16), dict(rot=64, scaling={"kind": "other"}), dict(rot=64, scaling={"scale": 4}),
           dict(rot=64, scaling={"kind": "linear", "scale": 0}), dict(rot=64, scaling={"kind": "linear", "scale": 2, "low": 1}),
           dict(rot=64, scaling={"kind": "yarn", "scale": 2}), dict(rot=64, scaling={"kind": "bands", "scale": 2, "original": 100, "low": 4, "high": 4}),
           dict(rot=64, theta=1.0, scaling={"kind": "yarn", "scale": 2, "original": 100})]
    for kw in bad:
        with pytest.raises(m.MoeError):
            m.Rope(device="cpu", **kw)


def test_other_device(m, monkeypatch):  # noqa: F811
    """The library launches on the current device: tensors of another one are refused before the call."""
    monkeypatch.setattr(m, "_device", lambda t: -1)
    monkeypatch.setattr(m, "_ptr", lambda t, dev: t.data_ptr())
    monkeypatch.setattr(m, "_current_device", lambda: 1)
    monkeypatch.setattr(m, "_raw_stream", lambda dev: pytest.fail("launched"))
    x, pos = torch.zeros((2, 2, 64)), torch.zeros(2, dtype=torch.int32)
    pool, table = m.kv8_pool(2, 2, 64, 32, device="cpu"), torch.zeros((1, 2), dtype=torch.int32)
    one, cu = torch.zeros(1, dtype=torch.int32), torch.tensor([0, 2], dtype=torch.int32)
    for f in (lambda: m.head_norm_rope(x, pos), lambda: m.kv8_append(x, x, pool, table, cu, one), lambda: m.token_logprobs(x[0])):
        with pytest.raises(m.MoeError, match="device"):
            f()


def test_copies_of_a_rope(m):  # noqa: F811
    """A copied or unpickled Rope names its own frequencies' memory, not that of the one it was made from."""
    import copy
    import pickle
    r = m.Rope(64, start=8, interleaved=True, factor=0.5, device="cpu")
    for c in (copy.copy(r), copy.deepcopy(r), pickle.loads(pickle.dumps(r))):
        assert torch.equal(c.turns, r.turns) and m._rope(c, -1, 128) == (c.turns.data_ptr(), 64, 8, 1, 0.5)
    assert copy.deepcopy(r).turns.data_ptr() != r.turns.data_ptr()
    r._device = 5  # as one saved on another device and loaded onto this one
    assert pickle.loads(pickle.dumps(r))._device == -1


def test_ranks_refused(m, monkeypatch):  # noqa: F811
    """Tensors with too few or too many dimensions are argument errors like any other."""
    monkeypatch.setattr(m, "_device", lambda t: -1)
    monkeypatch.setattr(m, "_ptr", lambda t, dev: t.data_ptr())
    monkeypatch.setattr(m, "_launch", lambda *a: pytest.fail("launched"))
    q, pos = torch.zeros((3, 4, 64)), torch.zeros(3, dtype=torch.int32)
    pool, table = m.kv8_pool(2, 2, 64, 32, device="cpu"), torch.zeros((1, 2), dtype=torch.int32)
    k, cu, start = torch.zeros((3, 2, 64)), torch.tensor([0, 3], dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
    one = torch.zeros(())
    for other in (one, q[0, 0], q[0], q[None]):
        for f in (lambda: m.head_norm_rope(other, pos), lambda: m.head_norm_rope(q, pos, k=other), lambda: m.head_norm_rope(q, pos, q_out=other),
                  lambda: m.head_norm_rope(q, pos, k=q, k_out=other), lambda: m.kv8_append(other, k, pool, table, cu, start), lambda: m.kv8_append(k, other, pool, table, cu, start),
                  lambda: m.kv8_append(k, k, pool, table, cu, start, q=other), lambda: m.kv8_append(k, k, pool, table, cu, start, q=q, q_out=other),
                  lambda: m.token_logprobs(other) if other.dim() != 2 else m.token_logprobs(q), lambda: m.token_logprobs(q[0, :2], other.int()),
                  lambda: m.head_norm_rope(q, pos, q_weight=other[..., None]), lambda: m.kv8_append(k, k, pool, table, cu, start, k_weight=other[..., None])):
            with pytest.raises(m.MoeError):
                f()
