"""What the cache, attention and norm calls refuse on the host, without a GPU: nothing is launched
when an argument error is returned."""
import pytest
import torch

OK, NULL, TYPE, SHAPE, CAP, SCRATCH, ALIGN = 0, -1, -2, -3, -4, -7, -6


@pytest.fixture(scope="module")
def m():
    from quantized_routed_expert_grouped_gb300 import build
    build.build()
    import quantized_routed_expert_grouped_gb300 as mod
    mod.lib()
    return mod


def cache(m, **kw):
    f = dict(pool=16, n_pages=4, n_kv_heads=2, head_dim=128, page_tokens=64, page_table=16, table_stride=4, max_pages=4, n_seqs=2)
    return m.KV8CacheC(**{**f, **kw})


BAD_CACHE = [
    (dict(pool=None), NULL), (dict(page_table=None), NULL), (dict(pool=24), ALIGN), (dict(page_table=18), ALIGN),
    (dict(head_dim=0), SHAPE), (dict(head_dim=100), SHAPE), (dict(head_dim=288), SHAPE), (dict(head_dim=-32), SHAPE),
    (dict(page_tokens=0), SHAPE), (dict(page_tokens=48), SHAPE), (dict(page_tokens=-32), SHAPE),
    (dict(n_pages=0), CAP), (dict(n_kv_heads=0), CAP), (dict(n_kv_heads=70000), CAP), (dict(max_pages=0), CAP),
    (dict(n_seqs=0), CAP), (dict(n_seqs=1 << 21), CAP), (dict(table_stride=3), CAP),
]


def test_block_bytes(m):
    assert [m.kv8_block_bytes(d) for d in (32, 128, 256)] == [2064, 8208, 16400]
    assert [m.kv8_block_bytes(d) for d in (0, -32, 16, 100, 288)] == [0] * 5


@pytest.mark.parametrize("name", ["moe_kv8_write", "moe_kv8_read"])
def test_rows_refusals(m, name):
    import ctypes
    f = getattr(m.lib(), name)
    ref = ctypes.byref

    def call(c=None, cu=16, start=16, **kw):
        r = m.KV8RowsC(**{**dict(k=16, v=16, type=0, n_tokens=8, k_token_stride=256, k_head_stride=128, v_token_stride=256, v_head_stride=128), **kw})
        return f(ref(c or cache(m)), ref(r), cu, start, None, None)
    for kw, rc in BAD_CACHE:
        assert call(cache(m, **kw)) == rc, kw
    assert f(None, None, 16, 16, None, None) == NULL
    assert call(cu=None) == NULL and call(start=None) == NULL and call(k=None) == NULL and call(v=None) == NULL
    assert call(type=3) == TYPE and call(type=-1) == TYPE
    assert call(n_tokens=-1) == SHAPE and call(n_tokens=1 << 31) == SHAPE
    assert call(k=18) == ALIGN and call(type=1, v=17) == ALIGN
    assert call(n_tokens=0, k=None, v=None) == OK  # nothing to do, nothing launched


def test_attention_refusals(m):
    import ctypes
    L = m.lib()
    ws = L.moe_kv8_attention_workspace_bytes(2, 4, 8, 2, 128)
    assert ws > 0
    for bad in [(0, 4, 8, 2, 128), (2, 0, 8, 2, 128), (2, 33, 8, 2, 128), (2, 4, 7, 2, 128), (2, 4, 8, 0, 128), (2, 4, 8, 2, 100)]:
        assert L.moe_kv8_attention_workspace_bytes(*bad) == 0, bad

    def call(c=None, **kw):
        f = dict(cache=c or cache(m), q=16, type=2, T=4, n_heads=8, q_seq_stride=4096, q_token_stride=1024, q_head_stride=128,
                 lens=16, window=0, scale=1.0, out=16, lse=None, workspace=16, workspace_bytes=ws)
        return L.moe_kv8_attention(ctypes.byref(m.KV8AttentionC(**{**f, **kw})), None)
    for kw, rc in BAD_CACHE:
        assert call(cache(m, **kw)) == rc, kw
    assert L.moe_kv8_attention(None, None) == NULL
    for p in ("q", "lens", "out", "workspace"):
        assert call(**{p: None}) == NULL, p
    assert call(type=7) == TYPE
    assert call(cache(m, max_pages=1 << 29, table_stride=1 << 29)) == CAP  # more blocks than 32 bits count
    for kw in (dict(T=0), dict(T=33), dict(n_heads=0), dict(n_heads=9), dict(window=-1)):
        assert call(**kw) == SHAPE, kw
    assert call(q=17) == ALIGN and call(out=24) == ALIGN and call(workspace=20) == ALIGN
    assert call(workspace_bytes=ws - 1) == SCRATCH


def test_norm_refusals(m):
    import ctypes
    L = m.lib()

    def call(**kw):
        f = dict(x=16, residual=16, weight=16, sum=16, y=16, xq=16, type=0, w_type=0, rows=4, x_stride=64, residual_stride=64, cols=64, eps=1e-6)
        return L.moe_add_rms_norm_q8_1(ctypes.byref(m.NormCallC(**{**f, **kw})), None)
    assert L.moe_add_rms_norm_q8_1(None, None) == NULL
    assert call(x=None) == NULL and call(weight=None) == NULL and call(sum=None, y=None, xq=None) == NULL
    assert call(type=3) == TYPE and call(w_type=-1) == TYPE
    for kw in (dict(cols=0), dict(cols=48), dict(cols=32800), dict(rows=-1), dict(x_stride=32), dict(residual_stride=0)):
        assert call(**kw) == SHAPE, kw
    for kw in (dict(x=20), dict(residual=8), dict(weight=4), dict(sum=24), dict(y=12), dict(xq=18), dict(x_stride=65), dict(residual_stride=66)):
        assert call(**kw) == ALIGN, kw
    assert call(rows=0) == OK
    assert L.moe_dequantize_q8_1(None, 1, 32, 16, 0, None) == NULL
    assert L.moe_dequantize_q8_1(16, 1, 33, 16, 0, None) == SHAPE and L.moe_dequantize_q8_1(16, -1, 32, 16, 0, None) == SHAPE
    assert L.moe_dequantize_q8_1(16, 1, 32, 16, 5, None) == TYPE
    assert L.moe_dequantize_q8_1(18, 1, 32, 16, 0, None) == ALIGN and L.moe_dequantize_q8_1(16, 1, 32, 24, 0, None) == ALIGN


def test_binding_refusals(m):
    """Tensors of the wrong kind never reach the library."""
    pool = m.kv8_pool(2, 2, 64, 32, device="cpu")
    assert pool.shape == (2, 2, 1, 4112)
    table = torch.zeros((1, 2), dtype=torch.int32)
    x = torch.zeros((3, 2, 64))
    cu, start = torch.tensor([0, 3], dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
    q = torch.zeros((1, 1, 4, 64))
    bad = [
        lambda: m.kv8_write(x, x, pool, table, cu, start),                       # not on a GPU
        lambda: m.kv8_write(x, x, pool.float(), table, cu, start),
        lambda: m.kv8_write(x, x, pool[..., :-1], table, cu, start),
        lambda: m.kv8_write(x, x, pool, table.long(), cu, start),
        lambda: m.kv8_pool(2, 2, 100, 32, device="cpu"),
        lambda: m.kv8_pool(2, 2, 64, 40, device="cpu"),
        lambda: m.kv8_attention(q, pool, table, start),
        lambda: m.add_rms_norm_q8_1(torch.zeros((2, 64)), torch.zeros(32)),
        lambda: m.add_rms_norm_q8_1(torch.zeros((2, 64)), torch.zeros(64), residual=torch.zeros((2, 64)).half()),
        lambda: m.dequantize_q8_1(torch.zeros((2, 2, 35), dtype=torch.uint8)),
        lambda: m.kv8_attention_workspace(1, 40, 4, 2, 64, device="cpu"),
    ]
    for f in bad:
        with pytest.raises(m.MoeError):
            f()


def test_binding_device(m, monkeypatch):
    """The library launches on the current device: tensors, or a stream, of another one are refused before the call."""
    class Stream:
        cuda_stream = 0

        def __init__(self, device):
            self.device_index = device
    calls = []

    def f(*args):
        calls.append(args)
        return 0
    monkeypatch.setattr(m, "_current_device", lambda: 0, raising=False)
    monkeypatch.setattr(m, "_raw_stream", lambda dev: 7)
    for dev, stream in ((1, None), (1, Stream(1)), (0, Stream(1))):
        with pytest.raises(m.MoeError):
            m._launch(f, dev, stream, (), 3)
    assert not calls
    m._launch(f, 0, None, (), 3)
    m._launch(f, 0, Stream(0), (), 3)
    assert calls == [(3, 7), (3, 0)]


def test_arrays_off_their_boundary(m):
    """int32 and fp32 arrays off 4 bytes are refused before a kernel would read them."""
    import ctypes
    L, ref = m.lib(), ctypes.byref
    rows = m.KV8RowsC(k=16, v=16, type=0, n_tokens=8, k_token_stride=256, k_head_stride=128, v_token_stride=256, v_head_stride=128)
    for f in (L.moe_kv8_write, L.moe_kv8_read):
        for cu, start, err in ((18, 16, 16), (16, 17, 16), (16, 16, 22)):
            assert f(ref(cache(m)), ref(rows), cu, start, err, None) == ALIGN
    call = dict(cache=cache(m), q=16, type=2, T=4, n_heads=8, q_seq_stride=4096, q_token_stride=1024, q_head_stride=128, lens=16, tree=16,
                scale=1.0, out=16, lse=16, err=16, workspace=16, workspace_bytes=L.moe_kv8_attention_workspace_bytes(2, 4, 8, 2, 128))
    for name in ("lens", "tree", "lse", "err"):
        assert L.moe_kv8_attention(ref(m.KV8AttentionC(**{**call, name: 18})), None) == ALIGN, name


def test_depth_refusals(m):
    import ctypes
    call = dict(cache=cache(m), q=16, type=2, T=4, n_heads=8, q_seq_stride=4096, q_token_stride=1024, q_head_stride=128, lens=16, tree=16,
                depth=16, window=5, scale=1.0, out=16, workspace=16, workspace_bytes=m.lib().moe_kv8_attention_workspace_bytes(2, 4, 8, 2, 128))
    f = lambda **kw: m.lib().moe_kv8_attention(ctypes.byref(m.KV8AttentionC(**{**call, **kw})), None)  # noqa: E731
    assert f(tree=None) == SHAPE and f(tree=None, window=0) == SHAPE and f(depth=18) == ALIGN


def test_two_descriptions_agree(m):
    """The binding packs the calls' structures by format; the ctypes structures say the same, field by field."""
    import ctypes
    import struct
    kinds = {ctypes.c_void_p: "P", ctypes.c_int32: "i", ctypes.c_int64: "q", ctypes.c_float: "f"}

    def flat(s, base=0):
        for name, t in s._fields_:
            at = base + getattr(s, name).offset
            if isinstance(t, type) and issubclass(t, ctypes.Structure):
                yield from flat(t, at)
            else:
                yield at, kinds[t]

    for s, pack in ((m.KV8CacheC, m._pack_rows[0]), (m.KV8RowsC, m._pack_rows[1]), (m.KV8AttentionC, m._pack_attn), (m.NormCallC, m._pack_norm)):
        fields = list(flat(s))
        values = [i + 1 for i in range(len(fields))]
        packed = pack(*values)
        assert ctypes.sizeof(s) - 8 < len(packed) <= ctypes.sizeof(s)
        for (at, kind), v in zip(fields, values):
            assert struct.unpack_from("@" + kind, packed, at)[0] == v


def test_no_sequences(m, monkeypatch):
    """An empty batch is nothing to do: no call of the library, empty results."""
    monkeypatch.setattr(m, "_device", lambda t: 0)
    monkeypatch.setattr(m, "_ptr", lambda t, dev: t.data_ptr())
    monkeypatch.setattr(m, "_current_device", lambda: 0)
    monkeypatch.setattr(m, "_raw_stream", lambda dev: 0)
    pool, table = m.kv8_pool(2, 2, 64, 32, device="cpu"), torch.zeros((0, 3), dtype=torch.int32)
    zero, none = torch.zeros(1, dtype=torch.int32), torch.zeros(0, dtype=torch.int32)
    x = torch.zeros((0, 2, 64))
    m.kv8_write(x, x, pool, table, zero, none)
    k, v = m.kv8_read(pool, table, zero, none, 0)
    assert k.shape == v.shape == (0, 2, 64) and k.dtype is torch.bfloat16
    out, lse = m.kv8_attention(torch.zeros((0, 4, 6, 64)), pool, table, none, with_lse=True)
    assert out.shape == (0, 4, 6, 64) and lse.shape == (0, 4, 6)
    with pytest.raises(m.MoeError):  # rows of no sequence
        m.kv8_write(torch.zeros((1, 2, 64)), torch.zeros((1, 2, 64)), pool, table, zero, none)


def test_numbers_out_of_range(m, monkeypatch):
    """Numbers that a field of the call does not hold raise the package's error."""
    monkeypatch.setattr(m, "_device", lambda t: 0)
    monkeypatch.setattr(m, "_ptr", lambda t, dev: t.data_ptr())
    monkeypatch.setattr(m, "_launch", lambda *a: pytest.fail("launched"))
    pool, table = m.kv8_pool(2, 2, 64, 32, device="cpu"), torch.zeros((1, 2), dtype=torch.int32)
    one = torch.zeros(1, dtype=torch.int32)
    q, x = torch.zeros((1, 1, 4, 64)), torch.zeros((2, 64))
    for f in (lambda: m.kv8_attention(q, pool, table, one, window=1 << 31), lambda: m.kv8_attention(q, pool, table, one, window=2.5),
              lambda: m.kv8_attention(q, pool, table, one, scale=10 ** 400), lambda: m.add_rms_norm_q8_1(x, torch.zeros(64), eps="1e-6")):
        with pytest.raises(m.MoeError):
            f()
