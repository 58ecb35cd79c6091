"""The steps of moe_decode.h as a decode loop runs them (examples/decode_layer.py with head norms, rotation and a vocabulary): over a prompt
and windows with rejected drafts, against plain formulas in 64 bits; draft trees; and calls on two streams at once. Tolerances: fp32
products of up to 512 terms add 1e-4 of the largest value at most, as in test_gpu_decode_layer.py."""
import importlib.util
import os

import numpy as np
import pytest
import torch

import decode_ref as D
from test_gpu_logprobs import check as check_logprobs

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def m():
    import quantized_routed_expert_grouped_gb300 as mod
    mod.lib()
    return mod


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("decode_layer", os.path.join(ROOT, "examples", "decode_layer.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def norm(h, w, eps=1e-6):
    return h / (h.square().mean(-1, keepdim=True) + eps).sqrt() * w.double().cpu()


def close(got, want, tol):
    assert ((got.double().cpu() - want).abs().amax() <= tol * want.abs().amax()).item()


def turned(x, places, weight, rope):
    y, _ = D.rope(x.numpy(), places, weight.double().cpu().numpy(), rope.inv_freq, float(np.float32(rope.factor)), rope.start, rope.interleaved)
    return torch.from_numpy(y)


@pytest.mark.parametrize("inter", [False, True])
def test_layer_with_rotation(m, example, inter):
    rope = m.Rope(48, theta=10000.0, start=8, interleaved=inter, scaling={"kind": "yarn", "scale": 4, "original": 256})
    L = example.DecodeLayer(rope=rope, head_norms=True, vocab=5003)
    g = torch.Generator("cuda").manual_seed(3)
    held = [0, 0]
    for T, keep in ((32, [32, 32]), (13, [13, 13]), (4, [1, 4]), (4, [2, 0]), (1, [1, 1]), (4, [4, 3])):
        rows = L.B * T
        update, residual = (torch.randn((rows, L.N), generator=g, device="cuda") for _ in range(2))
        start = L.start.clone()
        got, stream = L.window(update, residual.clone())
        assert int(L.err) == 0 and start.tolist() == held
        h = (update + residual).double().cpu()
        qkv = (norm(h, L.norm1) @ L.w_qkv.double().cpu()).view(rows, -1, L.D)
        places = np.concatenate([np.arange(n, n + T) for n in held])
        q = turned(qkv[:, :L.H], places, L.q_norm, rope).view(L.B, T, L.H, L.D)
        k_new = turned(qkv[:, L.H:L.H + L.HKV], places, L.k_norm, rope).view(L.B, T, L.HKV, L.D)
        attn = torch.zeros((L.B, T, L.H, L.D), dtype=torch.float64)
        cu = torch.tensor([0, held[0] + T, held[0] + held[1] + 2 * T], dtype=torch.int32, device="cuda")
        k, v = (t.double().cpu() for t in m.kv8_read(L.pool, L.table, cu, torch.zeros_like(start), int(cu[-1]), dtype=torch.float32))
        for b in range(L.B):
            n = held[b] + T
            kb, vb = (t[int(cu[b]):int(cu[b]) + n] for t in (k, v))
            # half a step of the block's scale, which earlier tokens may have set
            assert ((kb[-T:] - k_new[b]).abs() <= 0.51 * kb.abs().amax() / 127 + 1e-3 * k_new[b].abs().amax()).all()
            kb, vb = (t.repeat_interleave(L.H // L.HKV, 1) for t in (kb, vb))
            s = torch.einsum("thd,nhd->thn", q[b], kb) / L.D ** 0.5
            s.masked_fill_(torch.arange(n) > torch.arange(held[b], n)[:, None, None], -torch.inf)
            attn[b] = torch.einsum("thn,nhd->thd", s.softmax(-1), vb)
        close(stream, h + attn.view(rows, -1) @ L.w_o.double().cpu(), 1e-4)
        # the drafts: every second one is what the model would have said
        logits = ((got + stream) @ L.w_vocab).view(L.B, T, -1)
        drafts = torch.randint(0, 5003, (L.B, T), generator=g, device="cuda", dtype=torch.int32)
        best = logits.argmax(-1).int()
        if T > 1:
            drafts[0, 1:] = best[0, :-1]
            drafts[1, 1] = best[1, 0]
        stand, logprobs, top = L.verify(got + stream, drafts)
        assert torch.equal(top, best)
        ids = torch.cat([drafts[:, 1:], torch.full_like(drafts[:, :1], -1)], 1).view(-1, 1)
        check_logprobs(m, logits.view(rows, -1), ids.cpu().numpy(), 1)  # (an error of 2^-24 of a log probability of -100 alone is 6e-6)
        assert torch.equal(logprobs, m.token_logprobs(logits.view(rows, -1), ids, top=1)[0].view(L.B, T)[:, :-1])
        expect = [1 + int((best[b, :-1] == drafts[b, 1:]).long().cumprod(0).sum()) for b in range(L.B)]
        assert stand.tolist() == expect and (T == 1 or stand[0] == T)
        L.accept(torch.tensor(keep, dtype=torch.int32, device="cuda"))
        held = [a + b for a, b in zip(held, keep)]


def test_tree_is_its_paths(m):
    """Draft trees turned by their depth: each token's attention is what its path gives, decoded token by token."""
    B, T, H, HKV, d, ctx = 2, 6, 4, 2, 64, 70
    parent = [[-1, 0, 0, 1, 1, 2], [-1, 0, 1, 2, 3, 0]]
    g = torch.Generator().manual_seed(5)
    rope = m.Rope(64, theta=1000.0)
    w = 1 + 0.2 * torch.randn((2, d), generator=g)
    w = w.cuda()
    pre = torch.randn((B, ctx, H + 2 * HKV, d), generator=g).cuda()
    win = torch.randn((B, T, H + 2 * HKV, d), generator=g).cuda()
    ints = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731

    def fresh():
        return m.kv8_pool(B * 2, HKV, d), ints([[0, 1], [2, 3]])

    def append(pool, table, x, start, positions=None):
        n = x.shape[1]
        x = x.reshape(B * n, H + 2 * HKV, d)
        return m.kv8_append(x[:, H:H + HKV], x[:, H + HKV:], pool, table, ints([0, n, 2 * n]), ints([start] * B), rope, q=x[:, :H], q_weight=w[0], k_weight=w[1],
                            positions=positions).view(B, n, H, d)
    depth = [[0] * T for _ in range(B)]
    see = [[0] * T for _ in range(B)]
    for b in range(B):
        for t in range(T):
            p = parent[b][t]
            depth[b][t] = 0 if p < 0 else depth[b][p] + 1
            see[b][t] = (0 if p < 0 else see[b][p]) | 1 << t
    pool, table = fresh()
    append(pool, table, pre, 0)
    turn = ints([ctx + depth[b][t] for b in range(B) for t in range(T)])
    q = append(pool, table, win, ctx, turn)
    out = m.kv8_attention(q, pool, table, ints([ctx + T] * B), tree=ints(see))
    for t in range(T):
        # the paths of token t in both sequences may differ in length: each is decoded on its own
        for b in range(B):
            path = [i for i in range(T) if see[b][t] >> i & 1]
            p2, t2 = fresh()
            append(p2, t2, pre, 0)
            rows = win[:, path]
            q2 = append(p2, t2, rows, ctx)
            ref = m.kv8_attention(q2[:, -1:], p2, t2, ints([ctx + len(path)] * B))
            assert torch.equal(q2[b, -1], q[b, t])  # the same position, the same bits
            # blocks of the window hold other tokens too: other scales, half a step of the largest value apart at most
            step = float(win.abs().max()) * 1.5 / 127
            assert (out[b, t] - ref[b, 0]).abs().max() <= 4 * step


def test_two_streams_at_once(m):
    """Calls on two streams at the same time, from a shared Rope and shared weights, give what they give alone."""
    g = torch.Generator("cuda").manual_seed(7)
    x = [torch.randn((3000, 40, 64), generator=g, device="cuda").bfloat16() for _ in range(2)]
    logits = [torch.randn((64, 30001), generator=g, device="cuda") for _ in range(2)]
    pos = torch.arange(3000, dtype=torch.int32, device="cuda")
    rope, w = m.Rope(64), torch.ones(64, dtype=torch.bfloat16, device="cuda")
    pools = [m.kv8_pool(50, 4, 64) for _ in range(4)]
    table = torch.arange(50, dtype=torch.int32, device="cuda").view(1, 50)
    cu, zero = torch.tensor([0, 3000], dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")

    def run(i, pool, stream=None):
        a = m.head_norm_rope(x[i][:, :32], pos, rope, q_weight=w, stream=stream)[0]
        b = m.kv8_append(x[i][:, 32:36], x[i][:, 36:], pool, table, cu, zero, rope, q=x[i][:, :32], k_weight=w, stream=stream)
        return [a, b] + list(m.token_logprobs(logits[i], top=9, stream=stream)[1:])
    want = [run(i, pools[i]) for i in range(2)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(5):
        got = [run(i, pools[2 + i], streams[i]) for i in range(2)]
        torch.cuda.synchronize()
        for i in range(2):
            assert torch.equal(pools[i], pools[2 + i])
            assert all(torch.equal(a, b) for a, b in zip(got[i], want[i]))


def test_large_offsets(m):
    """Rows more than 2^31 elements from the first: norms, rotation and logits."""
    n, apart = 5, 3 << 29
    far = torch.empty(n * apart, dtype=torch.bfloat16, device="cuda")
    rows = far.as_strided((n, 2, 64), (apart, 64, 1))
    rows.copy_(torch.randn((n, 2, 64), device="cuda"))
    pos, rope = torch.arange(n, dtype=torch.int32, device="cuda"), m.Rope(64)
    want = m.head_norm_rope(rows.contiguous(), pos, rope)[0]
    assert torch.equal(m.head_norm_rope(rows, pos, rope)[0], want)
    m.head_norm_rope(rows, pos, rope, q_out=rows)
    assert torch.equal(rows, want)
    logits = far.as_strided((n, 5001), (apart, 1))
    logits.copy_(torch.randn((n, 5001), device="cuda"))
    # (not bit for bit against contiguous rows: what lies at another alignment is summed in another order)
    check_logprobs(m, logits, np.array([[0], [5000], [-1], [17], [2500]]), 5)
