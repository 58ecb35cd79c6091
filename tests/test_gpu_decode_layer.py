"""The example layer (examples/decode_layer.py) over a prompt and windows with rejected drafts, against plain
formulas in 64 bits: attention over keys and values as the cache holds them, the norms, and the experts
on dequantised weights and activations. Tolerances: fp32 products of up to 512 terms add 1e-4 at most;
the q8_1 codes of the gated activations may turn at a tie (one step in 127 of one value)."""
import importlib.util
import os

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("decode_layer", os.path.join(ROOT, "examples", "decode_layer.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def q8_0(blobs, rows, cols):
    b = blobs.cpu().numpy().reshape(blobs.shape[0], -1)[:, :rows * (cols // 32) * 34].reshape(-1, rows, cols // 32, 34)
    d = np.ascontiguousarray(b[..., :2]).view(np.float16).astype(np.float64)
    return torch.from_numpy(d * b[..., 2:].view(np.int8)).flatten(2)


def norm(h, w, eps=1e-6):
    return h / (h.square().mean(-1, keepdim=True) + eps).sqrt() * w.double().cpu()


def close(got, want, tol):
    assert ((got.double().cpu() - want).abs().amax() <= tol * want.abs().amax()).item()


def test_decode_layer(example):
    import quantized_routed_expert_grouped_gb300 as m
    L = example.DecodeLayer()
    gu_w, dn_w = q8_0(L.gate_up, 2 * L.F, L.N), q8_0(L.down, L.N, L.F)
    g = torch.Generator("cuda").manual_seed(3)
    held = [0, 0]
    for T, keep in ((32, [32, 32]), (13, [13, 13]), (4, [1, 4]), (4, [2, 0]), (1, [1, 1]), (4, [4, 3])):
        rows = L.B * T
        update, residual = (torch.randn((rows, L.N), generator=g, device="cuda") for _ in range(2))
        start = L.start.clone()
        got, stream = L.window(update, residual.clone())
        assert int(L.err) == 0 and start.tolist() == held
        # ---- plain
        h = (update + residual).double().cpu()
        x = norm(h, L.norm1)
        qkv = (x @ L.w_qkv.double().cpu()).view(L.B, T, -1, L.D)
        attn = torch.zeros((L.B, T, L.H, L.D), dtype=torch.float64)
        cu = torch.tensor([0, held[0] + T, held[0] + held[1] + 2 * T], dtype=torch.int32, device="cuda")
        k, v = m.kv8_read(L.pool, L.table, cu, torch.zeros_like(start), int(cu[-1]), dtype=torch.float32)
        for b in range(L.B):
            n = held[b] + T
            kb, vb = (t[int(cu[b]):int(cu[b]) + n].double().cpu().repeat_interleave(L.H // L.HKV, 1) for t in (k, v))
            new = qkv[b, :, L.H:L.H + L.HKV].repeat_interleave(L.H // L.HKV, 1)
            # half a step of the block's scale, which earlier tokens may have set
            assert ((kb[-T:] - new).abs() <= 0.51 * kb.abs().amax() / 127 + 1e-3 * new.abs().amax()).all()
            s = torch.einsum("thd,nhd->thn", qkv[b, :, :L.H], kb) / L.D ** 0.5
            s.masked_fill_(torch.arange(n) > torch.arange(held[b], n)[:, None, None], -torch.inf)
            attn[b] = torch.einsum("thn,nhd->thd", s.softmax(-1), vb)
        h = h + attn.view(rows, -1) @ L.w_o.double().cpu()
        close(stream, h, 1e-4)
        y = norm(stream.double().cpu(), L.norm2)
        _, y32, xq = m.add_rms_norm_q8_1(stream, L.norm2, with_y=True)
        close(y32, y, 1e-5)
        a = m.dequantize_q8_1(xq).double().cpu()
        ids, weights = (t.cpu() for t in m.router_topk(y32 @ L.w_router, L.k))
        want = torch.zeros((rows, L.N), dtype=torch.float64)
        for t in range(rows):
            for j, e in enumerate(ids[t].tolist()):
                gu = gu_w[e] @ a[t]
                act = gu[:L.F] * torch.sigmoid(gu[:L.F]) * gu[L.F:]
                hq = m.dequantize_q8_1(m.quantize_q8_1(act.float().view(1, -1).cuda()))[0].double().cpu()
                want[t] += weights[t, j].double() * (dn_w[e] @ hq)
        close(got, want, 5e-3)
        L.accept(torch.tensor(keep, dtype=torch.int32, device="cuda"))
        held = [a + b for a, b in zip(held, keep)]


def test_example_runs(example, capsys):
    example.main()
    assert "err 0" in capsys.readouterr().out
