"""One decoder layer over verify windows, from the residual stream back to it, on this library's calls:

    residual + norm (add_rms_norm_q8_1) -> projections (torch) -> keys and values into the 8-bit cache
    (kv8_write) -> attention of the window over it (kv8_attention) -> projection (torch) -> residual + norm + q8_1
    rows (add_rms_norm_q8_1) -> router (router_topk, route_group) -> the routed experts (ExpertCall)
    -> combine

A prompt goes through as windows of up to 32 tokens; then windows of draft tokens follow, of which some
are rejected: the next window starts at the first rejected position and writes over the rest.

    python examples/decode_layer.py            # on a GPU: a prompt, then windows of four drafts
"""
from __future__ import annotations

import os
import sys
import time

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import quantized_routed_expert_grouped_gb300 as m  # noqa: E402
import synth  # noqa: E402


class DecodeLayer:
    """Seeded weights; a cache of `max_tokens` positions for each of n_seqs sequences, pages handed out in order."""

    def __init__(self, n_embd=512, n_heads=8, n_kv_heads=2, head_dim=64, n_ff=256, n_experts=8, top_k=2, n_seqs=2,
                 max_tokens=1024, page_tokens=64, seed=1, device="cuda"):
        self.N, self.H, self.HKV, self.D, self.F, self.E, self.k = n_embd, n_heads, n_kv_heads, head_dim, n_ff, n_experts, top_k
        self.B, self.dev = n_seqs, device
        g = torch.Generator(device=device).manual_seed(seed)

        def w(*shape):
            return torch.randn(shape, generator=g, device=device) / shape[0] ** 0.5

        self.w_qkv, self.w_o, self.w_router = w(n_embd, (n_heads + 2 * n_kv_heads) * head_dim), w(n_heads * head_dim, n_embd), w(n_embd, n_experts)
        self.norm1, self.norm2 = 1 + 0.1 * torch.randn((2, n_embd), generator=g, device=device)
        self.gate_up = synth.weight_blobs(m.Q8_0, 2 * n_ff, n_embd, n_experts, synth.derive_key(seed, 1), device)
        self.down = synth.weight_blobs(m.Q8_0, n_embd, n_ff, n_experts, synth.derive_key(seed, 2), device)
        self.tables = [torch.tensor([b[x].data_ptr() for x in range(n_experts)], dtype=torch.int64, device=device)
                       for b in (self.gate_up, self.down)]
        pages = -(-max_tokens // page_tokens)
        self.pool = m.kv8_pool(n_seqs * pages, n_kv_heads, head_dim, page_tokens, device)
        self.table = torch.arange(n_seqs * pages, dtype=torch.int32, device=device).view(n_seqs, pages)
        self.workspace = m.kv8_attention_workspace(n_seqs, 32, n_heads, n_kv_heads, head_dim, device)
        self.err = torch.zeros(1, dtype=torch.int32, device=device)
        self.start = torch.zeros(n_seqs, dtype=torch.int32, device=device)  # positions held before the window

    def attention(self, x):
        """x: normed rows [B * T, N] of the windows -> attention output [B * T, N]."""
        T = x.shape[0] // self.B
        qkv = (x @ self.w_qkv).view(self.B * T, self.H + 2 * self.HKV, self.D)
        cu = torch.arange(self.B + 1, dtype=torch.int32, device=self.dev) * T
        # keys and values are read where the projection left them
        m.kv8_write(qkv[:, self.H:self.H + self.HKV], qkv[:, self.H + self.HKV:], self.pool, self.table, cu, self.start, err=self.err)
        q = qkv[:, :self.H].unflatten(0, (self.B, T))
        out = m.kv8_attention(q, self.pool, self.table, self.start + T, workspace=self.workspace, err=self.err)
        return out.view(self.B * T, self.H * self.D) @ self.w_o

    def experts(self, y, xq):
        """y: normed rows [rows, N], xq: their q8_1 rows -> the routed experts' combined output [rows, N]."""
        n = y.shape[0] * self.k
        ints = lambda c: torch.empty(c, dtype=torch.int32, device=self.dev)  # noqa: E731
        ids, weights = m.router_topk(y @ self.w_router, self.k)
        grp_expert, grp_start, n_groups, src, dst = ints(n), ints(n + 1), ints(1), ints(n), ints(n)
        m.route_group(ids, self.E, 0, grp_expert, grp_start, n_groups, src, dst, err=self.err)
        gu = torch.empty((n, 2 * self.F), device=self.dev)
        hq = torch.empty((n, self.F // 32, 36), dtype=torch.uint8, device=self.dev)
        out = torch.empty((n, self.N), device=self.dev)
        m.ExpertCall(m.Q8_0, None, m.Q8_0, None, self.N, self.F, *self.tables, self.E, grp_expert, grp_start, n_groups, min(n, self.E), 0, n, xq,
                     src, dst, gu, hq, out, self.err)()
        return m.combine(out, ids, weights, self.E)

    def window(self, update, residual):
        """One window: residual stream [B * T, N] (T tokens of each sequence) and the previous layer's update of
        it, 1 <= T <= 32 -> this layer's update and the stream that it belongs to. The cache holds the window's
        tokens afterwards, from position self.start on."""
        residual, x, _ = m.add_rms_norm_q8_1(update, self.norm1, residual=residual, with_y=True)
        attn = self.attention(x)
        # the stream is updated in place; the experts take the q8_1 rows, the router the norm itself
        residual, y, xq = m.add_rms_norm_q8_1(attn, self.norm2, residual=residual, sum_out=residual, with_y=True)
        return self.experts(y, xq), residual

    def accept(self, n):
        """Keep the first n tokens of the window just computed (per sequence: a number or an int32 tensor)."""
        self.start = self.start + n


def main():
    torch.manual_seed(0)
    layer = DecodeLayer(n_embd=1024, n_heads=16, n_kv_heads=4, head_dim=128, n_ff=512, n_experts=64, top_k=8, n_seqs=4, max_tokens=8192)
    prompt = 300
    for a in range(0, prompt, 32):
        T = min(32, prompt - a)
        layer.window(torch.zeros((4 * T, layer.N), device="cuda"), torch.randn((4 * T, layer.N), device="cuda"))
        layer.accept(T)
    torch.cuda.synchronize()
    t = time.perf_counter()
    steps = 50
    for i in range(steps):
        layer.window(torch.zeros((16, layer.N), device="cuda"), torch.randn((16, layer.N), device="cuda"))
        layer.accept(torch.tensor([1 + (i + b) % 4 for b in range(4)], dtype=torch.int32, device="cuda"))
    torch.cuda.synchronize()
    print(f"{steps} windows of 4 drafts for 4 sequences: {(time.perf_counter() - t) / steps * 1e6:.0f} us each, "
          f"{layer.start.tolist()} positions held, err {int(layer.err)}")


if __name__ == "__main__":
    main()
