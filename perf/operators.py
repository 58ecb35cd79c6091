"""Timing cases of the operators around a verify window's 8-bit key/value cache.

Four operators, each in a plain form (elementary torch operations in 32 bits) and as the package's own calls:

- ``write``: new keys and values quantised into the paged cache, then the touched positions read back;
- ``read``: a range of each sequence's cached keys and values read back as dense rows;
- ``attention``: a window of queries per sequence over the cache;
- ``norm``: residual addition, root-mean-square norm and the q8_1 rows that the routed experts take, read back as values.

A cache record holds 32 tokens (positions 32 j .. 32 j + 31) of one key/value head:
``f32 k_scale, f32 v_scale, 8 bytes unused, u8 k[32 D], u8 v[32 D]``, a code c standing for (c - 128) * scale.
Keys: ``[4 row groups][D / 32][8 rows][32 dims]``, token t at row group (t >> 1) & 3, row 2 (t >> 3) + (t & 1).
Values: ``[D dims][32 tokens]``. Pool: uint8 ``[pages, kv heads, page tokens / 32, 64 D + 16]``; page 0 stays a filler
page here, which unused page table entries name.
"""
import math
import random

import numpy as np
import torch

own = False

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
DEV = "cuda"


# ------------------------------------------------------------------------------------------------ cases

def _attn(name, B, T, hq, hkv, D, lo, hi, page, dtype, window=0, tree=False, empty=0):
    c = dict(op="attention", B=B, T=T, hq=hq, hkv=hkv, D=D, lo=lo, hi=hi, page=page, dtype=dtype, window=window, tree=tree, empty=empty)
    return dict(c, name=name) if name else c


def _write(name, B, n_lo, n_hi, s_lo, s_hi, hkv, D, page, dtype):
    c = dict(op="write", B=B, n_lo=n_lo, n_hi=n_hi, s_lo=s_lo, s_hi=s_hi, hkv=hkv, D=D, page=page, dtype=dtype)
    return dict(c, name=name) if name else c


def _read(name, B, n_lo, n_hi, s_lo, s_hi, hkv, D, page, dtype):
    return dict(_write(name, B, n_lo, n_hi, s_lo, s_hi, hkv, D, page, dtype), op="read")


def _norm(name, rows, cols, dtype, wdtype, residual=True):
    c = dict(op="norm", rows=rows, cols=cols, dtype=dtype, wdtype=wdtype, residual=residual)
    return dict(c, name=name) if name else c


def listed():
    return [
        # one user, one token, a short chat: latency only
        _attn("attn_one_token_short", 1, 1, 16, 4, 128, 777, 777, 64, "bf16"),
        # one user's verify window of 4 at a 131k-token context, in the engine's own fp32 activations
        _attn("attn_window4_131k_f32", 1, 4, 16, 4, 128, 131077, 131077, 64, "f32"),
        # a serving batch of single tokens, ragged lengths, three slots idle (rows that see nothing)
        _attn("attn_batch64_ragged", 64, 1, 32, 8, 128, 1, 16384, 64, "bf16", empty=3),
        # a draft tree of 8 tokens under a sliding window, one query head per key/value head, small heads
        _attn("attn_tree8_sliding", 24, 8, 12, 12, 64, 5, 9001, 32, "f16", window=1000, tree=True),
        # a million-token context, wide heads, two query tokens
        _attn("attn_window2_1M", 1, 2, 8, 1, 256, 1048579, 1048579, 128, "bf16"),
        # the largest: a full batch of windows of 4, eight query heads per key/value head
        _attn("attn_batch32_window4", 32, 4, 64, 8, 128, 8191, 32769, 64, "f16"),
        # a serving batch's window of 4 appended at odd places (kept tokens may need a wider scale)
        _write("write_window4_batch64", 64, 4, 4, 31, 16001, 8, 128, 64, "bf16"),
        # prompts of several users written at once, each from its own place
        _write("write_prompts", 7, 1, 20011, 0, 45, 8, 128, 64, "bf16"),
        # a small shared prefix read back in fp32
        _read("read_small_f32", 3, 33, 700, 0, 17, 4, 96, 32, "f32"),
        # long prefixes read back for another attention
        _read("read_prefixes", 5, 4097, 40001, 0, 64, 8, 128, 128, "bf16"),
        # a window of 4 tokens into the experts: latency only
        _norm("norm_window4", 4, 2560, "f32", "f32"),
        # a prompt's rows
        _norm("norm_prompt", 8191, 4096, "bf16", "bf16"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    top = max(work(c)["bytes"] for c in listed())
    while True:
        op = rng.choice(["attention", "attention", "write", "read", "norm"])
        page, dtype = rng.choice([32, 64, 128]), rng.choice(list(TYPES))
        D, hkv = rng.choice([64, 96, 128, 192, 256]), rng.choice([1, 2, 3, 4, 8, 12])
        if op == "attention":
            T = rng.randint(1, 8)
            hi = _log(rng, 1, 300000)
            c = _attn(None, _log(rng, 1, 96), T, hkv * rng.choice([1, 2, 3, 4, 5, 8, 16]), hkv, D, _log(rng, 1, hi), hi, page, dtype,
                      window=rng.choice([0, 0, _log(rng, 1, 5000)]), tree=T > 1 and rng.random() < 0.4, empty=0)
            c["empty"] = rng.randint(0, c["B"] // 4)
            # padded to the longest sequence, as the plain form holds it
            fits = c["B"] * c["hi"] * hkv * max(D, c["hq"] // hkv * T) <= 32 * 32769 * 8 * 128
        elif op == "norm":
            c = _norm(None, _log(rng, 1, 16384), 32 * _log(rng, 1, 512), dtype, rng.choice([dtype, "f32"]), rng.random() < 0.7)
            fits = c["rows"] * c["cols"] <= 1 << 26
        else:
            n_hi = rng.choice([rng.randint(1, 8), _log(rng, 8, 60000)])
            c = (_write if op == "write" else _read)(None, _log(rng, 1, 64), rng.randint(0, n_hi), n_hi, 0, _log(rng, 1, 20000), hkv, D, page, dtype)
            fits = sum(_spread(c["B"], c["n_lo"], c["n_hi"])) * hkv * D <= 1 << 28 and c["B"] * (c["s_hi"] + n_hi) * hkv * D <= 1 << 31
        if fits and work(c)["bytes"] <= top:
            return c


def _spread(n, lo, hi):
    """n whole numbers from lo to hi (over their logarithm), in a fixed order that is not theirs by size."""
    if n == 1:
        return [hi]
    v = [int(round((lo + 1) * ((hi + 1) / (lo + 1)) ** (i / (n - 1)))) - 1 for i in range(n)]
    random.Random(n).shuffle(v)
    return v


def _lens(c):
    v = _spread(c["B"] - c["empty"], c["lo"], c["hi"]) if c["B"] > c["empty"] else []
    return v + [0] * c["empty"]


def _back(start, n):
    """The whole-block range that a write of n tokens at start touches, up to the write's end."""
    return (start - start % 32, n + start % 32) if n else (start, 0)


def work(case):
    c = case
    if c["op"] == "norm":
        e, w, m = (4 if c["dtype"] == "f32" else 2), (4 if c["wdtype"] == "f32" else 2), c["rows"] * c["cols"]
        # x, residual; the sum, the norm, the q8_1 rows, their values in fp16
        return {"bytes": m * (e * (2 + c["residual"] + c["residual"]) + 36 / 32 + 2) + c["cols"] * w, "flops": 8 * m}
    e, hd = (4 if c["dtype"] == "f32" else 2), c["hkv"] * c["D"]
    code = 2 * hd + 16 / 32 * c["hkv"]  # cache bytes of a token, keys and values
    if c["op"] == "attention":
        seen = sum(min(n, c["window"] + c["T"] - 1) if c["window"] else n for n in _lens(c))
        rows = c["B"] * c["T"] * c["hq"]
        return {"bytes": seen * code + rows * (2 * c["D"] * e + 4), "flops": 4 * c["T"] * c["hq"] * c["D"] * seen}
    n, s = _spread(c["B"], c["n_lo"], c["n_hi"]), _spread(c["B"], c["s_lo"], c["s_hi"])
    if c["op"] == "read":
        return {"bytes": sum(n) * (code + 2 * hd * e), "flops": sum(n) * 2 * hd}
    back = sum(_back(a, b)[1] for a, b in zip(s, n))
    return {"bytes": sum(n) * (2 * hd * e + code) + back * (code + 2 * hd * e), "flops": (3 * sum(n) + back) * 2 * hd}


# ------------------------------------------------------------------------------------------------ inputs

def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def _cache(c, tokens, g, rng):
    """A pool of plausible records (codes about normal, scales by head) and a page table for `tokens` positions per sequence."""
    need = [-(-t // c["page"]) for t in tokens]
    n_pages = sum(need) + 3
    nb, rb = c["page"] // 32, 64 * c["D"] + 16
    pool = torch.empty((n_pages, c["hkv"], nb, rb), dtype=torch.uint8, device=DEV)
    flat = pool.view(-1, rb)
    for a in range(0, flat.shape[0], 1 << 16):
        part = flat[a:a + (1 << 16)]
        part.copy_((torch.randn(part.shape, generator=g, device=DEV, dtype=torch.float16) * 40 + 128).clamp_(1, 255).round_())
    scale = torch.exp(0.4 * torch.randn((n_pages, c["hkv"], nb, 2), generator=g, device=DEV)) * 0.03
    pool[..., :8] = scale.view(torch.uint8).view(n_pages, c["hkv"], nb, 8)
    pool[..., 8:16] = 0
    ids = list(range(1, n_pages))
    rng.shuffle(ids)
    table = torch.zeros((len(need), max(max(need), 1)), dtype=torch.int32)
    at = 0
    for b, m in enumerate(need):
        table[b, :m] = torch.tensor(ids[at:at + m], dtype=torch.int32)
        at += m
    return pool, table.to(DEV)


def prepare(case, seed):
    c, rng = case, random.Random(seed)
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    dt = TYPES[c["dtype"]]
    st = {"case": dict(c)}
    if c["op"] == "norm":
        R, N = c["rows"], c["cols"]
        st["x"] = torch.randn((R, N), generator=g, device=DEV).to(dt)
        # a residual stream: larger than its update, with a few strong channels
        ch = torch.exp(0.5 * torch.randn((N,), generator=g, device=DEV))
        st["residual"] = (torch.randn((R, N), generator=g, device=DEV) * (3 * ch)).to(dt) if c["residual"] else None
        st["weight"] = (1 + 0.3 * torch.randn((N,), generator=g, device=DEV)).to(TYPES[c["wdtype"]])
        st["eps"] = 1e-6
        return st
    if c["op"] == "attention":
        B, T, hq, hkv, D = c["B"], c["T"], c["hq"], c["hkv"], c["D"]
        lens = _lens(c)
        st["pool"], st["table"] = _cache(c, lens, g, rng)
        # the queries are the first heads of the fused projection's rows
        qkv = torch.randn((B, T, hq + 2 * hkv, D), generator=g, device=DEV)
        qkv *= torch.exp(0.5 * torch.randn((1, 1, hq + 2 * hkv, 1), generator=g, device=DEV))
        st["q"] = qkv.to(dt)[:, :, :hq]
        st["lens"] = _ints(lens)
        st["tree"] = None
        if c["tree"]:  # each draft token sees itself, its parent and what that sees; the last one of every third sequence nothing of the window
            rows = []
            for b in range(B):
                see = [1]
                for t in range(1, T):
                    see.append(see[rng.randrange(t)] | 1 << t)
                rows.append(see[:-1] + [0] if b % 3 == 2 else see)
            st["tree"] = _ints(rows)
        if own:  # a serving program keeps one workspace for its calls
            import quantized_routed_expert_grouped_gb300 as m
            st["ws"] = m.kv8_attention_workspace(B, T, hq, hkv, D)
        return st
    B, hkv, D = c["B"], c["hkv"], c["D"]
    n, s = _spread(B, c["n_lo"], c["n_hi"]), _spread(B, c["s_lo"], c["s_hi"])
    st["pool"], st["table"] = _cache(c, [a + b for a, b in zip(s, n)], g, rng)
    cu = lambda v: _ints(np.concatenate([[0], np.cumsum(v)]).astype(int).tolist())  # noqa: E731
    st["cu"], st["start"], st["N"] = cu(n), _ints(s), sum(n)
    if c["op"] == "write":
        # keys and values lie behind four query heads each in the fused projection's rows; some channels are strong
        ch = 1 + 3 * (torch.rand((1, hkv, D), generator=g, device=DEV) < 0.05)
        qkv = torch.randn((st["N"], 6 * hkv, D), generator=g, device=DEV, dtype=torch.float32 if dt is torch.float32 else torch.float16).to(dt)
        qkv[:, 4 * hkv:5 * hkv] *= ch.to(dt)
        st["k"], st["v"] = qkv[:, 4 * hkv:5 * hkv], qkv[:, 5 * hkv:]
        back = [_back(a, b) for a, b in zip(s, n)]
        st["back_start"], st["back_cu"], st["back_N"] = _ints([a for a, _ in back]), cu([b for _, b in back]), sum(b for _, b in back)
    return st


# ------------------------------------------------------------------------------------------------ plain forms

def _values(rec, D):
    """Records [..., 64 D + 16] -> keys and values [..., 32, D] in fp32."""
    lead = rec.shape[:-1]
    scale = rec[..., :8].contiguous().view(torch.float32)
    k = rec[..., 16:16 + 32 * D].reshape(*lead, 4, D // 32, 4, 2, 32)  # row group, dims / 32, t >> 3, t & 1, dims % 32
    n = len(lead)
    k = k.permute(*range(n), n + 2, n, n + 3, n + 1, n + 4).reshape(*lead, 32, D)
    v = rec[..., 16 + 32 * D:].reshape(*lead, D, 32).transpose(-1, -2)
    return (k.float() - 128) * scale[..., 0, None, None], (v.float() - 128) * scale[..., 1, None, None]


def _records(k, v, ks, vs):
    """Codes [..., 32, D] (centred at 0) and scales [...] -> records."""
    lead, D = k.shape[:-2], k.shape[-1]
    n = len(lead)
    k = (k + 128).to(torch.uint8).reshape(*lead, 4, 4, 2, D // 32, 32)
    k = k.permute(*range(n), n + 1, n + 3, n, n + 2, n + 4).reshape(*lead, 32 * D)
    v = (v + 128).to(torch.uint8).transpose(-1, -2).reshape(*lead, 32 * D)
    head = torch.stack([ks, vs, torch.zeros_like(ks), torch.zeros_like(ks)], -1).view(torch.uint8)
    return torch.cat([head, k, v], -1)


def _slots(cu, start, N, table, page):
    """Ragged rows -> 32-token blocks: sequence b's blocks are slots first[b], first[b] + 1, ..."""
    B = start.shape[0]
    cu, start = cu.long(), start.long()
    n = cu[1:] - cu[:-1]
    first = cu[:-1] // 32 + 2 * torch.arange(B, device=cu.device)
    j = torch.arange(N // 32 + 2 * B, device=cu.device)
    b = torch.searchsorted(first, j, right=True) - 1
    blk = start[b] // 32 + j - first[b]
    used = (n[b] > 0) & (blk * 32 < start[b] + n[b])
    pg = table[b, (blk * 32 // page).clamp(max=table.shape[1] - 1)].long()
    i = torch.arange(N, device=cu.device)
    bi = torch.searchsorted(cu[1:], i, right=True)
    p = start[bi] + i - cu[bi]
    # slots in no sequence go to the filler page
    return torch.where(used, pg, 0), blk * 32 % page // 32, (start[b] - blk * 32).clamp(0, 32), first[bi] + p // 32 - start[bi] // 32, p % 32


def _plain_read(pool, table, cu, start, N, dtype):
    D = (pool.shape[-1] - 16) // 64
    pg, nb, _, slot, t = _slots(cu, start, N, table, pool.shape[2] * 32)
    k, v = _values(pool[pg, :, nb], D)  # [slots, heads, 32, D]
    return k[slot, :, t].to(dtype), v[slot, :, t].to(dtype)


def _plain_quantise(x, old, kept, slot, t, first_kept):
    """One of keys or values: rows x, the blocks' old scales and codes -> new scales and codes."""
    S, H, _, D = kept.shape
    one27 = torch.full((), 127.0, device=x.device)
    new = torch.zeros((S, H, 32, D), device=x.device)
    new[slot, :, t] = x.float()
    fresh = torch.zeros((S, 32), dtype=torch.bool, device=x.device)
    fresh[slot, t] = True
    amax = new.abs().amax((2, 3))
    old = torch.where(first_kept[:, None] > 0, old, 0.0)
    scale = torch.maximum(old, torch.where(amax < 2.0 ** -100, 0.0, amax / one27))
    some = scale > 0
    ratio, inv = torch.where(some, old / scale, 0.0), torch.where(some, 1 / scale, 0.0)
    code = torch.where(fresh[:, None, :, None], torch.round(new * inv[..., None, None]).clamp(-127, 127), torch.round(kept * ratio[..., None, None]))
    return code, scale


def _plain_write(k, v, pool, table, cu, start):
    D, page = k.shape[-1], pool.shape[2] * 32
    pg, nb, keep, slot, t = _slots(cu, start, k.shape[0], table, page)
    rec = pool[pg, :, nb]
    scale = rec[..., :8].contiguous().view(torch.float32)
    unit = rec.clone()
    unit[..., :8] = torch.ones(2, device=k.device).view(torch.uint8)
    kc, vc = _values(unit, D)
    kc, ks = _plain_quantise(k, scale[..., 0], kc, slot, t, keep)
    vc, vs = _plain_quantise(v, scale[..., 1], vc, slot, t, keep)
    pool[pg, :, nb] = _records(kc, vc, ks, vs)


def _plain_attention(q, pool, table, lens, window, tree):
    B, T, hq, D = q.shape
    hkv, page = pool.shape[1], pool.shape[2] * 32
    rec = pool[table.long()].transpose(1, 2)  # [B, heads, pages, blocks, bytes]
    k, v = _values(rec, D)
    k, v = k.reshape(B, hkv, -1, D), v.reshape(B, hkv, -1, D)
    qh = q.float().reshape(B, T, hkv, hq // hkv, D).permute(0, 2, 3, 1, 4).reshape(B, hkv, -1, D)
    s = (qh @ k.transpose(-1, -2)).mul_(1 / math.sqrt(D)).view(B, hkv, hq // hkv, T, -1)
    j = torch.arange(s.shape[-1], device=q.device)
    at = lens.long()[:, None] - T + torch.arange(T, device=q.device)  # a query's position
    if tree is None:
        see = j <= at[..., None]
    else:
        w = j - (lens.long()[:, None, None] - T)  # a key's place in the window
        see = (w < 0) | ((tree.long()[..., None] >> w.clamp(0, 31)) & 1).bool()
    see &= (j < lens[:, None, None]) & (at[..., None] >= 0)
    if window:
        see &= j > at[..., None] - window
    s.masked_fill_(~see[:, None, None], -math.inf)
    m = s.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, 0.0, m)
    p = s.sub_(m).exp_()
    total = p.sum(-1, keepdim=True)
    o = (p.view(B, hkv, -1, p.shape[-1]) @ v).view(B, hkv, hq // hkv, T, D)
    o = torch.where(total > 0, o / total, 0.0)
    lse = (m + total.log())[..., 0]
    return o.permute(0, 3, 1, 2, 4).reshape(B, T, hq, D).to(q.dtype), lse.permute(0, 3, 1, 2).reshape(B, T, hq)


def _plain_norm(x, residual, weight, eps):
    h = x.float() if residual is None else x.float() + residual.float()
    y = h * torch.rsqrt(h.square().mean(-1, keepdim=True) + eps) * weight.float()
    blocks = y.view(x.shape[0], -1, 32)
    d = blocks.abs().amax(-1, keepdim=True) / torch.full((), 127.0, device=x.device)
    r = torch.where(d > 0, blocks / d, 0.0)
    code = torch.sign(r) * torch.floor(r.abs() + 0.5)
    return (None if residual is None else h.to(x.dtype)), y.to(x.dtype), (code * d.half().float()).half().view(x.shape)


def run(state):
    st, c = state, state["case"]
    op = c["op"]
    if own:
        import quantized_routed_expert_grouped_gb300 as m
        if op == "attention":
            out, lse = m.kv8_attention(st["q"], st["pool"], st["table"], st["lens"], window=c["window"], tree=st["tree"], workspace=st["ws"], with_lse=True)
            return {"out": out, "lse": lse}
        if op == "norm":
            total, y, xq = m.add_rms_norm_q8_1(st["x"], st["weight"], residual=st["residual"], eps=st["eps"], with_y=True)
            return {"sum": total, "y": y, "codes": m.dequantize_q8_1(xq, dtype=torch.float16)}
        if op == "write":
            m.kv8_write(st["k"], st["v"], st["pool"], st["table"], st["cu"], st["start"])
            k, v = m.kv8_read(st["pool"], st["table"], st["back_cu"], st["back_start"], st["back_N"], dtype=st["k"].dtype)
        else:
            k, v = m.kv8_read(st["pool"], st["table"], st["cu"], st["start"], st["N"], dtype=TYPES[c["dtype"]])
        return {"k": k, "v": v}
    if op == "attention":
        out, lse = _plain_attention(st["q"], st["pool"], st["table"], st["lens"], c["window"], st["tree"])
        return {"out": out, "lse": lse}
    if op == "norm":
        total, y, codes = _plain_norm(st["x"], st["residual"], st["weight"], st["eps"])
        return {"sum": total, "y": y, "codes": codes}
    if op == "write":
        _plain_write(st["k"], st["v"], st["pool"], st["table"], st["cu"], st["start"])
        k, v = _plain_read(st["pool"], st["table"], st["back_cu"], st["back_start"], st["back_N"], st["k"].dtype)
    else:
        k, v = _plain_read(st["pool"], st["table"], st["cu"], st["start"], st["N"], TYPES[c["dtype"]])
    return {"k": k, "v": v}


# ------------------------------------------------------------------------------------------------ 64 bits

def _tokens64(pool, table, b, p0, p1):
    """Keys and values [heads, p1 - p0, D] of sequence b in 64 bits, byte by byte from the record's definition; and their codes and scales."""
    page, D = pool.shape[2] * 32, (pool.shape[3] - 16) // 64
    p = torch.arange(p0, p1, device=pool.device)
    t, d = p % 32, torch.arange(D, device=pool.device)
    rec = pool[table[b].long()[p // page], :, p % page // 32]  # [tokens, heads, bytes]
    k_at = 16 + ((((t >> 1) & 3)[:, None] * (D // 32) + d // 32) * 8 + (2 * (t >> 3) + (t & 1))[:, None]) * 32 + d % 32
    v_at = 16 + 32 * D + d * 32 + t[:, None]
    scale = rec[..., :8].contiguous().view(torch.float32).double()
    pick = lambda at: rec.gather(2, at[:, None].expand(-1, rec.shape[1], -1)).double() - 128  # noqa: E731
    return pick(k_at), pick(v_at), scale


def _exact_attention(st, c):
    q, lens, tree = st["q"].double(), st["lens"].tolist(), None if st["tree"] is None else st["tree"].tolist()
    B, T, hq, D = q.shape
    hkv = c["hkv"]
    G = hq // hkv
    out, lse = torch.zeros((B, T, hq, D), dtype=torch.float64, device=q.device), torch.full((B, T, hq), -math.inf, dtype=torch.float64, device=q.device)
    for b, n in enumerate(lens):
        lo = max(0, n - T - c["window"]) if c["window"] else 0
        ctx = []
        for a in range(lo, n, 16384):
            kc, vc, sc = _tokens64(st["pool"], st["table"], b, a, min(n, a + 16384))
            k, v = kc * sc[..., :1], vc * sc[..., 1:]
            s = torch.einsum("thgd,nhd->thgn", q[b].view(T, hkv, G, D), k) / math.sqrt(D)
            pos = torch.arange(a, a + k.shape[0], device=q.device)
            for t in range(T):
                at = n - T + t
                if tree is None:
                    see = pos <= at
                else:
                    see = torch.tensor([i < n - T or bool(tree[b][t] >> (i - n + T) & 1) for i in range(a, a + k.shape[0])] if a + k.shape[0] > n - T else [True] * k.shape[0], device=q.device)
                if c["window"]:
                    see = see & (pos > at - c["window"])
                if at < 0:
                    see = see & False
                s[t].masked_fill_(~see, -math.inf)
            m = s.amax(-1)
            p = (s - torch.where(m == -math.inf, 0.0, m)[..., None]).exp()
            ctx.append((m, p.sum(-1), torch.einsum("thgn,nhd->thgd", p, v)))
        if not ctx:
            continue
        top = torch.stack([m for m, _, _ in ctx]).amax(0)
        base = torch.where(top == -math.inf, 0.0, top)
        total = sum(l * (m - base).exp() for m, l, _ in ctx)
        o = sum(a * (m - base).exp()[..., None] for m, _, a in ctx)
        out[b] = torch.where(total[..., None] > 0, o / total[..., None], 0.0).view(T, hq, D)
        lse[b] = (base + total.log()).view(T, hq)
    return {"out": out, "lse": lse}


def exact(case, seed):
    c = case
    st = prepare(case, seed)
    if c["op"] == "attention":
        return _exact_attention(st, c)
    if c["op"] == "norm":
        h = st["x"].double()
        if st["residual"] is not None:
            h = h + st["residual"].double()
        y = h / (h.square().mean(1, keepdim=True) + st["eps"]).sqrt() * st["weight"].double()
        d = y.view(c["rows"], -1, 32).abs().amax(2, keepdim=True) / 127
        q = y.view(c["rows"], -1, 32) / torch.where(d > 0, d, 1.0)
        codes = torch.where(q < 0, -torch.floor(0.5 - q), torch.floor(0.5 + q)) * d.half().double()
        return {"sum": None if st["residual"] is None else h, "y": y, "codes": codes.view(c["rows"], c["cols"])}
    n = (st["cu"][1:] - st["cu"][:-1]).tolist()
    got = {"k": [], "v": []}
    for b, (s, m) in enumerate(zip(st["start"].tolist(), n)):
        if not m:
            continue
        if c["op"] == "read":
            for a in range(s, s + m, 8192):
                kc, vc, sc = _tokens64(st["pool"], st["table"], b, a, min(s + m, a + 8192))
                got["k"].append(kc * sc[..., :1])
                got["v"].append(vc * sc[..., 1:])
            continue
        row = int(st["cu"][b])
        kept = _tokens64(st["pool"], st["table"], b, s - s % 32, s) if s % 32 else None
        for w, name in enumerate("kv"):
            x = st[name][row:row + m].double()
            edge = [0] + [i for i in range(32 - s % 32, m, 32)] + [m]
            if len(edge) < 3:
                edge = [0, m]
            size = torch.tensor([q - p for p, q in zip(edge, edge[1:])], device=x.device)
            of = torch.repeat_interleave(torch.arange(len(size), device=x.device), size)
            amax = torch.stack([x[p:q].abs().amax((0, 2)) for p, q in zip(edge, edge[1:])])
            scale = amax / 127
            if kept is not None:
                old = kept[2][0, :, w]
                scale[0] = torch.maximum(scale[0], old)
                got[name].append(torch.round(kept[w] * (old / scale[0])[:, None]) * scale[0][:, None])
            got[name].append(torch.round(x / scale[of][..., None]) * scale[of][..., None])
    none = torch.zeros((0, c["hkv"], c["D"]), dtype=torch.float64, device=DEV)
    return {x: torch.cat(got[x]) if got[x] else none for x in "kv"}
