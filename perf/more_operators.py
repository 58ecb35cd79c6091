"""Timing cases of the steps around a verify window's attention that a decode loop adds to the cache and the experts.

Three operators, each in a plain form (elementary torch operations in 32 bits, angles in 64) and as the package's own calls:

- ``rope``: a root-mean-square norm of each head's queries and keys and the rotation by position, in one pass;
- ``append``: new keys, normed and rotated on the way, and values quantised into the paged 8-bit cache, the queries of the
  same tokens normed and rotated beside them; the touched positions are read back;
- ``logprobs``: of rows of logits, the log probabilities of given tokens, the most likely tokens with theirs, the entropy
  and the log-sum-exp.

Rotation: dims start .. start + rot of a head form rot / 2 pairs, dims (start + i, start + i + rot / 2), or with ``inter``
(start + 2 i, start + 2 i + 1); pair i turns by position * f_i. f_i = theta^(-2 i / rot), scaled for long contexts:
``linear`` divides all by s; ``yarn`` divides those that turn less than slow times over the original length o, keeps
those that turn more than fast times, takes a line in i between, and multiplies the rotated dims by 0.1 log s + 1;
``bands`` does so by low and high times, with a line in the number of turns, and no factor.

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
EPS = 1e-6


# ------------------------------------------------------------------------------------------------ cases

def _named(name, c):
    return dict(c, name=name) if name else c


def _rope(name, N, T, hq, hkv, D, rot, dtype, start=0, inter=False, wdtype="none", scaling="none", far=4096):
    return _named(name, dict(op="rope", N=N, T=T, hq=hq, hkv=hkv, D=D, rot=rot, start=start, inter=inter, dtype=dtype, wdtype=wdtype, scaling=scaling, far=far))


def _append(name, B, n_lo, n_hi, s_lo, s_hi, hq, hkv, D, page, rot, dtype, start=0, inter=False, wdtype="none", scaling="none", tree=False):
    return _named(name, dict(op="append", B=B, n_lo=n_lo, n_hi=n_hi, s_lo=s_lo, s_hi=s_hi, hq=hq, hkv=hkv, D=D, page=page, rot=rot, start=start, inter=inter,
                             dtype=dtype, wdtype=wdtype, scaling=scaling, tree=tree))


def _logprobs(name, R, V, ids, top, dtype, scale=1.0, masked=0.0, pad=0):
    return _named(name, dict(op="logprobs", R=R, V=V, ids=ids, top=top, dtype=dtype, scale=scale, masked=masked, pad=pad))


def listed():
    return [
        # one user's next token: latency only
        _rope("rope_one_token", 1, 1, 16, 4, 128, 128, "bf16", wdtype="bf16"),
        # a serving batch's windows of 4 in fp32, half of each head rotated in pairs of neighbours, without norms
        _rope("rope_window4_batch64_f32", 256, 4, 32, 8, 128, 64, "f32", inter=True, scaling="linear", far=16001),
        # a prompt of odd-sized heads whose last dims are rotated
        _rope("rope_prompt_part_of_head", 1021, 1021, 12, 12, 80, 32, "f16", start=48, wdtype="f32", scaling="bands", far=9001),
        # a long prompt at far positions, many query heads
        _rope("rope_prompt_far", 8191, 8191, 64, 8, 128, 128, "bf16", wdtype="bf16", scaling="yarn", far=1048579),
        # one user's next token into the cache
        _append("append_one_token", 1, 1, 1, 777, 777, 16, 4, 128, 64, 128, "bf16", wdtype="bf16"),
        # a serving batch's window of 4 appended at odd places (kept tokens may need a wider scale)
        _append("append_window4_batch64", 64, 4, 4, 31, 16001, 32, 8, 128, 64, 128, "bf16", wdtype="bf16"),
        # prefixes in fp32, keys and values only, a third of each head rotated in pairs of neighbours
        _append("append_prefixes_f32", 5, 33, 4001, 0, 17, 0, 4, 96, 32, 32, "f32", inter=True, scaling="linear"),
        # prompts of several users at once, each from its own place: the largest
        _append("append_prompts", 7, 1, 20011, 0, 45, 32, 8, 128, 64, 128, "bf16", wdtype="bf16", scaling="yarn"),
        # one token's choice with its alternatives
        _logprobs("logprobs_one_row", 1, 32768, 1, 20, "f32"),
        # a verify window of 4: each draft's log probability, and what would have been likelier
        _logprobs("logprobs_window4", 4, 131072, 1, 5, "bf16"),
        # a serving batch under a grammar that leaves few tokens, at a temperature, several candidates a row, one row with none
        _logprobs("logprobs_batch_masked", 192, 65537, 3, 20, "f32", scale=1 / 0.7, masked=0.95, pad=3),
        # a prompt's tokens scored, rows at odd addresses
        _logprobs("logprobs_prompt", 2047, 131075, 1, 5, "bf16"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    top = max(work(c)["bytes"] for c in listed())
    while True:
        op, dtype = rng.choice(["rope", "append", "logprobs"]), rng.choice(list(TYPES))
        wdtype = rng.choice(["none", dtype, "f32"])
        scaling, inter = rng.choice(["none", "linear", "yarn", "bands"]), rng.random() < 0.4
        hkv = rng.choice([1, 2, 3, 4, 8, 12])
        if op == "logprobs":
            V = _log(rng, 5, 260000)
            c = _logprobs(None, _log(rng, 1, 8192), V, rng.randint(1, 4), rng.randint(0, min(32, V)), dtype, scale=rng.choice([1.0, 0.5, 1 / 0.7, 3.0]),
                          masked=rng.choice([0.0, 0.0, 0.5, 0.99]), pad=rng.choice([0, 0, 1, 8, 61]))
            fits = c["R"] * (c["V"] + c["pad"]) <= 1 << 28
        elif op == "rope":
            D = 16 * rng.randint(2, 16)
            rot = 16 * rng.randint(1, D // 16)
            N = _log(rng, 1, 20000)
            c = _rope(None, N, _log(rng, 1, N), rng.choice([1, 2, 5, 8, 16, 32, 64]), rng.choice([0, hkv]), D, rot, dtype, start=8 * rng.randint(0, (D - rot) // 8), inter=inter,
                      wdtype=wdtype, scaling=scaling, far=N + _log(rng, 1, 1 << 30))
            fits = N * (c["hq"] + 2 * c["hkv"]) * D <= 1 << 28
        else:
            D = rng.choice([32, 64, 96, 128, 160, 192, 256])
            rot = 16 * rng.randint(1, D // 16)
            n_hi = rng.choice([rng.randint(1, 8), _log(rng, 8, 30000)])
            c = _append(None, _log(rng, 1, 64), rng.randint(0, n_hi), n_hi, 0, _log(rng, 1, 20000), hkv * rng.choice([0, 1, 2, 4, 5, 8]), hkv, D, rng.choice([32, 64, 128]), rot, dtype,
                        start=8 * rng.randint(0, (D - rot) // 8), inter=inter, wdtype=wdtype, scaling=scaling, tree=n_hi <= 8 and rng.random() < 0.5)
            n = _spread(c["B"], c["n_lo"], c["n_hi"])
            fits = sum(n) * (c["hq"] + 2 * hkv) * D <= 1 << 28 and c["B"] * (c["s_hi"] + n_hi) * hkv * D <= 1 << 31
        if fits and work(c)["bytes"] <= top:
            return c


def _spread(n, lo, hi):
    """n whole numbers from lo to hi (over their logarithm), in a fixed order that is not theirs by size."""
    if n == 1:
        return [hi]
    v = [int(round((lo + 1) * ((hi + 1) / (lo + 1)) ** (i / (n - 1)))) - 1 for i in range(n)]
    random.Random(n).shuffle(v)
    return v


def _back(start, n):
    """The whole-block range that a write of n tokens at start touches, up to the write's end."""
    return (start - start % 32, n + start % 32) if n else (start, 0)


def work(case):
    c = case
    e = 4 if c["dtype"] == "f32" else 2
    if c["op"] == "logprobs":
        return {"bytes": c["R"] * (c["V"] * e + 8 * (c["ids"] + c["top"] + 1)), "flops": 6 * c["R"] * c["V"]}
    if c["op"] == "rope":
        m = c["N"] * (c["hq"] + c["hkv"]) * c["D"]
        return {"bytes": 2 * m * e + 4 * c["N"], "flops": 8 * m}
    n, s = _spread(c["B"], c["n_lo"], c["n_hi"]), _spread(c["B"], c["s_lo"], c["s_hi"])
    hd = c["hkv"] * c["D"]
    code = 2 * hd + 16 / 32 * c["hkv"]  # cache bytes of a token, keys and values
    back = sum(_back(a, b)[1] for a, b in zip(s, n))
    # keys and values in, codes out; queries in and out; the touched blocks read back in fp16
    return {"bytes": sum(n) * (2 * hd * e + code + 2 * c["hq"] * c["D"] * e) + back * (code + 4 * hd),
            "flops": sum(n) * (8 * c["hq"] * c["D"] + 14 * hd) + back * 2 * hd}


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


#: the parameters of each scaling, as the package's Rope takes them
SCALING = {
    "none": None,
    "linear": dict(kind="linear", scale=4.0),
    "yarn": dict(kind="yarn", scale=16.0, original=8192, fast=32.0, slow=1.0),
    "bands": dict(kind="bands", scale=8.0, original=8192, low=1.0, high=4.0),
}
THETA = 500000.0


def _frequencies(rot, scaling):
    """f_i in 64 bits and the factor of the rotated dims."""
    f, p = THETA ** (-np.arange(0, rot, 2, dtype=np.float64) / rot), SCALING[scaling]
    if p is None:
        return f, 1.0
    if p["kind"] == "linear":
        return f / p["scale"], 1.0
    turns = p["original"] * f / (2 * np.pi)  # over the original length
    if p["kind"] == "bands":
        keep = np.clip((turns - p["low"]) / (p["high"] - p["low"]), 0, 1)
        return f * keep + f / p["scale"] * (1 - keep), 1.0
    # the pairs between which the line runs: those that turn fast and slow times, outward to whole ones
    at = [rot * math.log(p["original"] / (2 * math.pi * r)) / (2 * math.log(THETA)) for r in (p["fast"], p["slow"])]
    lo, hi, i = max(math.floor(at[0]), 0), math.ceil(at[1]), np.arange(rot // 2)
    divided = np.clip((i - lo) / (hi - lo), 0, 1) if hi > lo else (i > lo) * 1.0
    return f * (1 - divided) + f / p["scale"] * divided, 0.1 * math.log(p["scale"]) + 1


def _rows(N, heads, D, g, dt):
    """Rows of a projection: heads of different sizes, a few strong dims."""
    x = torch.randn((N, heads, D), generator=g, device=DEV)
    x *= torch.exp(0.5 * torch.randn((1, heads, 1), generator=g, device=DEV)) * (1 + 3 * (torch.rand((1, heads, D), generator=g, device=DEV) < 0.05))
    return x.to(dt)


def prepare(case, seed):
    c, rng = case, random.Random(seed)
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    dt = TYPES[c["dtype"]]
    st = {"case": dict(c)}
    if c["op"] == "logprobs":
        R, V = c["R"], c["V"]
        x = torch.randn((R, V + c["pad"]), generator=g, device=DEV) * 2.5
        # a few likely tokens a row, more or less likely
        peaks = torch.randint(0, V, (R, 8), generator=g, device=DEV)
        x.scatter_add_(1, peaks, 10 * torch.rand((R, 8), generator=g, device=DEV) * torch.rand((R, 1), generator=g, device=DEV))
        if c["masked"]:
            for a in range(0, R, 256):
                x[a:a + 256].masked_fill_(torch.rand(x[a:a + 256].shape, generator=g, device=DEV) < c["masked"], -math.inf)
            if R > 2:
                x[R // 3] = -math.inf
        st["logits"] = x.to(dt)[:, :V]
        ids = torch.randint(0, V, (R, c["ids"]), generator=g, device=DEV)
        ids = torch.where(torch.rand(ids.shape, generator=g, device=DEV) < 0.5, peaks[:, :1], ids)
        # no token there: the draft was shorter
        st["ids"] = torch.where(torch.rand(ids.shape, generator=g, device=DEV) < 0.05, -1, ids).to(torch.int32)
        return st
    hq, hkv, D, rot = c["hq"], c["hkv"], c["D"], c["rot"]
    if c["wdtype"] == "none":
        st["q_weight"] = st["k_weight"] = None
    else:
        st["q_weight"], st["k_weight"] = (1 + 0.3 * torch.randn((2, D), generator=g, device=DEV)).to(TYPES[c["wdtype"]])
    f, st["factor"] = _frequencies(rot, c["scaling"])
    st["freq"] = torch.from_numpy(f).to(DEV)
    if own:  # a serving program keeps the rotation's frequencies
        import quantized_routed_expert_grouped_gb300 as m
        st["rope"] = m.Rope(rot, theta=THETA, start=c["start"], interleaved=c["inter"], scaling=SCALING[c["scaling"]], device=DEV)
    if c["op"] == "rope":
        # windows of T tokens at places of their own, the last one's last token the farthest
        N, T = c["N"], c["T"]
        first = [rng.randint(0, max(0, c["far"] - T)) for _ in range(-(-N // T) - 1)] + [max(0, c["far"] - T)]
        st["positions"] = (_ints(first)[:, None] + torch.arange(T, dtype=torch.int32, device=DEV)).view(-1)[-N:].contiguous()
        qkv = _rows(N, hq + 2 * hkv, D, g, dt)
        st["q"], st["k"] = qkv[:, :hq], qkv[:, hq:hq + hkv] if hkv else None
        return st
    B = c["B"]
    n, s = _spread(B, c["n_lo"], c["n_hi"]), _spread(B, c["s_lo"], c["s_hi"])
    st["pool"], st["table"] = _cache(c, [a + b for a, b in zip(s, n)], g, rng)
    cu = lambda v: _ints(np.concatenate([[0], np.cumsum(v)]).astype(int).tolist())  # noqa: E731
    st["cu"], st["start"], st["N"] = cu(n), _ints(s), sum(n)
    st["positions"] = None
    if c["tree"]:  # a draft token turns by its depth in the tree, not by its place in the cache
        st["positions"] = _ints([a + d for a, m in zip(s, n) for d in sorted(rng.randint(0, i) for i in range(m))])
    qkv = _rows(st["N"], hq + 2 * hkv, D, g, dt)
    st["q"], st["k"], st["v"] = qkv[:, :hq] if hq else None, qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
    back = [_back(a, b) for a, b in zip(s, n)]
    st["back_start"], st["back_cu"], st["back_N"] = _ints([a for a, _ in back]), cu([b for _, b in back]), sum(b for _, b in back)
    return st


# ------------------------------------------------------------------------------------------------ plain forms

def _plain_rope(x, positions, weight, freq, factor, start, inter):
    """Norm (where there is a weight) and rotation, in fp32; angles in 64 bits."""
    x = x.float()
    if weight is not None:
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * weight.float()
    a = positions.double()[:, None] * freq
    cos, sin = (a.cos() * factor).float()[:, None], (a.sin() * factor).float()[:, None]
    h = freq.shape[0]
    lo, part, hi = x[..., :start], x[..., start:start + 2 * h], x[..., start + 2 * h:]
    if inter:
        u, w = part[..., 0::2], part[..., 1::2]
        part = torch.stack([u * cos - w * sin, u * sin + w * cos], -1).flatten(-2)
    else:
        u, w = part[..., :h], part[..., h:]
        part = torch.cat([u * cos - w * sin, u * sin + w * cos], -1)
    return torch.cat([lo, part, hi], -1)


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
    """Ragged rows -> 32-token blocks: sequence b's blocks are slots first[b], first[b] + 1, ...; and each row's position."""
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
    return torch.where(used, pg, 0), blk * 32 % page // 32, (start[b] - blk * 32).clamp(0, 32), first[bi] + p // 32 - start[bi] // 32, p % 32, p


def _plain_read(pool, table, cu, start, N, dtype):
    D = (pool.shape[-1] - 16) // 64
    pg, nb, _, slot, t, _ = _slots(cu, start, N, table, pool.shape[2] * 32)
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


def _plain_append(st, c):
    pool, table, k, v = st["pool"], st["table"], st["k"], st["v"]
    pg, nb, keep, slot, t, place = _slots(st["cu"], st["start"], st["N"], table, c["page"])
    turn = place if st["positions"] is None else st["positions"]
    k = _plain_rope(k, turn, st["k_weight"], st["freq"], st["factor"], c["start"], c["inter"])
    rec = pool[pg, :, nb]
    scale = rec[..., :8].contiguous().view(torch.float32)
    unit = rec.clone()
    unit[..., :8] = torch.ones(2, device=k.device).view(torch.uint8)
    kc, vc = _values(unit, c["D"])
    kc, ks = _plain_quantise(k, scale[..., 0], kc, slot, t, keep)
    vc, vs = _plain_quantise(v, scale[..., 1], vc, slot, t, keep)
    pool[pg, :, nb] = _records(kc, vc, ks, vs)
    if st["q"] is None:
        return None
    return _plain_rope(st["q"], turn, st["q_weight"], st["freq"], st["factor"], c["start"], c["inter"]).to(st["q"].dtype)


def _plain_logprobs(logits, ids, top, scale):
    x = logits.float()
    V = x.shape[1]
    best = None
    if top:
        # one whole number orders by value (an order of the bits, -0 as 0), then by the lowest index
        bits = (x + 0.0).view(torch.int32).long()
        key = torch.where(bits < 0, -2147483648 - bits - 1, bits) * 4294967296 + (4294967295 - torch.arange(V, device=x.device))
        best = 4294967295 - (key.topk(top, -1)[0] & 4294967295)
        del bits, key
    m = x.amax(-1, keepdim=True)
    t = (x - torch.where(m == -math.inf, 0.0, m)) * scale
    e = t.exp()
    s = e.sum(-1, keepdim=True)
    u = (e * t.clamp(min=-1e30)).sum(-1, keepdim=True)
    some = s > 0
    entropy = torch.where(some, s.log() - u / s, 0.0)
    at = lambda i: torch.where(some, t.gather(1, i.clamp(0, V - 1)) - s.log(), -math.inf)  # noqa: E731
    i = ids.long()
    return {"logprobs": torch.where((i >= 0) & (i < V), at(i), -math.inf), "top": at(best) if top else None, "top_ids": best.int() if top else None,
            "entropy": entropy[:, 0], "lse": torch.where(some, m * scale + s.log(), -math.inf)[:, 0]}


def run(state):
    st, c = state, state["case"]
    op = c["op"]
    if own:
        import quantized_routed_expert_grouped_gb300 as m
        if op == "logprobs":
            logprobs, top, top_ids, entropy, lse = m.token_logprobs(st["logits"], st["ids"], top=c["top"], scale=c["scale"])
            return {"logprobs": logprobs, "top": top, "top_ids": top_ids, "entropy": entropy, "lse": lse}
        if op == "rope":
            q, k = m.head_norm_rope(st["q"], st["positions"], st["rope"], k=st["k"], q_weight=st["q_weight"], k_weight=st["k_weight"], eps=EPS)
            return {"q": q, "k": k}
        q = m.kv8_append(st["k"], st["v"], st["pool"], st["table"], st["cu"], st["start"], st["rope"], q=st["q"], q_weight=st["q_weight"], k_weight=st["k_weight"],
                         eps=EPS, positions=st["positions"])
        k, v = m.kv8_read(st["pool"], st["table"], st["back_cu"], st["back_start"], st["back_N"], dtype=torch.float16)
        return {"q": q, "k": k, "v": v}
    if op == "logprobs":
        return _plain_logprobs(st["logits"], st["ids"], c["top"], c["scale"])
    if op == "rope":
        rot = lambda x, w: _plain_rope(x, st["positions"], w, st["freq"], st["factor"], c["start"], c["inter"]).to(x.dtype)  # noqa: E731
        return {"q": rot(st["q"], st["q_weight"]), "k": None if st["k"] is None else rot(st["k"], st["k_weight"])}
    q = _plain_append(st, c)
    k, v = _plain_read(st["pool"], st["table"], st["back_cu"], st["back_start"], st["back_N"], torch.float16)
    return {"q": q, "k": k, "v": v}


# ------------------------------------------------------------------------------------------------ 64 bits

def _turned64(x, places, weight, c):
    """Norm and rotation in 64 bits, pairs as complex numbers; places: each row's position."""
    x = x.double()
    if weight is not None:
        x = x / (x.pow(2).sum(-1, keepdim=True) / c["D"] + EPS).sqrt() * weight.double()
    f, factor = _frequencies(c["rot"], c["scaling"])
    angle = torch.outer(places.double(), torch.tensor(f, dtype=torch.float64, device=x.device))
    first = torch.arange(c["rot"] // 2, device=x.device)
    first, second = (2 * first, 2 * first + 1) if c["inter"] else (first, first + c["rot"] // 2)
    z = torch.complex(x[..., c["start"] + first], x[..., c["start"] + second]) * (torch.exp(1j * angle) * factor)[:, None]
    y = x.clone()
    y[..., c["start"] + first], y[..., c["start"] + second] = z.real, z.imag
    return y


def _tokens64(pool, table, b, p0, p1):
    """Codes of keys and values [p1 - p0, heads, D] of sequence b, less 128, byte by byte from the record's definition; and their scales."""
    page, D = pool.shape[2] * 32, (pool.shape[3] - 16) // 64
    p = torch.arange(p0, p1, device=pool.device)
    t, d = p % 32, torch.arange(D, device=pool.device)
    rec = pool[table[b].long()[p // page], :, p % page // 32]  # [tokens, heads, bytes]
    k_at = 16 + ((((t >> 1) & 3)[:, None] * (D // 32) + d // 32) * 8 + (2 * (t >> 3) + (t & 1))[:, None]) * 32 + d % 32
    v_at = 16 + 32 * D + d * 32 + t[:, None]
    scale = rec[..., :8].contiguous().view(torch.float32).double()
    pick = lambda at: rec.gather(2, at[:, None].expand(-1, rec.shape[1], -1)).double() - 128  # noqa: E731
    return pick(k_at), pick(v_at), scale


def _exact_append(st, c):
    got = {"q": [], "k": [], "v": []}
    n = (st["cu"][1:] - st["cu"][:-1]).tolist()
    for b, (s, m) in enumerate(zip(st["start"].tolist(), n)):
        if not m:
            continue
        row = int(st["cu"][b])
        place = torch.arange(s, s + m, device=DEV) if st["positions"] is None else st["positions"][row:row + m]
        if c["hq"]:
            got["q"].append(_turned64(st["q"][row:row + m], place, st["q_weight"], c))
        kept = _tokens64(st["pool"], st["table"], b, s - s % 32, s) if s % 32 else None
        for w, name in enumerate("kv"):
            x = _turned64(st["k"][row:row + m], place, st["k_weight"], c) if name == "k" else st["v"][row:row + m].double()
            edge = [0] + [i for i in range(32 - s % 32, m, 32)] + [m]
            size = torch.tensor([q - p for p, q in zip(edge, edge[1:])], device=x.device)
            of = torch.repeat_interleave(torch.arange(len(size), device=x.device), size)
            amax = torch.stack([x[p:q].abs().amax((0, 2)) for p, q in zip(edge, edge[1:])])
            scale = amax / 127
            if kept is not None:
                old = kept[2][0, :, w]
                scale[0] = torch.maximum(scale[0], old)
                got[name].append(torch.round(kept[w] * (old / scale[0])[:, None]) * scale[0][:, None])
            got[name].append(torch.round(x / scale[of][..., None]) * scale[of][..., None])
    none = lambda h: torch.zeros((0, h, c["D"]), dtype=torch.float64, device=DEV)  # noqa: E731
    return {x: None if not h else torch.cat(v) if v else none(h) for (x, v), h in zip(got.items(), (c["hq"], c["hkv"], c["hkv"]))}


def _exact_logprobs(st, c):
    got = {"logprobs": [], "top": [], "entropy": [], "lse": []}
    for a in range(0, c["R"], 256):
        x = st["logits"][a:a + 256].double() * c["scale"]
        ids = st["ids"][a:a + 256].long()
        lse = torch.logsumexp(x, -1)
        lp = torch.where(lse[:, None] > -math.inf, x - lse[:, None], -math.inf)
        p = lp.exp()
        got["lse"].append(lse)
        got["entropy"].append(-torch.where(p > 0, p * lp, 0.0).sum(-1))
        lp1 = torch.cat([lp, torch.full_like(lp[:, :1], -math.inf)], 1)
        got["logprobs"].append(lp1.gather(1, torch.where(ids < 0, c["V"], ids)))
        if c["top"]:
            got["top"].append(lp.topk(c["top"], -1)[0])
    out = {k: torch.cat(v) if v else None for k, v in got.items()}
    out["top_ids"] = None
    return out


def exact(case, seed):
    c = case
    st = prepare(case, seed)
    if c["op"] == "append":
        return _exact_append(st, c)
    if c["op"] == "logprobs":
        return _exact_logprobs(st, c)
    return {"q": _turned64(st["q"], st["positions"], st["q_weight"], c), "k": None if st["k"] is None else _turned64(st["k"], st["positions"], st["k_weight"], c)}
