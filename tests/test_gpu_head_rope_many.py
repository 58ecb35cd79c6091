"""Norm and rotation of so many tokens that a CTA takes two, three or four of them, the last one fewer, against the formula in 64 bits (as in
test_gpu_head_rope.py), and against the same tokens in small calls, bit for bit."""
import pytest
import torch

import kv8_ref as K
from test_gpu_head_rope import check, ints, rows

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def m():
    import quantized_routed_expert_grouped_gb300 as mod
    mod.lib()
    return mod


CASES = [
    # tokens, query heads, key heads, dims, rotated, start, interleaved, layout
    (1823, 3, 1, 64, 32, 16, False, "dense"),
    (1825, 3, 1, 64, 64, 0, True, "odd"),
    (2735, 2, 2, 48, 16, 8, False, "fused"),
    (2737, 3, 1, 64, 64, 0, False, "dense"),
    (3001, 2, 0, 128, 64, 32, True, "heads"),
    (3646, 9, 2, 32, 32, 0, False, "odd"),
    (3649, 2, 1, 80, 48, 24, True, "fused"),
    (4003, 5, 3, 64, 32, 0, False, "heads"),
    (5003, 1, 1, 256, 16, 240, False, "dense"),
]


@pytest.mark.parametrize("dtype", list(K.TYPES))
@pytest.mark.parametrize("case", range(len(CASES)))
def test_tokens_of_a_block(m, case, dtype):
    N, hq, hk, D, rot, start, inter, layout = CASES[case]
    g = torch.Generator().manual_seed(case)
    q, k = rows(g, N, hq, D, dtype, layout), rows(g, N, hk, D, dtype, "dense") if hk else None
    qw, kw = (1 + 0.3 * torch.randn((2, D), generator=g)).cuda()
    rope = m.Rope(rot, theta=10000.0, start=start, interleaved=inter)
    pos = torch.randint(0, 64, (N,), generator=g).tolist()
    for a, b, r in ((qw, kw, rope), (None, kw, rope), (qw, None, None)):
        b = None if k is None else b
        y, z = m.head_norm_rope(q, ints(pos), r, k=k, q_weight=a, k_weight=b)
        check(y, q, pos, a, r, dtype)
        if k is not None:
            check(z, k, pos, b, r, dtype)
        for first in (0, 1000, N - 300):  # a token a CTA
            some = slice(first, first + 300)
            y1, z1 = m.head_norm_rope(q[some], ints(pos[some]), r, k=None if k is None else k[some], q_weight=a, k_weight=b)
            assert torch.equal(y1, y[some]) and (k is None or torch.equal(z1, z[some]))
