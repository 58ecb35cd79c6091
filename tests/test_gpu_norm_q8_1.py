"""Residual + norm + q8_1 (moe_add_rms_norm_q8_1) against the formula in 64 bits, its q8_1 rows
against the fp32 y that the kernel itself gives, bit for bit, and the reading back of q8_1 rows.

Tolerance of y: the sum of squares adds at most 32 terms per thread, 5 levels of lanes and 32 warps,
so its relative error is below 70 * 2^-24 and the factor's below 35 * 2^-24 + 3 roundings; with the
two products 40 * 2^-24. In 16 bits one rounding more."""
import numpy as np
import pytest
import torch

import kv8_ref as R

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def m():
    import quantized_routed_expert_grouped_gb300 as mod
    mod.lib()
    return mod


def q8_1_of(y):
    """fp32 [rows, cols] -> q8_1 bytes, one fp32 operation a step."""
    b = y.reshape(y.shape[0], -1, 32)
    amax = np.abs(b).max(-1)
    d = (amax / np.float32(127)).astype(np.float32)
    with np.errstate(all="ignore"):
        r = np.where(d[..., None] == 0, np.float32(0), b / d[..., None])
    q = (np.sign(r) * np.floor(np.abs(r).astype(np.float64) + 0.5)).astype(np.int8)
    s = (d * q.astype(np.int32).sum(-1).astype(np.float32)).astype(np.float32)
    out = np.zeros((*b.shape[:2], 36), np.uint8)
    out[..., 0:2] = d.astype(np.float16)[..., None].view(np.uint8)
    out[..., 2:4] = s.astype(np.float16)[..., None].view(np.uint8)
    out[..., 4:] = q.view(np.uint8)
    return out


def make(seed, rows, cols, dtype, wdtype):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((rows, cols), generator=g) * torch.exp(torch.randn((rows, 1), generator=g) * 2)
    r = 3 * torch.randn((rows, cols), generator=g)
    w = 1 + 0.5 * torch.randn((cols,), generator=g)
    return x.to(R.TYPES[dtype]).cuda(), r.to(R.TYPES[dtype]).cuda(), w.to(R.TYPES[wdtype]).cuda()


def expect(x, r, w, eps):
    h = x.double().cpu() + (r.double().cpu() if r is not None else 0)
    return h, h / torch.sqrt((h * h).mean(-1, keepdim=True) + eps) * w.double().cpu()


SHAPES = [(1, 32), (3, 64), (4, 2560), (1, 4096), (5, 1056), (2, 8192), (3, 16416), (2, 32768), (700, 96), (257, 800)]


@pytest.mark.parametrize("dtype", list(R.TYPES))
@pytest.mark.parametrize("shape", SHAPES)
def test_norm(m, shape, dtype):
    rows, cols = shape
    wdtype = dtype if rows % 2 else ["f32", "f16", "bf16"][cols // 32 % 3]
    x, r, w = make(rows * cols, rows, cols, dtype, wdtype)
    for residual in (r, None):
        total, y, xq = m.add_rms_norm_q8_1(x, w, residual=residual, eps=1e-5, with_y=True)
        h, want = expect(x, residual, w, 1e-5)
        if residual is None:
            assert total is None
        else:
            assert torch.equal(total, (x.float() + r.float()).to(x.dtype))
        far = (y.double().cpu() - want).abs() - (40 * 2.0 ** -24 + (0 if dtype == "f32" else R.HALF_ULP[dtype])) * want.abs()
        assert (far <= 2.0 ** -25).all()  # the smallest fp16 subnormals round by that
        if dtype == "f32":
            assert np.array_equal(xq.cpu().numpy(), q8_1_of(y.cpu().numpy()))
            values = m.dequantize_q8_1(xq)
        else:  # y is rounded, the codes are of the unrounded one: half a step and the roundings apart
            values = m.dequantize_q8_1(xq)
            d = want.reshape(rows, -1, 32).abs().amax(-1, keepdim=True) / 127
            near = (values.double().cpu() - want).reshape(rows, -1, 32).abs() - d * (0.5 + 127 * 2.0 ** -11 + 0.01) - 127 * 2.0 ** -25
            assert (near <= 0).all()
        # the same rows from the library's own quantizer of the fp32 y
        x32, r32 = x.float(), None if residual is None else r.float()
        _, y32, xq32 = m.add_rms_norm_q8_1(x32, w, residual=r32, eps=1e-5, with_y=True)
        assert torch.equal(xq32, xq)
        assert torch.equal(m.quantize_q8_1(y32), xq32)


def test_in_place_and_strided(m):
    """The sum over the residual, y over x, rows inside a wider buffer; outputs one at a time."""
    x, r, w = make(5, 9, 416, "bf16", "f32")
    want, y0, xq0 = m.add_rms_norm_q8_1(x, w, residual=r, with_y=True)
    wide = torch.full((9, 2, 416), float("nan"), dtype=x.dtype, device="cuda")
    wide[:, 0], wide[:, 1] = x, r
    total, y, xq = m.add_rms_norm_q8_1(wide[:, 0], w, residual=wide[:, 1], with_y=True)
    assert torch.equal(total, want) and torch.equal(y, y0) and torch.equal(xq, xq0)
    x2, r2 = x.clone(), r.clone()
    total, y, xq = m.add_rms_norm_q8_1(x2, w, residual=r2, sum_out=r2, y=x2)
    assert torch.equal(r2, want) and torch.equal(x2, y0) and torch.equal(xq, xq0)
    total, y, xq = m.add_rms_norm_q8_1(x, w, residual=r)
    assert y is None and torch.equal(xq, xq0)


def test_values(m):
    """A row of zeros, one of the type's largest values, one with a NaN, one with an infinity."""
    x = torch.randn((5, 64), generator=torch.Generator().manual_seed(1)).cuda()
    x[0] = 0
    x[1] *= 1e18
    x[2, 40] = float("nan")
    x[3, 3] = float("inf")
    w = torch.ones(64, device="cuda")
    _, y, xq = m.add_rms_norm_q8_1(x, w, with_y=True)
    v = m.dequantize_q8_1(xq)
    assert (y[0] == 0).all() and (v[0] == 0).all() and y[1].isfinite().all() and y[4].isfinite().all()
    assert y[2].isnan().all() and v[2].isnan().all()
    assert y[3, 3].isnan() and (y[3, :3] == 0).all() and v[3, :32].isnan().all() and (v[3, 32:] == 0).all()
    _, want = expect(x, None, w, 1e-6)
    assert ((y.double().cpu() - want).abs()[[1, 4]] <= 40 * 2.0 ** -24 * want.abs()[[1, 4]]).all()


@pytest.mark.parametrize("dtype", list(R.TYPES))
def test_dequantize(m, dtype):
    y = torch.randn((7, 352), generator=torch.Generator().manual_seed(2)).cuda()
    y[3] = 0
    xq = m.quantize_q8_1(y)
    b = xq.cpu().numpy()
    want = b[..., 0:2].copy().view(np.float16).astype(np.float32) * b[..., 4:].view(np.int8).astype(np.float32)
    got = m.dequantize_q8_1(xq, dtype=R.TYPES[dtype])
    assert torch.equal(got.cpu(), torch.from_numpy(want.reshape(7, 352)).to(R.TYPES[dtype]))


def test_no_rows(m):
    x = torch.empty((0, 64), device="cuda")
    total, y, xq = m.add_rms_norm_q8_1(x, torch.ones(64, device="cuda"), residual=x, with_y=True)
    assert total.shape == (0, 64) and xq.shape == (0, 2, 36) and m.dequantize_q8_1(xq).shape == (0, 64)


# more than 304 rows of 512 columns or more, and rows of 8,224 to 16,384 columns: two pieces a thread
@pytest.mark.parametrize("dtype", list(R.TYPES))
@pytest.mark.parametrize("shape", [(400, 512), (305, 4096), (321, 7200), (3, 8224), (2, 16384), (310, 16352)])
def test_two_pieces_a_thread(m, shape, dtype):
    test_norm(m, shape, dtype)
    rows, cols = shape
    x, r, w = make(rows + cols, rows, cols, dtype, dtype)
    want, y0, xq0 = m.add_rms_norm_q8_1(x, w, residual=r, with_y=True)
    x2, r2 = x.clone(), r.clone()
    _, _, xq = m.add_rms_norm_q8_1(x2, w, residual=r2, sum_out=r2, y=x2)
    assert torch.equal(r2, want) and torch.equal(x2, y0) and torch.equal(xq, xq0)


@pytest.mark.parametrize("dtype", list(R.TYPES))
@pytest.mark.parametrize("rows,cols", [(1217, 4096), (155, 32160), (622593, 32)])
def test_dequantize_many(m, rows, cols, dtype):
    """More than 622,592 pieces of eight values: two a thread, the last CTA's not all there."""
    y = torch.randn((rows, cols), generator=torch.Generator("cuda").manual_seed(3), device="cuda")
    xq = m.quantize_q8_1(y)
    got = m.dequantize_q8_1(xq, dtype=R.TYPES[dtype])
    d = xq[..., 0:2].contiguous().view(torch.float16).float()
    want = (d * xq[..., 4:].view(torch.int8).float()).to(R.TYPES[dtype])
    assert torch.equal(got, want.view(rows, cols))
