"""Microscaled FP4 (E2M1, one E8M0 scale per 32 channels) quantise-on-write, bit by bit against exact
rationals on the CPU's own rounding, its row maps, and the refusals.
"""
from fractions import Fraction

import numpy as np
import pytest
import torch

import compressed_sparse_attention_quantize_b200 as csa2
from compressed_sparse_attention_quantize_b200 import build as csa2_build
from tests._exact import e2m1_encode

INVALID, SHAPE = 1, 2


def mx_quantise(x):
    """Codes [rows, dim / 2] and scale bytes [rows, dim / 32] of fp32 rows, in exact rationals."""
    rows, dim = x.shape
    codes = np.zeros((rows, dim), np.uint8)
    scales = np.zeros((rows, dim // 32), np.uint8)
    for r in range(rows):
        for b in range(dim // 32):
            v = x[r, 32 * b:32 * b + 32]
            if not np.isfinite(v).all():
                scales[r, b] = 255
                continue
            top = max(abs(Fraction(float(a))) for a in v)
            e = -127
            if top:
                e = top.numerator.bit_length() - top.denominator.bit_length()
                e += 1 if Fraction(2) ** (e + 1) <= top else 0
                e -= 1 if Fraction(2) ** e > top else 0
                e = max(e - 2, -127)
            scales[r, b] = e + 127
            for k in range(32):
                codes[r, 32 * b + k] = e2m1_encode(Fraction(float(v[k])) / Fraction(2) ** e, bool(np.signbit(v[k])))
    return codes[:, 0::2] | (codes[:, 1::2] << 4), scales


def hard_rows(rng, rows, dim):
    """Random rows; blocks at and next to every midpoint, of extreme sizes, of zeros."""
    x = (rng.standard_normal((rows, dim)) * np.exp2(rng.integers(-30, 30, (rows, 1)))).astype(np.float32)
    mids = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, 7.0, 7.99], np.float32)
    x[0, :32] = 0.0
    x[0, 1] = -0.0
    for i, e in enumerate((0, -100, -140, 120)):
        r = 1 + i
        if r >= rows:
            break
        v = (rng.choice(mids, dim) * rng.choice([-1, 1], dim)).astype(np.float32)
        v = np.where(rng.random(dim) < 0.3, np.nextafter(v, np.float32(9)), v)
        v[::32] = 4.0
        x[r] = np.ldexp(v, e).astype(np.float32)
    if rows > 6:
        x[5] = np.float32(1e-45) * rng.integers(-3, 4, dim)          # subnormals
        x[6] = np.float32(3.4e38)
    return x


@pytest.mark.gpu
@pytest.mark.parametrize("rows,dim,dtype,pad", [(1, 32, "f32", 0), (9, 64, "f32", 0), (33, 512, "bf16", 0),
                                                (8, 96, "f32", 1), (7, 160, "bf16", 3), (300, 32, "bf16", 0)])
def test_mx_bit_exact(rows, dim, dtype, pad):
    rng = np.random.default_rng(rows + dim)
    x = hard_rows(rng, rows, dim)
    xt = torch.from_numpy(x)
    if dtype == "bf16":
        xt = xt.bfloat16()
        x = xt.float().numpy()
    wide = torch.zeros(rows, dim + pad, dtype=xt.dtype, device="cuda")
    wide[:, pad:] = xt.cuda()
    rc, rs = mx_quantise(x)
    dt = csa2.DTYPE_F32 if dtype == "f32" else csa2.DTYPE_BF16
    cs, ss = dim // 2 + (1 if pad else 0), dim // 32 + 2
    dst = torch.from_numpy(rng.permutation(rows + 5)[:rows].astype(np.int64))
    dst[rows // 2] = -1                                               # an unused place of a row map
    d = dst.numpy()
    for batch in (False, True):
        codes = torch.full((rows + 5, cs), 0xAB, dtype=torch.uint8, device="cuda")
        scales = torch.full((rows + 5, ss), 0xAB, dtype=torch.uint8, device="cuda")
        args = (csa2.FMT_MXFP4, wide[:, pad:], dt, rows, dim, dim + pad, codes, cs, scales, ss, dst.cuda())
        if batch:
            csa2.csa2_quantize_kv_batch([csa2.quant_job(*args)])
        else:
            csa2.csa2_quantize_kv(*args)
        ec = np.full((rows + 5, cs), 0xAB, np.uint8)
        es = np.full((rows + 5, ss), 0xAB, np.uint8)
        ec[d[d >= 0], :dim // 2] = rc[d >= 0]
        es[d[d >= 0], :dim // 32] = rs[d >= 0]
        assert np.array_equal(scales.cpu().numpy(), es)
        assert np.array_equal(codes.cpu().numpy(), ec)


@pytest.mark.gpu
def test_mx_non_finite_blocks():
    x = torch.randn(4, 96)
    x[0, 5], x[1, 40], x[2, 95] = float("nan"), float("inf"), -float("inf")
    rc, rs = mx_quantise(x.numpy())
    codes = torch.zeros(4, 48, dtype=torch.uint8, device="cuda")
    scales = torch.zeros(4, 3, dtype=torch.uint8, device="cuda")
    csa2.csa2_quantize_kv(csa2.FMT_MXFP4, x.cuda(), csa2.DTYPE_F32, 4, 96, 96, codes, 48, scales, 3)
    assert np.array_equal(codes.cpu().numpy(), rc) and np.array_equal(scales.cpu().numpy(), rs)
    assert (rs == 255).sum() == 3


@pytest.mark.gpu
@pytest.mark.parametrize("fmt,dim", [(csa2.FMT_FP4, 48), (csa2.FMT_FP8_TOKEN, 64), (csa2.FMT_FP8_TOKEN, 4096)])
@pytest.mark.parametrize("batch", [False, True])
def test_negative_destinations_are_skipped(fmt, dim, batch):
    """The other formats' rows: the same bytes where the destination is a row, none where it is negative."""
    x = torch.randn(6, dim, device="cuda")
    cs, ss = (dim // 2, dim // 16) if fmt == csa2.FMT_FP4 else (dim, 4)
    whole = [torch.zeros(6, cs, dtype=torch.uint8, device="cuda"), torch.zeros(6, ss, dtype=torch.uint8, device="cuda")]
    part = [torch.full_like(t, 0x5A) for t in whole]
    csa2.csa2_quantize_kv(fmt, x, 0, 6, dim, dim, whole[0], cs, whole[1], ss)
    dst = torch.tensor([3, -1, 0, -(1 << 40), 5, 1], device="cuda")
    args = (fmt, x, 0, 6, dim, dim, part[0], cs, part[1], ss, dst)
    if batch:
        csa2.csa2_quantize_kv_batch([csa2.quant_job(*args)])
    else:
        csa2.csa2_quantize_kv(*args)
    for w, p in zip(whole, part):
        assert torch.equal(p[[3, 0, 5, 1]], w[[0, 2, 4, 5]])
        assert (p[[2, 4]] == 0x5A).all()


@pytest.mark.gpu
def test_compress_skips_negative_destinations():
    x = torch.randn(12, 64, device="cuda")
    whole = [torch.zeros(3, 32, dtype=torch.uint8, device="cuda"), torch.zeros(3, 4, dtype=torch.uint8, device="cuda")]
    part = [torch.full_like(t, 0x5A) for t in whole]
    csa2.csa2_compress_quantize_kv(x, 0, 3, 4, 64, 64, None, 0, whole[0], 32, whole[1], 4)
    csa2.csa2_compress_quantize_kv(x, 0, 3, 4, 64, 64, None, 0, part[0], 32, part[1], 4,
                                   torch.tensor([2, -1, 0], device="cuda"))
    for w, p in zip(whole, part):
        assert torch.equal(p[[2, 0]], w[[0, 2]]) and (p[1] == 0x5A).all()


def test_mx_refusals():
    csa2_build.build()
    q = csa2.lib().csa2_quantize_kv
    assert q(2, 16, 0, 4, 48, 48, 16, 24, 16, 2, None, None) == SHAPE          # dim % 32
    assert q(2, 16, 0, 4, 64, 64, 16, 31, 16, 2, None, None) == SHAPE          # code stride
    assert q(2, 16, 0, 4, 64, 64, 16, 32, 16, 1, None, None) == SHAPE          # scale stride
    assert q(2, None, 0, 4, 64, 64, 16, 32, 16, 2, None, None) == INVALID
    assert q(3, 16, 0, 4, 64, 64, 16, 32, 16, 2, None, None) == INVALID        # unknown format
