"""csa2_fp4_matmul against 64-bit products of the dequantised values (GPU), and its refusals (CPU).

Tolerance, per output: the products of two E2M1 values and two block scales are exact; what rounds is
the fp32 accumulation.  Each 16-channel block sum enters a running sum (of a K slice, then of the
slices), and each such step loses at most 2^-23 of the magnitudes added so far (a truncation, twice a
rounding's half step), so |error| <= (K / 16 + 8 slices + 2) * 2^-23 * sum |a| |b|; bf16 output adds
half a step, 2^-8 relative.
"""
import ctypes

import numpy as np
import pytest
import torch

import compressed_sparse_attention_quantize_b200 as csa2
from compressed_sparse_attention_quantize_b200 import build as csa2_build

OK, INVALID, SHAPE, ALIGN, WS = 0, 1, 2, 3, 7
GRID = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, -0., -.5, -1, -1.5, -2, -3, -4, -6], dtype=torch.float64)


def block_of(fmt):
    return 16 if fmt == csa2.FMT_FP4 else 32


def values(codes, scales, fmt):
    """float64 values of code rows (uint8 [rows, K / 2]) and scale bytes."""
    c = torch.stack((codes & 15, codes >> 4), dim=2).reshape(codes.shape[0], -1).long()
    if fmt == csa2.FMT_FP4:
        s = scales.view(torch.float8_e4m3fn).double()
    else:
        s = torch.pow(torch.tensor(2.0, dtype=torch.float64), scales.double() - 127)
        s[scales == 255] = float("nan")
    v = GRID.to(codes.device)[c].reshape(codes.shape[0], -1, block_of(fmt)) * s[:, :, None]
    return v.reshape(codes.shape[0], -1)


def operand(g, rows, K, fmt, code_pad=0, scale_pad=0, wild=False):
    """Random code rows and scales in wider buffers; every code occurs, scales spread over octaves."""
    codes = torch.randint(0, 256, (rows, -(-(K // 2) // 16) * 16 + code_pad), generator=g, dtype=torch.uint8)
    nb = K // block_of(fmt)
    if fmt == csa2.FMT_FP4:
        lo, hi = (0, 127) if wild else (40, 72)
    else:
        lo, hi = (90, 165) if wild else (122, 133)
    scales = torch.randint(lo, hi, (rows, nb + scale_pad), generator=g, dtype=torch.uint8)
    return codes.cuda(), scales.cuda()


def check(M, N, K, fmt, out_dtype, seed=0, code_pad=0, scale_pad=0, out_pad=0, shift=0, alpha=1.0, wild=False):
    g = torch.Generator().manual_seed(1000 * seed + M + 7 * N + 13 * K)
    a, sa = operand(g, M, K, fmt, code_pad, scale_pad, wild)
    b, sb = operand(g, N, K, fmt, code_pad, scale_pad, wild)
    nb = K // block_of(fmt)
    td = torch.float32 if out_dtype == csa2.DTYPE_F32 else torch.bfloat16
    raw = torch.full((M * (N + out_pad) + shift + 64,), -777.0, dtype=td, device="cuda")
    size = csa2.csa2_fp4_matmul_workspace_size(M, N, K)
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")
    csa2.csa2_fp4_matmul(fmt, a, a.stride(0), sa, sa.stride(0), b, b.stride(0), sb, sb.stride(0), M, N, K, alpha,
                         raw[shift:], out_dtype, N + out_pad, ws, size)
    assert csa2.csa2_device_error() == 0
    rows = raw[shift:shift + M * (N + out_pad)].reshape(M, N + out_pad)
    got = rows[:, :N].double()
    assert (rows[:, N:] == -777).all() and (raw[:shift] == -777).all() and (raw[shift + rows.numel():] == -777).all()
    va, vb = values(a[:, :K // 2], sa[:, :nb], fmt), values(b[:, :K // 2], sb[:, :nb], fmt)
    ref = alpha * (va @ vb.t())
    tol = (K / 16 + 10) * 2.0 ** -23 * abs(alpha) * (va.abs() @ vb.abs().t())
    if td == torch.bfloat16:
        tol = tol * (1 + 2.0 ** -8) + 2.0 ** -8 * ref.abs()
    worst = ((got - ref).abs() / tol.clamp(min=1e-300)).max().item()
    assert worst <= 1, f"error is {worst:.3g} of what the accumulation allows"
    return raw


SIZES = [(1, 1, 32), (1, 16, 64), (2, 3, 96), (1, 4096, 2048), (3, 130, 256), (16, 17, 288), (17, 1000, 1504),
         (33, 520, 8192), (65, 129, 544), (64, 4000, 1024), (128, 256, 256), (129, 300, 512), (256, 512, 800),
         (333, 1000, 1504), (1000, 1000, 96), (2100, 1300, 512), (700, 5000, 2048)]


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", [csa2.FMT_FP4, csa2.FMT_MXFP4])
@pytest.mark.parametrize("M,N,K", SIZES)
def test_matmul(M, N, K, fmt):
    check(M, N, K, fmt, csa2.DTYPE_F32)
    check(M, N, K, fmt, csa2.DTYPE_BF16, seed=1, alpha=0.375)


@pytest.mark.gpu
@pytest.mark.parametrize("M,N,K", [(1, 40, 16), (5, 200, 48), (200, 333, 528)])
def test_matmul_sixteen_channel_tails(M, N, K):
    """K a multiple of 16 and not of 32: the codes' rows end inside a 16-byte piece."""
    check(M, N, K, csa2.FMT_FP4, csa2.DTYPE_F32)


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", [csa2.FMT_FP4, csa2.FMT_MXFP4])
@pytest.mark.parametrize("M,N,K", [(9, 150, 608), (300, 260, 1120)])
@pytest.mark.parametrize("code_pad,scale_pad,out_pad,shift", [(16, 0, 0, 0), (0, 3, 5, 1), (32, 1, 8, 8), (0, 16, 3, 0)])
def test_matmul_strides(M, N, K, fmt, code_pad, scale_pad, out_pad, shift):
    """Padded rows, scale rows off every alignment, an output off 16 bytes; nothing else is written."""
    for dt in (csa2.DTYPE_F32, csa2.DTYPE_BF16):
        check(M, N, K, fmt, dt, code_pad=code_pad, scale_pad=scale_pad, out_pad=out_pad, shift=shift)


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", [csa2.FMT_FP4, csa2.FMT_MXFP4])
@pytest.mark.parametrize("M,N,K,code_pad,scale_pad,out_pad,shift", [
    (1025, 3330, 2080, 0, 0, 0, 0), (1400, 2561, 4096, 16, 0, 7, 8), (3330, 1100, 2048, 0, 5, 0, 3), (2304, 2048, 1600, 0, 16, 2, 0)])
def test_matmul_large(M, N, K, code_pad, scale_pad, out_pad, shift, fmt):
    """Sizes that fill the GPU with 256 x 256 tiles, ragged in every direction."""
    for dt in (csa2.DTYPE_F32, csa2.DTYPE_BF16):
        check(M, N, K, fmt, dt, code_pad=code_pad, scale_pad=scale_pad, out_pad=out_pad, shift=shift, wild=True)


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", [csa2.FMT_FP4, csa2.FMT_MXFP4])
def test_matmul_every_scale(fmt):
    """Scales over their whole range, zero and subnormal ones among them."""
    check(40, 300, 1024, fmt, csa2.DTYPE_F32, wild=True)


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", [csa2.FMT_FP4, csa2.FMT_MXFP4])
@pytest.mark.parametrize("M,N,K", [(4, 200, 288), (300, 200, 288), (1200, 3100, 2080)])
def test_matmul_nan_scale(fmt, M, N, K):
    """A NaN scale spoils its row (column) and nothing else, past the ragged ends included."""
    g = torch.Generator().manual_seed(3)
    a, sa = operand(g, M, K, fmt)
    b, sb = operand(g, N, K, fmt)
    nan = 0x7F if fmt == csa2.FMT_FP4 else 0xFF
    sa[1, sa.shape[1] - 1] = nan
    sb[150, 0] = nan
    out = torch.zeros(M, N, device="cuda")
    ws = torch.empty(256, dtype=torch.uint8, device="cuda")
    csa2.csa2_fp4_matmul(fmt, a, a.stride(0), sa, sa.stride(0), b, b.stride(0), sb, sb.stride(0), M, N, K, 1.0, out, 0, N,
                         ws, 256)
    want = torch.zeros(M, N, dtype=torch.bool, device="cuda")
    want[1], want[:, 150] = True, True
    assert torch.equal(out.isnan(), want)


@pytest.mark.gpu
def test_matmul_reads_cache_rows():
    """Entries of a packed 288-byte cache as one operand (stride 288, scales at byte 256)."""
    kv = torch.randint(0, 256, (500, 288), dtype=torch.uint8).cuda()
    kv[:, 256:] = torch.randint(40, 72, (500, 32), dtype=torch.uint8).cuda()
    g = torch.Generator().manual_seed(1)
    a, sa = operand(g, 70, 512, csa2.FMT_FP4)
    out = torch.empty(70, 500, device="cuda")
    ws = torch.empty(256, dtype=torch.uint8, device="cuda")
    csa2.csa2_fp4_matmul(csa2.FMT_FP4, a, 256, sa, 32, kv, 288, kv[:, 256:], 288, 70, 500, 512, 1.0, out, 0, 500, ws, 256)
    va, vb = values(a, sa, csa2.FMT_FP4), values(kv[:, :256], kv[:, 256:].contiguous(), csa2.FMT_FP4)
    tol = (512 / 16 + 10) * 2.0 ** -23 * (va.abs() @ vb.abs().t())
    assert ((out.double() - va @ vb.t()).abs() <= tol).all()


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", [csa2.FMT_FP4, csa2.FMT_MXFP4])
def test_linear_in_a_graph_on_a_side_stream(fmt):
    """quantise -> product, captured on another stream and replayed on new inputs, twice the same."""
    M, N, K = 37, 700, 1024
    blk = block_of(fmt)
    x = torch.randn(M, K, device="cuda", dtype=torch.bfloat16)
    g = torch.Generator().manual_seed(2)
    w, sw = operand(g, N, K, fmt)
    xc = torch.empty(M, K // 2, dtype=torch.uint8, device="cuda")
    xs = torch.empty(M, K // blk, dtype=torch.uint8, device="cuda")
    out = torch.empty(M, N, device="cuda")
    ws = torch.empty(256, dtype=torch.uint8, device="cuda")

    def step():
        csa2.csa2_quantize_kv(fmt, x, csa2.DTYPE_BF16, M, K, K, xc, K // 2, xs, K // blk)
        csa2.csa2_fp4_matmul(fmt, xc, K // 2, xs, K // blk, w, K // 2, sw, K // blk, M, N, K, 1.0, out, 0, N, ws, 256)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step()
    for seed in (1, 2):
        torch.manual_seed(seed)
        x.copy_(torch.randn(M, K, device="cuda"))
        graph.replay()
        first = out.clone()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(first, out)
        va, vb = values(xc, xs, fmt), values(w, sw, fmt)
        tol = (K / 16 + 10) * 2.0 ** -23 * (va.abs() @ vb.abs().t())
        assert ((out.double() - va @ vb.t()).abs() <= tol).all()
        # the rows themselves are within half a step of E2M1 (or its saturation) of x
        assert ((va - x.double()).norm() / x.double().norm()).item() < 0.2


def test_matmul_refusals():
    csa2_build.build()
    L = csa2.lib()
    names = ("fmt", "a", "as_", "sa", "ss", "b", "bs", "sb", "sbs", "M", "N", "K", "alpha", "out", "dt", "os", "ws", "wb",
             "stream")
    good = dict(zip(names, (0, 16, 256, 16, 32, 16, 256, 16, 32, 4, 8, 512, ctypes.c_float(1), 16, 0, 8, 16, 4096, None)))

    def call(**kw):
        a = {**good, **kw}
        return L.csa2_fp4_matmul(*[a[n] for n in names])
    assert call(fmt=1) == INVALID and call(fmt=7) == INVALID and call(dt=3) == INVALID
    for k in ("a", "sa", "b", "sb", "out"):
        assert call(**{k: None}) == INVALID
    assert call(M=-1) == SHAPE and call(N=-1) == SHAPE and call(M=1 << 31) == SHAPE and call(M=1 << 30, N=1 << 30, os=1 << 30) == SHAPE
    assert call(K=0) == SHAPE and call(K=520) == SHAPE and call(K=(1 << 20) + 16) == SHAPE
    assert call(fmt=2, K=528, as_=272, bs=272) == SHAPE                            # K % 32
    assert call(as_=240) == SHAPE and call(bs=240) == SHAPE and call(ss=31) == SHAPE and call(sbs=31) == SHAPE
    assert call(os=7) == SHAPE
    assert call(a=24) == ALIGN and call(b=24) == ALIGN and call(as_=264) == ALIGN and call(bs=264) == ALIGN
    assert call(out=18) == ALIGN and call(out=17, dt=1) == ALIGN
    assert call(ws=None) == WS and call(wb=8) == WS
    assert call(M=0) == OK and call(N=0) == OK and call(M=0, a=None, K=5) == OK
    assert csa2.csa2_fp4_matmul_workspace_size(1, 1, 16) > 0
    with pytest.raises(csa2.CSA2Error, match="SHAPE"):
        csa2.csa2_fp4_matmul_workspace_size(1, 1, 0)


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", [csa2.FMT_FP4, csa2.FMT_MXFP4])
@pytest.mark.parametrize("M,N,K", [(3, 200, 1600), (300, 333, 1120), (1200, 3100, 1600)])
def test_matmul_padding_is_not_read(M, N, K, fmt):
    """Code and scale rows that end inside an aligned 16 bytes, with NaN scales and codes behind their ends."""
    blk = block_of(fmt)
    nb = K // blk
    g = torch.Generator().manual_seed(4)
    ops = []
    for rows in (M, N):
        c, s = operand(g, rows, K, fmt, code_pad=16, scale_pad=-nb % 16 + 16)
        assert s.stride(0) % 16 == 0
        c[:, K // 2:] = 0x77
        s[:, nb:] = 0x7F if fmt == csa2.FMT_FP4 else 0xFF
        ops += [c, s]
    a, sa, b, sb = ops
    out = torch.empty(M, N, device="cuda")
    ws = torch.empty(256, dtype=torch.uint8, device="cuda")
    csa2.csa2_fp4_matmul(fmt, a, a.stride(0), sa, sa.stride(0), b, b.stride(0), sb, sb.stride(0), M, N, K, 1.0, out, 0, N,
                         ws, 256)
    va, vb = values(a[:, :K // 2], sa[:, :nb].contiguous(), fmt), values(b[:, :K // 2], sb[:, :nb].contiguous(), fmt)
    tol = (K / 16 + 66) * 2.0 ** -23 * (va.abs() @ vb.abs().t())
    assert ((out.double() - va @ vb.t()).abs() <= tol).all()


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", [csa2.FMT_FP4, csa2.FMT_MXFP4])
def test_linear_far_rows(fmt):
    """Inputs and outputs beyond 2^31 elements: rows there equal the same rows near the start."""
    M, N, K = 70001, 32776, 64
    blk = block_of(fmt)
    g = torch.Generator().manual_seed(6)
    b, sb = operand(g, N, K, fmt)
    x = torch.randn(40, K, generator=g).bfloat16().cuda()
    wide = torch.empty(M, N, dtype=torch.bfloat16, device="cuda")
    wide[:40, :K], wide[M - 40:, :K] = x, x
    codes = torch.zeros(M, 32, dtype=torch.uint8, device="cuda")
    scales = torch.zeros(M, K // blk, dtype=torch.uint8, device="cuda")
    csa2.csa2_quantize_kv(fmt, wide[M - 40:], csa2.DTYPE_BF16, 40, K, N, codes[M - 40:], 32, scales[M - 40:], K // blk)
    whole, whole_s = torch.zeros_like(codes), torch.zeros_like(scales)
    csa2.csa2_quantize_kv(fmt, wide, csa2.DTYPE_BF16, M, K, N, whole, 32, whole_s, K // blk)
    assert torch.equal(whole[M - 40:], codes[M - 40:]) and torch.equal(whole_s[M - 40:], scales[M - 40:])
    codes[:40], scales[:40] = codes[M - 40:], scales[M - 40:]
    ws = torch.empty(256, dtype=torch.uint8, device="cuda")
    csa2.csa2_fp4_matmul(fmt, codes, 32, scales, K // blk, b, b.stride(0), sb, sb.stride(0), M, N, K, 1.0, wide,
                         csa2.DTYPE_BF16, N, ws, 256)
    va, vb = values(codes[:40], scales[:40], fmt), values(b[:, :K // 2], sb, fmt)
    ref, mag = va @ vb.t(), va.abs() @ vb.abs().t()
    assert torch.equal(wide[:40], wide[M - 40:])
    assert ((wide[:40].double() - ref).abs() <= 2.0 ** -8 * ref.abs() + (K / 16 + 10) * 2.0 ** -23 * mag).all()
    assert csa2.csa2_device_error() == 0


@pytest.mark.gpu
def test_matmul_after_copies_in_a_graph():
    """A captured product that follows memory copies, one of them on a joined stream, reads what they wrote."""
    M, N, K, fmt = 70, 600, 512, csa2.FMT_MXFP4
    g = torch.Generator().manual_seed(8)
    (a, sa), (b, sb) = operand(g, M, K, fmt), operand(g, N, K, fmt)
    a1, b1 = torch.zeros_like(a), torch.zeros_like(b)
    out = torch.empty(M, N, device="cuda")
    ws = torch.empty(256, dtype=torch.uint8, device="cuda")
    side, other, graph = torch.cuda.Stream(), torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        other.wait_stream(side)
        with torch.cuda.stream(other):
            b1.copy_(b)
        a1.copy_(a)
        side.wait_stream(other)
        csa2.csa2_fp4_matmul(fmt, a1, K // 2, sa, K // 32, b1, K // 2, sb, K // 32, M, N, K, 1.0, out, 0, N, ws, 256)
        a1.zero_()                                          # after the product has read it
    for _ in range(3):
        out.fill_(-1.0)
        a.random_(0, 256)
        graph.replay()
        torch.cuda.synchronize()
        va, vb = values(a, sa, fmt), values(b, sb, fmt)
        tol = (K / 16 + 66) * 2.0 ** -23 * (va.abs() @ vb.abs().t())
        assert ((out.double() - va @ vb.t()).abs() <= tol).all()
