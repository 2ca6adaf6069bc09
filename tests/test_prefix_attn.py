"""csa2_prefix_attn against 64-bit attention over the dequantised entries (GPU), and its refusals (CPU).

Tolerances, from the kernel's arithmetic (n entries, 128 to a tile; A = the weighted mean of |v|):
  logits     512 exact products accumulated in fp32, each step losing at most 2^-23 of the magnitudes so
             far: dz = 2^-14 * softmax_scale * max_j sum_c |q_c v_jc|  (plus one rounding of the scale)
  weights    2^-22 from the exponential; rounded to fp16 for the product: 2^-11 relative, or 2^-32 of
             the largest weight where the fp16 value is subnormal
  sums       fp32: at most 2^-23 per tile, piece and lane step, (n / 128 + 64) * 2^-23
  out        |error| <= A * (2^-11 + 2 dz + 2^-20 + 2 (n / 128 + 64) 2^-23) + n * 2^-32 * max |v|
             + half a step of the output type (2^-8, 2^-24) of |out|
  lse        |error| <= dz + 2^-20 + (n / 128 + 64) 2^-23 + 2^-22 |lse|
"""
import ctypes
import math

import pytest
import torch

import compressed_sparse_attention_quantize_b200 as csa2
from compressed_sparse_attention_quantize_b200 import build as csa2_build
from tests.test_fp4_matmul import values

INVALID, SHAPE, ALIGN, UNSUP, WS = 1, 2, 3, 4, 7
D = 512


def cache(g, rows):
    """Packed main-KV rows from random latents, quantised by the library."""
    x = torch.randn(max(rows, 1), D, generator=g, device="cuda")
    x[:, torch.randperm(D, generator=g, device="cuda")[:4]] *= 8
    kv = torch.zeros(max(rows, 1), 288, dtype=torch.uint8, device="cuda")
    csa2.csa2_quantize_kv(csa2.FMT_FP4, x, csa2.DTYPE_F32, x.shape[0], D, D, kv, 288, kv[:, 256:], 288)
    return kv


class Case:
    """One call's inputs; `run` and `check` share them."""

    def __init__(self, lens, starts, rows, H, page=None, own=True, seed=0, out_dtype=csa2.DTYPE_F32, scale=None,
                 stride=288, q_gain=1.0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.lens, self.starts, self.rows, self.H, self.page, self.out_dtype = lens, starts, rows, H, page, out_dtype
        G, most = len(lens), max(lens)
        self.max_n = most
        if page:
            width = max(-(-most // page), 1)
            pool = sum(-(-n // page) for n in lens) + 3
            order = torch.randperm(pool, generator=g, device="cuda").int()
            self.table = torch.full((G, width), -1, dtype=torch.int32, device="cuda")
            at = 0
            for i, n in enumerate(lens):
                k = -(-n // page)
                self.table[i, :k] = order[at:at + k]
                at += k
            self.seq = None
            total = pool * page
            ids = [self.table[i][torch.arange(n, device="cuda") // page].long() * page + torch.arange(n, device="cuda") % page
                   for i, n in enumerate(lens)]
        else:
            self.table = None
            offs = torch.tensor([0] + list(lens)).cumsum(0)[:-1]
            self.seq = offs.to(torch.int64).cuda()
            total = sum(lens)
            ids = [int(o) + torch.arange(n, device="cuda") for o, n in zip(offs, lens)]
        self.ids = ids
        kv = cache(g, total)
        self.kv_rows = kv.shape[0]
        wide = torch.full((kv.shape[0], stride), 0x77, dtype=torch.uint8, device="cuda")
        wide[:, :288] = kv
        self.kv, self.stride = wide, stride
        self.q = (torch.randn(rows, H, D, generator=g, device="cuda") * q_gain).bfloat16()
        self.own_out = torch.randn(rows, H, D, generator=g, device="cuda") * 0.2 if own else None
        self.own_lse = math.log(max(most, 1)) + torch.randn(rows, H, generator=g, device="cuda") if own else None
        self.scale = 1.0 / math.sqrt(D) if scale is None else scale
        self.out = torch.full((rows, H, D), float("nan"), device="cuda",
                              dtype=torch.float32 if out_dtype == csa2.DTYPE_F32 else torch.bfloat16)
        self.lse = torch.full((rows, H), float("nan"), device="cuda")
        self.row_start = torch.tensor(starts, dtype=torch.int32, device="cuda")
        self.n = torch.tensor(lens, dtype=torch.int32, device="cuda")
        self.ws_bytes = csa2.csa2_prefix_attn_workspace_size(rows, H, G, self.max_n)
        self.ws = torch.full((self.ws_bytes,), 0x7F, dtype=torch.uint8, device="cuda")

    def run(self, stream=None):
        csa2.csa2_prefix_attn(self.q, self.rows, self.H, D, self.row_start, len(self.lens), self.kv, self.stride,
                              self.kv_rows, self.seq, self.table, self.table.shape[1] if self.table is not None else 0,
                              self.page or 0, self.n, self.max_n, self.scale, self.own_out, self.own_lse, self.out,
                              self.out_dtype, self.lse, self.ws, self.ws_bytes, stream)

    def group_of(self, row):
        for i, (lo, hi) in enumerate(zip(self.starts[:-1], self.starts[1:])):
            if lo <= row < hi:
                return i
        return None

    def check(self, skip_rows=()):
        every = values(self.kv[:, :256], self.kv[:, 256:288].contiguous(), csa2.FMT_FP4)
        half = 2.0 ** -24 if self.out_dtype == csa2.DTYPE_F32 else 2.0 ** -8
        for r in range(self.rows):
            if r in skip_rows:
                continue
            i = self.group_of(r)
            ids = self.ids[i] if i is not None else self.ids[0][:0]
            v, n = every[ids], len(ids)
            q = self.q[r].double()
            z = q @ v.t() * self.scale
            dz = 2.0 ** -14 * self.scale * float((q.abs() @ v.abs().t()).max()) if n else 0.0
            vals, mags = v, v.abs()
            if self.own_out is not None:
                z = torch.cat((z, self.own_lse[r].double()[:, None]), dim=1)
            m = z.amax(dim=1, keepdim=True) if z.shape[1] else torch.full((self.H, 1), -math.inf, device="cuda").double()
            p = torch.where(m == -math.inf, torch.zeros_like(z), torch.exp(z - m))
            total = p.sum(dim=1, keepdim=True)
            out, mag = p[:, :n] @ vals, p[:, :n] @ mags
            if self.own_out is not None:
                own = torch.where(p[:, n:] > 0, self.own_out[r].double(), torch.zeros_like(self.own_out[r].double()))
                out, mag = out + p[:, n:] * own, mag + p[:, n:] * own.abs()
            safe = total.clamp(min=1e-300)
            out, mag = out / safe, mag / safe
            lse = torch.where(total[:, 0] > 0, m[:, 0] + torch.log(safe[:, 0]), torch.full_like(m[:, 0], -math.inf))
            steps = (n / 128 + 64) * 2.0 ** -23
            tol = mag * (2.0 ** -11 + 2 * dz + 2.0 ** -20 + 2 * steps) + n * 2.0 ** -32 * (vals.abs().max().item() if n else 0)
            tol = tol + half * out.abs() + 1e-30
            got = self.out[r].double()
            assert not got.isnan().any(), f"row {r}"
            worst = float(((got - out).abs() / tol).max())
            assert worst <= 1, f"row {r}: out is {worst:.3g} of the tolerance"
            lt = dz + 2.0 ** -20 + steps + 2.0 ** -22 * lse.abs()
            gl = self.lse[r].double()
            assert torch.equal(gl == -math.inf, lse == -math.inf), f"row {r}"
            fin = lse != -math.inf
            assert ((gl - lse).abs()[fin] <= lt[fin]).all(), f"row {r}: lse"


@pytest.mark.gpu
@pytest.mark.parametrize("n", [0, 1, 2, 127, 128, 129, 255, 1000, 5000])
@pytest.mark.parametrize("H,own", [(16, True), (64, False)])
def test_one_prefix(n, H, own):
    c = Case([n], [0, 3], 3, H, own=own, seed=n)
    c.run()
    assert csa2.csa2_device_error() == 0
    c.check()


@pytest.mark.gpu
@pytest.mark.parametrize("page", [1, 3, 16, 64, 100, 4096])
@pytest.mark.parametrize("H", [16, 48, 128])
def test_paged_groups(page, H):
    """Ragged groups, an empty prefix and an empty group among them, pages that end inside a tile."""
    c = Case([300, 0, 129, 77, 1300], [0, 2, 3, 3, 8, 11], 11, H, page=page, seed=page + H, out_dtype=csa2.DTYPE_BF16)
    c.run()
    assert csa2.csa2_device_error() == 0
    c.check()


@pytest.mark.gpu
def test_rows_outside_every_group():
    """Rows before the first and behind the last group have their own part alone."""
    c = Case([200, 50], [2, 5, 7], 10, 32, page=16, seed=5)
    c.run()
    assert csa2.csa2_device_error() == 0
    c.check()


@pytest.mark.gpu
@pytest.mark.parametrize("rows,H,n", [(1, 16, 40000), (5, 64, 20000), (40, 128, 700), (300, 64, 260), (64, 64, 4096)])
def test_shares_of_the_work(rows, H, n):
    """Few queries on a long prefix (a tile cut into many pieces), many queries (many tiles to a CTA)."""
    c = Case([n], [0, rows], rows, H, seed=rows, own=rows % 2 == 0)
    c.run()
    assert csa2.csa2_device_error() == 0
    c.check()


@pytest.mark.gpu
def test_many_groups():
    G = 70
    lens = [(37 * i) % 300 for i in range(G)]
    starts = [0]
    for i in range(G):
        starts.append(starts[-1] + i % 3)
    c = Case(lens, starts, starts[-1], 16, page=32, seed=9)
    c.run()
    assert csa2.csa2_device_error() == 0
    c.check()


@pytest.mark.gpu
@pytest.mark.parametrize("gain,scale", [(1.0, 1.0), (30.0, None), (1e-6, None), (2.0 ** 60, 2.0 ** -62), (2.0 ** -100, 2.0 ** 98)])
def test_peaked_and_flat_weights(gain, scale):
    """Logits from flat to hundreds apart (maxima that move late), queries far from fp16's range."""
    c = Case([3000], [0, 2], 2, 64, seed=3, scale=scale, q_gain=gain)
    c.run()
    assert csa2.csa2_device_error() == 0
    c.check()


@pytest.mark.gpu
def test_one_heavy_key_late_and_light_rest():
    """The last key has almost all weight for some queries, none for others: maxima move in the last tile
    after thousands of light keys have been summed."""
    c = Case([6000], [0, 2], 2, 16, seed=4, own=False)
    v = values(c.kv[:, :256], c.kv[:, 256:288].contiguous(), csa2.FMT_FP4)
    big = v[c.ids[0][-1]]
    c.q[0] = (big * 0.5).bfloat16()
    c.q[1] = (-big * 0.5).bfloat16()
    c.run()
    c.check()


@pytest.mark.gpu
def test_bad_rows_stay_with_themselves():
    """A query row of NaNs or infinities, and a NaN scale in one prefix, spoil their own outputs only."""
    c = Case([400, 300], [0, 4, 6], 6, 64, page=16, seed=8)
    c.q[1, 5] = float("nan")
    c.q[2, 7] = float("inf")
    c.kv[int(c.ids[1][17]), 256 + 3] = 0x7F                # NaN scale in the second prefix
    c.own_out[3, 0] = float("nan")
    c.own_lse[3, 0] = -math.inf                            # no own part: its output does not count
    c.run()
    assert csa2.csa2_device_error() == 0
    assert c.out[1, 5].isnan().all() and c.out[2, 7].isnan().any()
    assert c.out[4:, :].isnan().any(dim=2).all()
    keep = torch.ones(6, 64, dtype=torch.bool, device="cuda")
    keep[1, 5], keep[2, 7], keep[4:] = False, False, False
    assert not c.out[keep].isnan().any()
    out, lse = c.out.clone(), c.lse.clone()
    c.kv[int(c.ids[1][17]), 256 + 3] = 0x38
    c.q[1, 5], c.q[2, 7] = 0.0, 0.0
    c.run()
    assert torch.equal(out[keep], c.out[keep]) and torch.equal(lse[keep], c.lse[keep])
    c.check()


@pytest.mark.gpu
@pytest.mark.parametrize("what", ["page", "width", "row", "starts", "length", "overlap"])
def test_broken_contract(what):
    """Bad pages, rows and groups: an error word, the other groups' results, nothing read outside."""
    c = Case([300, 200, 260], [0, 2, 4, 7], 7, 16, page=16, seed=12)
    err, skip = csa2.CSA2_ERR_INVALID_ARG, set()
    if what == "page":
        c.table[1, 3] = -1
        c.ids[1] = torch.cat((c.ids[1][:48], c.ids[1][64:]))
    elif what == "width":
        c.table = c.table[:, :17].contiguous()             # 272 entries: the first prefix ends early
        c.ids[0] = c.ids[0][:272]
    elif what == "row":
        c.table[2, 0] = 1 << 25
        c.ids[2] = c.ids[2][16:]
    elif what == "starts":
        c.row_start[3] = 99
        err, c.ids[2] = csa2.CSA2_ERR_SHAPE, c.ids[2][:0]
    elif what == "length":
        c.n[1] = 301
        err, c.ids[1] = csa2.CSA2_ERR_SHAPE, c.ids[1][:0]
    else:
        c.row_start.copy_(torch.tensor([0, 4, 2, 7]))      # the second runs backwards, the third into the first
        err, skip = csa2.CSA2_ERR_SHAPE, set(range(4))
        c.starts, c.ids[1], c.ids[2] = [0, 4, 4, 7], c.ids[1][:0], c.ids[2][:0]
        skip = set()
    c.run()
    assert csa2.csa2_device_error() == err
    c.check(skip)
    assert csa2.csa2_device_error() == 0


@pytest.mark.gpu
def test_wide_rows_in_place_and_repeatable():
    """kv rows 320 bytes apart, out and lse over the own part, the same bits twice."""
    c = Case([777], [0, 5], 5, 32, stride=320, seed=2)
    c.run()
    c.check()
    first, lse = c.out.clone(), c.lse.clone()
    own_out, own_lse = c.own_out.clone(), c.own_lse.clone()
    c.out, c.lse = c.own_out, c.own_lse
    c.run()
    assert torch.equal(c.own_out, first) and torch.equal(c.own_lse, lse)
    c.own_out, c.own_lse, c.out, c.lse = own_out, own_lse, first, lse
    c.check()


@pytest.mark.gpu
def test_no_lse_output_and_two_streams():
    """Two calls at once on their own streams and workspaces; one without an lse output."""
    a, b = Case([2000], [0, 9], 9, 64, page=64, seed=1), Case([900, 1500], [0, 4, 8], 8, 128, seed=2)
    keep = b.lse
    b.lse = None
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(3):
        a.run(s1)
        b.run(s2)
    torch.cuda.synchronize()
    assert csa2.csa2_device_error() == 0
    a.check()
    b.lse = keep
    b.run()
    out = b.out.clone()
    b.check()
    assert torch.equal(out, b.out)


@pytest.mark.gpu
def test_captured_and_replayed_on_other_lengths():
    """A captured call replayed after lengths, groups and pages changed on the device."""
    c = Case([900, 1000], [0, 3, 8], 8, 64, page=32, seed=6)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        c.run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        c.run()
    for lens, starts in (([1000, 10], [0, 1, 8]), ([0, 555], [0, 6, 7]), ([900, 1000], [0, 3, 8])):
        full = [c.table[i][torch.arange(1000, device="cuda") // 32].long() * 32 + torch.arange(1000, device="cuda") % 32
                for i in range(2)]
        lens = [min(n, 900) if i == 0 else n for i, n in enumerate(lens)]
        c.n.copy_(torch.tensor(lens))
        c.row_start.copy_(torch.tensor(starts))
        c.lens, c.starts, c.ids = lens, starts, [f[:n] for f, n in zip(full, lens)]
        c.out.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert csa2.csa2_device_error() == 0
        c.check()


def test_prefix_refusals():
    csa2_build.build()
    L = csa2.lib()
    names = ("q", "rows", "H", "D", "row_start", "G", "kv", "stride", "kv_rows", "seq", "table", "max_pages", "page", "n",
             "max_n", "scale", "own_out", "own_lse", "out", "dt", "lse", "ws", "wb", "stream")
    good = dict(zip(names, (16, 4, 64, 512, 16, 1, 16, 288, 100, None, 16, 8, 64, 16, 100, ctypes.c_float(1), 16, 16, 16, 0, 16,
                            16, 1 << 40, None)))

    def call(**kw):
        a = {**good, **kw}
        return L.csa2_prefix_attn(*[a[k] for k in names])
    for k in ("q", "row_start", "kv", "n", "out", "own_out", "own_lse"):
        assert call(**{k: None}) == INVALID, k
    assert call(table=None) == INVALID and call(dt=4) == INVALID
    assert call(D=256) == UNSUP
    assert call(H=8) == SHAPE and call(H=40) == SHAPE and call(H=144) == SHAPE
    assert call(rows=0) == SHAPE and call(rows=1 << 20) == SHAPE
    assert call(G=0) == SHAPE and call(G=1025) == SHAPE
    assert call(max_n=-1) == SHAPE and call(max_n=(1 << 26) + 1) == SHAPE and call(G=1024, max_n=1 << 21) == SHAPE
    assert call(kv_rows=-1) == SHAPE and call(stride=272) == SHAPE
    assert call(page=0) == SHAPE and call(page=(1 << 20) + 1) == SHAPE and call(max_pages=0) == SHAPE
    for k in ("q", "kv", "own_out", "out"):
        assert call(**{k: 24}) == ALIGN, k
    assert call(stride=296) == ALIGN and call(table=None, seq=20) == ALIGN
    for k in ("row_start", "table", "n", "own_lse", "lse"):
        assert call(**{k: 18}) == ALIGN, k
    assert call(ws=None) == WS and call(wb=1000) == WS
    size = csa2.csa2_prefix_attn_workspace_size(32, 64, 1, 32768)
    assert size >= 32 * 64 * 1024 + 4 * 32768                     # queries in fp16, the entries' cache rows
    assert size < csa2.csa2_prefix_attn_workspace_size(32, 64, 1, 1 << 22)
    with pytest.raises(csa2.CSA2Error, match="SHAPE"):
        csa2.csa2_prefix_attn_workspace_size(32, 60, 1, 32768)


@pytest.mark.gpu
@pytest.mark.parametrize("paged", [False, True])
def test_far_rows(paged):
    """Entries more than 2^32 bytes into the cache: what the same entries give near its start."""
    near = Case([260, 100], [0, 2, 5], 5, 16, page=16 if paged else None, seed=21)
    near.run()
    out, lse = near.out.clone(), near.lse.clone()
    shift = 16 * 1000000                                       # rows, whole pages
    kv = torch.empty((shift + near.kv_rows, near.stride), dtype=torch.uint8, device="cuda")
    kv[shift:] = near.kv
    near.kv, near.kv_rows = kv, kv.shape[0]
    if paged:
        near.table = torch.where(near.table >= 0, near.table + shift // 16, near.table)
    else:
        near.seq = near.seq + shift
    near.run()
    assert csa2.csa2_device_error() == 0
    assert torch.equal(out, near.out) and torch.equal(lse, near.lse)
