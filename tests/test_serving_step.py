"""A serving step over a paged cache, its operators one after another: FP4 products make queries and
latents from hidden states, page maps place them, the quantisers write them, page ids carry a selection
to cache rows, sparse attention gives every request's own part and prefix attention merges it with the
prompt the requests of a group share.  GPU.
"""
import math

import numpy as np
import pytest
import torch

import compressed_sparse_attention_quantize_b200 as csa2
from tests.test_fp4_matmul import values
from tests.test_paged import maps_by_loops

pytestmark = pytest.mark.gpu

B, H, D, HID, E, RATIO, W, K, MAX_PAGES = 6, 64, 512, 256, 16, 4, 128, 64, 16
STARTS, LENS = [0, 3, 6], [300, 130]
CAP_T, CAP_E = 64, 24


class Step:
    """Buffers of a step, as a serving program keeps them; `run` enqueues the whole step."""

    def __init__(self, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        dev = dict(device="cuda")
        randn = lambda *s: torch.randn(*s, generator=g, **dev)                            # noqa: E731
        prefix_pages = [-(-n // E) for n in LENS]
        self.pool = sum(prefix_pages) + B * MAX_PAGES
        order = torch.randperm(self.pool, generator=g, **dev).int()
        self.table_prefix = torch.full((2, max(prefix_pages)), -1, dtype=torch.int32, **dev)
        at = 0
        for i, n in enumerate(prefix_pages):
            self.table_prefix[i, :n] = order[at:at + n]
            at += n
        self.free = order[at:].contiguous()
        self.table = torch.full((B, MAX_PAGES), -1, dtype=torch.int32, **dev)
        self.kv = torch.full((self.pool * E, 288), 0x7F, dtype=torch.uint8, **dev)        # NaN scales everywhere
        self.win = torch.full((B * W, D), 0x7F, dtype=torch.uint8, **dev)
        self.win_scale = torch.full((B * W,), float("nan"), **dev)
        for i, n in enumerate(LENS):                                                      # the prompts' entries
            rows = self.table_prefix[i][torch.arange(n, **dev) // E].long() * E + torch.arange(n, **dev) % E
            csa2.csa2_quantize_kv(csa2.FMT_FP4, randn(n, D), 0, n, D, D, self.kv, 288, self.kv[:, 256:], 288, rows)
        # weights, quantised once
        self.wq, self.wq_s = self.weights(randn(H * D, HID) / math.sqrt(HID))
        self.wk, self.wk_s = self.weights(randn(D, HID) / math.sqrt(HID))
        # the step's inputs
        self.hidden, self.hidden_e = randn(B, HID).bfloat16(), randn(CAP_E, HID).bfloat16()
        self.tokens = randn(CAP_T, D)
        i32 = lambda *s: torch.zeros(*s, dtype=torch.int32, **dev)                        # noqa: E731
        i64 = lambda *s: torch.zeros(*s, dtype=torch.int64, **dev)                        # noqa: E731
        self.old, self.new, self.next = i32(B), i32(B), i32(2)
        self.n, self.swa_len, self.eo, self.er = i32(B), i32(B), i64(B + 1), i64(CAP_E)
        self.to, self.wr, self.qp = i64(B + 1), i64(CAP_T), i32(CAP_T)
        self.xc, self.xs = torch.zeros(B, HID // 2, dtype=torch.uint8, **dev), torch.zeros(B, HID // 16, dtype=torch.uint8, **dev)
        self.ec, self.es = torch.zeros(CAP_E, HID // 2, dtype=torch.uint8, **dev), torch.zeros(CAP_E, HID // 16, dtype=torch.uint8, **dev)
        self.q = torch.zeros(B, H, D, dtype=torch.bfloat16, **dev)
        self.latent = torch.zeros(CAP_E, D, **dev)
        self.sel, self.rows = i32(B, K) - 1, i32(B, K)
        self.zero = i64(B)
        self.own, self.own_lse = torch.zeros(B, H, D, **dev), torch.zeros(B, H, **dev)
        self.out, self.lse = torch.zeros(B, H, D, **dev), torch.zeros(B, H, **dev)
        self.row_start = torch.tensor(STARTS, dtype=torch.int32, **dev)
        self.lens = torch.tensor(LENS, dtype=torch.int32, **dev)
        self.ws = torch.empty(max(csa2.csa2_prefix_attn_workspace_size(B, H, 2, max(LENS)),
                                  csa2.csa2_sparse_attn_workspace_size(B, H, K), 4096), dtype=torch.uint8, **dev)
        self.scale = 1 / math.sqrt(D)

    @staticmethod
    def weights(w):
        c = torch.empty(w.shape[0], HID // 2, dtype=torch.uint8, device="cuda")
        s = torch.empty(w.shape[0], HID // 16, dtype=torch.uint8, device="cuda")
        csa2.csa2_quantize_kv(csa2.FMT_FP4, w, 0, w.shape[0], HID, HID, c, HID // 2, s, HID // 16)
        return c, s

    def linear(self, x, xc, xs, w, ws, out, dt):
        m, n = x.shape[0], w.shape[0]
        csa2.csa2_quantize_kv(csa2.FMT_FP4, x, csa2.DTYPE_BF16, m, HID, HID, xc, HID // 2, xs, HID // 16)
        csa2.csa2_fp4_matmul(csa2.FMT_FP4, xc, HID // 2, xs, HID // 16, w, HID // 2, ws, HID // 16, m, n, HID, 1.0, out, dt, n,
                             self.ws, 4096)

    def run(self):
        self.linear(self.hidden, self.xc, self.xs, self.wq, self.wq_s, self.q, csa2.DTYPE_BF16)
        self.linear(self.hidden_e, self.ec, self.es, self.wk, self.wk_s, self.latent, csa2.DTYPE_F32)
        csa2.csa2_page_maps(self.old, self.new, B, RATIO, E, W, self.table, MAX_PAGES, self.free, self.free.numel(),
                            self.next, self.next[1:], self.n, self.swa_len, self.eo, self.er, CAP_E, self.to, self.wr,
                            self.qp, CAP_T)
        csa2.csa2_quantize_kv_batch([
            csa2.quant_job(csa2.FMT_FP4, self.latent, 0, CAP_E, D, D, self.kv, 288, self.kv[:, 256:], 288, self.er),
            csa2.quant_job(csa2.FMT_FP8_TOKEN, self.tokens, 0, CAP_T, D, D, self.win, D, self.win_scale, 4, self.wr)])
        csa2.csa2_page_ids(self.sel, B, 1, K, self.table, MAX_PAGES, E, self.rows)
        csa2.csa2_sparse_attn(self.q, B, 1, H, D, self.kv, 288, self.zero, None, self.rows, None, K, self.win, self.win_scale,
                              W, None, self.swa_len, self.scale, self.own, csa2.DTYPE_F32, self.own_lse, self.ws, self.ws.numel())
        csa2.csa2_prefix_attn(self.q, B, H, D, self.row_start, 2, self.kv, 288, self.kv.shape[0], None, self.table_prefix,
                              self.table_prefix.shape[1], E, self.lens, max(LENS), self.scale, self.own, self.own_lse,
                              self.out, csa2.DTYPE_F32, self.lse, self.ws, self.ws.numel())

    def begin(self, old, new, seed):
        """The host's part: lengths, inputs and the selection (every own entry) of the next step."""
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.old.copy_(torch.tensor(old))
        self.new.copy_(torch.tensor(new))
        self.next[0] = self.next[1]
        self.hidden.copy_(torch.randn(B, HID, generator=g, device="cuda"))
        self.hidden_e.copy_(torch.randn(CAP_E, HID, generator=g, device="cuda"))
        self.tokens.copy_(torch.randn(CAP_T, D, generator=g, device="cuda"))
        n = torch.tensor(new, device="cuda")[:, None] // RATIO
        ids = torch.arange(K, device="cuda")[None, :].expand(B, K)
        self.sel.copy_(torch.where(ids < n, ids, torch.full_like(ids, -1)))

    def check(self, old, new, latents, tokens):
        """Queries, writes and outputs against 64 bits.  `latents`, `tokens`: what every request has been
        given so far (lists of rows), to which this step's are added."""
        assert csa2.csa2_device_error() == 0
        # the product: one rounding to bf16 of the fp32 sum over 256 channels
        ref = values(self.xc, self.xs, csa2.FMT_FP4) @ values(self.wq, self.wq_s, csa2.FMT_FP4).t()
        mag = values(self.xc, self.xs, csa2.FMT_FP4).abs() @ values(self.wq, self.wq_s, csa2.FMT_FP4).abs().t()
        assert ((self.q.double().reshape(B, -1) - ref).abs() <= 2.0 ** -8 * ref.abs() + 30 * 2.0 ** -23 * mag).all()
        eo, to = self.eo.tolist(), self.to.tolist()
        for b in range(B):
            latents[b] += [self.latent[i].clone() for i in range(eo[b], eo[b + 1])]
            tokens[b] += [self.tokens[i].clone() for i in range(to[b], to[b + 1])]
        every = values(self.kv[:, :256], self.kv[:, 256:].contiguous(), csa2.FMT_FP4)
        win = self.win.view(torch.float8_e4m3fn).double() * self.win_scale.double()[:, None]
        for b in range(B):
            n = new[b] // RATIO
            assert len(latents[b]) == n and len(tokens[b]) == new[b] and int(self.n[b]) == n
            rows = self.table[b][torch.arange(n, device="cuda") // E].long() * E + torch.arange(n, device="cuda") % E
            assert torch.equal(self.rows[b, :n].long(), rows)
            # the cache holds the request's latents: E2M1 is within half a step (1/4 relative of the block's
            # largest / 6, plus the scale's 2^-4), so a quarter of the block's largest bounds every error
            own = every[rows]
            if n:
                x = torch.stack(latents[b]).double()
                amax = x.reshape(n, -1, 16).abs().amax(2, keepdim=True).expand(n, 32, 16).reshape(n, D)
                assert ((own - x).abs() <= 0.25 * amax).all()
            # the window holds the last tokens: E4M3 is within 2^-4 relative, or 2^-10 of the scale
            ring = win[b * W:(b + 1) * W]
            last = range(max(0, new[b] - W), new[b])
            wv = torch.stack([ring[p % W] for p in last]) if len(last) else ring[:0]
            if len(last):
                x = torch.stack([tokens[b][p] for p in last]).double()
                assert ((wv - x).abs() <= 2.0 ** -4 * x.abs() + 2.0 ** -9 * x.abs().amax(1, keepdim=True) / 448 * 1.01).all()
            # the own part within the library's stated bound, the whole within the prefix's
            g = 0 if b < STARTS[1] else 1
            pn = LENS[g]
            prows = self.table_prefix[g][torch.arange(pn, device="cuda") // E].long() * E + torch.arange(pn, device="cuda") % E
            pv, q = every[prows], self.q[b].double()
            ov = torch.cat((own, wv))
            if len(ov):
                z = q @ ov.t() * self.scale
                ref = torch.softmax(z, 1) @ ov
                err = self.own[b].double() - ref
                assert float(err.norm() / ref.norm()) <= 1e-3
                assert ((self.own_lse[b].double() - torch.logsumexp(z, 1)).abs() <= 1e-3).all()
            else:
                assert (self.own[b] == 0).all() and (self.own_lse[b] == -math.inf).all()
            z = torch.cat((q @ pv.t() * self.scale, self.own_lse[b].double()[:, None]), 1)
            p = torch.softmax(z, 1)
            ref = p[:, :pn] @ pv + p[:, pn:] * self.own[b].double()
            mag = p[:, :pn] @ pv.abs() + p[:, pn:] * self.own[b].double().abs()
            dz = 2.0 ** -14 * self.scale * float((q.abs() @ pv.abs().t()).max())
            tol = mag * (2.0 ** -11 + 2 * dz + 2.0 ** -18) + pn * 2.0 ** -32 * float(pv.abs().max()) + 2.0 ** -23 * ref.abs()
            assert ((self.out[b].double() - ref).abs() <= tol).all()
            assert ((self.lse[b].double() - torch.logsumexp(z, 1)).abs() <= dz + 2.0 ** -16).all()


STEPS = [([0] * B, [40, 7, 0, 3, 1, 0]), ([40, 7, 0, 3, 1, 0], [41, 8, 0, 7, 2, 5]), ([41, 8, 0, 7, 2, 5], [49, 9, 4, 8, 20, 6])]


@pytest.mark.parametrize("graph", [False, True])
def test_serving_steps(graph):
    """Three steps in a row, eagerly and as one captured graph replayed: both against 64 bits, and the
    maps against plain loops."""
    s = Step()
    latents, tokens = [[] for _ in range(B)], [[] for _ in range(B)]
    replay = None
    if graph:
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            s.run()                                        # no requests yet: nothing is written
        torch.cuda.synchronize()
        replay = torch.cuda.CUDAGraph()
        with torch.cuda.graph(replay, stream=side):
            s.run()
    table, free, nxt = s.table.cpu().numpy(), s.free.cpu().numpy(), 0
    for i, (old, new) in enumerate(STEPS):
        s.begin(old, new, 10 + i)
        if graph:
            replay.replay()
        else:
            s.run()
        torch.cuda.synchronize()
        ref, bad = maps_by_loops(np.array(old), np.array(new), RATIO, E, W, table, free, nxt, CAP_E, CAP_T)
        assert not bad
        table, nxt = ref["table"], ref["free_next"][0]
        assert np.array_equal(s.table.cpu().numpy(), table) and s.next.tolist()[1] == nxt
        assert np.array_equal(s.er.cpu().numpy(), ref["entry_rows"]) and np.array_equal(s.wr.cpu().numpy(), ref["window_rows"])
        s.check(old, new, latents, tokens)


def test_two_steps_at_once():
    """Two programs with buffers and workspaces of their own on two streams: bit for bit what each gives alone."""
    def fresh(seed):
        s = Step(seed)
        s.begin(*STEPS[0], 20 + seed)
        return s
    alone = [fresh(1), fresh(2)]
    for s in alone:
        s.run()
        torch.cuda.synchronize()
    both, streams = [fresh(1), fresh(2)], [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(5):                                      # the same step again: it writes the same bytes
        for s, st in zip(both, streams):
            with torch.cuda.stream(st):
                s.run()
    torch.cuda.synchronize()
    assert csa2.csa2_device_error() == 0
    for a, b in zip(alone, both):
        for name in ("q", "latent", "own", "own_lse", "out", "lse", "kv", "win", "er", "wr", "table"):
            assert torch.equal(getattr(a, name).view(torch.uint8), getattr(b, name).view(torch.uint8)), name
