"""Operators of a serving step over paged, quantised caches: their cases, inputs and plain forms.

Four operators, as a serving program calls them one after another:

  linear   y = (quantised x) . (quantised W)^T: the rows of x are quantised to microscaled FP4
           (E2M1 codes with one E8M0 scale per 32 channels, or one E4M3 scale per 16), then
           multiplied with FP4 weights.  This makes queries, latents and indexer rows from hidden
           states.
  maps     block table, cache rows, window slots and positions of a step's new tokens, from the
           request lengths and a list of free pages.
  ids      entry numbers (a top-K selection) to cache rows, through a block table.
  prefix   attention of a batch over a prefix that its requests share, read once for all of them
           from paged FP4 entries, merged with each request's own part (its output and its
           log-sum-exp).

``run`` computes the plain form (elementary torch operations in 32 bits) where ``own`` is false and
calls the library where it is true.  ``exact`` is written apart from both, in 64 bits.
"""
import math

import torch

own = False

LATENT = 512          # width of a cache entry: keys and values at once
KV_ROW = 288          # its bytes: 256 code bytes, then 32 E4M3 scales
WINDOW = 128          # sliding-window slots of a sequence
RATIO = 4             # tokens per compressed entry


# --------------------------------------------------------------------------------------------
# cases
# --------------------------------------------------------------------------------------------
def listed():
    return [
        # one decode token through a projection of hidden states: weight reads and launches count
        dict(name="linear mx 1x4096x2048", op="linear", fmt="mx", m=1, n=4096, k=2048),
        # a decode batch of 32 into 64 heads x 512 query channels: the weights' bytes count
        dict(name="linear mx 32x32768x4096", op="linear", fmt="mx", m=32, n=32768, k=4096),
        # an odd batch and odd output width, 16-channel scales, as for indexer rows (8 heads x 64)
        dict(name="linear e4m3 333x1000x1504", op="linear", fmt="e4m3", m=333, n=1000, k=1504),
        # a prefill chunk of 4096 tokens: the tensor cores count
        dict(name="linear e4m3 4096x8192x4096", op="linear", fmt="e4m3", m=4096, n=8192, k=4096),
        # a decode step of 32 requests, one token each
        dict(name="maps decode 32", op="maps", b=32, most_old=131072, most_new=1, page=64),
        # ragged prefill chunks for 256 requests, pages that end inside a chunk
        dict(name="maps prefill 256", op="maps", b=256, most_old=16384, most_new=8192, page=48),
        # a decode batch's selection of 2048 entries per row
        dict(name="ids 32x2048", op="ids", b=32, t=1, k=2048, page=64, n=32768),
        # a prefill chunk's selections: 4096 rows of one sequence
        dict(name="ids 4096x2048", op="ids", b=1, t=4096, k=2048, page=16, n=33792),
        # one request with 16 heads over a short prefix: latency counts
        dict(name="prefix 1x16 of 1000", op="prefix", groups=1, rows=1, heads=16, n=1000, page=16),
        # a decode batch in four groups, each with a prefix of its own length
        dict(name="prefix 32x64 of 4 x 8192", op="prefix", groups=4, rows=32, heads=64, n=8192, page=64),
        # 32 requests behind one 128K-token prompt
        dict(name="prefix 32x64 of 32768", op="prefix", groups=1, rows=32, heads=64, n=32768, page=64),
        # 128 requests behind it: the largest
        dict(name="prefix 128x64 of 32768", op="prefix", groups=1, rows=128, heads=64, n=32768, page=64),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("linear", "linear", "maps", "ids", "prefix", "prefix"))
    if op == "linear":
        while True:
            m, n, k = _log(rng, 1, 4096), _log(rng, 64, 32768), 32 * _log(rng, 8, 256)
            if m * n * k <= 4096 * 8192 * 4096 and n * k <= 32768 * 4096:
                return dict(op=op, fmt=rng.choice(("mx", "e4m3")), m=m, n=n, k=k)
    if op == "maps":
        most_new = rng.choice((1, _log(rng, 2, 8192)))
        return dict(op=op, b=_log(rng, 1, 256), most_old=_log(rng, 16, 131072), most_new=most_new,
                    page=rng.choice((1, 16, 48, 64, 100, 256)))
    if op == "ids":
        b, k = _log(rng, 1, 64), _log(rng, 1, 4096)
        t = _log(rng, 1, max(1, 4096 // b))
        return dict(op=op, b=b, t=t, k=min(k, 4096 * 2048 // (b * t)), page=rng.choice((1, 16, 48, 64, 256)),
                    n=_log(rng, 16, 65536))
    groups = rng.choice((1, 1, 1, 2, 3, 5))
    rows, heads = _log(rng, groups, 128), rng.choice((16, 32, 64, 128))
    rows = min(rows, 128 * 64 // heads)
    return dict(op=op, groups=groups, rows=max(rows, groups), heads=heads, n=_log(rng, 1, 32768),
                page=rng.choice((1, 16, 48, 64, 100, 256)))


# --------------------------------------------------------------------------------------------
# E2M1 with block scales, in 32 bits (inputs and plain forms)
# --------------------------------------------------------------------------------------------
_MIDPOINTS = ((0.25, False), (0.75, True), (1.25, False), (1.75, True), (2.5, False), (3.5, True), (5.0, False))


def _block(fmt):
    return 32 if fmt == "mx" else 16


def _quantise(x, fmt):
    """Codes (0..15), scale values and scale bytes of rows x in blocks: each code the exact quotient
    rounded once to nearest, ties to even, saturating at 6."""
    blk = _block(fmt)
    v = x.float().reshape(x.shape[0], -1, blk)
    amax = v.abs().amax(dim=2)
    if fmt == "mx":
        # the largest power of two at most amax, divided by 4 (the exponent of 6)
        e = (torch.frexp(amax).exponent - 3).clamp(-127, 127)
        e = torch.where(amax == 0, torch.full_like(e, -127), e)
        scale = torch.ldexp(torch.ones_like(amax), e)
        byte = (e + 127).to(torch.uint8)
    else:
        s = (amax / 6.0).clamp(max=448.0).to(torch.float8_e4m3fn)
        scale, byte = s.float(), s.view(torch.uint8)
    a, s = v.abs(), scale[:, :, None]
    code = torch.zeros_like(a, dtype=torch.uint8)
    # |x| against midpoint * scale: the products are exact, so the exact quotient decides
    for mid, tie_up in _MIDPOINTS:
        code += (a >= mid * s) if tie_up else (a > mid * s)
    code = torch.where(s == 0, torch.zeros_like(code), code + 8 * torch.signbit(v).to(torch.uint8))
    return code.reshape(x.shape), scale, byte


def _pack(code):
    return code[:, 0::2] | (code[:, 1::2] << 4)


def _values(code, scale):
    """Codes and block scale values to fp32 (exact)."""
    grid = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, 0, -.5, -1, -1.5, -2, -3, -4, -6], device=code.device)
    v = grid[code.int()].reshape(code.shape[0], scale.shape[1], -1)
    return (v * scale[:, :, None]).reshape(code.shape)


def _unpack(packed):
    return torch.stack((packed & 15, packed >> 4), dim=2).reshape(packed.shape[0], -1)


def _scale_values(byte, fmt):
    if fmt == "mx":
        return torch.ldexp(torch.ones(byte.shape, device=byte.device), byte.int() - 127)
    return byte.view(torch.float8_e4m3fn).float()


# --------------------------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------------------------
def _latents(g, rows):
    """Cache latents: N(0, 1) with 4 channels 8 times as large, the caches' distribution."""
    x = torch.randn(rows, LATENT, generator=g, device="cuda")
    x[:, torch.randperm(LATENT, generator=g, device="cuda")[:4]] *= 8
    return x


def _page_table(g, need, width, total):
    """Pages of each request in a random order of the pool, -1 behind them."""
    order = torch.randperm(total, generator=g, device="cuda").int()
    start = torch.cumsum(need, 0) - need
    col = torch.arange(width, device="cuda")[None, :]
    table = order[(start[:, None] + col).clamp(max=total - 1)]
    return torch.where(col < need[:, None], table, torch.full_like(table, -1))


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    c = dict(case)
    if c["op"] == "linear":
        x = torch.randn(c["m"], c["k"], generator=g, device="cuda")
        x[:, torch.randperm(c["k"], generator=g, device="cuda")[:4]] *= 8       # outlier channels
        w = torch.randn(c["n"], c["k"], generator=g, device="cuda") / math.sqrt(c["k"])
        code, _, byte = _quantise(w, c["fmt"])
        return dict(case=c, x=x.bfloat16(), w_codes=_pack(code), w_scales=byte.contiguous(),
                    x_codes=torch.empty(c["m"], c["k"] // 2, dtype=torch.uint8, device="cuda"),
                    x_scales=torch.empty(c["m"], c["k"] // _block(c["fmt"]), dtype=torch.uint8, device="cuda"),
                    out=torch.empty(c["m"], c["n"], dtype=torch.bfloat16, device="cuda"))
    if c["op"] == "maps":
        b, page = c["b"], c["page"]
        old = torch.randint(0, c["most_old"] + 1, (b,), generator=g, device="cuda", dtype=torch.int32)
        new = old + (1 if c["most_new"] == 1 else
                     torch.randint(0, c["most_new"] + 1, (b,), generator=g, device="cuda", dtype=torch.int32))
        have = (old // RATIO + page - 1) // page
        want = (new // RATIO + page - 1) // page
        # the arrays have room for the longest step of b requests; this step fills a part of them
        width = ((c["most_old"] + c["most_new"]) // RATIO + page - 1) // page
        held, fresh = b * width, int((want - have).sum())
        table = _page_table(g, have.long(), max(width, 1), held)
        free = held + torch.randperm(fresh + 7, generator=g, device="cuda").int()
        cap_tokens = b * c["most_new"]
        cap_entries = b * ((c["most_new"] + RATIO - 1) // RATIO)
        i32, i64 = dict(dtype=torch.int32, device="cuda"), dict(dtype=torch.int64, device="cuda")
        return dict(case=c, old=old, new=new, table=table.contiguous(), free=free.contiguous(),
                    cap_tokens=cap_tokens, cap_entries=cap_entries,
                    free_next=torch.full((1,), 3, **i32), free_next_out=torch.empty(1, **i32),
                    n_entries=torch.empty(b, **i32), swa_len=torch.empty(b, **i32),
                    entry_off=torch.empty(b + 1, **i64), entry_rows=torch.empty(cap_entries, **i64),
                    token_off=torch.empty(b + 1, **i64), window_rows=torch.empty(cap_tokens, **i64),
                    q_pos=torch.empty(cap_tokens, **i32))
    if c["op"] == "ids":
        b, t, k, page, n = c["b"], c["t"], c["k"], c["page"], c["n"]
        width = (n + page - 1) // page
        lens = torch.randint((n + 1) // 2, n + 1, (b,), generator=g, device="cuda", dtype=torch.int32)
        table = _page_table(g, ((lens + page - 1) // page).long(), width, b * width)
        ids = (torch.rand(b, t, k, generator=g, device="cuda") * lens[:, None, None]).int()
        ids = torch.minimum(ids, lens[:, None, None] - 1)
        keep = torch.randint(max(k // 2, 1), k + 1, (b, t, 1), generator=g, device="cuda")
        ids = torch.where(torch.arange(k, device="cuda") < keep, ids, torch.full_like(ids, -1))
        ids = ids.reshape(b * t, k).contiguous()
        return dict(case=c, ids=ids, table=table.contiguous(), out=torch.empty_like(ids))
    # prefix
    groups, rows, heads, n, page = c["groups"], c["rows"], c["heads"], c["n"], c["page"]
    cut = torch.randperm(rows - 1, generator=g, device="cuda")[:groups - 1].sort().values + 1 if groups > 1 else \
        torch.zeros(0, dtype=torch.int64, device="cuda")
    row_start = torch.cat((cut.new_zeros(1), cut, cut.new_full((1,), rows))).int()
    lens = torch.full((groups,), n, dtype=torch.int32, device="cuda")
    if groups > 1:                                     # the first group has the longest prefix
        lens[1:] = torch.randint((n + 1) // 2, n + 1, (groups - 1,), generator=g, device="cuda", dtype=torch.int32)
    width = (n + page - 1) // page
    total = groups * width
    table = _page_table(g, ((lens + page - 1) // page).long(), width, total)
    code, _, byte = _quantise(_latents(g, total * page), "e4m3")
    kv = torch.cat((_pack(code), byte), dim=1).contiguous()
    q = torch.randn(rows, heads, LATENT, generator=g, device="cuda").bfloat16()
    own_out = torch.randn(rows, heads, LATENT, generator=g, device="cuda") * 0.2
    own_lse = 8.0 + torch.randn(rows, heads, generator=g, device="cuda")
    most_rows = int((row_start[1:] - row_start[:-1]).max())
    return dict(case=c, q=q, row_start=row_start, most_rows=most_rows, lens=lens, table=table.contiguous(), kv=kv,
                scale=1.0 / math.sqrt(LATENT), own_out=own_out, own_lse=own_lse,
                out=torch.empty(rows, heads, LATENT, dtype=torch.bfloat16, device="cuda"),
                lse=torch.empty(rows, heads, device="cuda"))


# --------------------------------------------------------------------------------------------
# plain forms
# --------------------------------------------------------------------------------------------
def _linear(s):
    fmt = s["case"]["fmt"]
    code, scale, _ = _quantise(s["x"], fmt)
    w = _values(_unpack(s["w_codes"]), _scale_values(s["w_scales"], fmt))
    return (_values(code, scale) @ w.t()).bfloat16()


def _maps(s):
    page = s["case"]["page"]
    old, new, dev = s["old"].long(), s["new"].long(), s["old"].device
    b, width = s["table"].shape
    e0, e1 = old // RATIO, new // RATIO
    have, want = (e0 + page - 1) // page, (e1 + page - 1) // page
    need = want - have
    first = torch.cumsum(need, 0) - need + s["free_next"].long()
    # the new pages into the table
    col = torch.arange(width, device=dev)[None, :]
    fresh = (col >= have[:, None]) & (col < want[:, None])
    at = (first[:, None] + col - have[:, None]).clamp(0, s["free"].numel() - 1)
    table = torch.where(fresh, s["free"][at], s["table"])
    zero = old.new_zeros(1)
    # rows of the new entries
    entry_off = torch.cat((zero, torch.cumsum(e1 - e0, 0)))
    i = torch.arange(s["cap_entries"], device=dev)
    r = torch.searchsorted(entry_off[1:], i, right=True).clamp(max=b - 1)
    e = e0[r] + i - entry_off[r]
    rows = table[r, (e // page).clamp(max=width - 1)].long() * page + e % page
    entry_rows = torch.where(i < entry_off[b], rows, torch.full_like(rows, -1))
    # window slots and positions of the new tokens
    token_off = torch.cat((zero, torch.cumsum(new - old, 0)))
    i = torch.arange(s["cap_tokens"], device=dev)
    r = torch.searchsorted(token_off[1:], i, right=True).clamp(max=b - 1)
    p = old[r] + i - token_off[r]
    live = i < token_off[b]
    window_rows = torch.where(live & (p >= new[r] - WINDOW), r * WINDOW + p % WINDOW, torch.full_like(p, -1))
    q_pos = torch.where(live, p, torch.full_like(p, -1)).int()
    return dict(table=table, free_next=(s["free_next"] + need.sum()).int(), n_entries=e1.int(),
                swa_len=new.clamp(max=WINDOW).int(), entry_off=entry_off, entry_rows=entry_rows,
                token_off=token_off, window_rows=window_rows, q_pos=q_pos)


def _ids(s):
    c, ids = s["case"], s["ids"].long()
    seq = torch.arange(ids.shape[0], device=ids.device)[:, None] // c["t"]
    at = ids.clamp(min=0)
    rows = s["table"][seq, at // c["page"]].long() * c["page"] + at % c["page"]
    return torch.where(ids < 0, ids, rows).int()


def _prefix(s):
    c, q = s["case"], s["q"].float()
    rows, heads, _ = q.shape
    lens, start = s["lens"].long(), s["row_start"].long()
    width, page = s["table"].shape[1], c["page"]
    # every group's entries, as far as the longest prefix; the query rows of each group, padded
    j = torch.arange(width * page, device=q.device)
    cache = (s["table"].long()[:, j // page] * page + j % page).clamp(min=0)
    packed = s["kv"][cache.reshape(-1)]
    v = _values(_unpack(packed[:, :256]), _scale_values(packed[:, 256:].contiguous(), "e4m3"))
    v = v.reshape(cache.shape[0], -1, LATENT)
    count = start[1:] - start[:-1]
    i = torch.arange(rows, device=q.device)
    group = torch.searchsorted(start[1:], i, right=True)
    place = i - start[group]
    padded = q.new_zeros(count.shape[0], s["most_rows"], heads, LATENT)
    padded[group, place] = q
    z = padded.reshape(count.shape[0], -1, LATENT) @ v.transpose(1, 2) * s["scale"]
    z = z.masked_fill(j[None, None, :] >= lens[:, None, None], -math.inf)
    m = z.amax(dim=2, keepdim=True)
    p = torch.exp(z - m)
    total = p.sum(dim=2, keepdim=True)
    out = ((p @ v) / total).reshape(count.shape[0], -1, heads, LATENT)[group, place]
    lse = (m + torch.log(total)).reshape(count.shape[0], -1, heads)[group, place]
    # with the rows' own part
    top = torch.maximum(lse, s["own_lse"])
    a, b = torch.exp(lse - top), torch.exp(s["own_lse"] - top)
    out = (out * a[:, :, None] + s["own_out"] * b[:, :, None]) / (a + b)[:, :, None]
    return dict(out=out.bfloat16(), lse=top + torch.log(a + b))


# --------------------------------------------------------------------------------------------
# the library's calls
# --------------------------------------------------------------------------------------------
def _own(s):
    import compressed_sparse_attention_quantize_b200 as csa2
    c = s["case"]
    if c["op"] == "linear":
        m, n, k = c["m"], c["n"], c["k"]
        fmt = csa2.FMT_MXFP4 if c["fmt"] == "mx" else csa2.FMT_FP4
        blocks = k // _block(c["fmt"])
        if "ws" not in s:                                  # a program keeps its workspace
            size = csa2.csa2_fp4_matmul_workspace_size(m, n, k)
            s["ws_bytes"], s["ws"] = size, torch.empty(size, dtype=torch.uint8, device="cuda")
        csa2.csa2_quantize_kv(fmt, s["x"], csa2.DTYPE_BF16, m, k, k, s["x_codes"], k // 2, s["x_scales"], blocks)
        csa2.csa2_fp4_matmul(fmt, s["x_codes"], k // 2, s["x_scales"], blocks, s["w_codes"], k // 2,
                             s["w_scales"], blocks, m, n, k, 1.0, s["out"], csa2.DTYPE_BF16, n,
                             s["ws"], s["ws_bytes"])
        return s["out"]
    if c["op"] == "maps":
        csa2.csa2_page_maps(s["old"], s["new"], c["b"], RATIO, c["page"], WINDOW, s["table"], s["table"].shape[1],
                            s["free"], s["free"].numel(), s["free_next"], s["free_next_out"], s["n_entries"],
                            s["swa_len"], s["entry_off"], s["entry_rows"], s["cap_entries"], s["token_off"],
                            s["window_rows"], s["q_pos"], s["cap_tokens"])
        return dict(table=s["table"], free_next=s["free_next_out"], n_entries=s["n_entries"], swa_len=s["swa_len"],
                    entry_off=s["entry_off"], entry_rows=s["entry_rows"], token_off=s["token_off"],
                    window_rows=s["window_rows"], q_pos=s["q_pos"])
    if c["op"] == "ids":
        csa2.csa2_page_ids(s["ids"], c["b"], c["t"], c["k"], s["table"], s["table"].shape[1], c["page"], s["out"])
        return s["out"]
    rows, heads = c["rows"], c["heads"]
    if "ws" not in s:
        size = csa2.csa2_prefix_attn_workspace_size(rows, heads, c["groups"], c["n"])
        s["ws_bytes"], s["ws"] = size, torch.empty(size, dtype=torch.uint8, device="cuda")
    csa2.csa2_prefix_attn(s["q"], rows, heads, LATENT, s["row_start"], c["groups"], s["kv"], KV_ROW,
                          s["kv"].shape[0], None, s["table"], s["table"].shape[1], c["page"], s["lens"], c["n"],
                          s["scale"], s["own_out"], s["own_lse"], s["out"], csa2.DTYPE_BF16, s["lse"],
                          s["ws"], s["ws_bytes"])
    return dict(out=s["out"], lse=s["lse"])


def run(state):
    if own:
        return _own(state)
    return {"linear": _linear, "maps": _maps, "ids": _ids, "prefix": _prefix}[state["case"]["op"]](state)


# --------------------------------------------------------------------------------------------
# work
# --------------------------------------------------------------------------------------------
def work(case):
    c = case
    if c["op"] == "linear":
        m, n, k = c["m"], c["n"], c["k"]
        return dict(bytes=2 * m * k + n * (k // 2 + k // _block(c["fmt"])) + 2 * m * n, flops=2 * m * n * k)
    if c["op"] == "maps":
        # lengths and per-request results, new pages, and every place of the maps (written to the
        # end); a step's new tokens are half of the most on average
        b, most = c["b"], c["most_new"]
        pages = b * most // (2 * RATIO * c["page"])
        return dict(bytes=b * (8 + 8 + 16) + 8 * pages + b * most * 12 + b * ((most + RATIO - 1) // RATIO) * 8,
                    flops=0)
    if c["op"] == "ids":
        return dict(bytes=c["b"] * (c["t"] * c["k"] * 8 + 4 * ((c["n"] + c["page"] - 1) // c["page"])), flops=0)
    # groups share the rows evenly, prefixes behind the first are three quarters as long, on average
    g, rows, heads, n = c["groups"], c["rows"], c["heads"], c["n"]
    share = (1 + 0.75 * (g - 1)) / g
    return dict(bytes=rows * heads * (LATENT * (2 + 4 + 2) + 8) + share * g * n * KV_ROW,
                flops=4 * rows * heads * share * n * LATENT)


# --------------------------------------------------------------------------------------------
# 64 bits
# --------------------------------------------------------------------------------------------
def _exact_scales(byte, fmt):
    b = byte.to(torch.int64)
    if fmt == "mx":
        return torch.pow(torch.tensor(2.0, dtype=torch.float64, device=b.device), (b - 127).double())
    e, m = b // 8, (b % 8).double()
    return torch.where(e == 0, m / 512, (1 + m / 8) * torch.pow(2.0, (e - 7).double()))


def _exact_codes(packed):
    """Packed E2M1 to float64: sign, two exponent bits with bias 1, one mantissa bit."""
    c = torch.empty(packed.shape[0], 2 * packed.shape[1], dtype=torch.int64, device=packed.device)
    c[:, 0::2], c[:, 1::2] = (packed % 16).long(), (packed // 16).long()
    e, m = (c // 2) % 4, (c % 2).double()
    mag = torch.where(e == 0, m / 2, (1 + m / 2) * torch.pow(2.0, (e - 1).double()))
    return torch.where(c >= 8, -mag, mag)


def _exact_rows(packed, byte, fmt):
    s = _exact_scales(byte, fmt)
    v = _exact_codes(packed)
    return (v.reshape(v.shape[0], s.shape[1], -1) * s[:, :, None]).reshape(v.shape)


def _exact_quantised(x, fmt):
    """x rounded to the format's values: the nearest of the grid, the even code where two are as near."""
    grid = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device=x.device)
    v = x.double().reshape(x.shape[0], -1, _block(fmt))
    top = v.abs().amax(dim=2)
    if fmt == "mx":
        # every scale's power of two, the largest of them at most top / 4
        every = torch.tensor([2.0 ** e for e in range(-127, 128)], dtype=torch.float64, device=x.device)
        s = every[(torch.searchsorted(every, top / 4, right=True) - 1).clamp(min=0)]
    else:
        # every non-negative E4M3 value, the nearest of them to top / 6
        every = _exact_scales(torch.arange(127, dtype=torch.uint8, device=x.device), fmt)
        up = torch.searchsorted(every, top / 6).clamp(1, 126)
        low, high = every[up - 1], every[up]
        d = (top / 6 - low) - (high - top / 6)
        s = torch.where((d > 0) | ((d == 0) & (up % 2 == 0)), high, low)
    a = torch.where(s[:, :, None] > 0, v.abs() / s[:, :, None].clamp(min=1e-300), torch.zeros_like(v))
    up = torch.searchsorted(grid, a.clamp(max=6.0)).clamp(1, 7)
    low, high = grid[up - 1], grid[up]
    d = (a.clamp(max=6.0) - low) - (high - a.clamp(max=6.0))
    mag = torch.where((d > 0) | ((d == 0) & (up % 2 == 0)), high, low)
    return (torch.sign(v) * mag * s[:, :, None]).reshape(x.shape)


def exact(case, seed):
    s = prepare(case, seed)
    c = s["case"]
    if c["op"] == "linear":
        return _exact_quantised(s["x"], c["fmt"]) @ _exact_rows(s["w_codes"], s["w_scales"], c["fmt"]).t()
    if c["op"] in ("maps", "ids"):
        return None                                     # whole numbers: equal or not
    if 4.0 * c["rows"] * c["heads"] * c["n"] * LATENT > 3e11:
        return None                                     # too long in 64 bits
    out, lse = torch.empty(s["q"].shape, dtype=torch.float64, device="cuda"), s["own_lse"].double()
    for i in range(c["groups"]):
        lo, hi, n = int(s["row_start"][i]), int(s["row_start"][i + 1]), int(s["lens"][i])
        j = torch.arange(n, device="cuda")
        rows = s["kv"][s["table"][i, j // c["page"]].long() * c["page"] + j % c["page"]]
        v = _exact_rows(rows[:, :256], rows[:, 256:], "e4m3")
        for r in range(lo, hi):                         # a row's heads at a time bounds the memory
            z = s["q"][r].double() @ v.t() * s["scale"]
            every = torch.cat((z, s["own_lse"][r].double()[:, None]), dim=1)
            p = torch.softmax(every, dim=1)
            out[r] = p[:, :n] @ v + p[:, n:] * s["own_out"][r].double()
            lse[r] = torch.logsumexp(every, dim=1)
    return dict(out=out, lse=lse)
