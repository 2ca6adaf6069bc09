"""csa2_page_maps and csa2_page_ids against plain loops (GPU), and their refusals (CPU).

Every result is a whole number and has to be equal.
"""
import numpy as np
import pytest
import torch

import compressed_sparse_attention_quantize_b200 as csa2
from compressed_sparse_attention_quantize_b200 import build as csa2_build

OK, INVALID, SHAPE, ALIGN = 0, 1, 2, 3


# ---------------------------------------------------------------------------------------------
# plain loops
# ---------------------------------------------------------------------------------------------
def maps_by_loops(old, new, ratio, E, window, table, free, nxt, cap_entries, cap_tokens):
    """The step's maps; also whether anything broke the contract."""
    table = table.copy()
    B, width = table.shape
    entry_rows, window_rows, q_pos = [], [], []
    entry_off, token_off, n_entries, swa_len = [0], [0], [], []
    taken, bad = 0, not 0 <= nxt <= len(free)
    left = len(free) - nxt if not bad else 0
    for b in range(B):
        o, n = int(old[b]), int(new[b])
        bad |= o < 0 or n < o
        o = max(o, 0)
        n = max(n, o)
        e0, e1 = o // ratio, n // ratio
        have, want = -(-e0 // E), -(-e1 // E)
        bad |= want > width
        have, want = min(have, width), min(want, width)
        for p in range(have, want):
            if taken < left:
                table[b, p] = free[nxt + taken]
                taken += 1
            else:
                table[b, p] = -1
                bad = True
        mapped = have + sum(1 for p in range(have, want) if table[b, p] >= 0)
        n_entries.append(min(e1, mapped * E))
        swa_len.append(min(n, window))
        for e in range(e0, e1):
            page = table[b, e // E] if e // E < width else -1
            bad |= page < 0
            entry_rows.append(page * E + e % E if page >= 0 else -1)
        for p in range(o, n):
            window_rows.append(b * window + p % window if p >= n - window else -1)
            q_pos.append(p)
        entry_off.append(len(entry_rows))
        token_off.append(len(q_pos))
    bad |= len(entry_rows) > cap_entries or len(q_pos) > cap_tokens

    def cut(v, cap):
        return np.array((v + [-1] * cap)[:cap], np.int64)
    return dict(table=table, free_next=[nxt + taken if 0 <= nxt <= len(free) else nxt], n_entries=n_entries,
                swa_len=swa_len, entry_off=entry_off, entry_rows=cut(entry_rows, cap_entries), token_off=token_off,
                window_rows=cut(window_rows, cap_tokens), q_pos=cut(q_pos, cap_tokens)), bad


def run_maps(old, new, ratio, E, window, table, free, nxt, cap_entries, cap_tokens, shift=0, optional=True):
    """The call on fresh device buffers (`shift`: element offset of the maps, against 16-byte bases)."""
    dev = dict(device="cuda")
    B = len(old)
    i32 = lambda v: torch.tensor(np.asarray(v), dtype=torch.int32, **dev)                 # noqa: E731
    t = i32(table)
    out = {"table": t, "free_next": torch.full((1,), -77, dtype=torch.int32, **dev),
           "n_entries": torch.full((B,), -77, dtype=torch.int32, **dev),
           "swa_len": torch.full((B,), -77, dtype=torch.int32, **dev) if optional else None,
           "entry_off": torch.full((B + 1,), -77, dtype=torch.int64, **dev),
           "token_off": torch.full((B + 1,), -77, dtype=torch.int64, **dev),
           "entry_rows": torch.full((cap_entries + shift + 3,), -77, dtype=torch.int64, **dev),
           "window_rows": torch.full((cap_tokens + shift + 3,), -77, dtype=torch.int64, **dev),
           "q_pos": torch.full((cap_tokens + shift + 3,), -77, dtype=torch.int32, **dev)}
    cut = {k: out[k][shift:] for k in ("entry_rows", "window_rows", "q_pos")}
    csa2.csa2_page_maps(i32(old), i32(new), B, ratio, E, window, t, t.shape[1], i32(free), len(free), i32([nxt]),
                        out["free_next"], out["n_entries"], out["swa_len"], out["entry_off"], cut["entry_rows"],
                        cap_entries, out["token_off"], cut["window_rows"] if optional else None,
                        cut["q_pos"] if optional else None, cap_tokens)
    err = csa2.csa2_device_error()
    got = {k: v.cpu().numpy() for k, v in out.items() if v is not None}
    for k, cap in (("entry_rows", cap_entries), ("window_rows", cap_tokens), ("q_pos", cap_tokens)):
        assert (got[k][:shift] == -77).all() and (got[k][shift + cap:] == -77).all(), f"{k}: written outside"
        got[k] = got[k][shift:shift + cap]
    return got, err


def check_maps(got, ref, optional=True):
    for k, v in ref.items():
        if optional or k not in ("swa_len", "window_rows", "q_pos"):
            assert np.array_equal(got[k], np.asarray(v)), k


def random_step(rng, B, most_old, most_new, ratio, E, spare=5):
    old = rng.integers(0, most_old + 1, B)
    new = old + rng.integers(0, most_new + 1, B)
    have = -(-(old // ratio) // E)
    want = -(-(new // ratio) // E)
    width = max(int(want.max()), 1)
    pages = rng.permutation(int(have.sum() + (want - have).sum()) + spare + 4)
    table = np.full((B, width), -1, np.int64)
    at = 0
    for b in range(B):
        table[b, :have[b]] = pages[at:at + have[b]]
        at += have[b]
    free = pages[at:]
    return old, new, table, free


@pytest.mark.gpu
@pytest.mark.parametrize("B,most_old,most_new,ratio,E,window", [
    (1, 0, 1, 4, 64, 128), (1, 0, 0, 4, 16, 128), (1, 3, 1, 4, 1, 128), (32, 5000, 1, 4, 64, 128),
    (7, 300, 500, 4, 5, 128), (33, 100, 40, 1, 3, 7), (257, 60, 9, 64, 2, 1), (300, 2000, 300, 4, 48, 128),
    (4096, 20, 6, 4, 2, 128), (3, 20000, 9000, 4, 100, 128)])
def test_maps(B, most_old, most_new, ratio, E, window):
    rng = np.random.default_rng(B * 1000 + most_new)
    old, new, table, free = random_step(rng, B, most_old, most_new, ratio, E)
    tokens, entries = int((new - old).sum()), int((new // ratio - old // ratio).sum())
    for shift, more in ((0, 0), (1, 9)):                   # 16-byte bases and not; exact and longer maps
        args = (old, new, ratio, E, window, table, free, 2, entries + more, tokens + more)
        ref, bad = maps_by_loops(*args)
        got, err = run_maps(*args, shift=shift)
        assert not bad and err == 0
        check_maps(got, ref)
    got, err = run_maps(*args, optional=False)
    assert err == 0
    check_maps(got, ref, optional=False)


@pytest.mark.gpu
@pytest.mark.parametrize("what", ["pages", "width", "shrinks", "negative", "caps", "next", "next-neg", "hole"])
def test_maps_broken_contract(what):
    """Nothing outside the buffers is written, the error word says SHAPE and the call after it is clean."""
    rng = np.random.default_rng(5)
    old, new, table, free = random_step(rng, 9, 200, 90, 4, 4)
    nxt = 2
    tokens, entries = int((new - old).sum()), int((new // 4 - old // 4).sum())
    cap_e, cap_t = entries, tokens
    if what == "pages":
        free = free[:nxt + 3]
    elif what == "width":
        table = table[:, :max(table.shape[1] // 2, 1)]
    elif what == "shrinks":
        new[3] = old[3] - 1
    elif what == "negative":
        old[3], new[3] = -5, 10
        table[3] = -1
    elif what == "caps":
        cap_e, cap_t = entries - 5, tokens - 6
    elif what == "next":
        nxt = len(free) + 1
    elif what == "next-neg":
        nxt = -1
    else:                                                  # a held page that is not there
        b = int(np.argmax((old // 4) % 4 * (new // 4 > old // 4)))
        table[b, (old[b] // 4) // 4] = -1
    args = (old, new, 4, 4, 128, table, free, nxt, cap_e, cap_t)
    ref, bad = maps_by_loops(*args)
    got, err = run_maps(*args)
    assert bad and err == csa2.CSA2_ERR_SHAPE
    if what in ("caps", "hole"):
        ref["n_entries"] = got["n_entries"] if what == "hole" else ref["n_entries"]
    check_maps(got, ref)
    assert csa2.csa2_device_error() == 0


@pytest.mark.gpu
def test_maps_two_steps_in_a_graph():
    """Two steps captured one after the other, the second reading the first's list position; the
    replay on other lengths equals the loops, with the maps' unused ends at -1."""
    rng = np.random.default_rng(11)
    B, E, W, cap_t, cap_e = 12, 3, 128, 700, 200
    dev = dict(device="cuda")
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32, **dev)                            # noqa: E731
    i64 = lambda *s: torch.zeros(*s, dtype=torch.int64, **dev)                            # noqa: E731
    lens, table, free, nxt = i32(3, B), i32(B, 64), i32(400), i32(3)
    outs = [dict(n=i32(B), sl=i32(B), eo=i64(B + 1), er=i64(cap_e), to=i64(B + 1), wr=i64(cap_t), qp=i32(cap_t))
            for _ in range(2)]

    def step(i):
        o = outs[i]
        csa2.csa2_page_maps(lens[i], lens[i + 1], B, 4, E, W, table, 64, free, 400, nxt[i:], nxt[i + 1:], o["n"],
                            o["sl"], o["eo"], o["er"], cap_e, o["to"], o["wr"], o["qp"], cap_t)
    g = torch.cuda.CUDAGraph()
    step(0)
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        step(0)
        step(1)
    for seed in (1, 2):
        rng = np.random.default_rng(seed)
        L0 = rng.integers(0, 300, B)
        L1 = L0 + rng.integers(0, 50, B)
        L2 = L1 + rng.integers(0, 50, B)
        pages = rng.permutation(B * 64 + 400)
        T, F = pages[:B * 64].reshape(B, 64), pages[B * 64:]
        lens.copy_(torch.tensor(np.stack([L0, L1, L2])))
        table.copy_(torch.tensor(T))
        free.copy_(torch.tensor(F))
        nxt.copy_(torch.tensor([4, 0, 0]))
        g.replay()
        torch.cuda.synchronize()
        r1, bad1 = maps_by_loops(L0, L1, 4, E, W, T, F, 4, cap_e, cap_t)
        r2, bad2 = maps_by_loops(L1, L2, 4, E, W, r1["table"], F, r1["free_next"][0], cap_e, cap_t)
        assert not bad1 and not bad2 and csa2.csa2_device_error() == 0
        assert np.array_equal(table.cpu().numpy(), r2["table"])
        assert nxt.cpu().tolist() == [4] + list(r1["free_next"]) + list(r2["free_next"])
        for o, r in zip(outs, (r1, r2)):
            assert np.array_equal(o["er"].cpu().numpy(), r["entry_rows"])
            assert np.array_equal(o["wr"].cpu().numpy(), r["window_rows"])
            assert np.array_equal(o["qp"].cpu().numpy(), r["q_pos"])


@pytest.mark.gpu
@pytest.mark.parametrize("B,T,K,E,width", [(1, 1, 1, 1, 1), (32, 1, 2048, 64, 512), (3, 5, 37, 48, 9), (2, 300, 64, 7, 11),
                                           (1, 2, 4096, 1 << 20, 3), (5, 1, 1028, 3, 700), (1, 70000, 4, 16, 2)])
def test_ids(B, T, K, E, width):
    rng = np.random.default_rng(K)
    table = rng.permutation(min(B * width + 3, 2047))[:B * width].reshape(B, width) if B * width <= 2047 else \
        rng.integers(0, 2047, (B, width))
    ids = rng.integers(0, min(width * E, 2 ** 31 - 1), (B * T, K))
    ids[rng.random((B * T, K)) < 0.2] = -1
    ref = np.where(ids < 0, -1, table[np.arange(B * T)[:, None] // T, np.maximum(ids, 0) // E] * E + np.maximum(ids, 0) % E)
    fits = ref <= 2 ** 31 - 1
    for shift in (0, 1):                                   # 16-byte bases and not
        raw = torch.full((B * T * K + shift + 4,), -9, dtype=torch.int32, device="cuda")
        raw[shift:shift + B * T * K] = torch.tensor(ids.reshape(-1), dtype=torch.int32)
        view = raw[shift:]
        csa2.csa2_page_ids(view, B, T, K, torch.tensor(table, dtype=torch.int32, device="cuda"), width, E, view)
        assert csa2.csa2_device_error() == (0 if fits.all() else csa2.CSA2_ERR_INVALID_ARG)
        got = raw.cpu().numpy()
        assert np.array_equal(got[shift:shift + B * T * K].reshape(B * T, K), np.where(fits, ref, -1))
        assert (got[:shift] == -9).all() and (got[shift + B * T * K:] == -9).all()


@pytest.mark.gpu
def test_ids_division_at_its_ends():
    """Every page size's quotients next to multiples, up to the largest id."""
    rng = np.random.default_rng(3)
    for E in [1, 2, 3, 5, 7, 11, 64, 641, 65535, 65536, 65537, (1 << 20) - 1, 1 << 20] + list(rng.integers(2, 1 << 20, 20)):
        E = int(E)
        width = min(1 << 16, (2 ** 31 - 1) // E + 1)
        top = min(width * E, 2 ** 31) - 1
        k = rng.integers(0, top // E + 1, 500) * E
        ids = np.clip(np.concatenate([k - 1, k, k + 1, [0, top, top - 1]]), 0, top)
        table = np.arange(width)                           # identity: the row of an id is the id
        out = torch.empty(ids.size, dtype=torch.int32, device="cuda")
        csa2.csa2_page_ids(torch.tensor(ids, dtype=torch.int32, device="cuda"), 1, 1, ids.size,
                           torch.tensor(table, dtype=torch.int32, device="cuda"), width, E, out)
        assert np.array_equal(out.cpu().numpy(), ids), E
    assert csa2.csa2_device_error() == 0


@pytest.mark.gpu
def test_ids_bad_ids_and_pages():
    table = torch.tensor([[5, -1, 7]], dtype=torch.int32, device="cuda")
    ids = torch.tensor([[0, 9, 10, 29, 30, -4, 2 ** 31 - 1]], dtype=torch.int32, device="cuda")
    out = torch.empty_like(ids)
    csa2.csa2_page_ids(ids, 1, 1, 7, table, 3, 10, out)
    assert out.tolist() == [[50, 59, -1, 79, -1, -1, -1]]
    assert csa2.csa2_device_error() == csa2.CSA2_ERR_INVALID_ARG
    assert csa2.csa2_device_error() == 0


# ---------------------------------------------------------------------------------------------
# refusals (no launch)
# ---------------------------------------------------------------------------------------------
@pytest.fixture(scope="module")
def L():
    csa2_build.build()
    return csa2.lib()


def test_maps_refusals(L):
    names = ("old", "new", "B", "ratio", "E", "window", "table", "max_pages", "free", "n_free", "next", "next_out",
             "n_entries", "swa_len", "entry_off", "entry_rows", "cap_entries", "token_off", "window_rows", "q_pos",
             "cap_tokens", "stream")
    good = dict(zip(names, (16, 16, 4, 4, 64, 128, 16, 8, 16, 8, 16, 32, 48, 64, 16, 16, 9, 16, 16, 16, 9, None)))

    def call(**kw):
        a = {**good, **kw}
        return L.csa2_page_maps(*[a[n] for n in names])
    for k in ("B", "ratio", "E", "window", "max_pages"):
        assert call(**{k: 0}) == SHAPE
    assert call(B=4097) == SHAPE
    assert call(E=(1 << 20) + 1) == SHAPE and call(window=(1 << 20) + 1) == SHAPE
    for k in ("n_free", "cap_entries", "cap_tokens"):
        assert call(**{k: -1}) == SHAPE
    for k in ("old", "new", "table", "free", "next", "next_out", "n_entries", "entry_off", "entry_rows", "token_off"):
        assert call(**{k: None}) == INVALID
    assert call(next_out=16) == INVALID                     # the position's two words are one
    assert call(n_entries=16) == INVALID and call(swa_len=16) == INVALID and call(swa_len=48) == INVALID
    for k in ("old", "new", "table", "free", "next", "next_out", "n_entries", "swa_len", "q_pos"):
        assert call(**{k: 18}) == ALIGN
    for k in ("entry_off", "entry_rows", "token_off", "window_rows"):
        assert call(**{k: 20}) == ALIGN


def test_ids_refusals(L):
    def call(ids=16, B=2, T=1, K=8, table=16, max_pages=4, E=64, out=16):
        return L.csa2_page_ids(ids, B, T, K, table, max_pages, E, out, None)
    assert call(ids=None) == INVALID and call(table=None) == INVALID and call(out=None) == INVALID
    assert call(B=0) == SHAPE and call(T=0) == SHAPE and call(K=0) == SHAPE and call(max_pages=0) == SHAPE
    assert call(E=0) == SHAPE and call(E=(1 << 20) + 1) == SHAPE and call(B=1 << 16, T=1 << 16) == SHAPE
    assert call(ids=18) == ALIGN and call(table=18) == ALIGN and call(out=18) == ALIGN
