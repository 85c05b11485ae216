"""The paged KV cache: single-token attention over it (attn_decode_paged) and the writes into it
(attn_cache_append) against the fp64 oracle and plain indexing; and packed prompts, cache and decode steps
run together as a server runs them."""
import math

import numpy as np
import pytest

import oracle
import synth
from packed import (EXP, SUM, U16, assert_lse, assert_within, draw_packed, f64, gpu, host, offsets, reference,
                    score_error)

pytestmark = pytest.mark.gpu


def make_cache(seed, lens, page, Hkv, d, width=None, spare=2, fill=None):
    """A pool with its pages in shuffled order; rows behind a sequence's end and spare pages hold `fill`
    (default: NaN and infinities). Returns device tensors and the contiguous caches in fp64."""
    import torch

    rng = np.random.default_rng(seed)
    need = [-(-n // page) for n in lens]
    width = max(1, max(need)) if width is None else width
    n_pages = sum(need) + spare
    order = rng.permutation(n_pages)
    table = np.full((len(lens), width), -1, dtype=np.int32)
    kc = synth.normal_bf16(seed, synth.STREAM_K, (max(1, sum(lens)), Hkv, d))
    vc = synth.normal_bf16(seed, synth.STREAM_V, (max(1, sum(lens)), Hkv, d))
    bad = gpu(np.array([0x7FC0, 0x7F80, 0xFF80], dtype=np.uint16))  # NaN, inf, -inf
    pool = [torch.empty((n_pages, page, Hkv, d), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    for p in pool:
        if fill is None:
            p.view(-1)[:] = bad[torch.arange(p.numel(), device="cuda") % 3]
        else:
            p.fill_(fill)
    at = row = 0
    for b, n in enumerate(lens):
        ids = order[at:at + need[b]]
        at += need[b]
        table[b, :need[b]] = ids
        for p, c in zip(pool, (kc, vc)):
            flat = torch.full((need[b] * page, Hkv, d), 0.0, dtype=torch.bfloat16, device="cuda")
            idx = torch.from_numpy(ids.astype(np.int64)).cuda()
            if need[b]:
                flat = p[idx].reshape(-1, Hkv, d)
                flat[:n] = gpu(c[row:row + n])
                p[idx] = flat.view(need[b], page, Hkv, d)
        row += n
    return (pool[0], pool[1], torch.from_numpy(table).cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda"),
            f64(kc), f64(vc))


def decode_reference(q, kc, vc, lens, scale):
    """O, LSE and bounds: a packed call with one query per sequence."""
    O, L, bO, bL = reference(q, kc, vc, [1] * len(lens), list(lens), scale, False)
    return O, L.T, bO, bL.T


def _check_decode(lib, seed, lens, page, Hq, Hkv, d, width=None, scale=None):
    import torch

    sc = 1.0 / math.sqrt(d) if scale is None else scale
    kp, vp, table, kv_lens, kc, vc = make_cache(seed, lens, page, Hkv, d, width)
    qb = synth.normal_bf16(seed, synth.STREAM_Q, (len(lens), Hq, d))
    o, lse = lib.attn_decode_paged(gpu(qb), kp, vp, table, kv_lens, scale=sc)
    torch.cuda.synchronize()
    assert lib.attn_get_last_error() == lib.ATTN_OK
    O, L, bO, bL = decode_reference(f64(qb), kc, vc, lens, sc)
    what = f"paged d{d} Hq{Hq} Hkv{Hkv} page{page} {lens[:8]}"
    assert_within(host(o), O, bO, what)
    assert_lse(lse.cpu().numpy().astype(np.float64), L, bL, what)


EDGES = [0, 1, 15, 16, 17, 63, 64, 65, 127, 128, 129, 300]


@pytest.mark.parametrize("d", [32, 64, 128, 256])
@pytest.mark.parametrize("page", [16, 32, 48, 64, 128, 208])
def test_decode_lengths_and_pages(lib, d, page):
    _check_decode(lib, 8000 + d + page, EDGES, page, 8, 2, d)


@pytest.mark.parametrize("d", [32, 64, 128, 256])
@pytest.mark.parametrize("group", [1, 2, 3, 5, 7, 8, 9, 12, 16])
def test_decode_groups(lib, d, group):
    _check_decode(lib, 8100 + d + group, [70, 1, 517, 0], 32, 2 * group, 2, d)


@pytest.mark.parametrize("d,Hkv", [(128, 8), (256, 1), (64, 3)])
def test_decode_long_and_short_together(lib, d, Hkv):
    _check_decode(lib, 8200 + d, [9001, 3, 0, 4097, 64, 1, 2500], 16, 4 * Hkv, Hkv, d, width=4096)


def test_decode_one_long_sequence(lib):
    _check_decode(lib, 8300, [70001], 64, 4, 1, 128)


def test_decode_many_sequences(lib):
    rng = np.random.default_rng(5)
    _check_decode(lib, 8350, [int(x) for x in rng.integers(0, 90, size=1500)], 16, 2, 1, 64)


def test_decode_large_scores(lib):
    _check_decode(lib, 8360, [1000, 33], 16, 4, 2, 128, scale=3.0)


def test_decode_strided_queries_and_shared_pages(lib):
    import torch

    lens, Hq, Hkv, d, page = [200, 200, 130], 8, 2, 128, 16
    kp, vp, table, kv_lens, kc, vc = make_cache(8400, lens, page, Hkv, d)
    table[1] = table[0]  # the second sequence reads the first one's pages
    fused = gpu(synth.normal_bf16(8400, synth.STREAM_Q, (3, Hq + 2 * Hkv, d)))
    q = fused[:, :Hq]
    o, lse = lib.attn_decode_paged(q, kp, vp, table, kv_lens)
    o1, lse1 = lib.attn_decode_paged(q.contiguous(), kp, vp, table, kv_lens)
    assert torch.equal(o, o1) and torch.equal(lse, lse1)
    kc = np.concatenate([kc[:200], kc[:200], kc[400:]])
    vc = np.concatenate([vc[:200], vc[:200], vc[400:]])
    O, L, bO, bL = decode_reference(host(q), kc, vc, lens, 1 / math.sqrt(d))
    assert_within(host(o), O, bO, "shared pages")
    assert_lse(lse.cpu().numpy().astype(np.float64), L, bL, "shared pages")


def test_decode_pool_beyond_32_bit_offsets(lib):
    """A pool of more than 2^31 elements, the sequences' pages at its far end."""
    import torch

    page, Hkv, d = 64, 8, 128
    n_pages = (1 << 31) // (page * Hkv * d) + 40
    lens = [500, 64, 129]
    small = make_cache(8450, lens, page, Hkv, d, spare=0)
    far = n_pages - small[0].shape[0]
    kp = torch.empty((n_pages, page, Hkv, d), dtype=torch.bfloat16, device="cuda")
    vp = torch.empty_like(kp)
    kp[far:], vp[far:] = small[0], small[1]
    table = torch.where(small[2] >= 0, small[2] + far, small[2])
    q = gpu(synth.normal_bf16(8450, synth.STREAM_Q, (3, 16, d)))
    o, lse = lib.attn_decode_paged(q, kp, vp, table, small[3])
    o1, lse1 = lib.attn_decode_paged(q, small[0], small[1], small[2], small[3])
    assert torch.equal(o, o1) and torch.equal(lse, lse1)
    k_new = torch.randn((3, Hkv, d), device="cuda").to(torch.bfloat16)
    lib.attn_cache_append(k_new, -k_new, kp, vp, table, small[3])
    for b, n in enumerate(lens):
        p = int(table[b, (n - 1) // page])
        assert torch.equal(kp[p, (n - 1) % page], k_new[b]) and torch.equal(vp[p, (n - 1) % page], -k_new[b])
    assert lib.attn_get_last_error() == lib.ATTN_OK


def test_decode_bad_lengths_and_pages_are_clamped_and_flagged(lib):
    import torch

    lens, Hq, Hkv, d, page = [40, 100], 4, 2, 64, 16
    kp, vp, table, kv_lens, kc, vc = make_cache(8500, lens, page, Hkv, d, fill=0.0)
    q = gpu(synth.normal_bf16(8500, synth.STREAM_Q, (2, Hq, d)))
    O, _, bO, _ = decode_reference(host(q), kc, vc, lens, 1 / math.sqrt(d))

    def other_row_is_right(o):
        # (the other sequence's length moves the split, so its last bits may move)
        assert_within(host(o)[1], O[1], bO[1], "the other sequence")

    o, _ = lib.attn_decode_paged(q, kp, vp, table, kv_lens)
    assert lib.attn_get_last_error() == lib.ATTN_OK
    other_row_is_right(o)
    low = kv_lens.clone()
    low[0] = -5
    o, lse = lib.attn_decode_paged(q, kp, vp, table, low)
    assert lib.attn_get_last_error() == lib.ATTN_ERR_INVALID_ARG
    assert bool((o[0] == 0).all()) and bool(torch.isneginf(lse[0]).all())
    other_row_is_right(o)
    full = table.clone()
    full[0] = full[1]  # every entry of the row names a page
    high = kv_lens.clone()
    high[0] = 10 ** 9
    o, lse = lib.attn_decode_paged(q, kp, vp, full, high)
    assert lib.attn_get_last_error() == lib.ATTN_ERR_INVALID_ARG
    assert torch.isfinite(o.float()).all()
    other_row_is_right(o)
    for wrong in (-1, kp.shape[0], 2 ** 31 - 1, -2 ** 31):
        t = table.clone()
        t[0, 1] = wrong
        o, _ = lib.attn_decode_paged(q, kp, vp, t, kv_lens)
        assert lib.attn_get_last_error() == lib.ATTN_ERR_INVALID_ARG
        other_row_is_right(o)


def _append_plain(kp, vp, k_new, v_new, table, lens, new):
    page, row = kp.shape[1], 0
    for b, n in enumerate(new):
        for i in range(n):
            t = lens[b] - n + i
            p = int(table[b, t // page])
            kp[p, t % page], vp[p, t % page] = k_new[row], v_new[row]
            row += 1


@pytest.mark.parametrize("page,Hkv,d", [(16, 2, 64), (1, 3, 128), (7, 1, 32), (64, 8, 256), (33, 1, 8)])
def test_append(lib, page, Hkv, d):
    import torch

    lens, new = [40, 0, 129, 1, 65], [40, 0, 2, 1, 64]
    kp, vp, table, kv_lens, _, _ = make_cache(8600 + page, lens, page, Hkv, d, fill=3.0)
    want = [kp.clone(), vp.clone()]
    T = sum(new) + 4  # rows 0 and 1 and the last two belong to nobody
    k_new = torch.randn((T, Hkv, d), device="cuda").to(torch.bfloat16)
    v_new = torch.randn((T, Hkv, d), device="cuda").to(torch.bfloat16)
    lib.attn_cache_append(k_new, v_new, kp, vp, table, kv_lens, cu_seqlens=offsets(new, 2))
    _append_plain(want[0], want[1], k_new[2:], v_new[2:], table, lens, new)
    assert lib.attn_get_last_error() == lib.ATTN_OK
    assert torch.equal(kp, want[0]) and torch.equal(vp, want[1])


@pytest.mark.parametrize("n,Hkv,d", [(120000, 1, 32), (5000, 1, 64), (30000, 1, 128), (9000, 3, 40), (700, 16, 256)])
def test_append_many_rows_of_every_width(lib, n, Hkv, d):
    """Blocks of one row up to as many as they have threads; the last sequences and rows end inside a block."""
    import torch

    page, lens = 16, [n - 1500 if n > 3000 else n - 400, 1, 0, 377]
    table = torch.randperm(-(-n // page) + 8, device="cuda").to(torch.int32)
    need = [-(-x // page) for x in lens]
    rows = torch.full((4, max(need)), -1, dtype=torch.int32, device="cuda")
    for b, m in enumerate(need):
        rows[b, :m] = table[sum(need[:b]):sum(need[:b]) + m]
    kv_lens = torch.tensor(lens, dtype=torch.int32, device="cuda")
    pools = [torch.full((table.numel(), page, Hkv, d), 3.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    want = [p.clone() for p in pools]
    new = [torch.randn((sum(lens) + 5, Hkv, d), device="cuda").to(torch.bfloat16) for _ in range(2)]  # 5 of nobody
    lib.attn_cache_append(*new, *pools, rows, kv_lens, cu_seqlens=offsets(lens))
    at = 0
    for b, m in enumerate(lens):
        t = torch.arange(m, device="cuda")
        for w, x in zip(want, new):
            w[rows[b, t // page].long(), t % page] = x[at:at + m]
        at += m
    assert lib.attn_get_last_error() == lib.ATTN_OK
    assert torch.equal(pools[0], want[0]) and torch.equal(pools[1], want[1])


def test_append_one_row_per_sequence_from_a_fused_projection(lib):
    import torch

    lens, Hkv, d, page = [1, 17, 300, 64], 4, 128, 16
    kp, vp, table, kv_lens, _, _ = make_cache(8700, lens, page, Hkv, d, fill=3.0)
    want = [kp.clone(), vp.clone()]
    fused = torch.randn((4, 16, d), device="cuda").to(torch.bfloat16)
    k_new, v_new = fused[:, 8:12], fused[:, 12:]
    lib.attn_cache_append(k_new, v_new, kp, vp, table, kv_lens)
    _append_plain(want[0], want[1], k_new, v_new, table, lens, [1] * 4)
    assert torch.equal(kp, want[0]) and torch.equal(vp, want[1])


def test_append_leaves_out_and_flags_rows_without_a_place(lib):
    import torch

    lens, Hkv, d, page = [20, 20, 20, 20], 1, 64, 16
    kp, vp, table, kv_lens, _, _ = make_cache(8800, lens, page, Hkv, d, fill=3.0)
    new = torch.ones((4, Hkv, d), dtype=torch.bfloat16, device="cuda")
    assert lib.attn_get_last_error() == lib.ATTN_OK
    for place, wrong in (("len", 0), ("len", -7), ("len", 10 ** 9), ("page", -1), ("page", kp.shape[0])):
        t, n = table.clone(), kv_lens.clone()
        if place == "len":
            n[1] = wrong
        else:
            t[1, 1] = wrong
        got = [kp.clone(), vp.clone()]
        want = [kp.clone(), vp.clone()]
        lib.attn_cache_append(new, new, *got, t, n)
        assert lib.attn_get_last_error() == lib.ATTN_ERR_INVALID_ARG
        for b in (0, 2, 3):
            for w in want:
                w[int(table[b, 1]), 3] = 1.0
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_append_on_another_stream_and_captured(lib):
    """Eager on a side stream, and captured once and replayed with new rows, lengths and pages."""
    import torch

    lens, new, Hkv, d, page = [70, 5, 33], [7, 5, 1], 2, 64, 16
    kp, vp, table, kv_lens, _, _ = make_cache(8850, lens, page, Hkv, d, fill=3.0)
    start, cu = [kp.clone(), vp.clone()], offsets(new)
    rows = [torch.randn((sum(new), Hkv, d), device="cuda").to(torch.bfloat16) for _ in range(2)]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    lib.attn_cache_append(*rows, kp, vp, table, kv_lens, cu_seqlens=cu, stream=side)
    side.synchronize()
    want = [t.clone() for t in start]
    _append_plain(*want, *rows, table, lens, new)
    assert torch.equal(kp, want[0]) and torch.equal(vp, want[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        lib.attn_cache_append(*rows, kp, vp, table, kv_lens, cu_seqlens=cu)
    for lens, new in (([70, 5, 33], [7, 5, 1]), ([64, 6, 1], [12, 0, 1]), ([13, 4, 40], [9, 4, 0])):
        for t in rows:
            t.normal_()
        kv_lens.copy_(torch.tensor(lens, dtype=torch.int32))
        cu.copy_(offsets(new))
        kp.copy_(start[0])
        vp.copy_(start[1])
        graph.replay()
        want = [t.clone() for t in start]
        _append_plain(*want, *rows, table, lens, new)
        assert torch.equal(kp, want[0]) and torch.equal(vp, want[1])
    assert lib.attn_get_last_error() == lib.ATTN_OK
    del graph


def test_decode_on_another_stream_and_in_graphs_that_share_a_workspace(lib):
    """Two graphs over one workspace, replayed one after the other, and eager calls on a side stream."""
    import torch

    Hq, Hkv, d, page = 8, 2, 128, 16
    a = make_cache(8900, [3000, 10, 700], page, Hkv, d)
    b = make_cache(8901, [5, 0, 4000, 64], page, Hkv, d)
    q = [gpu(synth.normal_bf16(8900 + i, synth.STREAM_Q, (n, Hq, d))) for i, n in enumerate((3, 4))]
    want = [lib.attn_decode_paged(x, *c[:4]) for x, c in zip(q, (a, b))]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for x, c, w in zip(q, (a, b), want):
        o, lse = lib.attn_decode_paged(x, *c[:4], stream=side)
        side.synchronize()
        assert torch.equal(o, w[0]) and torch.equal(lse, w[1])
    ws = torch.empty(max(lib.attn_decode_paged_workspace_bytes(n, Hq, Hkv, d) for n in (3, 4)), dtype=torch.uint8,
                     device="cuda")
    graphs, outs = [], []
    for x, c in zip(q, (a, b)):
        g = torch.cuda.CUDAGraph()
        o, lse = torch.empty_like(x), torch.empty((x.shape[0], Hq), device="cuda")
        with torch.cuda.graph(g):
            lib.attn_decode_paged(x, *c[:4], workspace=ws, out=o, lse=lse)
        graphs.append(g)
        outs.append((o, lse))
    for i in (0, 1, 0, 0, 1):
        for t in outs[i]:
            t.zero_()
        graphs[i].replay()
        assert torch.equal(outs[i][0], want[i][0]) and torch.equal(outs[i][1], want[i][1])
    assert lib.attn_get_last_error() == lib.ATTN_OK
    del graphs


def test_prompts_cache_and_decode_steps_together(lib):
    """What a server does: packed prompts through attn_fwd_varlen, their K and V into the cache, then tokens
    one by one (append, decode). Every output equals the oracle's attention over the whole sequence."""
    import torch

    Hq, Hkv, d, page, steps = 8, 2, 128, 16, 5
    prompt = [33, 1, 160]
    total = [n + steps for n in prompt]
    qb, kb, vb = draw_packed(9000, total, total, Hq, Hkv, d)
    first = np.concatenate([[0], np.cumsum(total)])
    _, _, table, _, _, _ = make_cache(9000, total, page, Hkv, d)
    kp = torch.full((int(table.max()) + 1, page, Hkv, d), float("nan"), dtype=torch.bfloat16, device="cuda")
    vp = kp.clone()
    sc = 1 / math.sqrt(d)
    O, L, bO, bL = reference(f64(qb), f64(kb), f64(vb), total, total, sc, True)

    rows = np.concatenate([first[b] + np.arange(n) for b, n in enumerate(prompt)])
    q, k, v = gpu(qb[rows]), gpu(kb[rows]), gpu(vb[rows])
    cu = offsets(prompt)
    lens = torch.tensor(prompt, dtype=torch.int32, device="cuda")
    o, lse = lib.attn_fwd_varlen(q, k, v, cu, causal=True)
    lib.attn_cache_append(k, v, kp, vp, table, lens, cu_seqlens=cu)
    assert_within(host(o), O[rows], bO[rows], "prompts")
    assert_lse(lse.cpu().numpy().astype(np.float64), L[:, rows], bL[:, rows], "prompts")
    for s in range(steps):
        rows = np.array([first[b] + n + s for b, n in enumerate(prompt)])
        lens += 1
        lib.attn_cache_append(gpu(kb[rows]), gpu(vb[rows]), kp, vp, table, lens)
        o, lse = lib.attn_decode_paged(gpu(qb[rows]), kp, vp, table, lens)
        assert_within(host(o), O[rows], bO[rows], f"step {s}")
        assert_lse(lse.cpu().numpy().astype(np.float64), L[:, rows].T, bL[:, rows].T, f"step {s}")
    assert lib.attn_get_last_error() == lib.ATTN_OK
