"""Packed sequences of different lengths (attn_fwd_varlen, attn_bwd_varlen) against the fp64 oracle,
sequence by sequence: lengths from zero up, ragged tiles, Nq != Nkv, every head dim, strided operands,
rows that belong to nobody, offsets out of order, graphs and streams."""
import math

import numpy as np
import pytest

import oracle
import synth
from packed import (assert_lse, assert_within, draw_packed, f64, gpu, grad_bounds, host, offsets, reference,
                    sequences)
from parity import assert_grad_parity

pytestmark = pytest.mark.gpu

STREAM_DO = 5


def _check_forward(lib, seed, ql, kl, Hq, Hkv, d, causal, scale=None):
    import torch

    sc = 1.0 / math.sqrt(d) if scale is None else scale
    qb, kb, vb = draw_packed(seed, ql, kl, Hq, Hkv, d)
    cu_q = offsets(ql)
    cu_k = cu_q if ql == kl else offsets(kl)
    o, lse = lib.attn_fwd_varlen(gpu(qb), gpu(kb), gpu(vb), cu_q, cu_k, scale=sc, causal=causal)
    torch.cuda.synchronize()
    assert lib.attn_get_last_error() == lib.ATTN_OK
    O, L, bO, bL = reference(f64(qb), f64(kb), f64(vb), ql, kl, sc, causal)
    what = f"packed d{d} Hq{Hq} Hkv{Hkv} {ql} {kl} causal={causal}"
    n = sum(ql)
    assert_within(host(o)[:n], O[:n], bO[:n], what)
    assert_lse(lse.cpu().numpy().astype(np.float64)[:, :n], L[:, :n], bL[:, :n], what)


SAME = [
    ([1], 2, 1),
    ([1, 17, 64, 0, 129], 4, 2),
    ([128, 127, 256, 257, 255, 1], 2, 2),
    ([0, 0, 3, 0], 3, 1),
    ([700, 33], 2, 1),
]


@pytest.mark.parametrize("d", [32, 64, 128, 256])
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("case", range(len(SAME)))
def test_forward(lib, d, causal, case):
    lens, Hq, Hkv = SAME[case]
    _check_forward(lib, 7000 + 10 * case + d + int(causal), lens, lens, Hq, Hkv, d, causal)


MIXED = [
    ([1, 1, 1], [1, 130, 500], 4, 1),           # single tokens over earlier keys
    ([300, 5, 129], [100, 260, 0], 2, 1),       # more queries than keys: rows that see none; no keys at all
    ([0, 64, 200], [77, 640, 201], 4, 4),       # keys without queries
    ([513], [1025], 8, 1),
    ([384, 300], [10, 300], 2, 2),              # a whole first query tile without keys
]


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("case", range(len(MIXED)))
def test_forward_more_or_fewer_keys_than_queries(lib, d, causal, case):
    ql, kl, Hq, Hkv = MIXED[case]
    _check_forward(lib, 7200 + 10 * case + d + int(causal), ql, kl, Hq, Hkv, d, causal)


@pytest.mark.parametrize("d", [64, 128])
def test_forward_many_short_sequences(lib, d):
    rng = np.random.default_rng(d)
    lens = [int(x) for x in rng.integers(0, 6, size=3000)]
    _check_forward(lib, 7300 + d, lens, lens, 2, 1, d, True)


CUT = [
    ([40, 300], [9000, 4500], 2, 1),            # two blocks with many keys: each cut into parts
    ([1], [20011], 1, 1),                       # one query: as many parts as there are shares
    ([512, 3, 256], [2600, 129, 6000], 4, 2),   # whole blocks and cut ones together
    ([2000], [2100], 3, 1),                     # causal: early blocks short, late ones cut
    ([700], [5000], 16, 4),
]


@pytest.mark.parametrize("d", [32, 64, 128, 256])
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("case", range(len(CUT)))
def test_forward_keys_cut_into_parts(lib, d, causal, case):
    ql, kl, Hq, Hkv = CUT[case]
    _check_forward(lib, 7350 + 10 * case + d + int(causal), ql, kl, Hq, Hkv, d, causal)


PLANNED = [
    [5] * 40 + [2600] + [1] * 3,                # 8 threads of the plan to a sequence, one of 11 blocks
    [8300, 3],                                  # a warp to a sequence, one of 33 blocks
    [1] * 127 + [300],
    [2] * 129 + [2400],                         # a thread to a sequence, a warp to the long one
]


@pytest.mark.parametrize("case", range(len(PLANNED)))
def test_forward_plans_of_every_kind(lib, case):
    _check_forward(lib, 7140 + case, PLANNED[case], PLANNED[case], 1, 1, 64, True)


FEW_QUERIES = [
    ([64], [6000], 8, 1),                       # one block, units of two heads: their keys in many parts
    ([1, 0, 126, 1], [2500, 40, 1999, 3], 6, 3),
    ([128], [3000], 4, 4),                      # no second head in the group
    ([3] * 40, [50] * 39 + [2000], 16, 2),      # more blocks than CTAs, fewer units than twice that
]


@pytest.mark.parametrize("d", [32, 64, 128, 256])
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("case", range(len(FEW_QUERIES)))
def test_forward_few_queries_over_many_keys(lib, d, causal, case):
    ql, kl, Hq, Hkv = FEW_QUERIES[case]
    _check_forward(lib, 7150 + 10 * case + d + int(causal), ql, kl, Hq, Hkv, d, causal)


@pytest.mark.parametrize("d", [128, 256])
def test_parts_do_not_take_rows_of_others(lib, d):
    """Blocks cut into parts beside sequences of NaN, and rows that see keys of the last part only (more queries
    than keys would give none): finite results, the rows of nobody left as they were."""
    import torch

    ql, kl, Hq, Hkv, pad = [130, 64], [5000, 3003], 2, 1, 3
    qb, kb, vb = draw_packed(7390 + d, ql, kl, Hq, Hkv, d)

    def surrounded(bits, heads):
        t = torch.full((bits.shape[0] + 2 * pad, heads, d), float("nan"), dtype=torch.bfloat16, device="cuda")
        t[pad:-pad] = gpu(bits)
        return t

    q, k, v = surrounded(qb, Hq), surrounded(kb, Hkv), surrounded(vb, Hkv)
    k[pad:pad + kl[0]], v[pad:pad + kl[0]] = float("nan"), float("inf")  # the first sequence: NaN throughout
    o = torch.full_like(q, 7.0)
    lse = torch.full((Hq, q.shape[0]), 7.0, device="cuda")
    lib.attn_fwd_varlen(q, k, v, offsets(ql, pad), offsets(kl, pad), causal=True, out=o, lse=lse)
    sc = 1 / math.sqrt(d)
    a, b = list(sequences(ql, kl))[1]
    O, L, bO, bL = reference(f64(qb)[a], f64(kb)[b], f64(vb)[b], [64], [3003], sc, True)
    own = slice(pad + a.start, pad + a.stop)
    assert_within(host(o[own].contiguous()), O, bO, "beside NaN")
    assert_lse(lse[:, own].cpu().numpy().astype(np.float64), L, bL, "beside NaN")
    for x in (o[:pad], o[-pad:], lse[:, :pad], lse[:, -pad:]):
        assert bool((x == 7.0).all())
    assert bool(torch.isnan(o[pad:pad + 130].float()).all())  # NaN keys give NaN, not a number
    assert lib.attn_get_last_error() == lib.ATTN_OK


def test_forward_large_scores_and_groups(lib):
    _check_forward(lib, 7400, [260, 70], [260, 70], 16, 1, 128, True, scale=2.0)


def _backward(lib, qb, kb, vb, dob, ql, kl, sc, causal):
    import torch

    cu_q, cu_k = offsets(ql), offsets(kl)
    q, k, v, do = gpu(qb), gpu(kb), gpu(vb), gpu(dob)
    o, lse = lib.attn_fwd_varlen(q, k, v, cu_q, cu_k, scale=sc, causal=causal)
    grads = lib.attn_bwd_varlen(q, k, v, o, lse, do, cu_q, cu_k, scale=sc, causal=causal)
    torch.cuda.synchronize()
    assert lib.attn_get_last_error() == lib.ATTN_OK
    return [host(g) for g in grads]


BACKWARD = [
    ([1], [1], 1, 1),
    ([1, 17, 64, 0, 129], [1, 17, 64, 0, 129], 4, 2),
    ([128, 127, 256, 257, 1], [128, 127, 256, 257, 1], 2, 2),
    ([300, 5, 129], [100, 260, 0], 2, 1),
    ([0, 64, 200, 3], [77, 640, 201, 129], 4, 1),
    ([384, 300], [10, 300], 2, 1),
    ([1500], [1400], 8, 1),                     # few key blocks with many steps: each cut into parts
    ([2500, 3], [130, 40], 2, 2),
    ([40] * 300, [40] * 300, 2, 2),             # many blocks, none of them cut
    ([30] * 40, [20] * 39 + [1500], 1, 1),      # 8 threads of the plan to a sequence, one of 12 blocks
]


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("case", range(len(BACKWARD)))
def test_backward(lib, causal, case):
    ql, kl, Hq, Hkv = BACKWARD[case]
    d, sc = 128, 1.0 / math.sqrt(128)
    seed = 7500 + 10 * case + int(causal)
    qb, kb, vb = draw_packed(seed, ql, kl, Hq, Hkv, d)
    dob = synth.normal_bf16(seed, STREAM_DO, qb.shape)
    got = _backward(lib, qb, kb, vb, dob, ql, kl, sc, causal)
    q, k, v, do = f64(qb), f64(kb), f64(vb), f64(dob)
    O, _, bO, _ = reference(q, k, v, ql, kl, sc, causal)
    want, bounds = grad_bounds(q, k, v, do, O, bO, ql, kl, sc, causal)
    for name, g, w, b, n in zip(("dQ", "dK", "dV"), got, want, bounds, (sum(ql), sum(kl), sum(kl))):
        what = f"{name} {ql} {kl} Hq{Hq} Hkv{Hkv} causal={causal}"
        assert_within(g[:n], w[:n], b[:n], what)
        # the RMS gate has a slack of 1e-7 only, below the fp32 sums' own error (d 2^-23 sum |dO V|, about 1e-3 at
        # worst) where a gradient vanishes altogether (every row sees one key: dS = P (dP - D) = 0)
        if n and np.abs(w[:n]).max() > 0.1:
            assert_grad_parity(g[:n], w[:n], what)


def test_backward_against_differences(lib):
    """The directional derivative of sum(O dO) along random directions, from fp64 differences of the oracle."""
    ql, kl, Hq, Hkv, d, sc = [70, 131], [90, 131], 2, 1, 128, 0.1
    qb, kb, vb = draw_packed(7601, ql, kl, Hq, Hkv, d)
    dob = synth.normal_bf16(7601, STREAM_DO, qb.shape)
    got = _backward(lib, qb, kb, vb, dob, ql, kl, sc, True)
    x, do = [f64(qb), f64(kb), f64(vb)], f64(dob)

    def loss(q, k, v):
        return float((reference(q, k, v, ql, kl, sc, True)[0] * do).sum())

    rng = np.random.default_rng(3)
    O, _, bO, _ = reference(*x, ql, kl, sc, True)
    _, bounds = grad_bounds(*x, do, O, bO, ql, kl, sc, True)
    h = 2.0 ** -14
    for i in range(3):
        u = rng.standard_normal(x[i].shape)
        plus, minus = [list(x), list(x)]
        plus[i], minus[i] = x[i] + h * u, x[i] - h * u
        slope = (loss(*plus) - loss(*minus)) / (2 * h)
        # central differences: relative error about h^2 (2^-28) times third derivatives of order 10^2
        slack = 1e-5 * np.abs(got[i]).sum() + (bounds[i] * np.abs(u)).sum()
        # every element's error may have any sign against u; independent ones add as the root of squares
        spread = 8 * np.sqrt(((bounds[i] * u) ** 2).sum()) + 1e-5 * np.abs(slope) + 1e-3
        assert abs((got[i] * u).sum() - slope) <= min(slack, spread), ("dq", "dk", "dv")[i]


@pytest.mark.parametrize("d", [64, 128, 256])
def test_other_sequences_never_reach_a_result(lib, d):
    """NaN and infinities in every other sequence and in rows of nobody: the sequence's own rows come out as
    they do alone, bit for bit, and the rows of nobody are left as they were."""
    import torch

    lens, Hq, Hkv = [100, 77, 300], 4, 2
    qb, kb, vb = draw_packed(7700 + d, lens, lens, Hq, Hkv, d)
    rows = list(sequences(lens, lens))[1][0]
    pad = 5  # rows before the first and after the last sequence
    bad = torch.tensor([float("nan"), float("inf"), -float("inf")], dtype=torch.bfloat16, device="cuda")

    def spoiled(bits, heads):
        t = bad[torch.arange(sum(lens) + 2 * pad, device="cuda") % 3][:, None, None].expand(-1, heads, d).contiguous()
        t[pad + rows.start:pad + rows.stop] = gpu(bits)[rows]
        return t

    q, k, v = spoiled(qb, Hq), spoiled(kb, Hkv), spoiled(vb, Hkv)
    cu = offsets(lens, pad)
    one = offsets([77])
    alone = [gpu(x)[rows].contiguous() for x in (qb, kb, vb)]
    own = slice(pad + rows.start, pad + rows.stop)
    grown = sum(lens) + pad
    for causal in (False, True):
        o = torch.full((sum(lens) + 2 * pad, Hq, d), 7.0, dtype=torch.bfloat16, device="cuda")
        lse = torch.full((Hq, sum(lens) + 2 * pad), 7.0, dtype=torch.float32, device="cuda")
        lib.attn_fwd_varlen(q, k, v, cu, causal=causal, out=o, lse=lse)
        o1, lse1 = lib.attn_fwd_varlen(*alone, one, causal=causal)
        assert torch.equal(o[own], o1) and torch.equal(lse[:, own], lse1)
        for x in (o[:pad], o[grown:], lse[:, :pad], lse[:, grown:]):
            assert bool((x == 7.0).all())
        if d != 128:
            continue
        do = spoiled(synth.normal_bf16(7700, STREAM_DO, qb.shape), Hq)
        g = [torch.full((sum(lens) + 2 * pad, h, d), 7.0, dtype=torch.bfloat16, device="cuda") for h in (Hq, Hkv, Hkv)]
        lib.attn_bwd_varlen(q, k, v, o, lse, do, cu, causal=causal, dq=g[0], dk=g[1], dv=g[2])
        g1 = lib.attn_bwd_varlen(*alone, o1, lse1, do[own].contiguous(), one, causal=causal)
        # one sequence below 128 rows: every sum is made by one product, in the same order
        for a, b in zip(g, g1):
            assert torch.equal(a[own], b)
            assert bool((a[:pad] == 7.0).all()) and bool((a[grown:] == 7.0).all())
    assert lib.attn_get_last_error() == lib.ATTN_OK


@pytest.mark.parametrize("d", [64, 128, 256])
def test_slices_of_a_fused_projection(lib, d):
    import torch

    lens, Hq, Hkv = [130, 1, 259], 4, 2
    qb, kb, vb = draw_packed(7800 + d, lens, lens, Hq, Hkv, d)
    q, k, v = gpu(qb), gpu(kb), gpu(vb)
    fused = torch.cat([q, k, v], 1)
    sq, sk, sv = fused[:, :Hq], fused[:, Hq:Hq + Hkv], fused[:, Hq + Hkv:]
    cu = offsets(lens)
    o, lse = lib.attn_fwd_varlen(q, k, v, cu, causal=True)
    o2, lse2 = lib.attn_fwd_varlen(sq, sk, sv, cu, causal=True)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    if d == 128:
        do = torch.ones_like(o)
        a = lib.attn_bwd_varlen(q, k, v, o, lse, do, cu, causal=True)
        b = lib.attn_bwd_varlen(sq, sk, sv, o, lse, do, cu, causal=True)
        # dQ is summed over key blocks in the order they finish: fp32 sums in another order, rounded to bf16
        assert torch.allclose(a[0].float(), b[0].float(), rtol=2.0 ** -7, atol=1e-4)
        assert torch.equal(a[1], b[1]) and torch.equal(a[2], b[2])


@pytest.mark.parametrize("bad", [[0, 50, 40, 60], [-1, 10, 20, 60], [0, 10, 20, 61], [5, 4, 5, 60]])
def test_offsets_out_of_order_write_nothing(lib, bad):
    import torch

    H, d, T = 2, 128, 60
    x = torch.ones((T, H, d), dtype=torch.bfloat16, device="cuda")
    good = offsets([20, 20, 20])
    wrong = torch.tensor(bad, dtype=torch.int32, device="cuda")
    assert lib.attn_get_last_error() == lib.ATTN_OK
    for cu_q, cu_k in ((wrong, good), (good, wrong)):
        o = torch.full_like(x, 7.0)
        lse = torch.full((H, T), 7.0, device="cuda")
        lib.attn_fwd_varlen(x, x, x, cu_q, cu_k, out=o, lse=lse)
        assert lib.attn_get_last_error() == lib.ATTN_ERR_INVALID_ARG
        g = [torch.full_like(x, 7.0) for _ in range(3)]
        lib.attn_bwd_varlen(x, x, x, x, lse, x, cu_q, cu_k, dq=g[0], dk=g[1], dv=g[2])
        assert lib.attn_get_last_error() == lib.ATTN_ERR_INVALID_ARG
        for t in (o, lse, *g):
            assert bool((t == 7.0).all())


def test_graph_replays_with_new_offsets(lib):
    """Captured once, replayed with other offsets and inputs in the same buffers: each replay equals an eager
    call (dQ up to the order of its fp32 sums)."""
    import torch

    T, Hq, Hkv, d = 600, 4, 2, 128
    q, k, v, do = (torch.empty((T, h, d), dtype=torch.bfloat16, device="cuda") for h in (Hq, Hkv, Hkv, Hq))
    cu = offsets([200, 200, 200])
    ws = torch.empty(lib.attn_fwd_varlen_workspace_bytes(3, T, T, Hq, d), dtype=torch.uint8, device="cuda")
    ws_b = torch.empty(lib.attn_bwd_varlen_workspace_bytes(3, T, T, Hq, Hkv, d), dtype=torch.uint8, device="cuda")
    o, lse = torch.empty_like(q), torch.empty((Hq, T), device="cuda")
    g = [torch.empty_like(t) for t in (q, k, v)]

    def call():
        lib.attn_fwd_varlen(q, k, v, cu, causal=True, workspace=ws, out=o, lse=lse)
        lib.attn_bwd_varlen(q, k, v, o, lse, do, cu, causal=True, workspace=ws_b, dq=g[0], dk=g[1], dv=g[2])

    for t in (q, k, v, do):
        t.normal_()
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for lens in ([600, 0, 0], [1, 300, 299], [129, 129, 130]):
        for t in (q, k, v, do):
            t.normal_()
        cu.copy_(offsets(lens))
        graph.replay()
        got = [t.clone() for t in (o, lse, *g)]
        call()
        assert torch.equal(got[0][:sum(lens)], o[:sum(lens)]) and torch.equal(got[1][:, :sum(lens)], lse[:, :sum(lens)])
        n = sum(lens)
        assert torch.allclose(got[2][:n].float(), g[0][:n].float(), rtol=2.0 ** -7, atol=1e-3)
        assert torch.equal(got[3][:n], g[1][:n]) and torch.equal(got[4][:n], g[2][:n])
    assert lib.attn_get_last_error() == lib.ATTN_OK
    del graph


def test_two_streams_at_once(lib):
    import torch

    lens, Hq, Hkv, d = [1500, 700, 300], 8, 2, 128
    sets = []
    for seed in (7901, 7902):
        qb, kb, vb = draw_packed(seed, lens, lens, Hq, Hkv, d)
        sets.append([gpu(x) for x in (qb, kb, vb)])
    cu = offsets(lens)
    alone = [lib.attn_fwd_varlen(*s, cu, causal=True) for s in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(5):
        got = []
        for s, st in zip(sets, streams):
            got.append(lib.attn_fwd_varlen(*s, cu, causal=True, stream=st))
        torch.cuda.synchronize()
        for (o, lse), (o1, lse1) in zip(got, alone):
            assert torch.equal(o, o1) and torch.equal(lse, lse1)


def test_backward_on_another_stream_and_in_graphs_that_share_workspaces(lib):
    """Two graphs (one with few blocks, cut into parts, one with many) over the same workspaces, replayed in turn, and
    eager calls on a side stream. dQ is a sum of fp32 atomics: equal up to one bf16 step."""
    import torch

    Hq, Hkv, d = 4, 2, 128
    sets = []
    for i, lens in enumerate(([900, 1, 300], [60] * 150)):
        qb, kb, vb = draw_packed(7980 + i, lens, lens, Hq, Hkv, d)
        sets.append(([gpu(x) for x in (qb, kb, vb)], gpu(synth.normal_bf16(7980 + i, STREAM_DO, qb.shape)), offsets(lens)))

    def same(got, want):
        assert torch.allclose(got[0].float(), want[0].float(), rtol=2.0 ** -7, atol=1e-3)
        assert torch.equal(got[1], want[1]) and torch.equal(got[2], want[2])

    fwd = [lib.attn_fwd_varlen(*x, cu, causal=True) for x, _, cu in sets]
    want = [lib.attn_bwd_varlen(*x, *f, do, cu, causal=True) for (x, do, cu), f in zip(sets, fwd)]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for (x, do, cu), f, w in zip(sets, fwd, want):
        got = lib.attn_bwd_varlen(*x, *f, do, cu, causal=True, stream=side)
        side.synchronize()
        same(got, w)
    sizes = [(cu.numel() - 1, x[0].shape[0], x[1].shape[0]) for x, _, cu in sets]
    ws_f = torch.empty(max(lib.attn_fwd_varlen_workspace_bytes(*n, Hq, d) for n in sizes), dtype=torch.uint8,
                       device="cuda")
    ws_b = torch.empty(max(lib.attn_bwd_varlen_workspace_bytes(*n, Hq, Hkv, d) for n in sizes), dtype=torch.uint8,
                       device="cuda")
    graphs, outs = [], []
    for x, do, cu in sets:
        o, lse = torch.empty_like(x[0]), torch.empty((Hq, x[0].shape[0]), device="cuda")
        g = [torch.empty_like(t) for t in x]
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            lib.attn_fwd_varlen(*x, cu, causal=True, workspace=ws_f, out=o, lse=lse)
            lib.attn_bwd_varlen(*x, o, lse, do, cu, causal=True, workspace=ws_b, dq=g[0], dk=g[1], dv=g[2])
        graphs.append(graph)
        outs.append((o, lse, g))
    for i in (0, 1, 0, 0, 1):
        o, lse, g = outs[i]
        for t in (o, lse, *g):
            t.zero_()
        graphs[i].replay()
        assert torch.equal(o, fwd[i][0]) and torch.equal(lse, fwd[i][1])
        same(g, want[i])
    assert lib.attn_get_last_error() == lib.ATTN_OK
    del graphs


def test_rows_beyond_32_bit_offsets(lib):
    """The last sequence lies more than 2^31 elements behind the start of q, o, dq: its rows equal the oracle's."""
    import torch

    Hq, Hkv, d, n = 128, 8, 128, 130
    lens = [128] * 1024 + [n]  # 131072 rows of 16384 elements before it
    T = sum(lens)
    qb, kb, vb = draw_packed(7990, [n], [n], Hq, Hkv, d)
    dob = synth.normal_bf16(7990, STREAM_DO, qb.shape)
    q, do = (torch.zeros((T, Hq, d), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    k, v = (torch.zeros((T, Hkv, d), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    for t, x in ((q, qb), (k, kb), (v, vb), (do, dob)):
        t[T - n:] = gpu(x)
    cu, sc = offsets(lens), 1 / math.sqrt(d)
    o, lse = lib.attn_fwd_varlen(q, k, v, cu, scale=sc, causal=True)
    grads = lib.attn_bwd_varlen(q, k, v, o, lse, do, cu, scale=sc, causal=True)
    torch.cuda.synchronize()
    assert lib.attn_get_last_error() == lib.ATTN_OK
    x = [f64(b) for b in (qb, kb, vb, dob)]
    O, L, bO, bL = reference(*x[:3], [n], [n], sc, True)
    assert_within(host(o[T - n:]), O, bO, "O")
    assert_lse(lse[:, T - n:].cpu().numpy().astype(np.float64), L, bL, "LSE")
    want, bounds = grad_bounds(*x, O, bO, [n], [n], sc, True)
    for name, g, w, b in zip(("dQ", "dK", "dV"), grads, want, bounds):
        assert_within(host(g[T - n:].contiguous()), w, b, name)
    # zero inputs before it: O and every gradient are zero there
    assert not bool(o[:T - n].any()) and not any(bool(g[:T - n].any()) for g in grads)


def test_single_sequence_agrees_with_the_dense_entry_point(lib):
    """One sequence: the same tiles in the same order as attn_fwd."""
    import torch

    for d in (64, 128, 256):
        qb, kb, vb = draw_packed(7950 + d, [700], [700], 4, 2, d)
        q, k, v = gpu(qb), gpu(kb), gpu(vb)
        o, lse = lib.attn_fwd_varlen(q, k, v, offsets([700]), causal=True)
        o1, lse1 = lib.attn_fwd(q[None], k[None], v[None], causal=True)
        # both are within their bounds of the oracle: a difference of at most two roundings per element
        A = reference(f64(qb), f64(kb), np.abs(f64(vb)), [700], [700], 1 / math.sqrt(d), True)[0]
        assert np.all(np.abs(host(o) - host(o1[0])) <= 2 * (2.0 ** -8 + 2.0 ** -10) * 2 * A)
        assert torch.allclose(lse, lse1[0], rtol=0, atol=2.0 ** -10)
