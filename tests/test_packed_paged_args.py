"""What the packed-sequence and paged-cache entry points refuse, before any CUDA call (no GPU needed), the
workspace sizes, and the error bounds of the tests themselves against a model of the kernels' roundings."""
import math

import numpy as np
import pytest

P = 1 << 20  # an aligned address that is never dereferenced
BIG = 1 << 45


@pytest.fixture(scope="module")
def c():
    import exact_io_aware_41_b200 as pkg

    return pkg, pkg.lib_handle()


def test_packed_forward_refusals(c):
    pkg, lib = c

    def call(q=P, k=P, v=P, cu_q=P, cu_k=P, o=P, lse=P, S=2, Tq=16, Tk=16, Hq=4, Hkv=2, d=64, qs=256, ks=128, vs=128,
             scale=0.1, causal=1, ws=P, n=BIG):
        return lib.attn_fwd_varlen(q, k, v, cu_q, cu_k, o, lse, S, Tq, Tk, Hq, Hkv, d, qs, ks, vs, scale, causal, ws, n,
                                   None)

    for name in ("q", "k", "v", "cu_q", "cu_k", "o", "lse"):
        assert call(**{name: 0}) == pkg.ATTN_ERR_INVALID_ARG, name
    for name in ("q", "k", "v", "o"):
        assert call(**{name: P + 8}) == pkg.ATTN_ERR_INVALID_ARG, name
    for name in ("cu_q", "cu_k", "lse"):
        assert call(**{name: P + 2}) == pkg.ATTN_ERR_INVALID_ARG, name
    for bad in (dict(S=0), dict(Tq=0), dict(Tk=0), dict(Hq=3), dict(Hkv=0), dict(scale=0.0), dict(scale=math.nan),
                dict(causal=2), dict(qs=255), dict(qs=248), dict(ks=132), dict(vs=120), dict(ks=1 << 31), dict(qs=-256)):
        assert call(**bad) == pkg.ATTN_ERR_INVALID_ARG, bad
    assert call(d=48) == pkg.ATTN_ERR_UNSUPPORTED
    assert call(S=1000001) == pkg.ATTN_ERR_UNSUPPORTED
    need = lib.attn_fwd_varlen_workspace_bytes(2, 16, 16, 4, 64)
    for bad in (dict(ws=0), dict(ws=P + 16), dict(n=need - 1)):
        assert call(**bad) == pkg.ATTN_ERR_WORKSPACE, bad


def test_packed_backward_refusals(c):
    pkg, lib = c

    def call(S=2, Tq=16, Tk=16, Hq=4, Hkv=2, d=128, qs=512, ks=256, vs=256, scale=0.1, causal=0, ws=P, n=BIG, **ptr):
        names = ("q", "k", "v", "o", "lse", "dout", "cu_q", "cu_k", "dq", "dk", "dv")
        return lib.attn_bwd_varlen(*[ptr.get(x, P) for x in names], S, Tq, Tk, Hq, Hkv, d, qs, ks, vs, scale, causal, ws,
                                   n, None)

    for name in ("q", "k", "v", "o", "dout", "dq", "dk", "dv"):
        assert call(**{name: 0}) == pkg.ATTN_ERR_INVALID_ARG, name
        assert call(**{name: P + 8}) == pkg.ATTN_ERR_INVALID_ARG, name
    for name in ("lse", "cu_q", "cu_k"):
        assert call(**{name: 0}) == pkg.ATTN_ERR_INVALID_ARG, name
        assert call(**{name: P + 1}) == pkg.ATTN_ERR_INVALID_ARG, name
    for bad in (dict(S=0), dict(Tq=0), dict(Tk=0), dict(Hq=5), dict(scale=-1.0), dict(causal=-1), dict(qs=500)):
        assert call(**bad) == pkg.ATTN_ERR_INVALID_ARG, bad
    assert call(d=64, qs=256, ks=128, vs=128) == pkg.ATTN_ERR_UNSUPPORTED
    need = lib.attn_bwd_varlen_workspace_bytes(2, 16, 16, 4, 2, 128)
    for bad in (dict(ws=0), dict(ws=P + 128), dict(n=need - 1)):
        assert call(**bad) == pkg.ATTN_ERR_WORKSPACE, bad


def test_paged_decode_refusals(c):
    pkg, lib = c

    def call(n_pages=8, page=16, width=4, B=2, Hq=4, Hkv=2, d=64, qs=256, scale=0.1, ws=P, n=BIG, **ptr):
        names = ("q", "k", "v", "table", "lens")
        return lib.attn_decode_paged(*[ptr.get(x, P) for x in names], n_pages, page, width, ptr.get("o", P),
                                     ptr.get("lse", P), B, Hq, Hkv, d, qs, scale, ws, n, None)

    for name in ("q", "k", "v", "o"):
        assert call(**{name: 0}) == pkg.ATTN_ERR_INVALID_ARG, name
        assert call(**{name: P + 8}) == pkg.ATTN_ERR_INVALID_ARG, name
    for name in ("table", "lens", "lse"):
        assert call(**{name: 0}) == pkg.ATTN_ERR_INVALID_ARG, name
        assert call(**{name: P + 2}) == pkg.ATTN_ERR_INVALID_ARG, name
    for bad in (dict(n_pages=0), dict(page=0), dict(width=0), dict(B=0), dict(Hq=3), dict(scale=math.inf), dict(qs=8),
                dict(qs=260)):
        assert call(**bad) == pkg.ATTN_ERR_INVALID_ARG, bad
    for bad in (dict(d=96, qs=512), dict(page=8), dict(page=20), dict(page=65552), dict(Hq=34, qs=34 * 64)):
        assert call(**bad) == pkg.ATTN_ERR_UNSUPPORTED, bad
    need = lib.attn_decode_paged_workspace_bytes(2, 4, 2, 64)
    assert need > 0
    for bad in (dict(ws=0), dict(ws=P + 4), dict(n=need - 1)):
        assert call(**bad) == pkg.ATTN_ERR_WORKSPACE, bad


def test_cache_append_refusals(c):
    pkg, lib = c

    def call(B=2, T=5, n_pages=8, page=16, width=4, Hkv=2, d=64, ks=128, vs=128, **ptr):
        names = ("k", "v", "cu", "table", "lens", "kp", "vp")
        return lib.attn_cache_append(*[ptr.get(x, P) for x in names], B, T, n_pages, page, width, Hkv, d, ks, vs, None)

    for name in ("k", "v", "kp", "vp"):
        assert call(**{name: 0}) == pkg.ATTN_ERR_INVALID_ARG, name
        assert call(**{name: P + 8}) == pkg.ATTN_ERR_INVALID_ARG, name
    for name in ("table", "lens"):
        assert call(**{name: 0}) == pkg.ATTN_ERR_INVALID_ARG, name
    for bad in (dict(B=0), dict(T=0), dict(n_pages=0), dict(page=0), dict(width=0), dict(Hkv=0), dict(d=0),
                dict(Hkv=1, d=12, ks=16, vs=16), dict(ks=120), dict(vs=129), dict(cu=0), dict(cu=P + 2)):
        assert call(**bad) == pkg.ATTN_ERR_INVALID_ARG, bad


def test_workspace_sizes(c):
    pkg, _ = c
    assert pkg.attn_fwd_varlen_workspace_bytes(0, 16, 16, 4, 64) == 0
    assert pkg.attn_fwd_varlen_workspace_bytes(3, 0, 16, 4, 64) == 0
    assert pkg.attn_bwd_varlen_workspace_bytes(1, 0, 1, 1, 1, 128) == 0
    assert pkg.attn_bwd_varlen_workspace_bytes(1, 1, 1, 3, 2, 128) == 0
    assert pkg.attn_decode_paged_workspace_bytes(2, 3, 2, 64) == 0
    # a list of 3 + 300 blocks of 32 bytes (and the counters); room for parts only with few blocks and many keys
    assert pkg.attn_fwd_varlen_workspace_bytes(300, 1000, 1000, 8, 64) == 256 + 256 * math.ceil(303 * 32 / 256)
    assert pkg.attn_fwd_varlen_workspace_bytes(3, 100000, 100000, 8, 64) < 1 << 20
    assert 1 << 20 < pkg.attn_fwd_varlen_workspace_bytes(3, 1000, 100000, 8, 64) < 41 << 20


def test_binding_refusals():
    import torch

    import exact_io_aware_41_b200 as pkg

    x = torch.zeros((4, 2, 64), dtype=torch.bfloat16)
    cu = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        pkg.attn_fwd_varlen(x, x, x, cu)
    with pytest.raises(ValueError):
        pkg.attn_decode_paged(x, x[None], x[None], cu[None], cu)
    with pytest.raises(ValueError):
        pkg.attn_cache_append(x, x, x[None].float(), x[None].float(), cu[None], cu[:1])


def _bf16(x):
    import torch

    return torch.from_numpy(np.asarray(x, dtype=np.float32)).to(torch.bfloat16).double().numpy()


@pytest.mark.parametrize("plant", [None, "mask", "scale", "group"])
def test_the_bounds_hold_for_the_roundings_and_catch_mistakes(plant):
    """P and dS rounded to bf16, O from the rounded P, results rounded: within the derived bounds. The same
    with one planted mistake (a key too many visible, a wrong scale, a wrong kv head): outside."""
    import oracle
    from packed import draw_packed, f64, grad_bounds, reference, sequences

    ql, kl, Hq, Hkv, d, sc = [37, 1, 64], [40, 9, 64], 4, 2, 128, 1 / math.sqrt(128)
    q, k, v = (f64(x) for x in draw_packed(42, ql, kl, Hq, Hkv, d))
    do = f64(draw_packed(43, ql, kl, Hq, Hkv, d)[0])
    O, L, bO, bL = reference(q, k, v, ql, kl, sc, True)
    want, bounds = grad_bounds(q, k, v, do, O, bO, ql, kl, sc, True)
    got = [np.zeros_like(q), np.zeros_like(k), np.zeros_like(v)]
    o, lse = np.zeros_like(q), np.zeros_like(L)
    s2 = sc * 1.01 if plant == "scale" else sc
    for a, b in sequences(ql, kl):
        for h in range(Hq):
            g = (h % Hkv) if plant == "group" else h // (Hq // Hkv)
            n = b.stop - b.start - (a.stop - a.start)
            S = s2 * (q[a, h] @ k[b, g].T)
            i, j = np.arange(S.shape[0])[:, None], np.arange(S.shape[1])[None]
            S[j > i + n + (1 if plant == "mask" else 0)] = -np.inf
            m = S.max(1, keepdims=True)
            e = np.exp(S - m)
            z = e.sum(1, keepdims=True)
            lse[h, a] = (m + np.log(z))[:, 0]
            o[a, h] = _bf16((_bf16(e) @ v[b, g]) / z)
            p = e / z
            dp = do[a, h] @ v[b, g].T
            ds = _bf16(p * (dp - (do[a, h] * o[a, h]).sum(1, keepdims=True)))
            got[0][a, h] = s2 * (ds @ k[b, g])
            got[1][b, g] += s2 * (ds.T @ q[a, h])
            got[2][b, g] += _bf16(p).T @ do[a, h]
    inside = [np.all(np.abs(x - w) <= b) for x, w, b in ((o, O, bO), (lse, L, bL))]
    inside += [np.all(np.abs(_bf16(x) - w) <= b) for x, w, b in zip(got, want, bounds)]
    # 1 % of the scale moves O by about as much as the roundings may: LSE, which is not rounded, shows it
    assert all(inside) if plant is None else not all(inside[:2])
