"""The decode calls refuse wrong arguments on the host, before any GPU work (runs
without a GPU), and the fp64 oracle of the decode step is what it says."""
import ctypes

import numpy as np
import pytest
import torch

from oracle import decode_oracle as D

EINVAL, EUNSUPPORTED, EWORKSPACE, EALIGN = -1, -2, -3, -6
WS, PTR = 1 << 20, 1 << 24


def _cache(**kw):
    from vlm_visual_token_b200.decode import _CCache
    c = _CCache(2, 100, 8, 64, 128, 16, 20, *([PTR] * 8))
    for k, v in kw.items():
        setattr(c, k, v)
    return ctypes.byref(c)


def _lib():
    import vlm_visual_token_b200 as ivc
    return ivc.lib()


BAD_CACHES = [
    (dict(layers=0), EINVAL), (dict(pages=0), EINVAL), (dict(kv_heads=-1), EINVAL),
    (dict(max_seqs=0), EINVAL), (dict(max_pages=0), EINVAL), (dict(k=None), EINVAL),
    (dict(table=None), EINVAL), (dict(free_count=None), EINVAL),
    (dict(page_tokens=48), EUNSUPPORTED), (dict(page_tokens=256), EUNSUPPORTED),
    (dict(head_dim=96), EUNSUPPORTED), (dict(pages=(1 << 20) + 1), EUNSUPPORTED),
    (dict(max_seqs=65537), EUNSUPPORTED), (dict(pages=1 << 20, kv_heads=64), EUNSUPPORTED),
    (dict(max_pages=1 << 25), EUNSUPPORTED),
    (dict(k=PTR + 8), EALIGN), (dict(v=PTR + 2), EALIGN), (dict(length=PTR + 1), EALIGN),
]


@pytest.mark.parametrize("change,code", BAD_CACHES)
def test_every_cache_call_checks_the_descriptor(change, code):
    L, c = _lib(), _cache(**change)
    assert L.ivc_cache_init(c, None) == code
    assert L.ivc_cache_reserve(c, PTR, None, 1, WS, 1 << 30, None) == code
    assert L.ivc_cache_fork(c, PTR, PTR, 1, 1, WS, 1 << 30, None) == code
    assert L.ivc_cache_compact(c, PTR, None, 0, None, None, 1, WS, 1 << 30, None) == code
    assert L.ivc_cache_free(c, PTR, 1, WS, 1 << 30, None) == code
    assert L.ivc_cache_workspace_size(c, 1, 1) == 0
    assert L.ivc_tree_attention_workspace_size(c, 1, 8, 1) == 0
    assert L.ivc_qk_norm_rope(c, 0, PTR, 4096, 1, 16, PTR, PTR, 1e-6, 1e6, PTR, PTR, None, 1, PTR, WS,
                              256, None) == code
    assert L.ivc_tree_attention(c, 0, PTR, 2048, 1, 16, 0.1, None, PTR, None, 1, PTR, WS, 1 << 40,
                                None) == code


def test_cache_calls_check_their_arguments():
    L, c = _lib(), _cache()
    assert L.ivc_cache_init(None, None) == EINVAL
    for n, tokens, ws, size, code in ((-1, PTR, WS, 256, EINVAL), (17, PTR, WS, 256, EINVAL),
                                      (1, None, WS, 256, EINVAL), (1, PTR, None, 256, EINVAL),
                                      (1, PTR, WS + 64, 256, EALIGN), (1, PTR, WS, 255, EWORKSPACE),
                                      (0, None, WS, 256, 0)):
        assert L.ivc_cache_reserve(c, tokens, None, n, ws, size, None) == code
    assert L.ivc_cache_free(c, None, 17, WS, 256, None) == EINVAL
    assert L.ivc_cache_free(c, PTR, 1, WS, 128, None) == EWORKSPACE
    assert L.ivc_cache_free(c, None, 0, WS, 256, None) == 0
    need = L.ivc_cache_workspace_size(c, 3, 0)
    assert need >= 512 + 3 * 20 * 16                       # a job for every page of three sequences
    assert L.ivc_cache_workspace_size(c, 16, 0) <= 1024 + 100 * 16  # but no more than there are pages
    assert L.ivc_cache_workspace_size(c, 3, 1000) >= 3 * 1000 * 8
    assert L.ivc_cache_workspace_size(c, 17, 0) == 0
    assert L.ivc_cache_workspace_size(c, 1, -1) == 0
    assert L.ivc_cache_fork(c, None, PTR, 1, 1, WS, 1 << 30, None) == EINVAL
    assert L.ivc_cache_fork(c, PTR, None, 1, 1, WS, 1 << 30, None) == EINVAL
    assert L.ivc_cache_fork(c, PTR, PTR, 3, 0, WS, 512, None) == EWORKSPACE
    assert L.ivc_cache_compact(c, None, None, 0, None, None, 1, WS, 1 << 30, None) == EINVAL
    assert L.ivc_cache_compact(c, PTR, PTR, -1, None, None, 1, WS, 1 << 30, None) == EINVAL
    assert L.ivc_cache_compact(c, PTR, PTR, 1000, None, None, 3, WS, 3 * 8000, None) == EWORKSPACE
    assert L.ivc_cache_compact(c, PTR, PTR, 4, None, None, 0, WS, 4096, None) == 0


def test_qk_norm_rope_checks_its_arguments():
    L, c = _lib(), _cache()
    ok = dict(layer=1, qkv=PTR, ld=32 * 128, N=4, heads=16, gq=PTR, gk=PTR, eps=1e-6, theta=1e6, pos=PTR,
              off=PTR, B=2, out=PTR, ws=WS, size=256)

    def call(**kw):
        a = {**ok, **kw}
        return L.ivc_qk_norm_rope(c, a["layer"], a["qkv"], a["ld"], a["N"], a["heads"], a["gq"], a["gk"],
                                  a["eps"], a["theta"], a["pos"], a["off"], None, a["B"], a["out"],
                                  a["ws"], a["size"], None)

    for bad in (dict(layer=-1), dict(layer=2), dict(N=-1), dict(B=-1), dict(heads=0), dict(eps=-1.0),
                dict(eps=float("nan")), dict(eps=float("inf")), dict(theta=0.0), dict(theta=-2.0),
                dict(theta=float("nan")), dict(theta=float("inf")), dict(qkv=None), dict(gq=None),
                dict(gk=None), dict(pos=None), dict(off=None), dict(out=None), dict(ws=None)):
        assert call(**bad) == EINVAL, bad
    for bad in (dict(heads=12), dict(ld=32 * 128 - 8), dict(ld=32 * 128 + 4)):
        assert call(**bad) == EUNSUPPORTED, bad
    for bad in (dict(qkv=PTR + 8), dict(gq=PTR + 4), dict(out=PTR + 2), dict(ws=WS + 16)):
        assert call(**bad) == EALIGN, bad
    assert call(size=255) == EWORKSPACE
    assert call(N=0) == 0 and call(B=0) == 0


def test_tree_attention_checks_its_arguments():
    L, c = _lib(), _cache()
    need = L.ivc_tree_attention_workspace_size(c, 4, 16, 2)
    ok = dict(layer=1, q=PTR, ld=16 * 128, N=4, heads=16, scale=0.1, off=PTR, B=2, out=PTR, ws=WS, size=need)

    def call(**kw):
        a = {**ok, **kw}
        return L.ivc_tree_attention(c, a["layer"], a["q"], a["ld"], a["N"], a["heads"], a["scale"], None,
                                    a["off"], None, a["B"], a["out"], a["ws"], a["size"], None)

    for bad in (dict(layer=-1), dict(layer=2), dict(N=-1), dict(B=-1), dict(heads=0), dict(scale=0.0),
                dict(scale=-1.0), dict(scale=float("nan")), dict(scale=float("inf")), dict(q=None),
                dict(off=None), dict(out=None), dict(ws=None)):
        assert call(**bad) == EINVAL, bad
    for bad in (dict(heads=12), dict(heads=8 * 65, ld=8 * 65 * 128), dict(ld=16 * 128 - 8), dict(B=4097)):
        assert call(**bad) == EUNSUPPORTED, bad
    for bad in (dict(q=PTR + 8), dict(out=PTR + 2), dict(ws=WS + 16)):
        assert call(**bad) == EALIGN, bad
    assert call(size=need - 1) == EWORKSPACE
    assert call(N=0) == 0 and call(B=0) == 0
    assert L.ivc_tree_attention_workspace_size(c, 4, 16, 4097) == 0


def test_verify_drafts_checks_its_arguments():
    L = _lib()
    ok = dict(p=PTR, p_ld=50, q=PTR, q_ld=50, N=4, V=50, tok=PTR, off=PTR, B=2, u=PTR, un=PTR, path=PTR,
              stride=4, n_path=PTR, token=PTR, ws=WS, size=256)

    def call(**kw):
        a = {**ok, **kw}
        return L.ivc_verify_drafts(a["p"], a["p_ld"], a["q"], a["q_ld"], a["N"], a["V"], a["tok"], None,
                                   a["off"], a["B"], a["u"], a["un"], a["path"], a["stride"], a["n_path"],
                                   a["token"], a["ws"], a["size"], None)

    for bad in (dict(N=-1), dict(V=0), dict(B=-1), dict(stride=0), dict(p_ld=49), dict(q_ld=49), dict(p=None),
                dict(tok=None), dict(off=None), dict(u=None), dict(un=None), dict(path=None),
                dict(n_path=None), dict(token=None), dict(ws=None)):
        assert call(**bad) == EINVAL, bad
    assert call(V=(1 << 28) + 1, p_ld=1 << 29, q_ld=1 << 29) == EUNSUPPORTED
    assert call(ws=WS + 128) == EALIGN
    assert call(size=64) == EWORKSPACE
    assert call(B=0) == 0


def test_python_binding_refuses_wrong_tensors():
    """Types, ranks, devices and sizes, before the library is called."""
    import vlm_visual_token_b200 as ivc
    i = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
    kv = torch.zeros(2, 5, 2, 16, 64, dtype=torch.bfloat16)
    meta = dict(table=i(3, 4), length=i(3), n_pages=i(3), ref=i(5), free_list=i(5), free_count=i(1))
    c = ivc.Cache(kv, kv.clone(), **meta)
    assert (c.layers, c.pages, c.kv_heads, c.page_tokens, c.head_dim, c.max_seqs, c.max_pages) == \
        (2, 5, 2, 16, 64, 3, 4)
    for bad in (dict(table=i(3, 4).long()), dict(length=i(4)), dict(ref=i(4)), dict(free_count=i(2)),
                dict(table=i(4, 3).t())):
        with pytest.raises(ivc.IvcError):
            ivc.Cache(kv, kv.clone(), **{**meta, **bad})
    for k, v in ((kv.float(), kv.float()), (kv, kv[:, :4]), (kv[0], kv[0]), (kv.transpose(1, 2), kv)):
        with pytest.raises(ivc.IvcError):
            ivc.Cache(k, v, **meta)
    one, off = torch.ones(64, dtype=torch.bfloat16), i(2)
    q = torch.zeros(4, 4, 64, dtype=torch.bfloat16)
    x = torch.zeros(4, 8 * 64, dtype=torch.bfloat16)
    p = torch.zeros(4, 9)
    calls = [
        lambda: ivc.cache_reserve(c, i(2).float()), lambda: ivc.cache_reserve(c, i(2), i(3)),
        lambda: ivc.cache_fork(c, i(2), i(1)), lambda: ivc.cache_compact(c, i(2), i(3, 2)),
        lambda: ivc.cache_compact(c, i(2), None, i(1)), lambda: ivc.cache_free(c, i(2, 2)),
        lambda: ivc.qk_norm_rope(c, 0, x[:, 8:], one, one, i(4), off),           # not whole heads
        lambda: ivc.qk_norm_rope(c, 0, x[:, :256], one, one, i(4), off),         # no query head
        lambda: ivc.qk_norm_rope(c, 0, x.t(), one, one, i(4), off),
        lambda: ivc.qk_norm_rope(c, 0, x, one[:32], one, i(4), off),
        lambda: ivc.qk_norm_rope(c, 0, x, one, one, i(3), off),
        lambda: ivc.qk_norm_rope(c, 0, x, one, one, i(4), off, out=q[:3]),
        lambda: ivc.tree_attention(c, 0, q.float(), None, off),
        lambda: ivc.tree_attention(c, 0, q.transpose(0, 1), None, off),
        lambda: ivc.tree_attention(c, 0, q[:, :, :32], None, off),
        lambda: ivc.tree_attention(c, 0, q, i(3), off),
        lambda: ivc.tree_attention(c, 0, q, None, off, seqs=i(2)),
        lambda: ivc.verify_drafts(p.double(), None, i(4), None, off, p[:, 0].clone(), p[0, :1].clone()),
        lambda: ivc.verify_drafts(p, p[:3], i(4), None, off, p[:, 0].clone(), p[0, :1].clone()),
        lambda: ivc.verify_drafts(p, None, i(3), None, off, p[:, 0].clone(), p[0, :1].clone()),
        lambda: ivc.verify_drafts(p, None, i(4), None, off, p[:, 0].clone(), p[0, :2].clone()),
        lambda: ivc.cache_reserve(c, i(2)),                                       # all right, but not on a GPU
        lambda: ivc.tree_attention(c, 0, q, None, off),
    ]
    for k, call in enumerate(calls):
        with pytest.raises(ivc.IvcError) as e:
            call()
        assert e.value.code in (EINVAL, EUNSUPPORTED), k


# ------------------------------------------------------------------ the oracle itself
def test_oracle_attention_is_softmax_attention():
    """A chain over a context is torch's causal attention in float64; a tree's
    node sees what its mask says."""
    g = torch.Generator().manual_seed(0)
    n, m, H, kv, Dh = 5, 7, 4, 2, 8
    q = torch.randn(n, H, Dh, generator=g, dtype=torch.float64)
    k, v = (torch.randn(m + n, kv, Dh, generator=g, dtype=torch.float64) for _ in range(2))
    for parents in ([-1, 0, 1, 2, 3], [-1, 0, 0, 1, -1]):
        see = torch.zeros(n, m + n, dtype=torch.bool)
        see[:, :m] = True
        for i in range(n):
            for a in D.ancestors(parents, i):
                see[i, m + a] = True
        kk, vv = (t.repeat_interleave(H // kv, 1).transpose(0, 1) for t in (k, v))
        want = torch.nn.functional.scaled_dot_product_attention(q.transpose(0, 1), kk, vv, attn_mask=see,
                                                                scale=0.3)
        got = D.tree_attend(q.numpy(), k.numpy(), v.numpy(), m, parents, 0.3)
        np.testing.assert_allclose(got, want.transpose(0, 1).numpy(), rtol=1e-12, atol=1e-13)


def test_oracle_rotation_keeps_norms_and_depends_on_distance():
    rng = np.random.RandomState(1)
    x, y = rng.randn(1, 1, 16), rng.randn(1, 1, 16)
    rot = lambda z, t: D.norm_rope(z, 1.0, [t], 1e4, 0.0)[0, 0]  # noqa: E731
    assert np.isclose(np.linalg.norm(rot(x, 12345)), 4.0)        # sqrt(D) after the norm
    assert np.isclose(rot(x, 40) @ rot(y, 33), rot(x, 1007) @ rot(y, 1000))
    np.testing.assert_allclose(rot(x, 0), x[0, 0] / np.sqrt(np.mean(x ** 2)))


@pytest.mark.parametrize("dense", [False, True])
def test_oracle_verification_draws_from_the_target(dense):
    """With children drawn from q without replacement (dense) or fixed, the token
    after the root is distributed as p: its expectation over u and u_next, taken
    exactly over the intervals in which the answer is constant."""
    p = np.array([[0.40, 0.05, 0.30, 0.25]])
    q = np.array([[0.10, 0.55, 0.20, 0.15]])
    share = np.zeros(4)
    drafts = [(a, b, q[0, a] * q[0, b] / (1 - q[0, a])) for a in range(4) for b in range(4) if a != b] \
        if dense else [(1, 3, 1.0)]
    G = 80
    grid = (np.arange(G) + 0.5) / G
    for a, b, weight in drafts:
        for u1 in grid:
            for u2 in grid if dense else grid:
                path, t = D.verify(np.repeat(p, 3, 0), np.repeat(q, 3, 0) if dense else None, [0, a, b],
                                   [-1, 0, 0], [0, u1, u2], 0.5)
                if len(path) == 2:
                    share[(a, b)[path[1] - 1]] += weight / G ** 2
                else:  # the draw over u_next, exactly: the residual's shares
                    z1 = np.maximum(p[0] - q[0], 0) if dense else np.where(np.arange(4) == a, 0, p[0])
                    z1 = z1 / z1.sum()
                    q2 = np.where(np.arange(4) == a, 0, q[0]) / (1 - q[0, a])
                    z2 = np.maximum(z1 - q2, 0) if dense else np.where(np.arange(4) == b, 0, z1)
                    share += weight / G ** 2 * z2 / z2.sum()
    # each of two acceptance borders moves by at most one grid cell
    assert np.abs(share - p[0]).max() <= 2.0 / G


def test_oracle_cache_refuses_without_changing_anything():
    c = D.PagedCache(1, 6, 1, 16, 64, 4, 4)
    c.reserve([40, 20], [0, 1])
    before = (c.table.copy(), list(c.free), c.n_pages.copy())
    for call in (lambda: c.reserve([1, 1], [2, 2]), lambda: c.reserve([200], [2]),
                 lambda: c.fork([0], [1], True), lambda: c.compact([99], None, [0], [0]),
                 lambda: c.drop([0, 0])):
        with pytest.raises(ValueError):
            call()
    assert np.array_equal(c.table, before[0]) and c.free == before[1] and np.array_equal(c.n_pages, before[2])
