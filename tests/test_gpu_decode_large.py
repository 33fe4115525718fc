"""The decode step at the sizes its kernels are laid out for: attention with many key
tiles per CTA and a maximum that keeps rising, verification over vocabularies that a
cluster of CTAs shares, compactions in which a CTA moves several heads.

Attention tolerance: weights and output rounded to bf16 (2^-8 relative each). A score is
a sum of at most 128 fp32 products; with |q||k| scale below 2^9 it is off by less than
2^9 * 2^-24 * 16 = 2^-11, its exponent (a product with scale * log2 e, rounded) by as
much again, so that weights and their sum are off by 2^-10 relative each: 2^-9 of the
weighted mean of |v|.
"""
import numpy as np
import pytest
import torch

from oracle import decode_oracle as D
from tests.test_gpu_decode import BF, Pair, _ivc, _tree, _verify_case, _verify_check, dev

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------ attention
def _long_case(lens, counts, Hq, kv, D_, pt, seed, rise):
    """A cache whose keys grow along each context, so that a row's maximum rises by
    2^8 and more again and again; the tokens of a page shuffled over the cache."""
    ivc = _ivc()
    B, N = len(lens), sum(counts)
    need = [-(-(a + n) // pt) for a, n in zip(lens, counts)]
    c = ivc.Cache.empty(1, sum(need) + 3, kv, pt, D_, B, max(need) + 1)
    g = torch.Generator(device="cuda").manual_seed(seed)
    c.free_list.copy_(torch.randperm(c.pages, generator=g, device="cuda"))
    for name in ("k", "v"):
        getattr(c, name).copy_(torch.randn(c.k.shape, generator=g, device="cuda"))
    ivc.cache_reserve(c, dev(lens))
    ivc.cache_compact(c, dev(lens))
    ivc.cache_reserve(c, dev(counts))
    for b in range(B):
        pages = c.table[b, :need[b]].long()
        t = torch.arange(need[b] * pt, device="cuda") / (lens[b] + counts[b])
        grow = 0.05 * 2.0 ** (9 * t.clamp_max(1.0)) if rise else torch.ones_like(t)
        c.k[0, pages] = (c.k[0, pages].float() * grow.view(-1, 1, pt, 1)).bfloat16()
    q = torch.randn(N, Hq, D_, generator=g, device="cuda").bfloat16()
    rng = np.random.RandomState(seed)
    trees = [_tree(rng, n, "tree") for n in counts]
    off = dev(np.concatenate([[0], np.cumsum(counts)]))
    ws = ivc.new_workspace(ivc.tree_attention_workspace_size(c, N, Hq, B))
    return ivc, c, q, trees, off, need, ws


def _sees(tree, m):
    n = len(tree)
    see = torch.zeros(n, m + n, dtype=torch.bool)
    see[:, :m] = True
    for i in range(n):
        see[i, [m + a for a in D.ancestors(tree, i)]] = True
    return see.cuda()


def _check_long(c, got, q, trees, lens, counts, need, Hq, kv, D_):
    row = 0
    for b, (m, n) in enumerate(zip(lens, counts)):
        see = _sees(trees[b], m)
        k, v = (x[0, c.table[b, :need[b]].long()].transpose(1, 2).reshape(-1, kv, D_)[:m + n].double()
                for x in (c.k, c.v))
        G = Hq // kv
        for h in range(kv):
            s = torch.einsum("ngd,ld->gnl", q[row:row + n, h * G:(h + 1) * G].double(), k[:, h]) * D_ ** -0.5
            w = torch.softmax(s.masked_fill(~see, float("-inf")), -1)
            want = torch.einsum("gnl,ld->ngd", w, v[:, h])
            size = torch.einsum("gnl,ld->ngd", w, v[:, h].abs())
            err = (got[row:row + n, h * G:(h + 1) * G].double() - want).abs()
            assert bool((err <= BF * want.abs() + (BF + 2.0 ** -9) * size).all()), \
                (b, h, float((err / size).max()))
        row += n


@pytest.mark.parametrize("lens,counts,Hq,kv,D_,pt", [
    ([6100, 6000, 5900, 6333], [1] * 4, 32, 8, 128, 64),              # plain decoding
    ([6100, 6000, 5900, 6333], [27, 1, 32, 9], 32, 8, 128, 16),       # up to 128 rows
    ([6100, 6000, 5900, 6333], [64, 50, 33, 40], 32, 8, 128, 128),    # more than 128 rows
    ([6100, 6000, 5901, 6333], [128, 100, 128, 77], 16, 8, 64, 32),   # drafted nodes over three tiles
    ([6100, 6000, 5901], [128, 127, 90], 40, 8, 128, 64),             # 25 nodes of 5 heads a block
    ([1200 + 17 * i for i in range(40)], [1 + i % 5 for i in range(40)], 8, 4, 64, 64),
    ([2000 + 31 * i for i in range(36)], [33 + i % 40 for i in range(36)], 8, 2, 128, 64),
])
@pytest.mark.parametrize("rise", [True, False])
def test_attention_with_many_tiles_per_cta(lens, counts, Hq, kv, D_, pt, rise):
    tiles = sum(-(-(a + n) // 64) for a, n in zip(lens, counts)) * kv
    assert tiles >= 8 * 148
    ivc, c, q, trees, off, need, ws = _long_case(lens, counts, Hq, kv, D_, pt, 7, rise)
    par = dev(sum(trees, []))
    got = ivc.tree_attention(c, 0, q, par, off, workspace=ws)
    assert ivc.device_status(ws) == 0
    _check_long(c, got, q, trees, lens, counts, need, Hq, kv, D_)
    for _ in range(3):                       # the order of the work does not matter
        assert torch.equal(ivc.tree_attention(c, 0, q, par, off, workspace=ws), got)


@pytest.mark.parametrize("Hq,kv,D_", [(40, 8, 128), (32, 8, 64), (6, 2, 128)])
def test_a_row_does_not_depend_on_the_rows_beside_it(Hq, kv, D_):
    """Every other node's queries replaced, by larger, smaller and non-finite ones: the
    bits of the nodes between them stay, although they share the tiles' rows."""
    lens, counts = [6100, 6000, 5901, 12000], [40, 27, 33, 5]
    ivc, c, q, trees, off, need, ws = _long_case(lens, counts, Hq, kv, D_, 64, 3, True)
    par = dev(sum(trees, []))
    want = ivc.tree_attention(c, 0, q, par, off, workspace=ws)
    for other in (20.0, 0.0, float("inf"), float("nan")):
        changed = q.clone()
        changed[::2] *= other
        got = ivc.tree_attention(c, 0, changed, par, off, workspace=ws)
        assert torch.equal(got[1::2], want[1::2]), other


@pytest.mark.parametrize("Hq,counts", [(32, [64, 50, 33, 40]), (8, [64, 50, 33, 40]), (16, [128, 100, 128, 77])])
def test_unseen_values_with_many_tiles_per_cta(Hq, counts):
    """Every third node's value is not finite: only the rows that see it show it."""
    lens, kv, D_ = [6100, 6000, 5901, 6333], 8, 64
    ivc, c, q, trees, off, need, ws = _long_case(lens, counts, Hq, kv, D_, 32, 11, False)
    trees = [[-1] + [0] * (n - 1) for n in counts]       # a star: a node is seen by itself alone
    par = dev(sum(trees, []))
    clean = ivc.tree_attention(c, 0, q, par, off, workspace=ws)
    want = torch.zeros_like(clean, dtype=torch.bool)
    bad, row = [float("nan"), float("inf"), -float("inf")], 0
    for b, (m, n) in enumerate(zip(lens, counts)):
        for i in range(2, n, 3):
            page, slot = int(c.table[b, (m + i) // 32]), (m + i) % 32
            c.v[0, page, :, slot, i % D_] = bad[i % 7 % 3]
            want[row + i, :, i % D_] = True
        row += n
    got = ivc.tree_attention(c, 0, q, par, off, workspace=ws)
    assert ivc.device_status(ws) == 0
    assert torch.equal(~torch.isfinite(got.float()), want)
    assert torch.equal(got[~want], clean[~want])


# ------------------------------------------------------------------ verification
@pytest.mark.parametrize("dense", [False, True])
@pytest.mark.parametrize("V", [4096, 4097, 32000, 151001, 300001])
def test_verification_over_large_vocabularies(V, dense):
    """Rejections and draws at the ends and in the middle of the random numbers' range."""
    rng = np.random.RandomState(V % 1000 + dense)
    counts = [1, 6, 5, 0, 7, 2, 4]
    p, q, tok, trees, off, u, un = _verify_case(rng, counts, V, dense, "tree")
    top = float(np.nextafter(np.float32(1), np.float32(0)))
    for us, draws in ((u, un), (np.full_like(u, top), np.full_like(un, 0.5)),
                      (np.full_like(u, top), np.full_like(un, top)), (0.5 + u / 2, np.zeros_like(un)),
                      (np.zeros_like(u), np.full_like(un, 1e-7))):
        _verify_check(_ivc(), p, q, tok, trees, off, us, draws)


@pytest.mark.parametrize("dense", [False, True])
def test_verification_of_wide_trees_and_strided_rows_over_a_large_vocabulary(dense):
    rng = np.random.RandomState(13)
    case = _verify_case(rng, [128, 100], 5003, dense, "tree", peaked=0.3)
    _verify_check(_ivc(), *case, width=128, ld=5010)
    star = _verify_case(rng, [128, 3], 4999, dense, "star", peaked=0.1)
    _verify_check(_ivc(), *star, width=128)
    *most, u, un = star
    _verify_check(_ivc(), *most, np.nextafter(np.ones_like(u), np.float32(0)), un, width=128)


@pytest.mark.parametrize("at", [[0, 1, 2, 3], [4999, 0, 625, 624], [10, 2600, 4374, 4375]])
def test_verification_borders_over_a_large_vocabulary(at):
    """Certain tokens, equal distributions and rows that leave nothing, wherever the few
    tokens that have a probability stand in the CTAs' slices."""
    ivc, V = _ivc(), 5000
    chain, off = [[-1, 0, 1]], np.array([0, 3], np.int32)
    u0, un = np.zeros(3, np.float32), np.array([0.0], np.float32)
    top = np.full(3, np.nextafter(np.float32(1), np.float32(0)), np.float32)
    t = lambda *x: np.array([0] + [at[i] for i in x], np.int32)  # noqa: E731

    def rows(x):
        big = np.zeros((len(x), V), np.float32)
        big[:, at] = x
        return big

    one = rows(np.eye(4, dtype=np.float32))
    _verify_check(ivc, one[[1, 2, 3]], None, t(1, 2), chain, off, top, un)
    _verify_check(ivc, one[[2, 2, 3]], None, t(1, 2), chain, off, u0, un)
    flat = rows(np.array([[0.5, 0.5, 0, 0]] * 3))
    _verify_check(ivc, flat, flat, t(1, 0), chain, off, top, un)
    _verify_check(ivc, flat, flat, t(2, 0), chain, off, u0, un)
    _verify_check(ivc, flat, None, t(2, 3), [[-1, 0, 0]], off, u0, un)
    for last in (0.0, 0.49999997, 0.5, float(top[0])):
        _verify_check(ivc, flat[:1], None, t(), [[-1]], off[:1].tolist() + [1], u0[:1],
                      np.array([last], np.float32))
    four = rows(np.array([[0.1, 0.2, 0.3, 0.4]] * 4))
    back = rows(np.array([[0.4, 0.3, 0.2, 0.1]] * 4))
    for q in (None, back):
        _verify_check(ivc, four, q, t(1, 1, 1), [[-1, 0, 0, 0]], np.array([0, 4], np.int32),
                      np.full(4, 0.9, np.float32), np.array([0.6], np.float32))


def test_verification_of_bad_rows_over_a_large_vocabulary():
    ivc, V = _ivc(), 5000
    rng = np.random.RandomState(2)
    p, q, tok, trees, off, u, un = _verify_case(rng, [3, 3], V, True, "chain")
    f = lambda x: dev(x, torch.float32)  # noqa: E731
    ws = ivc.new_workspace(256)

    def run(p=p, tok=tok, off=off):
        r = ivc.verify_drafts(f(p), f(q), dev(tok), None, dev(off), f(u), f(un), path_width=4, workspace=ws)
        return [x.cpu() for x in r], ivc.device_status(ws)

    good, st = run()
    assert st == 0
    zero = p.copy()
    zero[3:] = 0
    (path, m, t), st = run(p=zero)
    assert st == 256 and int(t[1]) == -1 and int(m[1]) == 1 and int(t[0]) == int(good[2][0])
    for x in (np.nan, -1.0):
        odd = p.copy()
        odd[:3] = x
        odd[:3, 4990] = 0.25
        (path, m, t), st = run(p=odd)
        assert st == 0 and int(t[0]) == 4990
    odd = p.copy()
    odd[:3, 2600] = np.inf
    (path, m, t), st = run(p=odd, tok=np.zeros_like(tok))
    assert st == 256 and int(t[0]) == -1
    wrong = tok.copy()
    wrong[1], wrong[4] = V, -3
    (path, m, t), st = run(tok=wrong)
    assert st == 256 and m.tolist() == [1, 1] and (t >= 0).all()
    (path, m, t), st = run(off=np.array([0, 5, 3], np.int32))
    assert st & 128 and int(m[1]) == 0 and int(t[1]) == -1


# ------------------------------------------------------------------ compaction
@pytest.mark.parametrize("kv,layers,n,D_", [(5, 12, 48, 64), (8, 10, 64, 64), (7, 6, 60, 128)])
def test_compaction_with_several_heads_per_cta(kv, layers, n, D_):
    """Many sequences and layers: a CTA moves a group of heads (the last group smaller,
    or all heads), over more than one chunk of rows."""
    ivc, pt = _ivc(), 16
    p = Pair(ivc, layers=layers, pages=6 * n, kv_heads=kv, pt=pt, D_=D_, seqs=n, max_pages=6)
    p.ws = ivc.new_workspace(ivc.cache_workspace_size(p.gpu, n, 70))
    rng = np.random.RandomState(1)
    lens = rng.randint(0, 20, n).tolist()
    seqs = rng.permutation(n).tolist()
    p.reserve(lens, seqs)
    p.compact(lens, seqs=seqs)
    p.reserve([70] * n, seqs)
    keep = [sorted(rng.permutation(70)[:60].tolist()) for _ in range(n)]
    count = [int(x) for x in rng.randint(0, 61, n)]
    p.compact(count, keep, None, seqs)


def test_the_largest_cache():
    """2^20 pages, the most that a cache may have: all of them taken, shared, given back."""
    ivc = _ivc()
    if torch.cuda.mem_get_info()[0] < 8 << 30:
        pytest.skip("needs 4 GB of device memory")
    pages, row = 1 << 20, 1 << 16            # a sequence's 65536 pages of 16 tokens
    c = ivc.Cache.empty(1, pages, 1, 16, 64, 20, row)
    ws = ivc.new_workspace(ivc.cache_workspace_size(c, 16, 0))
    full = dev([16 * row] * 16)
    ivc.cache_reserve(c, full, workspace=ws)
    ivc.cache_compact(c, full, workspace=ws)
    assert ivc.device_status(ws) == 0 and int(c.free_count) == 0
    held = torch.arange(pages, dtype=torch.int32, device="cuda")
    assert torch.equal(c.table[:16].reshape(-1), held) and (c.ref == 1).all()
    ivc.cache_reserve(c, dev([1]), dev([16]), workspace=ws)
    assert ivc.device_status(ws) == 64
    ivc.cache_fork(c, dev([3, 3]), dev([16, 17]), workspace=ws)     # every page is full: none is needed
    ivc.cache_fork(c, dev([3]), dev([18]), False, workspace=ws)     # and none is there to copy to
    assert ivc.device_status(ws) == 64
    assert torch.equal(c.table[16], c.table[3]) and (c.ref[3 * row:4 * row] == 3).all()
    ivc.cache_free(c, dev([3, 0, 15, 16]), workspace=ws)
    assert ivc.device_status(ws) == 0 and int(c.free_count) == 2 * row
    assert torch.equal(c.free_list[:2 * row], torch.cat([held[15 * row:].flip(0), held[:row].flip(0)]))
    ivc.cache_fork(c, dev([17, 7]), dev([18, 19]), False, workspace=ws)
    assert ivc.device_status(ws) == 0 and int(c.free_count) == 0
    assert torch.equal(c.table[18], held[:row]) and torch.equal(c.table[19], held[15 * row:])
    ivc.cache_free(c, dev([17, 18, 19, 1, 2, 4, 5, 6, 7, 8, 9, 10, 11, 12, 13, 14]), workspace=ws)
    assert ivc.device_status(ws) == 0 and int(c.free_count) == pages and (c.ref == 0).all()
    assert torch.equal(c.free_list.sort().values, held) and (c.table == -1).all()
