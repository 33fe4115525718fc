"""The decode step on the GPU against its fp64 oracle: paged cache operations
(equal, to the page number), per-head norms and rotation, attention of drafted
trees, verification of drafted tokens, and a run of them together.

Tolerances. norm + rotation: one bf16 rounding (2^-8 relative) of an fp32 value
whose two terms carry about 8 fp32 roundings and an angle rounded to fp32
(2^-23 of a half turn): under 2^-20 of the head's largest value. Attention: the
weights are rounded to bf16 (2^-8 relative each, so at most 2^-8 of the weighted
mean of |v|), then the output once (2^-8 relative); scores and sums in fp32 add
under 2^-14 of the mean of |v| for scores below 64.
"""
import numpy as np
import pytest
import torch

from oracle import decode_oracle as D

pytestmark = pytest.mark.gpu
BF = 2.0 ** -8


def _ivc():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import vlm_visual_token_b200 as ivc
    return ivc


def dev(x, dtype=torch.int32):
    return torch.as_tensor(np.asarray(x), dtype=dtype).cuda()


def np64(t):
    return t.detach().double().cpu().numpy()


class Pair:
    """The library's cache and the oracle's, changed together and compared."""

    def __init__(self, ivc, layers=2, pages=64, kv_heads=2, pt=16, D_=64, seqs=8, max_pages=24, seed=0):
        self.ivc = ivc
        self.gpu = ivc.Cache.empty(layers, pages, kv_heads, pt, D_, seqs, max_pages)
        self.ref = D.PagedCache(layers, pages, kv_heads, pt, D_, seqs, max_pages)
        g = torch.Generator().manual_seed(seed)
        for name in ("k", "v"):
            x = torch.randn(getattr(self.gpu, name).shape, generator=g).bfloat16()
            getattr(self.gpu, name).copy_(x)
            setattr(self.ref, name, np64(x))
        self.ws = ivc.new_workspace(ivc.cache_workspace_size(self.gpu, seqs, 512))

    def same(self, pages=True):
        c, r = self.gpu, self.ref
        np.testing.assert_array_equal(c.length.cpu().numpy(), r.length)
        np.testing.assert_array_equal(c.n_pages.cpu().numpy(), r.n_pages)
        np.testing.assert_array_equal(c.ref.cpu().numpy(), r.ref)
        np.testing.assert_array_equal(c.table.cpu().numpy(), r.table)
        free = int(c.free_count.cpu())
        assert c.free_list.cpu().numpy()[:free].tolist() == r.free
        assert (c.free_list.cpu().numpy()[free:] == -1).all()
        np.testing.assert_array_equal(np64(c.k), r.k)
        np.testing.assert_array_equal(np64(c.v), r.v)

    def both(self, gpu, ref, refused=0):
        """Run both; the status bits have to be `refused`, the states equal."""
        if refused:
            with pytest.raises(ValueError):
                ref()
        else:
            ref()
        gpu()
        assert self.ivc.device_status(self.ws) == refused
        self.same()

    def reserve(self, tokens, seqs, refused=0):
        self.both(lambda: self.ivc.cache_reserve(self.gpu, dev(tokens), dev(seqs), workspace=self.ws),
                  lambda: self.ref.reserve(tokens, seqs), refused)

    def fork(self, src, dst, share, refused=0):
        self.both(lambda: self.ivc.cache_fork(self.gpu, dev(src), dev(dst), share, workspace=self.ws),
                  lambda: self.ref.fork(src, dst, share), refused)

    def compact(self, count, keep=None, start=None, seqs=None, refused=0):
        self.both(lambda: self.ivc.cache_compact(
            self.gpu, dev(count), None if keep is None else dev(keep),
            None if start is None else dev(start), None if seqs is None else dev(seqs),
            workspace=self.ws), lambda: self.ref.compact(count, keep, start, seqs), refused)

    def free(self, seqs, refused=0):
        self.both(lambda: self.ivc.cache_free(self.gpu, dev(seqs), workspace=self.ws),
                  lambda: self.ref.drop(seqs), refused)


BAD, FULL = 32, 64


@pytest.mark.parametrize("pt,D_,kv", [(16, 64, 1), (32, 128, 3), (64, 64, 2), (128, 128, 8)])
def test_cache_life_of_forked_sequences(pt, D_, kv):
    p = Pair(_ivc(), layers=3, kv_heads=kv, pt=pt, D_=D_)
    n0, n1 = 3 * pt + 5, 2 * pt
    p.reserve([n0, n1, 0], [4, 1, 0])
    p.compact([n0, n1], seqs=[4, 1])              # committed: no keep list, start = length
    p.fork([4, 1, 4, 0], [0, 2, 3, 5], True)      # shared full pages, an empty source too
    p.reserve([7, pt + 1], [0, 2])
    p.compact([3, 2], [[0, 2, 6, 0], [0, pt, 0, 0]], None, [0, 2])
    p.free([4])                                   # its full pages live on in 0 and 3
    p.fork([0], [4], False)                       # every page copied
    p.compact([2 * pt + 1], [list(range(1, 2 * pt + 2))], [1], [4])
    p.free([0, 3, 4])
    p.free([1, 2, 5, 0])
    assert len(p.ref.free) == 64


@pytest.mark.parametrize("seed", range(6))
def test_cache_random_walk(seed):
    """Sixty random operations, refusals among them."""
    rng = np.random.RandomState(seed)
    p = Pair(_ivc(), layers=1, pages=40, kv_heads=2, seqs=8, max_pages=9, seed=seed)
    calls = {"reserve": (lambda t, s: p.ivc.cache_reserve(p.gpu, dev(t), dev(s), workspace=p.ws),
                         lambda t, s: p.ref.reserve(t, s)),
             "fork": (lambda a, b, c: p.ivc.cache_fork(p.gpu, dev(a), dev(b), c, workspace=p.ws),
                      lambda a, b, c: p.ref.fork(a, b, c)),
             "compact": (lambda m, k, a, s: p.ivc.cache_compact(p.gpu, dev(m), dev(k), dev(a), dev(s),
                                                                workspace=p.ws),
                         lambda m, k, a, s: p.ref.compact(m, k, a, s)),
             "free": (lambda s: p.ivc.cache_free(p.gpu, dev(s), workspace=p.ws),
                      lambda s: p.ref.drop(s))}
    done = 0
    for _ in range(60):
        what = rng.choice(["reserve", "reserve", "fork", "compact", "compact", "free"])
        s = rng.permutation(8)[:rng.randint(1, 4)].tolist()
        if what == "reserve":
            args = ([int(rng.randint(0, 60)) for _ in s], s)
        elif what == "fork":
            args = ([int(x) for x in rng.randint(0, 8, len(s))], s, bool(rng.randint(2)))
        elif what == "compact":
            start = [int(rng.randint(0, p.ref.length[x] + 1)) for x in s]
            keep, m = [], []
            for x, a in zip(s, start):
                room = int(p.ref.n_pages[x]) * 16 - a
                k = sorted(rng.permutation(room)[:rng.randint(0, room + 1)].tolist()) if room > 0 else []
                m.append(len(k))
                keep.append((k + [0] * 160)[:160])
            args = (m, keep, start, s)
        else:
            args = (s[:2],)
        want = 0
        try:
            calls[what][1](*args)
            done += 1
        except ValueError as e:
            want = BAD if str(e) == "bad" else FULL
        calls[what][0](*args)
        got = p.ivc.device_status(p.ws)
        # several sequences may be wrong in several ways: the first that the oracle names is among them
        assert got & want == want and (got == 0) == (want == 0), (what, args, got, want)
        p.same()
    assert done > 15


def test_cache_refusals_leave_everything():
    p = Pair(_ivc())
    p.reserve([40, 20], [0, 1])
    p.compact([40, 20], seqs=[0, 1])
    p.reserve([1, 1], [2, 2], refused=BAD)               # the same sequence twice
    p.reserve([1], [8], refused=BAD)                     # outside the cache
    p.reserve([-1], [2], refused=BAD)
    p.reserve([16 * 24 + 1], [2], refused=FULL)          # longer than a table row
    p.reserve([16 * 24, 16 * 24, 16 * 24], [2, 3, 4], refused=FULL)  # more than the free pages
    p.fork([0], [1], True, refused=BAD)                  # the target is not empty
    p.fork([0, 1], [2, 2], True, refused=BAD)
    p.fork([9], [2], True, refused=BAD)
    p.compact([9], [[0] * 9], None, [0], refused=BAD)    # not rising
    p.compact([1], [[8]], None, [0], refused=BAD)        # behind the pages
    p.compact([1], [[-1]], None, [0], refused=BAD)
    p.compact([1], [[0]], [41], [0], refused=BAD)        # a start behind the length
    p.compact([49], None, [0], [0], refused=BAD)
    p.fork([0], [3], True)
    p.compact([2], [[0, 3]], [0], [3], refused=BAD)      # would write a shared page
    p.compact([20], None, [0], [3], refused=BAD)         # would leave a shared page partly filled
    p.compact([16], None, [0], [3])                      # a full shared page may be the last
    p.free([-1], refused=BAD)
    p.free([0, 0], refused=BAD)
    p.fork([1, 3, 0], [4, 5, 6], False)


def test_cache_two_sequences_dropping_one_page_in_one_call():
    p = Pair(_ivc())
    p.reserve([64], [0])
    p.compact([64], seqs=[0])
    p.fork([0, 0, 0], [1, 2, 3], True)
    p.compact([32, 32, 16], None, [0, 0, 0], [1, 0, 2])
    p.free([3, 0, 1, 2])


def test_cache_bad_pages_are_not_followed():
    """Page numbers that are none: refused, nothing read or written through them."""
    p = Pair(_ivc())
    p.reserve([40], [0])
    p.compact([40], seqs=[0])
    good = p.gpu.table.clone()
    k = p.gpu.k.clone()
    for bad in (-1, 64, 1 << 30):
        p.gpu.table[0, 1] = bad
        for call in (lambda: p.ivc.cache_fork(p.gpu, dev([0]), dev([1]), False, workspace=p.ws),
                     lambda: p.ivc.cache_compact(p.gpu, dev([20]), dev([list(range(10, 30))]), dev([0]),
                                                 dev([0]), workspace=p.ws)):
            call()
            assert p.ivc.device_status(p.ws) == BAD
            assert torch.equal(p.gpu.k, k) and int(p.gpu.n_pages[0]) == 3 and int(p.gpu.n_pages[1]) == 0
    p.gpu.table.copy_(good)
    p.same()


# ------------------------------------------------------------------ norms and rotation
def _filled(ivc, lens, counts, layers=1, kv_heads=2, pt=16, D_=64, seed=1, order=None):
    """A cache holding lens tokens and pages for counts more, sequences in `order`."""
    order = list(range(len(lens))) if order is None else order
    need = [-(-(a + b) // pt) for a, b in zip(lens, counts)]
    p = Pair(ivc, layers, sum(need) + 2, kv_heads, pt, D_, max(order) + 1, max(need) + 1, seed)
    for tokens, commit in ((lens, True), (counts, False)):
        p.ref.reserve(tokens, order)
        ivc.cache_reserve(p.gpu, dev(tokens), dev(order))
        if commit:
            p.ref.compact(lens, seqs=order)
            ivc.cache_compact(p.gpu, dev(lens), seqs=dev(order))
    p.same()
    return p


@pytest.mark.parametrize("lens,counts,Hq,kv,pt,D_,pad", [
    ([0], [1], 1, 1, 16, 64, 0),
    ([15, 16, 0, 31], [1, 3, 17, 0], 4, 2, 16, 128, 3),
    ([100, 63], [70, 1], 15, 3, 64, 64, 0),
    ([5], [130], 40, 8, 128, 128, 1),
    ([0, 200], [33, 2], 71, 1, 32, 128, 0),
])
def test_qk_norm_rope(lens, counts, Hq, kv, pt, D_, pad):
    ivc = _ivc()
    order = list(range(len(lens)))[::-1]
    p = _filled(ivc, lens, counts, 2, kv, pt, D_, order=order)
    N = sum(counts)
    g = torch.Generator().manual_seed(3)
    width = (Hq + 2 * kv) * D_
    wide = torch.randn(N + pad, width + 24, generator=g).bfloat16()
    wide[0, :D_] = 0                         # a head of zeros: eps alone
    gam = [(1 + 0.3 * torch.randn(D_, generator=g)).bfloat16() for _ in range(2)]
    pos = np.random.RandomState(4).randint(0, 41000, N + pad).astype(np.int32)
    pos[0] = 2 ** 31 - 1
    off = np.concatenate([[0], np.cumsum(counts)])
    out = torch.full((N + pad, Hq, D_), 7.0, dtype=torch.bfloat16, device="cuda")
    ws = ivc.new_workspace(256)
    x = wide.cuda()[:, 8:8 + width]          # strided rows
    ivc.qk_norm_rope(p.gpu, 1, x, gam[0].cuda(), gam[1].cuda(), dev(pos), dev(off), 1e6, 1e-6,
                     seqs=dev(order), out=out, workspace=ws)
    assert ivc.device_status(ws) == 0
    h = np64(wide[:N, 8:8 + width]).reshape(N, Hq + 2 * kv, D_)
    q = D.norm_rope(h[:, :Hq], np64(gam[0]), pos, 1e6, 1e-6)
    k = D.norm_rope(h[:, Hq:Hq + kv], np64(gam[1]), pos, 1e6, 1e-6)
    close = lambda a, b: np.all(np.abs(a - b) <= BF * np.abs(b) + 2.0 ** -20 * np.abs(b).max(-1, keepdims=True))  # noqa: E731,E501
    assert close(np64(out[:N]), q)
    assert (out[N:] == 7.0).all()
    for i, s in enumerate(order):
        for t in range(counts[i]):
            page, slot = p.ref._slot(s, lens[i] + t)
            assert close(np64(p.gpu.k[1, page, :, slot]), k[off[i] + t])
            p.ref.k[1, page, :, slot] = np64(p.gpu.k[1, page, :, slot])
            p.ref.v[1, page, :, slot] = h[off[i] + t, Hq + kv:]
    p.same()                                 # nothing else was written


def test_qk_norm_rope_tokens_behind_the_pages_are_not_stored():
    ivc = _ivc()
    p = _filled(ivc, [10, 3], [6, 13])       # both end exactly with their page
    x = torch.randn(9, 4 * 64, dtype=torch.bfloat16, device="cuda")
    one = torch.ones(64, dtype=torch.bfloat16, device="cuda")
    ws = ivc.new_workspace(256)
    full = p.gpu.k.clone()
    ivc.qk_norm_rope(p.gpu, 0, x[:1, :5 * 64].repeat(1, 2)[:, :6 * 64].contiguous(), one, one, dev([0]),
                     dev([0, 0, 1]), seqs=dev([0, 7]), workspace=ws)
    assert ivc.device_status(ws) == BAD      # no such sequence
    assert torch.equal(full, p.gpu.k)
    x = torch.randn(7, 6 * 64, dtype=torch.bfloat16, device="cuda")
    q = ivc.qk_norm_rope(p.gpu, 0, x, one, one, dev(range(7)), dev([0, 7, 7]), workspace=ws)
    assert ivc.device_status(ws) == BAD      # the seventh token has no page
    assert torch.isfinite(q).all()
    changed = (p.gpu.k != full).any(-1).any(2)[0]  # [pages, slots]
    page = int(p.gpu.table[0, 0])
    assert changed[page].nonzero().flatten().tolist() == list(range(10, 16))
    changed[page] = False
    assert not changed.any()


# ------------------------------------------------------------------ attention
def _tree(rng, n, kind):
    if kind == "chain":
        return [i - 1 for i in range(n)]
    if kind == "star":
        return [-1] + [0] * (n - 1)
    if kind == "roots":
        return [-1] * n
    return [-1] + [int(rng.randint(max(-1, i - 6), i)) for i in range(1, n)]


def _attend_case(lens, counts, Hq, kv, pt, D_, kind, seed=5, order=None, spread=1.0):
    ivc = _ivc()
    p = _filled(ivc, lens, counts, 2, kv, pt, D_, seed=seed, order=order)
    N = sum(counts)
    g = torch.Generator().manual_seed(seed)
    q = (spread * torch.randn(N, Hq, D_, generator=g)).bfloat16().cuda()
    rng = np.random.RandomState(seed)
    trees = [_tree(rng, n, kind) for n in counts]
    off = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    return ivc, p, q, trees, off


def _attend_ref(p, q, trees, off, lens, counts, order, layer, scale):
    want, size = [], []
    for i, n in enumerate(counts):
        k, v = p.ref.tokens(order[i], lens[i] + n, layer)
        qq = np64(q[off[i]:off[i + 1]])
        want.append(D.tree_attend(qq, k, v, lens[i], trees[i], scale))
        size.append(D.tree_attend(qq, k, np.abs(v), lens[i], trees[i], scale))
    return np.concatenate(want), np.concatenate(size)


def _attend_close(got, want, size):
    err = np.abs(np64(got) - want)
    assert np.all(err <= BF * np.abs(want) + (BF + 2.0 ** -14) * size), float((err / size).max())


@pytest.mark.parametrize("lens,counts,Hq,kv,pt,D_,kind", [
    ([0], [1], 1, 1, 16, 64, "chain"),
    ([1], [1], 4, 1, 16, 128, "chain"),
    ([127, 128, 129, 0], [1, 1, 1, 1], 8, 2, 64, 128, "chain"),
    ([300, 17, 64, 1000], [1, 1, 0, 1], 8, 8, 16, 64, "chain"),
    ([120], [20], 4, 4, 128, 128, "tree"),
    ([200, 5, 250], [27, 3, 6], 8, 2, 32, 64, "tree"),
    ([0, 90], [128, 100], 4, 2, 16, 128, "tree"),
    ([31], [128], 8, 1, 64, 128, "star"),
    ([50], [37], 10, 2, 16, 64, "roots"),
    ([700], [33], 21, 3, 128, 128, "chain"),
    ([260], [7], 64, 1, 64, 128, "tree"),
    ([140], [65], 12, 4, 32, 128, "tree"),
])
def test_tree_attention(lens, counts, Hq, kv, pt, D_, kind):
    order = list(range(len(lens)))[::-1]
    ivc, p, q, trees, off = _attend_case(lens, counts, Hq, kv, pt, D_, kind, order=order)
    N = sum(counts)
    ws = ivc.new_workspace(ivc.tree_attention_workspace_size(p.gpu, N + 2, Hq, len(lens)))
    out = torch.full((N + 2, Hq, D_), 7.0, dtype=torch.bfloat16, device="cuda")
    qq = torch.zeros(N + 2, Hq + 2, D_, dtype=torch.bfloat16, device="cuda")
    qq[:N, 1:-1] = q
    par = dev(sum(trees, []) + [-1, -1])
    ivc.tree_attention(p.gpu, 1, qq[:, 1:-1], par, dev(off), seqs=dev(order), out=out, workspace=ws)
    assert ivc.device_status(ws) == 0
    want, size = _attend_ref(p, q, trees, off, lens, counts, order, 1, D_ ** -0.5)
    _attend_close(out[:N], want, size)
    assert (out[N:] == 7.0).all()
    if kind == "chain":
        same = ivc.tree_attention(p.gpu, 1, q, None, dev(off), seqs=dev(order))
        assert torch.equal(same, out[:N])


def test_tree_attention_long_context_many_splits():
    lens, counts = [9001, 40], [5, 2]
    ivc, p, q, trees, off = _attend_case(lens, counts, 8, 2, 64, 128, "tree", spread=3.0)
    got = ivc.tree_attention(p.gpu, 0, q, dev(sum(trees, [])), dev(off), scale=0.11)
    want, size = _attend_ref(p, q, trees, off, lens, counts, [0, 1], 0, 0.11)
    _attend_close(got, want, size)


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("Hq", [2, 16])
def test_tree_attention_is_not_touched_by_what_it_does_not_see(bad, Hq):
    """Unseen siblings, slots behind the sequence in its last page, pages of others:
    non-finite values there change nothing, and in a seen node they show."""
    lens, counts = [130, 20], [20, 9]
    ivc, p, q, trees, off = _attend_case(lens, counts, Hq, 2, 32, 128, "tree")
    trees = [[-1] + [0] * 19, [-1, 0, 0, 1, 1, 2, 2, 3, 3]]
    par = dev(sum(trees, []))
    clean = ivc.tree_attention(p.gpu, 0, q, par, dev(off))
    used = torch.zeros(p.gpu.k.shape[1], 32, dtype=torch.bool)
    for s in range(2):
        for t in range(lens[s] + counts[s]):
            page, slot = p.ref._slot(s, t)
            used[page, slot] = True
    for x in (p.gpu.k, p.gpu.v):
        x[0].masked_fill_(~used.cuda()[:, None, :, None], bad)
    assert torch.equal(ivc.tree_attention(p.gpu, 0, q, par, dev(off)), clean)
    page, slot = p.ref._slot(0, 130 + 7)     # node 7 of the star: only itself sees it
    p.gpu.v[0, page, 1, slot, 5] = bad
    got = ivc.tree_attention(p.gpu, 0, q, par, dev(off))
    touched = got.float().isnan() | got.float().isinf()
    want = torch.zeros_like(touched)
    want[7, Hq // 2:, 5] = True              # kv head 1
    assert torch.equal(touched, want)
    assert torch.equal(got[~want], clean[~want])
    p.gpu.v[0, page, 1, slot, 5] = 0
    p.gpu.k[0, page, 0, slot, 3] = bad
    got = ivc.tree_attention(p.gpu, 0, q, par, dev(off))
    rows = torch.ones(q.shape[0], Hq, dtype=torch.bool)
    rows[7, :Hq // 2] = False
    base = ivc.tree_attention(p.gpu, 0, q, par, dev(off))
    assert torch.equal(got[rows.cuda()], base[rows.cuda()])
    assert torch.isfinite(got[rows.cuda()].float()).all()


def test_tree_attention_large_scores_and_one_dominant_key():
    """Scores of +-1000 (after scale): the running maximum keeps every exponent at most 0."""
    lens, counts = [400], [3]
    ivc, p, q, trees, off = _attend_case(lens, counts, 4, 2, 16, 64, "chain", spread=400.0)
    got = ivc.tree_attention(p.gpu, 0, q, None, dev(off))
    want, size = _attend_ref(p, q, trees, off, lens, counts, [0], 0, 0.125)
    # fp32 scores of up to 2^11 with 64 products: an absolute error below 2^11 * 2^-24 * 16 = 2^-9
    err = np.abs(np64(got) - want)
    assert np.all(err <= BF * np.abs(want) + (BF + 2.0 ** -8) * size)


def test_tree_attention_bad_device_data():
    ivc = _ivc()
    p = _filled(ivc, [40, 20], [6, 6])
    q = torch.randn(12, 4, 64, dtype=torch.bfloat16, device="cuda")
    ws = ivc.new_workspace(ivc.tree_attention_workspace_size(p.gpu, 200, 4, 2))
    good = ivc.tree_attention(p.gpu, 0, q, None, dev([0, 6, 12]))

    def run(par, off, seqs=None, qq=q):
        out = torch.full((qq.shape[0], 4, 64), 7.0, dtype=torch.bfloat16, device="cuda")
        ivc.tree_attention(p.gpu, 0, qq, par, dev(off), seqs=seqs, out=out, workspace=ws)
        return out, ivc.device_status(ws)

    chain = [-1, 0, 1, 2, 3, 4]
    out, st = run(dev([-1, 0, 1, 3, 3, 4] + chain), [0, 6, 12])       # a node as its own parent
    assert st == 128 and torch.equal(out[6:], good[6:]) and torch.equal(out[:3], good[:3])
    out, st = run(None, [0, 6, 12], dev([0, 9]))
    assert st == BAD and torch.equal(out[:6], good[:6]) and (out[6:] == 7).all()
    out, st = run(None, [0, 12, 6])
    assert st & 128
    lone = ivc.tree_attention(p.gpu, 0, q[:2], None, dev([0, 1, 2]))
    out, st = run(dev([0, -1]), [0, 1, 2], qq=q[:2])                  # a single node with a parent
    assert st == 128 and torch.equal(out, lone)
    big = torch.randn(140, 4, 64, dtype=torch.bfloat16, device="cuda")
    out, st = run(None, [0, 6, 140], qq=big)                          # more than 128 nodes
    assert st & 128 and (out[6:] == 7).all() and torch.isfinite(out[:6].float()).all()
    out, st = run(None, [0, 12, 12])                                  # tokens without pages
    assert st & BAD and (out == 7).all()
    p.gpu.table[1, 0] = 1 << 20
    out, st = run(None, [0, 6, 12])
    assert st & BAD and torch.equal(out[:6], good[:6])


# ------------------------------------------------------------------ verification
def _verify_case(rng, counts, V, dense, kind, peaked=2.0):
    N = sum(counts)
    soft = lambda x: (np.exp(x) / np.exp(x).sum(-1, keepdims=True)).astype(np.float32)  # noqa: E731
    base = peaked * rng.randn(N, V)
    p = soft(base)
    q = soft(base + rng.randn(N, V))
    trees = [_tree(rng, n, kind) if n else [] for n in counts]
    trees = [[-1] + [max(0, x) for x in t[1:]] if t else [] for t in trees]
    tok = np.zeros(N, np.int32)
    off = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    for b, t in enumerate(trees):
        for j in range(1, len(t)):
            w = q[off[b] + t[j]].astype(np.float64)
            tok[off[b] + j] = rng.choice(V, p=w / w.sum())
    return p, (q if dense else None), tok, trees, off, rng.rand(N).astype(np.float32), \
        rng.rand(len(counts)).astype(np.float32)


def _verify_check(ivc, p, q, tok, trees, off, u, un, width=12, status=0, ld=None):
    B = len(trees)
    f = lambda x: None if x is None else dev(x, torch.float32)  # noqa: E731
    ws = ivc.new_workspace(256)
    pp, qq = f(p), f(q)
    if ld:
        room = torch.full((p.shape[0], ld), float("nan"), device="cuda")
        room[:, 1:1 + p.shape[1]] = pp
        pp = room[:, 1:1 + p.shape[1]]
    path, m, t = ivc.verify_drafts(pp, qq, dev(tok), dev(sum(trees, [])), dev(off), f(u), f(un),
                                   path_width=width, workspace=ws)
    assert ivc.device_status(ws) == status
    for b in range(B):
        a, e = off[b], off[b + 1]
        if a == e:
            assert int(m[b]) == 0 and int(t[b]) == -1 and (path[b] == -1).all()
            continue
        want, nxt = D.verify(p[a:e].astype(np.float64), None if q is None else q[a:e].astype(np.float64),
                             tok[a:e], trees[b], u[a:e].astype(np.float64), float(un[b]))
        assert int(m[b]) == len(want), b
        assert path[b].tolist() == want + [-1] * (width - len(want))
        assert int(t[b]) == nxt
    return path, m, t


@pytest.mark.parametrize("dense", [False, True])
@pytest.mark.parametrize("kind", ["chain", "star", "tree"])
@pytest.mark.parametrize("V", [1, 2, 37, 1024, 5003])
def test_verify_drafts(dense, kind, V):
    rng = np.random.RandomState(V + 7 * dense)
    case = _verify_case(rng, [1, 9, 4, 0, 12, 2, 7, 12], V, dense, kind)
    _verify_check(_ivc(), *case)


@pytest.mark.parametrize("dense", [False, True])
def test_verify_drafts_wide_trees_and_strided_rows(dense):
    rng = np.random.RandomState(11)
    case = _verify_case(rng, [128, 100], 211, dense, "tree", peaked=0.3)
    _verify_check(_ivc(), *case, width=128, ld=260)
    star = _verify_case(rng, [128], 97, dense, "star", peaked=0.1)
    _verify_check(_ivc(), *star, width=128)


def test_verify_drafts_borders():
    """u = 0, certain tokens, equal distributions, rows that leave nothing."""
    ivc = _ivc()
    one = np.eye(4, dtype=np.float32)
    chain = [[-1, 0, 1]]
    off = np.array([0, 3], np.int32)
    u0, un = np.zeros(3, np.float32), np.array([0.0], np.float32)
    # the target is certain of the drafted tokens: all stand, also at the largest u below 1
    top = np.full(3, np.nextafter(np.float32(1), np.float32(0)), np.float32)
    _verify_check(ivc, one[[1, 2, 3]], None, np.array([0, 1, 2], np.int32), chain, off, top, un)
    # certain of others: none stands, u = 0 included
    _verify_check(ivc, one[[2, 2, 3]], None, np.array([0, 1, 2], np.int32), chain, off, u0, un)
    # draft and target equal: always stands; a token that neither gives never does
    flat = np.array([[0.5, 0.5, 0, 0]] * 3, np.float32)
    _verify_check(ivc, flat, flat, np.array([0, 1, 0], np.int32), chain, off, top, un)
    _verify_check(ivc, flat, flat, np.array([0, 2, 0], np.int32), chain, off, u0, un)
    # every sibling rejected until nothing is left: drawn from the node's own row
    _verify_check(ivc, flat, None, np.array([0, 2, 3], np.int32), [[-1, 0, 0]], off, u0, un)
    for last in (0.0, 0.49999997, 0.5, float(top[0])):
        _verify_check(ivc, flat[:1], None, np.array([0], np.int32), [[-1]],
                      np.array([0, 1], np.int32), u0[:1], np.array([last], np.float32))
    # the same token twice among siblings
    p = np.array([[0.1, 0.2, 0.3, 0.4]] * 4, np.float32)
    half = np.full(4, 0.9, np.float32)
    for q in (None, p[:, ::-1].copy()):
        _verify_check(ivc, p, q, np.array([0, 1, 1, 1], np.int32), [[-1, 0, 0, 0]],
                      np.array([0, 4], np.int32), half, np.array([0.6], np.float32))


def test_verify_drafts_bad_device_data():
    ivc = _ivc()
    rng = np.random.RandomState(2)
    p, q, tok, trees, off, u, un = _verify_case(rng, [3, 3], 50, True, "chain")
    f = lambda x: dev(x, torch.float32)  # noqa: E731
    ws = ivc.new_workspace(256)

    def run(p=p, tok=tok, par=None, off=off):
        r = ivc.verify_drafts(f(p), f(q), dev(tok), par, dev(off), f(u), f(un), path_width=4, workspace=ws)
        return [x.cpu() for x in r], ivc.device_status(ws)

    good, st = run()
    assert st == 0
    zero = p.copy()
    zero[3:] = 0
    (path, m, t), st = run(p=zero)
    assert st == 256 and int(t[1]) == -1 and int(m[1]) == 1 and int(t[0]) == int(good[2][0])
    for x in (np.nan, -1.0):                       # count as nothing
        odd = p.copy()
        odd[:3] = x
        odd[:3, 7] = 0.25
        (path, m, t), st = run(p=odd)
        assert st == 0 and int(t[0]) == 7
    odd = p.copy()
    odd[:3, 8] = np.inf
    (path, m, t), st = run(p=odd, tok=np.zeros_like(tok))
    assert st == 256 and int(t[0]) == -1
    wrong = tok.copy()
    wrong[1], wrong[4] = 50, -3
    (path, m, t), st = run(tok=wrong)
    assert st == 256 and m.tolist() == [1, 1] and (t >= 0).all()
    (path, m, t), st = run(off=np.array([0, 5, 3], np.int32))
    assert st & 128 and int(m[1]) == 0 and int(t[1]) == -1
    (path, m, t), st = run(par=dev([-1, 1, 0, -1, 0, 1]))
    assert st == 128                               # a bad parent counts as a root: never reached
    assert int(m[1]) == int(good[1][1])


def test_verify_drafts_draws_from_the_target():
    """Over a fine grid of the random numbers the next token after a rejected or
    accepted draft is distributed as the target: each token's share of the grid
    is off by at most its cells at interval borders."""
    ivc = _ivc()
    p = np.array([[0.40, 0.05, 0.30, 0.25]], np.float32)
    q = np.array([[0.10, 0.55, 0.20, 0.15]], np.float32)
    G = 64
    grid = ((np.arange(G) + 0.5) / G).astype(np.float32)
    share = np.zeros(4)
    for c in range(4):  # the drafted token c has probability q[c]
        rows = G * G
        u = np.repeat(grid, G)
        un = np.tile(grid, G)
        P = np.repeat(p, 2 * rows, 0)
        off = np.arange(0, 2 * rows + 1, 2)
        tok = np.tile(np.array([0, c], np.int32), rows)
        uu = np.zeros(2 * rows, np.float32)
        uu[1::2] = u
        path, m, t = ivc.verify_drafts(dev(P, torch.float32), dev(np.repeat(q, 2 * rows, 0), torch.float32),
                                       dev(tok), None, dev(off), dev(uu, torch.float32),
                                       dev(un, torch.float32), path_width=2)
        first = torch.where(m == 2, c, t).cpu().numpy()
        share += q[0, c] * np.bincount(first, minlength=4) / rows
    # a border moves at most one of G columns of u and one of G of u_next per draft
    assert np.abs(share - p[0]).max() <= 2.0 / G


# ------------------------------------------------------------------ the step as a whole
def _step_inputs(B, Hq, kv, D_, V, n, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    N = B * n
    return {"qkv": r(2, N, (Hq + 2 * kv) * D_).bfloat16(), "gam": (1 + 0.1 * r(2, D_)).bfloat16(),
            "p": torch.softmax(2 * r(N, V), -1), "q": torch.softmax(2 * r(N, V), -1),
            "tok": torch.randint(0, V, (N,), generator=g, device="cuda", dtype=torch.int32),
            "u": torch.rand(N, generator=g, device="cuda"), "un": torch.rand(B, generator=g, device="cuda")}


def _one_step(ivc, c, x, par, off, n_new, lens_pos, ws):
    ivc.cache_reserve(c, n_new, workspace=ws)
    outs = []
    for layer in range(2):
        q = ivc.qk_norm_rope(c, layer, x["qkv"][layer], x["gam"][0], x["gam"][1], lens_pos, off,
                             workspace=ws)
        outs.append(ivc.tree_attention(c, layer, q, par, off, workspace=ws))
    path, m, t = ivc.verify_drafts(x["p"], x["q"], x["tok"], par, off, x["u"], x["un"], path_width=8,
                                   workspace=ws)
    ivc.cache_compact(c, m, path, workspace=ws)
    return outs, path, m, t


def test_decode_steps_together_eager_and_captured():
    """Prefix, fork, three speculative steps: what the cache holds afterwards is
    what storing the accepted tokens one after the other gives, and a captured
    graph replayed on the same state gives the same bits."""
    ivc = _ivc()
    B, Hq, kv, D_, V, n, pt = 3, 8, 2, 64, 300, 7, 16
    tree = [-1, 0, 0, 1, 1, 2, 3]
    par, off = dev(tree * B), dev([n * i for i in range(B + 1)])
    n_new = dev([n] * B)

    def fresh():
        c = ivc.Cache.empty(2, 40, kv, pt, D_, B, 12)
        pre = dev([37, 0, 0])
        ivc.cache_reserve(c, pre)
        x = _step_inputs(1, Hq, kv, D_, V, 37, 1)
        for layer in range(2):
            ivc.qk_norm_rope(c, layer, x["qkv"][layer], x["gam"][0], x["gam"][1],
                             dev(range(37)), dev([0, 37, 37, 37]))
        ivc.cache_compact(c, pre)
        ivc.cache_fork(c, dev([0, 0]), dev([1, 2]))
        return c

    steps = [_step_inputs(B, Hq, kv, D_, V, n, 10 + i) for i in range(3)]
    depth = dev([len(D.ancestors(tree, i)) - 1 for i in range(n)])
    a, log = fresh(), []
    ws = ivc.new_workspace(max(ivc.tree_attention_workspace_size(a, B * n, Hq, B),
                               ivc.cache_workspace_size(a, B, 8)))
    for x in steps:
        pos = (a.length[:, None] + depth).reshape(-1).to(torch.int32).contiguous()
        log.append(_one_step(ivc, a, x, par, off, n_new, pos, ws))
    assert ivc.device_status(ws) == 0

    # the same tokens stored one after the other
    b = fresh()
    for x, (outs, path, m, t) in zip(steps, log):
        pos = (b.length[:, None] + depth).reshape(-1).to(torch.int32)
        for s in range(B):
            k = int(m[s])
            rows = (s * n + path[s, :k]).long()
            one = torch.zeros(B, dtype=torch.int32, device="cuda")
            one[s] = k
            ivc.cache_reserve(b, one)
            o = torch.cat([torch.zeros(1, device="cuda"), one.cumsum(0)]).to(torch.int32)
            for layer in range(2):
                q = ivc.qk_norm_rope(b, layer, x["qkv"][layer][rows].contiguous(), x["gam"][0], x["gam"][1],
                                     pos[rows].contiguous(), o)
                chain = ivc.tree_attention(b, layer, q, None, o)
                d = (chain.float() - outs[layer][rows].float()).abs().max()
                assert d <= 2 * (2 * BF + 2.0 ** -13) * 6  # two roundings each of values below 6
            ivc.cache_compact(b, one)
    assert torch.equal(a.length, b.length)
    for s in range(B):
        L = int(a.length[s])
        for x in ("k", "v"):
            get = lambda c: getattr(c, x)[:, c.table[s, :-(-L // pt)].long()].transpose(2, 3).reshape(2, -1, kv, D_)[:, :L]  # noqa: E731,E501
            assert torch.equal(get(a), get(b))

    # one step captured, replayed on the same state
    c = fresh()
    x = steps[0]
    pos = (c.length[:, None] + depth).reshape(-1).to(torch.int32).contiguous()
    state = [t.clone() for t in (c.k, c.v, c.table, c.length, c.n_pages, c.ref, c.free_list, c.free_count)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        _one_step(ivc, c, x, par, off, n_new, pos, ws)     # first use outside the capture
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs, path, m, t = _one_step(ivc, c, x, par, off, n_new, pos, ws)
    for _ in range(2):
        for dst, src in zip((c.k, c.v, c.table, c.length, c.n_pages, c.ref, c.free_list, c.free_count), state):
            dst.copy_(src)
        graph.replay()
        torch.cuda.synchronize()
        for u, v in zip([*outs, path, m, t], [*log[0][0], *log[0][1:]]):
            assert torch.equal(u, v)
    assert ivc.device_status(ws) == 0


def test_calls_on_another_stream_and_without_workspaces():
    ivc = _ivc()
    p = _filled(ivc, [50, 40], [3, 3])
    q = torch.randn(6, 4, 64, dtype=torch.bfloat16, device="cuda")
    want = ivc.tree_attention(p.gpu, 0, q, None, dev([0, 3, 6]))
    off = dev([0, 3, 6])
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for _ in range(3):
        got = ivc.tree_attention(p.gpu, 0, q, None, off, stream=s)
    s.synchronize()
    assert torch.equal(got, want)


def test_pages_beyond_32_bit_offsets():
    """A cache of 5 GB a layer: the same step in its last pages of layer 1 and in a
    small cache gives the same bits."""
    ivc = _ivc()
    if torch.cuda.mem_get_info()[0] < 30 << 30:
        pytest.skip("needs 22 GB of device memory")
    Hq, kv, pt, D_ = 8, 8, 128, 128
    par, off = dev([-1, 0, 0, 1, 1, 2, -1, 0, 1]), dev([0, 6, 9])

    def step(pages, first):
        c = ivc.Cache.empty(2, pages, kv, pt, D_, 3, 8)
        order = torch.arange(first, first + 8, dtype=torch.int32, device="cuda")
        c.free_list[-8:] = order            # taken from the last one down
        ws = ivc.new_workspace(ivc.tree_attention_workspace_size(c, 9, Hq, 2))
        pre = dev([300, 100])
        g = torch.Generator(device="cuda").manual_seed(9)
        outs = []
        for counts, parents, offs in ((pre, None, dev([0, 300, 400])), (dev([6, 3]), par, off)):
            n = int(offs[-1])
            ivc.cache_reserve(c, counts, workspace=ws)
            for layer in (0, 1):
                x = torch.randn(n, (Hq + 2 * kv) * D_, generator=g, device="cuda").bfloat16()
                one = torch.ones(D_, dtype=torch.bfloat16, device="cuda")
                q = ivc.qk_norm_rope(c, layer, x, one, one, dev(range(n)), offs, workspace=ws)
                if parents is not None:
                    outs.append(ivc.tree_attention(c, layer, q, parents, offs, workspace=ws))
            if parents is None:
                ivc.cache_compact(c, counts)
        ivc.cache_compact(c, dev([3, 1]), dev([[0, 2, 5], [1, 0, 0]]))
        ivc.cache_fork(c, dev([0]), dev([2]), False)
        for s, n in ((0, 303), (1, 101), (2, 303)):
            pages_of = c.table[s, :-(-n // pt)].long()
            for x in (c.k, c.v):
                outs.append(x[1, pages_of].transpose(1, 2).reshape(-1, kv, D_)[:n])
        assert ivc.device_status(ws) == 0
        return outs

    small = step(12, 4)
    far = step(20000, 19992)
    assert all(torch.equal(a, b) for a, b in zip(small, far))
    assert torch.equal(far[2], far[6])


def test_two_streams_with_their_own_workspaces_and_two_graphs():
    """Attention over one cache from two streams at once, eager and as replayed
    graphs, each with its own workspace."""
    lens, counts = [900, 77, 300], [9, 1, 20]
    ivc, p, q, trees, off = _attend_case(lens, counts, 16, 2, 32, 128, "tree")
    par, off = dev(sum(trees, [])), dev(off)
    want = ivc.tree_attention(p.gpu, 0, q, par, off), ivc.tree_attention(p.gpu, 1, q, par, off)
    size = ivc.tree_attention_workspace_size(p.gpu, 30, 16, 3)
    spaces = [ivc.new_workspace(size) for _ in range(2)]
    outs = [torch.empty_like(want[0]) for _ in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    graphs = []
    torch.cuda.synchronize()
    for layer, (s, ws, o) in enumerate(zip(streams, spaces, outs)):
        for _ in range(4):
            ivc.tree_attention(p.gpu, layer, q, par, off, out=o, workspace=ws, stream=s)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(outs, want))
    for layer, (ws, o) in enumerate(zip(spaces, outs)):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            ivc.tree_attention(p.gpu, layer, q, par, off, out=o, workspace=ws)
        graphs.append(g)
        o.zero_()
    torch.cuda.synchronize()
    for _ in range(4):
        for s, g in zip(streams, graphs):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(outs, want))
    assert [ivc.device_status(ws) for ws in spaces] == [0, 0]


@pytest.mark.parametrize("B,Hq,kv,D_,pt", [(300, 4, 2, 64, 16), (4096, 2, 1, 64, 32), (70, 24, 8, 128, 64)])
def test_tree_attention_many_short_sequences(B, Hq, kv, D_, pt):
    """More items than CTAs, empty sequences among them, against torch in float64."""
    ivc = _ivc()
    rng = np.random.RandomState(B)
    lens, counts = rng.randint(0, 150, B), rng.randint(0, 4, B)
    need = -(-(lens + counts) // pt)
    c = ivc.Cache.empty(1, int(need.sum()) + 1, kv, pt, D_, B, int(need.max()) + 1)
    c.k.normal_()
    c.v.normal_()
    ivc.cache_reserve(c, dev(lens))
    ivc.cache_compact(c, dev(lens))
    ivc.cache_reserve(c, dev(counts))
    N = int(counts.sum())
    q = torch.randn(N, Hq, D_, device="cuda").bfloat16()
    off = dev(np.concatenate([[0], np.cumsum(counts)]))
    ws = ivc.new_workspace(ivc.tree_attention_workspace_size(c, N, Hq, B))
    got = ivc.tree_attention(c, 0, q, None, off, workspace=ws)
    assert ivc.device_status(ws) == 0
    row = 0
    for b in range(B):
        n, m = int(counts[b]), int(lens[b])
        if n == 0:
            continue
        pages = c.table[b, :need[b]].long()
        k, v = (x[0, pages].transpose(1, 2).reshape(-1, kv, D_)[:m + n].double()
                .repeat_interleave(Hq // kv, 1) for x in (c.k, c.v))
        s = torch.einsum("nhd,lhd->hnl", q[row:row + n].double(), k) * D_ ** -0.5
        see = torch.ones(n, m + n, dtype=torch.bool, device="cuda").tril(m)
        w = torch.softmax(s.masked_fill(~see, float("-inf")), -1)
        want, size = torch.einsum("hnl,lhd->nhd", w, v), torch.einsum("hnl,lhd->nhd", w, v.abs())
        err = (got[row:row + n].double() - want).abs()
        assert bool((err <= BF * want.abs() + (BF + 2.0 ** -14) * size).all()), b
        row += n


def test_cache_many_sequences_in_one_call():
    """More sequences than a CTA has threads: one reserve, fork, compact and free."""
    ivc = _ivc()
    n, pt = 1500, 16
    p = Pair(ivc, layers=1, pages=4 * n, kv_heads=1, pt=pt, seqs=2 * n, max_pages=3)
    p.ws = ivc.new_workspace(ivc.cache_workspace_size(p.gpu, n, 8))
    rng = np.random.RandomState(0)
    seqs = rng.permutation(2 * n)[:n].tolist()
    rest = [s for s in range(2 * n) if s not in set(seqs)]
    lens = rng.randint(0, 3 * pt, n).tolist()
    p.reserve(lens, seqs)
    p.compact(lens, seqs=seqs)
    p.fork(seqs, rest, True)
    # every third copy keeps up to eight tokens of what it alone holds
    start = [x // pt * pt for x in lens]
    keep = [sorted(rng.permutation(max(x - a, 1))[:8].tolist()) for x, a in zip(lens, start)]
    count = [0 if x == a else min(len(k), 8) for x, a, k in zip(lens, start, keep)]
    keep = [(k + [0] * 8)[:8] for k in keep]
    p.compact(count, keep, start, rest)
    p.free(rest[:n // 2] + seqs[n // 2:])
    p.free(rest[n // 2:] + seqs[:n // 2])
    assert len(p.ref.free) == 4 * n
