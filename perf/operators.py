"""Cases of the decode-step operators over a paged cache, with their plain forms.

Kinds of cases:
  norm      qk_norm_rope: per-head norms and rotation of q and k, k and v stored in the pages
  attend    tree_attention: drafted tokens (a tree; one token = plain decoding) over the pages
  verify    verify_drafts: the drafted tree against the target's probabilities
  pages     cache_free, cache_fork, cache_reserve, cache_compact: the life of a forked sequence
"""
import math

import torch

own = False
DEV = "cuda"
THETA, EPS = 1e6, 1e-6


# ---------------------------------------------------------------------------- cases
def listed():
    return [
        # one new token of one conversation: a launch's latency
        dict(name="norm_1tok", kind="norm", B=1, n=1, q_heads=32, kv_heads=8, D=128, page=64, ctx=3400),
        # 32-node drafts of 16 conversations
        dict(name="norm_16x32", kind="norm", B=16, n=32, q_heads=32, kv_heads=8, D=128, page=64, ctx=4000),
        # prefill of four spliced image prompts
        dict(name="norm_prefill", kind="norm", B=4, n=3500, q_heads=32, kv_heads=8, D=128, page=64, ctx=0),
        # one short conversation, one token
        dict(name="attend_short", kind="attend", B=1, n=1, q_heads=32, kv_heads=8, D=128, page=64, ctx=333),
        # plain decoding of a batch behind image prompts
        dict(name="attend_decode", kind="attend", B=48, n=1, q_heads=32, kv_heads=8, D=128, page=64, ctx=4500),
        # drafted trees of a batch, small pages, ragged contexts
        dict(name="attend_tree", kind="attend", B=24, n=27, q_heads=32, kv_heads=8, D=128, page=16, ctx=6000),
        # wide trees near the end of a 40960-token context
        dict(name="attend_long", kind="attend", B=4, n=64, q_heads=32, kv_heads=8, D=128, page=128, ctx=40800),
        # one conversation, a short draft given without probabilities
        dict(name="verify_one", kind="verify", B=1, n=6, V=32000, dense=False, wide=False, agree=0.6),
        # a batch of wide trees drafted with probabilities
        dict(name="verify_trees", kind="verify", B=48, n=16, V=151001, dense=True, wide=True, agree=0.7),
        # several answers branched off image prompts: full pages shared
        dict(name="pages_branch", kind="pages", n=8, layers=36, kv_heads=8, D=128, page=64, ctx=3401,
             share=True, draft=16, keep=5, thin=False),
        # a batch's accepted drafts moved together in every layer
        dict(name="pages_accept", kind="pages", n=48, layers=36, kv_heads=8, D=128, page=16, ctx=200,
             share=True, draft=32, keep=7, thin=False),
        # copies of image prompts thinned from 256 to 64 tokens a tile
        dict(name="pages_thin", kind="pages", n=3, layers=36, kv_heads=8, D=128, page=64, ctx=3390,
             share=False, draft=1, keep=0, thin=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["norm", "attend", "attend", "verify", "pages"])
    D = rng.choice([64, 128, 128])
    page = rng.choice([16, 32, 64, 128])
    kv = rng.choice([1, 2, 4, 8, 8])
    heads = kv * rng.choice([1, 2, 4, 4, 5, 7, 8])
    if kind == "norm":
        B = _log(rng, 1, 64)
        most = 500000 // (heads + 2 * kv)
        return dict(kind=kind, B=B, n=_log(rng, 1, max(1, most // B)), q_heads=heads, kv_heads=kv, D=D,
                    page=page, ctx=rng.choice([0, _log(rng, 1, 4000)]))
    if kind == "attend":
        B = _log(rng, 1, 64)
        n = rng.choice([1, _log(rng, 2, 128)])
        heads = max(kv, min(heads, 2048 // n // kv * kv))
        return dict(kind=kind, B=B, n=n, q_heads=heads, kv_heads=kv, D=D, page=page,
                    ctx=_log(rng, 1, min(40000, 160000 // B)))
    if kind == "verify":
        B = _log(rng, 1, 48)
        return dict(kind=kind, B=B, n=rng.randint(1, 16), V=_log(rng, 50, 151000),
                    dense=rng.random() < 0.6, wide=rng.random() < 0.5, agree=round(rng.random(), 3))
    n = _log(rng, 1, 32)
    thin = rng.random() < 0.4
    return dict(kind=kind, n=n, layers=rng.randint(1, 36), kv_heads=kv, D=D, page=page,
                ctx=_log(rng, 1, 8000 // n) + 2, share=(not thin) or rng.random() < 0.5,
                draft=rng.randint(1, 32), keep=rng.randint(0, 8), thin=thin) | (
                    {"share": False} if thin else {})


# ---------------------------------------------------------------------------- inputs
def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed & 0x7fffffff)
    return g


def _ints(lo, hi, shape, g):
    return torch.randint(lo, max(hi, lo + 1), shape, generator=g, device=DEV)


def _bf(shape, g):
    return torch.randn(shape, generator=g, device=DEV, dtype=torch.bfloat16)


def _ragged(n, B):
    """B counts spread over n/2 .. n, the first one n."""
    return [n - (i * i * 7 + i * 3) % (n // 2 + 1) for i in range(B)]


def _on(counts):
    return torch.tensor(counts, device=DEV)


def _offsets(c):
    return torch.cat([torch.zeros_like(c[:1]), c.cumsum(0)]).to(torch.int32)


def _trees(counts, total, wide, g):
    """A parent for every node: the one before it (a chain), or (wide) a random one among the
    last few; -1 for the first node of each sequence."""
    off = _offsets(counts)[:-1].long()
    seq = torch.repeat_interleave(torch.arange(counts.numel(), device=DEV), counts, output_size=total)
    i = torch.arange(total, device=DEV) - off[seq]
    back = 1 + (torch.rand(total, generator=g, device=DEV) * (8 if wide else 1)).long()
    return torch.where(i == 0, -1, (i - back).clamp_min(0)).to(torch.int32)


def _cache(layers, kv_heads, D, page, lens, room, seqs, g, spare=0):
    """Pages of `seqs` sequences: the first lens.numel() hold lens[s] tokens and have pages for
    room[s] tokens, the others are empty; the page numbers are shuffled. Keys and values ~ N(0, 1)."""
    n = lens.numel()
    need = (room + page - 1) // page
    total, widest = int(need.sum()), int(need.max())
    width = widest + 2 + spare // max(1, seqs - n)
    pages = total + spare + 3
    order = torch.randperm(pages, generator=g, device=DEV).to(torch.int32)
    table = torch.full((seqs, width), -1, dtype=torch.int32, device=DEV)
    owned = torch.zeros(seqs, dtype=torch.int32, device=DEV)
    owned[:n] = need.to(torch.int32)
    length = torch.zeros(seqs, dtype=torch.int32, device=DEV)
    length[:n] = lens.to(torch.int32)
    col = torch.arange(width, device=DEV)
    first = need.cumsum(0) - need
    at = first[:, None] + col
    table[:n] = torch.where(col < need[:, None], order[at.clamp_max(pages - 1)], table[:n])
    ref = torch.zeros(pages, dtype=torch.int32, device=DEV)
    ref[order[:total].long()] = 1
    left = order[total:].sort(descending=True).values
    free = torch.cat([left, torch.full((total,), -1, dtype=torch.int32, device=DEV)])
    count = torch.tensor([pages - total], dtype=torch.int32, device=DEV)
    shape = (layers, pages, kv_heads, page, D)
    c = dict(k=_bf(shape, g), v=_bf(shape, g), table=table, length=length, n_pages=owned, ref=ref,
             free_list=free, free_count=count)
    return c


def _handle(s):
    """The handle and scratch memory that a program keeps beside the cache's tensors."""
    import vlm_visual_token_b200 as ivc
    s["ivc"], size, kind = ivc, ivc.STEP_WORKSPACE_BYTES, s["case"]["kind"]
    if "c" in s:
        s["cache"] = ivc.Cache(**s["c"])
    if kind == "attend":
        size = ivc.tree_attention_workspace_size(s["cache"], s["N"], s["case"]["q_heads"], s["case"]["B"])
    if kind == "pages":
        size = ivc.cache_workspace_size(s["cache"], s["case"]["n"], s["keep"].shape[1])
    s["ws"] = ivc.new_workspace(size)


def prepare(case, seed):
    g = _gen(seed)
    s = dict(case=case)
    k = case["kind"]
    if k in ("norm", "attend"):
        B, n, D, Hq, Hkv = case["B"], case["n"], case["D"], case["q_heads"], case["kv_heads"]
        counts = _on(_ragged(n, B))
        lens = _on(_ragged(case["ctx"], B))
        s["c"] = _cache(1, Hkv, D, case["page"], lens, lens + counts, B, g)
        s["offsets"] = _offsets(counts)
        N, s["n_max"], s["len_max"] = (int(v) for v in
                                       torch.stack([counts.sum(), counts.max(), lens.max()]).tolist())
        s["N"] = N
        s["parents"] = _trees(counts, N, True, g)
        if k == "norm":
            s["qkv"] = _bf((N, (Hq + 2 * Hkv) * D), g)
            s["q_gamma"], s["k_gamma"] = (1 + 0.2 * _bf((D,), g) for _ in range(2))
            seq = torch.repeat_interleave(torch.arange(B, device=DEV), counts, output_size=N)
            s["positions"] = (lens[seq] + torch.arange(N, device=DEV)
                              - s["offsets"][seq]).to(torch.int32)
        else:
            s["q"] = _bf((N, Hq, D), g)
        s["out"] = torch.zeros(N, Hq, D, dtype=torch.bfloat16, device=DEV)
    elif k == "verify":
        B, n, V = case["B"], case["n"], case["V"]
        counts = _on(_ragged(n, B))
        s["offsets"] = _offsets(counts)
        N, s["n_max"] = (int(v) for v in torch.stack([counts.sum(), counts.max()]).tolist())
        s["N"] = N
        s["parents"] = _trees(counts, N, case["wide"], g)
        logits = 2.5 * torch.randn(N, V, generator=g, device=DEV)
        s["p"] = torch.softmax(logits, -1)
        s["q"] = None
        other = torch.randn(N, V, generator=g, device=DEV)
        drafts = torch.softmax(logits + 1.5 * (1 - case["agree"]) * other, -1)
        if case["dense"]:
            s["q"] = drafts
        # a child's token is drawn from its parent's draft row
        first = torch.repeat_interleave(s["offsets"][:-1].long(), counts, output_size=N)
        row = first + s["parents"].long().clamp_min(0)
        cdf = drafts.double().cumsum(-1)
        z = torch.rand(N, 1, generator=g, device=DEV).double()
        tok = torch.searchsorted(cdf[row], z * cdf[row][:, -1:], right=True)[:, 0].clamp_max(V - 1)
        s["tokens"] = tok.to(torch.int32)
        s["u"] = torch.rand(N, generator=g, device=DEV)
        s["u_next"] = torch.rand(B, generator=g, device=DEV)
        s["path"] = torch.zeros(B, s["n_max"], dtype=torch.int32, device=DEV)
        s["n_path"] = torch.zeros(B, dtype=torch.int32, device=DEV)
        s["token"] = torch.zeros(B, dtype=torch.int32, device=DEV)
    else:
        n, draft, page = case["n"], case["draft"], case["page"]
        lens = _on(_ragged(case["ctx"], n))
        top = case["ctx"] + draft
        per = (top + page - 1) // page + 1
        s["c"] = _cache(case["layers"], case["kv_heads"], case["D"], page, lens, lens, 2 * n, g,
                        spare=n * per)
        s["src"] = torch.arange(n, dtype=torch.int32, device=DEV)
        s["dst"] = s["src"] + n
        s["draft"] = torch.full((n,), draft, dtype=torch.int32, device=DEV)
        s["len_max"] = top
        if case["thin"]:  # of every 256 tokens the first 64 stay
            at = torch.arange(case["ctx"], device=DEV)
            kept = at[at % 256 < 64]
            s["keep"] = kept.expand(n, -1).to(torch.int32).contiguous()
            s["start"] = torch.zeros(n, dtype=torch.int32, device=DEV)
            s["count"] = (kept < lens[:, None]).sum(1).to(torch.int32)
        else:  # an accepted path: the first node, then rising ones
            m = min(case["keep"], draft)
            pick = torch.rand(n, draft, generator=g, device=DEV)
            pick[:, 0] = -1
            s["keep"] = pick.argsort(1)[:, :max(m, 1)].sort(1).values.to(torch.int32).contiguous()
            s["start"] = lens.to(torch.int32)
            s["count"] = torch.full((n,), m, dtype=torch.int32, device=DEV)
            s["count"][1:] = _ints(min(1, m), m + 1, (n - 1,), g).to(torch.int32)
    if own:
        _handle(s)
    return s


# ---------------------------------------------------------------------------- plain forms
def _pad(offsets, n_max):
    """Row numbers [B, n_max] of each sequence's tokens, and which of them there are."""
    i = torch.arange(n_max, device=DEV)
    count = offsets[1:] - offsets[:-1]
    there = i < count[:, None]
    return torch.where(there, offsets[:-1, None] + i, 0).long(), there


def plain_norm(s):
    case, c = s["case"], s["c"]
    D, Hq, Hkv, N = case["D"], case["q_heads"], case["kv_heads"], s["N"]
    x = s["qkv"].float().view(N, Hq + 2 * Hkv, D)
    gamma = torch.cat([s["q_gamma"].float().expand(Hq, D), s["k_gamma"].float().expand(Hkv, D)])
    y = x[:, :Hq + Hkv]
    y = y * torch.rsqrt((y * y).mean(-1, keepdim=True) + EPS) * gamma
    freq = THETA ** (-torch.arange(0, D, 2, device=DEV, dtype=torch.float64) / D)
    angle = s["positions"].double()[:, None] * freq
    cos, sin = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]
    a, b = y[..., :D // 2], y[..., D // 2:]
    y = torch.cat([a * cos - b * sin, b * cos + a * sin], -1).to(torch.bfloat16)
    rows = torch.arange(N, device=DEV, dtype=torch.int32)
    seq = torch.searchsorted(s["offsets"], rows, right=True) - 1
    pos = (c["length"][seq] + rows - s["offsets"][seq]).long()
    page = c["table"][seq, pos // case["page"]].long()
    c["k"][0][page, :, pos % case["page"]] = y[:, Hq:]
    c["v"][0][page, :, pos % case["page"]] = x[:, Hq + Hkv:].to(torch.bfloat16)
    return y[:, :Hq], c["k"], c["v"]


def plain_attend(s):
    case, c = s["case"], s["c"]
    D, Hq, Hkv, P = case["D"], case["q_heads"], case["kv_heads"], case["page"]
    B, G = case["B"], case["q_heads"] // case["kv_heads"]
    rows, there = _pad(s["offsets"], s["n_max"])
    n, L = s["n_max"], s["len_max"] + s["n_max"]
    q = s["q"].float()[rows].view(B, n, Hkv, G, D)
    pos = torch.arange(L, device=DEV)
    page = c["table"][:, (pos // P).clamp_max(c["table"].shape[1] - 1)].long().clamp_min(0)
    k = c["k"][0][page, :, pos % P].float()  # [B, L, Hkv, D]
    v = c["v"][0][page, :, pos % P].float()
    par = torch.where(there, s["parents"][rows], -1).long()
    eye = torch.eye(n, device=DEV, dtype=torch.float64)
    up = (par[:, :, None] == torch.arange(n, device=DEV)).double()
    anc = torch.linalg.matrix_power(up + eye, max(n - 1, 1)) > 0  # node i sees its ancestors and itself
    node = pos - c["length"][:, None]  # which node of the tree stands at a position
    seen = anc.gather(2, node.clamp(0, n - 1)[:, None, :].expand(B, n, L).long())
    seen = torch.where(node[:, None] < 0, True, seen & (node[:, None] < n))
    x = torch.einsum("bnhgd,blhd->bhgnl", q, k) / math.sqrt(D)
    x = x.masked_fill(~seen[:, None, None], float("-inf"))
    x = torch.exp(x - x.amax(-1, keepdim=True))
    x = x / x.sum(-1, keepdim=True)
    o = torch.einsum("bhgnl,blhd->bnhgd", x, v.masked_fill((node >= n)[..., None, None], 0))
    return o.reshape(B, n, Hq, D)[there].to(torch.bfloat16)


def plain_verify(s):
    case = s["case"]
    B, V, n = case["B"], case["V"], s["n_max"]
    rows, there = _pad(s["offsets"], n)
    b = torch.arange(B, device=DEV)
    tok = s["tokens"][rows].long()
    par = torch.where(there, s["parents"][rows], -2)
    u = s["u"][rows].double()
    cur = torch.zeros(B, dtype=torch.int32, device=DEV)
    r = s["p"][rows[:, 0]].double()
    q = s["q"][rows[:, 0]].double() if case["dense"] else None
    z = torch.ones(B, dtype=torch.float64, device=DEV)  # r / z is what is left of the target
    w = torch.ones_like(z)                              # q / w is what is left of the draft
    path = torch.full((B, n), -1, dtype=torch.int32, device=DEV)
    path[:, 0] = 0
    count = torch.ones(B, dtype=torch.int32, device=DEV)
    for j in range(1, n):
        tried = (par[:, j] == cur) & (z > 0)
        c = tok[:, j]
        rc = r[b, c]
        qc = q[b, c] if case["dense"] else torch.ones_like(z)
        yes = tried & (u[:, j] * qc * z < rc * w)
        no = tried & ~yes
        if case["dense"]:
            t = torch.where(w > 0, 1 / w, 0)
            left = (r * (1 / z)[:, None] - q * t[:, None]).clamp_min(0)
            r = torch.where(no[:, None], left, r)
            z = torch.where(no, r.sum(-1), z)
            q[b, c] = torch.where(no, 0, qc)
            w = torch.where(no, w - qc, w)
        else:
            z = torch.where(no, z - rc, z)
            r[b, c] = torch.where(no, 0, rc)
        cur = torch.where(yes, j, cur)
        path[b, count.long().clamp_max(n - 1)] = torch.where(yes, j, path[b, count.long().clamp_max(n - 1)])
        count = count + yes.int()
        r = torch.where(yes[:, None], s["p"][rows[:, j]].double(), r)
        z = torch.where(yes, 1.0, z)
        w = torch.where(yes, 1.0, w)
        if case["dense"]:
            q = torch.where(yes[:, None], s["q"][rows[:, j]].double(), q)
    empty = r.sum(-1) <= 0
    r = torch.where(empty[:, None], s["p"][rows[b, cur.long()]].double(), r)
    cdf = r.cumsum(-1)
    t = s["u_next"].double()[:, None] * cdf[:, -1:]
    last = (V - 1 - (r.flip(-1) > 0).int().argmax(-1))[:, None]
    token = torch.minimum(torch.searchsorted(cdf, t, right=True), last)[:, 0].to(torch.int32)
    return path, count, token


def _push(c, freed):
    """The pages marked in `freed` go back on the free list, the lowest number on top."""
    P = freed.numel()
    k = freed.sum()
    order = torch.where(freed, torch.arange(P, device=DEV), -1).sort(descending=True).values
    at = c["free_count"].long() + torch.arange(P, device=DEV)
    old = c["free_list"].clone()
    keep = torch.arange(P, device=DEV) < k
    at = torch.where(keep, at, P)
    big = torch.cat([old, old[:1]])
    big[at] = torch.where(keep, order.to(torch.int32), old[0])
    c["free_list"].copy_(big[:P])
    c["free_count"].add_(k.to(torch.int32))


def _drop(c, seqs, keep_pages):
    """Pages of `seqs` from number keep_pages on are given up."""
    rows = c["table"][seqs]
    col = torch.arange(rows.shape[1], device=DEV)
    gone = (col >= keep_pages[:, None]) & (col < c["n_pages"][seqs][:, None])
    P = c["ref"].numel()
    hits = torch.zeros(P + 1, dtype=torch.int32, device=DEV)
    hits.index_add_(0, torch.where(gone, rows, P).reshape(-1).long(),
                    torch.ones(gone.numel(), dtype=torch.int32, device=DEV))
    before = c["ref"].clone()
    c["ref"].sub_(hits[:P])
    _push(c, (before > 0) & (c["ref"] == 0))
    c["table"][seqs] = torch.where(gone, -1, rows)
    c["n_pages"][seqs] = torch.minimum(c["n_pages"][seqs], keep_pages)


def _pop(c, seqs, need):
    """need[i] new pages behind those of sequence seqs[i], in this order off the top."""
    rows = c["table"][seqs]
    col = torch.arange(rows.shape[1], device=DEV)
    have = c["n_pages"][seqs]
    new = (col >= have[:, None]) & (col < (have + need)[:, None])
    order = need.cumsum(0) - need
    nth = order[:, None] + col - have[:, None]
    got = c["free_list"][(c["free_count"] - 1 - nth).clamp_min(0).long()]
    P = c["ref"].numel()
    ref = torch.cat([c["ref"], c["ref"][:1]])
    ref[torch.where(new, got, P).reshape(-1).long()] = 1
    c["ref"].copy_(ref[:P])
    c["free_list"].copy_(torch.where(torch.arange(P, device=DEV) >= c["free_count"] - need.sum(), -1,
                                     c["free_list"]))
    c["table"][seqs] = torch.where(new, got, rows)
    c["n_pages"][seqs] = (have + need).to(torch.int32)
    c["free_count"].sub_(need.sum().to(torch.int32))


def plain_pages(s):
    case, c = s["case"], s["c"]
    page, src, dst = case["page"], s["src"].long(), s["dst"].long()
    # free: every page of the earlier branch
    _drop(c, dst, torch.zeros_like(s["dst"]))
    c["length"][dst] = 0
    # fork: full pages shared (or all copied), the last partial page copied
    length = c["length"][src]
    used = (length + page - 1) // page
    full = length // page if case["share"] else torch.zeros_like(length)
    rows = c["table"][src]
    col = torch.arange(rows.shape[1], device=DEV)
    P = c["ref"].numel()
    shared = col < full[:, None]
    c["table"][dst] = torch.where(shared, rows, -1)
    hits = torch.zeros(P + 1, dtype=torch.int32, device=DEV)
    hits.index_add_(0, torch.where(shared, rows, P).reshape(-1).long(),
                    torch.ones(shared.numel(), dtype=torch.int32, device=DEV))
    c["ref"].add_(hits[:P])
    c["n_pages"][dst] = full.to(torch.int32)
    _pop(c, dst, used - full)
    c["length"][dst] = length
    if case["share"]:  # at most one page of each is copied: the one that its last token is in
        pos = (full * page)[:, None] + torch.arange(page, device=DEV)
    else:
        pos = torch.arange(s["len_max"], device=DEV).expand(dst.numel(), -1)
    _move(c, src, pos, dst, pos, pos < length[:, None], page)
    # reserve: room for the drafted tokens
    have = c["n_pages"][dst]
    need = ((c["length"][dst] + s["draft"] + page - 1) // page - have).clamp_min(0)
    _pop(c, dst, need)
    # compact: kept tokens behind start, the pages after them given up
    j = torch.arange(s["keep"].shape[1], device=DEV)
    to = s["start"][:, None] + j
    _move(c, dst, s["start"][:, None] + s["keep"], dst, to, j < s["count"][:, None], page)
    now = s["start"] + s["count"]
    c["length"][dst] = now
    _drop(c, dst, (now + page - 1) // page)
    return [c[k] for k in ("k", "v", "table", "length", "n_pages", "ref", "free_list", "free_count")]


def _move(c, src, from_pos, dst, to_pos, there, page):
    """Tokens of all layers, from_pos of sequence src to to_pos of sequence dst."""
    last = c["table"].shape[1] - 1
    a = c["table"][src[:, None], (from_pos // page).clamp_max(last).long()].long()
    b = c["table"][dst[:, None], (to_pos // page).clamp_max(last).long()].long()
    P = c["ref"].numel()
    H, D = c["k"].shape[2], c["k"].shape[4]
    # token slots as rows [layers, pages * page]: a slot past the end takes what is not moved
    i, t = (a * page + from_pos % page).reshape(-1), (b * page + to_pos % page).reshape(-1)
    ok = there.reshape(-1)
    safe = torch.where(ok, i, 0)
    # an unmoved entry writes its target back unchanged: into the first moved one, whose value it takes
    first = ok.int().argmax()
    safe = torch.where(ok, safe, safe[first])
    t = torch.where(ok, t, t[first])
    some = ok.any()
    for x in (c["k"], c["v"]):
        rows = x[:, safe // page, :, safe % page]
        here = x[:, t // page, :, t % page]
        x[:, t // page, :, t % page] = torch.where(some, rows, here)


# ---------------------------------------------------------------------------- one pass
def run(s):
    k = s["case"]["kind"]
    if not own:
        return {"norm": plain_norm, "attend": plain_attend, "verify": plain_verify,
                "pages": plain_pages}[k](s)
    ivc, ws = s["ivc"], s["ws"]
    if k == "norm":
        ivc.qk_norm_rope(s["cache"], 0, s["qkv"], s["q_gamma"], s["k_gamma"], s["positions"],
                         s["offsets"], theta=THETA, eps=EPS, out=s["out"], workspace=ws)
        return s["out"], s["c"]["k"], s["c"]["v"]
    if k == "attend":
        return ivc.tree_attention(s["cache"], 0, s["q"], s["parents"], s["offsets"], out=s["out"],
                                  workspace=ws)
    if k == "verify":
        return ivc.verify_drafts(s["p"], s["q"], s["tokens"], s["parents"], s["offsets"], s["u"],
                                 s["u_next"], out=(s["path"], s["n_path"], s["token"]), workspace=ws)
    c = s["cache"]
    ivc.cache_free(c, s["dst"], workspace=ws)
    ivc.cache_fork(c, s["src"], s["dst"], share=s["case"]["share"], workspace=ws)
    ivc.cache_reserve(c, s["draft"], s["dst"], workspace=ws)
    ivc.cache_compact(c, s["count"], s["keep"], s["start"], s["dst"], workspace=ws)
    return [s["c"][k] for k in ("k", "v", "table", "length", "n_pages", "ref", "free_list", "free_count")]


# ---------------------------------------------------------------------------- cost and definition
def work(case):
    k = case["kind"]
    if k == "norm":
        t = sum(_ragged(case["n"], case["B"]))
        row = (case["q_heads"] + 2 * case["kv_heads"]) * case["D"]
        return {"bytes": t * row * 4, "flops": t * row * 6}
    if k == "attend":
        n, m = _ragged(case["n"], case["B"]), _ragged(case["ctx"], case["B"])
        row = case["q_heads"] * case["D"]
        return {"bytes": sum(a + b for a, b in zip(n, m)) * case["kv_heads"] * case["D"] * 4 + sum(n) * row * 4,
                "flops": 4 * row * sum(a * (a + b) for a, b in zip(n, m))}
    if k == "verify":  # the row of probabilities in which a walk ends
        return {"bytes": case["B"] * case["V"] * (8 if case["dense"] else 4), "flops": 0}
    token = case["layers"] * case["kv_heads"] * case["D"] * 2 * 2 * 2  # read and written, k and v
    lens = _ragged(case["ctx"], case["n"])
    moved = sum(m % case["page"] if case["share"] else m for m in lens)
    if case["thin"]:
        moved += sum(max(0, m // 256 * 64 + min(64, m % 256) - 64) for m in lens)
    else:
        moved += case["n"] * max(0, min(case["keep"], case["draft"]) - 1) // 2
    return {"bytes": max(1, token * moved), "flops": 0}


def exact(case, seed):
    """From the definitions, sequence by sequence, in 64 bits."""
    global own
    was, own = own, False
    s = prepare(case, seed)
    own = was
    k = case["kind"]
    if k == "pages":  # moved rows and whole numbers: no computed value
        return None
    off = s["offsets"].tolist()
    if k == "norm":
        return _exact_norm(case, s, off)
    if k == "attend":
        return _exact_attend(case, s, off)
    return None  # whole numbers


def _exact_norm(case, s, off):
    c, D, Hq, Hkv = s["c"], case["D"], case["q_heads"], case["kv_heads"]
    x = s["qkv"].double().reshape(s["N"], -1, D)
    out = torch.empty(s["N"], Hq, D, dtype=torch.float64, device=DEV)
    ck, cv = c["k"].double(), c["v"].double()
    table, lens = c["table"].tolist(), c["length"].tolist()
    z = torch.polar(torch.ones(s["N"], D // 2, dtype=torch.float64, device=DEV),
                    s["positions"].double()[:, None]
                    * torch.exp(-math.log(THETA) * 2 / D * torch.arange(D // 2, device=DEV, dtype=torch.float64)))

    def turned(h, gamma):
        h = h / (h.pow(2).sum(-1, keepdim=True) / D + EPS).sqrt() * gamma.double()
        w = torch.complex(h[..., :D // 2].contiguous(), h[..., D // 2:].contiguous()) * z[:, None]
        return torch.cat([w.real, w.imag], -1)

    out = turned(x[:, :Hq], s["q_gamma"])
    key = turned(x[:, Hq:Hq + Hkv], s["k_gamma"])
    for b in range(case["B"]):
        i = 0
        while i < off[b + 1] - off[b]:  # page by page
            pos = lens[b] + i
            m = min(case["page"] - pos % case["page"], off[b + 1] - off[b] - i)
            pg, r0, t0 = table[b][pos // case["page"]], pos % case["page"], off[b] + i
            ck[0, pg, :, r0:r0 + m] = key[t0:t0 + m].transpose(0, 1)
            cv[0, pg, :, r0:r0 + m] = x[t0:t0 + m, Hq + Hkv:].transpose(0, 1)
            i += m
    return out, ck, cv


def _exact_attend(case, s, off):
    c, D, Hq, Hkv = s["c"], case["D"], case["q_heads"], case["kv_heads"]
    lens, parents = c["length"].tolist(), s["parents"].tolist()
    out = torch.empty(s["N"], Hq, D, dtype=torch.float64, device=DEV)
    for b in range(case["B"]):
        n, m = off[b + 1] - off[b], lens[b]
        pages = c["table"][b][: -(-(m + n) // case["page"])].long()
        k, v = (c[x][0][pages].transpose(1, 2).reshape(-1, Hkv, D)[: m + n].double() for x in "kv")
        see = torch.zeros(n, m + n, dtype=torch.bool)
        see[:, :m] = True
        for i in range(n):
            j = i
            while j >= 0:
                see[i, m + j] = True
                j = parents[off[b] + j]
        see = see.to(DEV)
        for h in range(Hkv):
            G = Hq // Hkv
            q = s["q"][off[b]:off[b + 1], h * G:(h + 1) * G].double()
            w = torch.einsum("ngd,ld->gnl", q, k[:, h]) * D ** -0.5
            w = torch.softmax(w.masked_fill(~see, -math.inf), -1)
            out[off[b]:off[b + 1], h * G:(h + 1) * G] = torch.einsum("gnl,ld->ngd", w, v[:, h])
    return out
