"""A prompt from the splice of its visual rows into the cache: the positions and
offsets of assemble_sequence go on to the norms, and its attention goes through in
pieces of at most MAX_TREE tokens, each committed before the next."""
import numpy as np
import pytest
import torch

import oracle as O
from oracle import decode_oracle as D
from tests.test_gpu_decode import BF, _ivc, dev, np64
from tests.test_gpu_parity import _prompt_ids

pytestmark = pytest.mark.gpu


def test_spliced_prompts_into_the_cache():
    ivc = _ivc()
    V, H, img, kv, Hq, D_, pt = 600, 64, 599, 2, 4, 64, 16
    mask = np.array([1, 0, 1], np.uint8)
    v_offs = O.compaction_offsets(mask)
    g = torch.Generator().manual_seed(5)
    table = torch.randn(V, H, generator=g).bfloat16().cuda()
    visual = torch.randn(int(v_offs[-1]), H, generator=g).bfloat16().cuda()
    ids, offs = _prompt_ids((2, 0, 1), img, V, seed=3)
    seq = ivc.assemble_sequence(dev(ids), dev(offs), img, table, visual, dev(mask, torch.uint8), dev(v_offs))
    assert ivc.device_status(seq["workspace"]) == 0
    offsets, positions = seq["seq_offsets"], seq["positions"]
    counts = (offsets[1:] - offsets[:-1]).tolist()
    B, L, total = len(counts), len(ids), int(offsets[-1])
    assert total < L and max(counts) > 2 * ivc.MAX_TREE
    seq["embeds"][total:] = 0                # rows of the capacity that the splice did not fill
    w = (torch.randn(H, (Hq + 2 * kv) * D_, generator=g) * H ** -0.5).bfloat16().cuda()
    qkv = seq["embeds"] @ w
    gam = [(1 + 0.3 * torch.randn(D_, generator=g)).bfloat16().cuda() for _ in range(2)]
    c = ivc.Cache.empty(1, sum(-(-n // pt) for n in counts), kv, pt, D_, B, -(-max(counts) // pt))
    ws = ivc.new_workspace(ivc.tree_attention_workspace_size(c, L, Hq, B))

    # the norms alone, all rows of the capacity at once: keys and values where they belong
    ivc.cache_reserve(c, offsets.diff(), workspace=ws)
    q = ivc.qk_norm_rope(c, 0, qkv, *gam, positions, offsets, workspace=ws)
    x = np64(qkv[:total]).reshape(total, Hq + 2 * kv, D_)
    pos = positions[:total].cpu().numpy()
    close = lambda a, b: np.all(np.abs(a - b) <= BF * np.abs(b) + 2.0 ** -20 * np.abs(b).max(-1, keepdims=True))  # noqa: E731,E501
    assert close(np64(q[:total]), D.norm_rope(x[:, :Hq], np64(gam[0]), pos, 1e6, 1e-6))
    keys = D.norm_rope(x[:, Hq:Hq + kv], np64(gam[1]), pos, 1e6, 1e-6)

    # the layer by pieces, as a program that runs every layer on a piece would
    out = torch.zeros_like(q)
    done = [0] * B
    first = offsets.tolist()
    while done != counts:
        now = [min(ivc.MAX_TREE, n - m) for n, m in zip(counts, done)]
        rows = torch.cat([torch.arange(a + m, a + m + k) for a, m, k in zip(first, done, now)]).cuda()
        o = dev(np.concatenate([[0], np.cumsum(now)]))
        ivc.cache_reserve(c, dev(now), workspace=ws)
        part = ivc.qk_norm_rope(c, 0, qkv[rows], *gam, positions[rows], o, workspace=ws)
        out[rows] = ivc.tree_attention(c, 0, part, None, o, workspace=ws)
        ivc.cache_compact(c, dev(now), workspace=ws)
        done = [m + k for m, k in zip(done, now)]
    assert ivc.device_status(ws) == 0
    assert c.length.tolist() == counts

    for b, n in enumerate(counts):
        pages = c.table[b, :-(-n // pt)].long()
        k, v = (t[0, pages].transpose(1, 2).reshape(-1, kv, D_)[:n].double() for t in (c.k, c.v))
        assert close(k.cpu().numpy(), keys[first[b]:first[b] + n])
        assert torch.equal(v, qkv[first[b]:first[b] + n].double().view(n, -1, D_)[:, Hq + kv:])
        see = torch.ones(n, n, dtype=torch.bool, device="cuda").tril()
        qq = q[first[b]:first[b] + n].double()
        kk, vv = k.repeat_interleave(Hq // kv, 1), v.repeat_interleave(Hq // kv, 1)
        s = torch.einsum("nhd,lhd->hnl", qq, kk) * D_ ** -0.5
        weight = torch.softmax(s.masked_fill(~see, float("-inf")), -1)
        want, size = torch.einsum("hnl,lhd->nhd", weight, vv), torch.einsum("hnl,lhd->nhd", weight, vv.abs())
        err = (out[first[b]:first[b] + n].double() - want).abs()
        assert bool((err <= BF * want.abs() + (BF + 2.0 ** -14) * size).all()), b
