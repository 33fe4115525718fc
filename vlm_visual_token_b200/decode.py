"""Decoding behind the spliced sequence: the paged cache and the calls of one
decode step (include/ivc.h, "Decoding behind the spliced sequence").

    cache = Cache.empty(layers, pages, kv_heads, page_tokens, head_dim, max_seqs, max_pages)
    ws = new_workspace(max(tree_attention_workspace_size(cache, N, q_heads, B),
                           cache_workspace_size(cache, B, MAX_TREE)))
    cache_reserve(cache, tokens, workspace=ws)    # pages for the new tokens
    q = qk_norm_rope(cache, layer, qkv, q_gamma, k_gamma, positions, offsets, workspace=ws)
    out = tree_attention(cache, layer, q, parents, offsets, workspace=ws)
    path, n_path, token = verify_drafts(p, draft_p, tokens, parents, offsets, u, u_next, workspace=ws)
    cache_compact(cache, n_path, path, workspace=ws)  # the accepted tokens stay, the rest is freed
    bits = device_status(ws)                      # 0, or what went wrong since the last look

Argument marshalling only, as in the rest of the package. A call runs on
`stream` (default: the current stream of the cache's device), its outputs and
an omitted workspace are made on that stream. A wrong argument raises IvcError
before anything is enqueued. Wrong device data, and a cache without enough free
pages, set bits of the workspace's status word (device_status) and nothing else
tells of them: a call without a workspace drops its bits. Outputs that a call
makes itself are zero where it writes nothing.
"""
from __future__ import annotations

import contextlib
import ctypes
from typing import Optional, Tuple

import torch

_vp, _i, _ll, _sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_longlong, ctypes.c_size_t
STEP_WORKSPACE_BYTES = 256
MAX_TREE = 128


class _CCache(ctypes.Structure):
    _fields_ = [(n, _i) for n in ("layers", "pages", "kv_heads", "page_tokens", "head_dim",
                                  "max_seqs", "max_pages")] + \
               [(n, _vp) for n in ("k", "v", "table", "length", "n_pages", "ref", "free_list",
                                   "free_count")]


def _declare(L) -> None:
    P = ctypes.POINTER(_CCache)
    for name, res, args in (
            ("ivc_cache_init", _i, [P, _vp]),
            ("ivc_cache_workspace_size", _sz, [P, _i, _i]),
            ("ivc_cache_reserve", _i, [P, _vp, _vp, _i, _vp, _sz, _vp]),
            ("ivc_cache_fork", _i, [P, _vp, _vp, _i, _i, _vp, _sz, _vp]),
            ("ivc_cache_compact", _i, [P, _vp, _vp, _i, _vp, _vp, _i, _vp, _sz, _vp]),
            ("ivc_cache_free", _i, [P, _vp, _i, _vp, _sz, _vp]),
            ("ivc_qk_norm_rope", _i, [P, _i, _vp, _ll, _i, _i, _vp, _vp, ctypes.c_float,
                                      ctypes.c_double, _vp, _vp, _vp, _i, _vp, _vp, _sz, _vp]),
            ("ivc_tree_attention_workspace_size", _sz, [P, _i, _i, _i]),
            ("ivc_tree_attention", _i, [P, _i, _vp, _ll, _i, _i, ctypes.c_float, _vp, _vp, _vp, _i,
                                        _vp, _vp, _sz, _vp]),
            ("ivc_verify_drafts", _i, [_vp, _ll, _vp, _ll, _i, _i, _vp, _vp, _vp, _i, _vp, _vp, _vp,
                                       _i, _vp, _vp, _vp, _sz, _vp])):
        f = getattr(L, name)
        f.restype, f.argtypes = res, args


_ivc = None  # the package, once loaded


def _pkg():
    global _ivc
    if _ivc is None:
        import vlm_visual_token_b200 as ivc
        ivc.lib()
        _ivc = ivc
    return _ivc


def _refuse(what: str, code: int = -1):
    raise _pkg().IvcError(code, what)


def _need(t, what: str, dtype, dims: int, device, n: int = -1) -> int:
    """t is a dense tensor of this type, rank and device (with n values); its address."""
    try:
        if t.dtype is dtype and t.dim() == dims and t.device == device and t.is_contiguous() and \
                (n < 0 or t.numel() == n):
            return t.data_ptr()
    except AttributeError:
        pass
    count = f" of {n} values" if n >= 0 else ""
    _refuse(f"{what}: a contiguous {dims}-dimensional {dtype} tensor{count} on {device} is needed")


def _maybe(t, what: str, dtype, dims: int, device, n: int = -1) -> Optional[int]:
    return None if t is None else _need(t, what, dtype, dims, device, n)


def _rows(t, what: str, dtype, device) -> int:
    """t is a matrix whose rows are dense; the elements between them."""
    if not isinstance(t, torch.Tensor) or t.dtype != dtype or t.dim() != 2 or t.device != device:
        _refuse(f"{what}: a 2-dimensional {dtype} tensor on {device} is needed")
    rows, width = t.shape
    if width > 1 and t.stride(1) != 1:
        _refuse(f"{what}: rows are not dense")
    return t.stride(0) if rows > 1 else max(width, 1)


# (the public forms build objects and take over a microsecond of each call)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _elsewhere(device, stream):
    """None where a call can run as it is; else the context to repeat it in, which
    makes `device` and `stream` current."""
    if stream is not None:
        if stream.device != device:
            _refuse("stream: it is another device's")
        return _other(device, stream)
    index = device.index  # None: not a GPU, which _call refuses
    return None if index is None or index == _current_device() else torch.cuda.device(device)


@contextlib.contextmanager
def _other(device, stream):
    with torch.cuda.device(device), torch.cuda.stream(stream):
        yield


def _call(name: str, device, *args) -> None:
    if device.index is None:
        _refuse(f"{name}: the tensors are not on a GPU")
    ivc = _pkg()
    rc = getattr(ivc._LIB, name)(*args, _raw_stream(device.index))
    if rc != 0:
        raise ivc.IvcError(rc, name)


def _workspace(ws, need: int, device):
    if ws is None:
        ws = torch.empty(need, dtype=torch.uint8, device=device)
        ws[:STEP_WORKSPACE_BYTES].zero_()
    else:
        _need(ws, "workspace", torch.uint8, 1, device)
    return ws


class Cache:
    """Keys and values of many sequences in pages, and the C descriptor.

    k, v: bf16 [layers, pages, kv_heads, page_tokens, head_dim]; the int32 tensors
    as in include/ivc.h (ivc_cache). Cache.empty() allocates all of them. The
    tensors are the caller's: the calls below change them in place."""

    def __init__(self, k: torch.Tensor, v: torch.Tensor, table: torch.Tensor, length: torch.Tensor,
                 n_pages: torch.Tensor, ref: torch.Tensor, free_list: torch.Tensor,
                 free_count: torch.Tensor):
        dev = k.device
        for name, t in (("k", k), ("v", v)):
            _need(t, name, torch.bfloat16, 5, dev)
        if k.shape != v.shape:
            _refuse("k and v differ in shape")
        _need(table, "table", torch.int32, 2, dev)
        seqs = table.shape[0]
        for name, t, n in (("length", length, seqs), ("n_pages", n_pages, seqs),
                           ("ref", ref, k.shape[1]), ("free_list", free_list, k.shape[1]),
                           ("free_count", free_count, 1)):
            _need(t, name, torch.int32, 1, dev, n)
        self.k, self.v, self.table, self.length, self.n_pages = k, v, table, length, n_pages
        self.ref, self.free_list, self.free_count = ref, free_list, free_count
        self.device = dev
        self.layers, self.pages, self.kv_heads, self.page_tokens, self.head_dim = k.shape
        self.max_seqs, self.max_pages = table.shape
        self.c = _CCache(*k.shape, *table.shape, *(t.data_ptr() for t in (
            k, v, table, length, n_pages, ref, free_list, free_count)))
        self._p = ctypes.byref(self.c)

    @classmethod
    def empty(cls, layers: int, pages: int, kv_heads: int, page_tokens: int, head_dim: int,
              max_seqs: int, max_pages: int, device="cuda", stream=None) -> "Cache":
        """A cache whose sequences are all empty (ivc_cache_init)."""
        dev = torch.device(device)
        if dev.type == "cuda" and dev.index is None:
            dev = torch.device("cuda", torch.cuda.current_device())
        with _elsewhere(dev, stream) or contextlib.nullcontext():
            shape = (layers, pages, kv_heads, page_tokens, head_dim)
            k, v = (torch.empty(shape, dtype=torch.bfloat16, device=dev) for _ in range(2))
            ints = [torch.empty(s, dtype=torch.int32, device=dev)
                    for s in ((max_seqs, max_pages), max_seqs, max_seqs, pages, pages, 1)]
            cache = cls(k, v, *ints)
            _call("ivc_cache_init", dev, cache._p)
        return cache


def cache_workspace_size(cache: Cache, n: int, keep_width: int = 0) -> int:
    """Bytes that cache_fork and cache_compact of n sequences need."""
    ivc = _pkg()
    size = ivc.lib().ivc_cache_workspace_size(cache._p, n, keep_width)
    if size == 0:
        raise ivc.IvcError(-2, "ivc_cache_workspace_size")
    return size


def cache_reserve(cache: Cache, tokens: torch.Tensor, seqs: Optional[torch.Tensor] = None,
                  workspace=None, stream=None) -> None:
    """Pages for tokens[i] more tokens of sequence seqs[i] (default: i)."""
    dev = cache.device
    other = _elsewhere(dev, stream)
    if other is not None:
        with other:
            return cache_reserve(cache, tokens, seqs, workspace)
    t = _need(tokens, "tokens", torch.int32, 1, dev)
    n = tokens.shape[0]
    s = _maybe(seqs, "seqs", torch.int32, 1, dev, n)
    ws = _workspace(workspace, STEP_WORKSPACE_BYTES, dev)
    _call("ivc_cache_reserve", dev, cache._p, t, s, n, ws.data_ptr(), ws.shape[0])


def cache_fork(cache: Cache, src: torch.Tensor, dst: torch.Tensor, share: bool = True,
               workspace=None, stream=None) -> None:
    """Empty sequence dst[i] becomes a copy of src[i]: its full pages shared, or
    (share=False) every page copied."""
    dev = cache.device
    other = _elsewhere(dev, stream)
    if other is not None:
        with other:
            return cache_fork(cache, src, dst, share, workspace)
    a = _need(src, "src", torch.int32, 1, dev)
    n = src.shape[0]
    b = _need(dst, "dst", torch.int32, 1, dev, n)
    ws = _workspace(workspace, 0 if workspace is not None else cache_workspace_size(cache, n), dev)
    _call("ivc_cache_fork", dev, cache._p, a, b, n, 1 if share else 0, ws.data_ptr(), ws.shape[0])


def cache_compact(cache: Cache, count: torch.Tensor, keep: Optional[torch.Tensor] = None,
                  start: Optional[torch.Tensor] = None, seqs: Optional[torch.Tensor] = None,
                  workspace=None, stream=None) -> None:
    """Tokens start[i] + keep[i, j], j < count[i], become tokens start[i] + j, and
    the last of them the sequence's last (keep None: the first count[i]; start
    None: the committed length). Pages behind that are freed."""
    dev = cache.device
    other = _elsewhere(dev, stream)
    if other is not None:
        with other:
            return cache_compact(cache, count, keep, start, seqs, workspace)
    m = _need(count, "count", torch.int32, 1, dev)
    n = count.shape[0]
    k, width = None, 0
    if keep is not None:
        k = _need(keep, "keep", torch.int32, 2, dev)
        if keep.shape[0] != n:
            _refuse("keep: one row for each count is needed")
        width = keep.shape[1]
        k = k or m  # rows of no tokens have no address; none of them is read
    a = _maybe(start, "start", torch.int32, 1, dev, n)
    s = _maybe(seqs, "seqs", torch.int32, 1, dev, n)
    ws = _workspace(workspace, 0 if workspace is not None else cache_workspace_size(cache, n, width),
                    dev)
    _call("ivc_cache_compact", dev, cache._p, m, k, width, a, s, n, ws.data_ptr(), ws.shape[0])


def cache_free(cache: Cache, seqs: torch.Tensor, workspace=None, stream=None) -> None:
    """The sequences become empty; pages that no other sequence holds are freed."""
    dev = cache.device
    other = _elsewhere(dev, stream)
    if other is not None:
        with other:
            return cache_free(cache, seqs, workspace)
    s = _need(seqs, "seqs", torch.int32, 1, dev)
    ws = _workspace(workspace, STEP_WORKSPACE_BYTES, dev)
    _call("ivc_cache_free", dev, cache._p, s, seqs.shape[0], ws.data_ptr(), ws.shape[0])


def _out(out, N: int, q_heads: int, D: int, device):
    if out is None:  # zeros: rows of skipped sequences and behind the last one are not written
        return torch.zeros(N, q_heads, D, dtype=torch.bfloat16, device=device)
    _need(out, "out", torch.bfloat16, 3, device)
    if out.shape != (N, q_heads, D):
        _refuse("out: [N, q_heads, head_dim] is needed")
    return out


def qk_norm_rope(cache: Cache, layer: int, qkv: torch.Tensor, q_gamma: torch.Tensor,
                 k_gamma: torch.Tensor, positions: torch.Tensor, offsets: torch.Tensor,
                 theta: float = 1e6, eps: float = 1e-6, seqs: Optional[torch.Tensor] = None,
                 out: Optional[torch.Tensor] = None, workspace=None, stream=None) -> torch.Tensor:
    """Per-head norms and rotation of the packed projections qkv [N, (q_heads + 2
    kv_heads) * head_dim] (rows may be strided); keys and values go to the cache
    behind the committed tokens, the queries [N, q_heads, head_dim] are returned
    (in `out`; without it, rows behind the last sequence are zero)."""
    dev, D = cache.device, cache.head_dim
    other = _elsewhere(dev, stream)
    if other is not None:
        with other:
            return qk_norm_rope(cache, layer, qkv, q_gamma, k_gamma, positions, offsets, theta, eps,
                                seqs, out, workspace)
    ld = _rows(qkv, "qkv", torch.bfloat16, dev)
    N, width = qkv.shape
    heads, rest = divmod(width, D)
    q_heads = heads - 2 * cache.kv_heads
    if rest or q_heads < 1:
        _refuse("qkv: q_heads + 2 kv_heads heads of head_dim are needed", -2)
    gq = _need(q_gamma, "q_gamma", torch.bfloat16, 1, dev, D)
    gk = _need(k_gamma, "k_gamma", torch.bfloat16, 1, dev, D)
    pos = _need(positions, "positions", torch.int32, 1, dev, N)
    off = _need(offsets, "offsets", torch.int32, 1, dev)
    B = offsets.shape[0] - 1
    s = _maybe(seqs, "seqs", torch.int32, 1, dev, B)
    out = _out(out, N, q_heads, D, dev)
    ws = _workspace(workspace, STEP_WORKSPACE_BYTES, dev)
    _call("ivc_qk_norm_rope", dev, cache._p, layer, qkv.data_ptr(), ld, N, q_heads, gq, gk, eps,
          theta, pos, off, s, B, out.data_ptr(), ws.data_ptr(), ws.shape[0])
    return out


def tree_attention_workspace_size(cache: Cache, N: int, q_heads: int, B: int) -> int:
    """Bytes that tree_attention needs for N rows of q_heads heads in B sequences."""
    ivc = _pkg()
    with _elsewhere(cache.device, None) or contextlib.nullcontext():
        size = ivc.lib().ivc_tree_attention_workspace_size(cache._p, N, q_heads, B)
    if size == 0:
        raise ivc.IvcError(-2, "ivc_tree_attention_workspace_size")
    return size


def tree_attention(cache: Cache, layer: int, q: torch.Tensor, parents: Optional[torch.Tensor],
                   offsets: torch.Tensor, seqs: Optional[torch.Tensor] = None,
                   scale: Optional[float] = None, out: Optional[torch.Tensor] = None,
                   workspace=None, stream=None) -> torch.Tensor:
    """Attention of the trees' nodes q [N, q_heads, head_dim] (tokens may be
    strided) over their committed tokens, ancestors and themselves. parents None:
    chains. scale: 1 / sqrt(head_dim) by default. Rows of sequences that are skipped
    (device_status tells) and behind the last one stay as they are in `out`;
    without `out` they are zero."""
    dev, D = cache.device, cache.head_dim
    other = _elsewhere(dev, stream)
    if other is not None:
        with other:
            return tree_attention(cache, layer, q, parents, offsets, seqs, scale, out, workspace)
    if not isinstance(q, torch.Tensor) or q.dtype != torch.bfloat16 or q.dim() != 3 or \
            q.device != dev or q.shape[2] != D:
        _refuse(f"q: a bf16 tensor [N, q_heads, {D}] on {dev} is needed")
    N, q_heads, _ = q.shape
    if N and q_heads and (q.stride(2) != 1 or (q_heads > 1 and q.stride(1) != D)):
        _refuse("q: a token's heads are not dense")
    ld = q.stride(0) if N > 1 else q_heads * D
    par = _maybe(parents, "parents", torch.int32, 1, dev, N)
    off = _need(offsets, "offsets", torch.int32, 1, dev)
    B = offsets.shape[0] - 1
    s = _maybe(seqs, "seqs", torch.int32, 1, dev, B)
    out = _out(out, N, q_heads, D, dev)
    ws = _workspace(workspace, 0 if workspace is not None else
                    tree_attention_workspace_size(cache, N, q_heads, B), dev)
    _call("ivc_tree_attention", dev, cache._p, layer, q.data_ptr(), ld, N, q_heads,
          D ** -0.5 if scale is None else scale, par, off, s, B, out.data_ptr(), ws.data_ptr(),
          ws.shape[0])
    return out


def verify_drafts(p: torch.Tensor, q: Optional[torch.Tensor], tokens: torch.Tensor,
                  parents: Optional[torch.Tensor], offsets: torch.Tensor, u: torch.Tensor,
                  u_next: torch.Tensor, out: Optional[Tuple[torch.Tensor, ...]] = None,
                  path_width: int = MAX_TREE, workspace=None, stream=None):
    """Drafted trees against the target's probabilities p [N, V] (rows may be
    strided), q the probabilities they were drafted from, or None. Returns
    (path [B, path_width] int32, n_path [B], next_token [B])."""
    dev = p.device
    other = _elsewhere(dev, stream)
    if other is not None:
        with other:
            return verify_drafts(p, q, tokens, parents, offsets, u, u_next, out, path_width, workspace)
    p_ld = _rows(p, "p", torch.float32, dev)
    N, V = p.shape
    q_ld, q_at = 0, None
    if q is not None:
        q_ld, q_at = _rows(q, "q", torch.float32, dev), q.data_ptr()
        if q.shape != p.shape:
            _refuse("p and q differ in shape")
    tok = _need(tokens, "tokens", torch.int32, 1, dev, N)
    par = _maybe(parents, "parents", torch.int32, 1, dev, N)
    uu = _need(u, "u", torch.float32, 1, dev, N)
    off = _need(offsets, "offsets", torch.int32, 1, dev)
    B = offsets.shape[0] - 1
    un = _need(u_next, "u_next", torch.float32, 1, dev, max(B, 0))
    if out is None:
        out = (torch.empty(max(B, 0), path_width, dtype=torch.int32, device=dev),
               torch.empty(max(B, 0), dtype=torch.int32, device=dev),
               torch.empty(max(B, 0), dtype=torch.int32, device=dev))
    path, n_path, token = out
    at = _need(path, "path", torch.int32, 2, dev)
    if path.shape[0] != B:
        _refuse("path: one row for each sequence is needed")
    m, t = _need(n_path, "n_path", torch.int32, 1, dev, B), _need(token, "next_token", torch.int32, 1,
                                                                dev, B)
    ws = _workspace(workspace, STEP_WORKSPACE_BYTES, dev)
    _call("ivc_verify_drafts", dev, p.data_ptr(), p_ld, q_at, q_ld, N, V, tok, par, off, B, uu, un,
          at, path.shape[1], m, t, ws.data_ptr(), ws.shape[0])
    return out
