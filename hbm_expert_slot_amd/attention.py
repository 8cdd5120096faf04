"""Attention over prompts and over a key/value cache held in 4 bits.

The half of a decoder layer that the expert operators leave open: HBM that the
cache does not need is HBM for expert slots.  `ops` has both names; streams,
allocation, graphs and gradients are as described there.
"""
import ctypes
import math

import torch

from . import binding as B
from .ops import _FORMAT, _TYPE, _Fixed, _ForInference, _need, _On, _record, _wants_grad

PAGE = B.SC_KV4_PAGE
HEAD_DIMS = (64, 128, 256)
_NARROW = (torch.bfloat16, torch.float16)
_INT = torch.int32


# What is wrong is only put into words once something is: a call spends less time on its checks.

def _rows3(t, name, dtypes, dev):
    """[tokens, heads, head_dim] with the last dimension contiguous."""
    if not (t.dim() == 3 and t.dtype in dtypes and t.device == dev and t.is_cuda and t.stride(2) == 1
            and t.shape[2] in HEAD_DIMS):
        _need(t.dim() == 3, "%s must be [tokens, heads, head_dim]" % name)
        _need(t.dtype in dtypes, "%s has type %s" % (name, t.dtype))
        _need(t.is_cuda and t.device == dev, "%s must be on the GPU, with the others" % name)
        _need(t.shape[2] in HEAD_DIMS, "%s: head_dim must be one of %s" % (name, HEAD_DIMS))
        _need(False, "%s must be contiguous along head_dim" % name)


def _ints(t, name, n, dev):
    if not (t.dtype == _INT and t.dim() == 1 and t.shape[0] == n and t.device == dev and (n < 2 or t.stride(0) == 1)):
        raise ValueError("%s must be a contiguous int32 vector of %d on %s" % (name, n, dev))


def _scale_of(scale, dim):
    if scale is None:
        return 1.0 / math.sqrt(dim)
    scale = float(scale)
    _need(0.0 < scale <= 2.3e38, "scale must be positive and at most 2.3e38")
    return scale


def _writable(t, name):
    """Rows of an output may not lie over each other."""
    spans = sorted((st, n) for n, st in zip(t.shape, t.stride()) if n > 1)
    reach = 1
    for st, n in spans:
        _need(st >= reach, "%s has elements that overlap" % name)
        reach = st * n if st * n > reach else reach


def prompt_attention(q, k, v, starts, key_starts=None, scale=None, out=None, return_lse=False, stream=None):
    """Causal attention over packed sequences.

    q [rows, heads, head_dim], k and v [keys, kv_heads, head_dim] (bfloat16 or
    float16; head_dim 64, 128 or 256; any strides but along head_dim); heads is a
    multiple of kv_heads.  starts int32 [n + 1] has the first row of each sequence
    and the end of the last; key_starts the same of its keys (default: starts).
    With fewer rows than keys the rows are the last ones: row i of Lq sees the keys
    below Lk - Lq + i + 1.  scale defaults to 1 / sqrt(head_dim).

    Returns out [rows, heads, head_dim], with return_lse also the natural logarithm
    of each row's sum of exponentials (float32 [rows, heads]).  A row that sees
    nothing gets 0 and -inf.  Rows outside of the sequences are not written.  out,
    if given, must not overlap q, k or v (and takes no part in a gradient)."""
    if out is None and _wants_grad(q, k, v):
        return _ForInference.apply("prompt_attention", lambda: prompt_attention(
            q, k, v, starts, key_starts, scale, None, return_lse, stream), q, k, v)
    dev = q.device
    _rows3(q, "q", _NARROW, dev)
    _rows3(k, "k", (q.dtype,), dev)
    _rows3(v, "v", (q.dtype,), dev)
    rows, heads, dim = q.shape
    keys, kv_heads, kdim = k.shape
    if not (kdim == dim and k.shape == v.shape):
        raise ValueError("q %s, k %s and v %s do not fit" % (tuple(q.shape), tuple(k.shape), tuple(v.shape)))
    _need(kv_heads > 0 and heads > 0 and heads % kv_heads == 0, "heads must be a multiple of kv_heads")
    _need(starts.dim() == 1 and starts.shape[0] >= 1, "starts must be [sequences + 1]")
    n = starts.shape[0] - 1
    _ints(starts, "starts", n + 1, dev)
    if key_starts is None:
        if keys != rows:
            raise ValueError("%d rows and %d keys: key_starts are needed" % (rows, keys))
        key_starts = starts
    else:
        _ints(key_starts, "key_starts", n + 1, dev)
    scale = _scale_of(scale, dim)
    with _On(dev, stream) as s:
        if out is None:
            out = torch.empty((rows, heads, dim), dtype=q.dtype, device=dev)
        else:
            _rows3(out, "out", (q.dtype,), dev)
            _need(out.shape == q.shape, "out does not fit q")
            _writable(out, "out")
        lse = torch.empty((rows, heads), dtype=torch.float32, device=dev) if return_lse else None
        qs, ks, vs, os = q.stride(), k.stride(), v.stride(), out.stride()
        # a single key has no next one, whatever stride it has
        kt, vt = (ks[0], vs[0]) if keys > 1 else (0, 0)
        if kt > B.SC_PROMPT_MAX_STRIDE or vt > B.SC_PROMPT_MAX_STRIDE:
            raise ValueError("keys and values must be at most %d elements apart" % B.SC_PROMPT_MAX_STRIDE)
        p = B.PROMPT.pack(_TYPE[q.dtype], dim, heads, kv_heads, n, rows, keys, scale, q.data_ptr(), k.data_ptr(),
                          v.data_ptr(), out.data_ptr(), 0 if lse is None else lse.data_ptr(), starts.data_ptr(),
                          key_starts.data_ptr(), qs[0], qs[1], kt, ks[1], vt, vs[1], os[0], os[1])
        ws = None
        if keys >= 2 * B.SC_PROMPT_PART_KEYS * n:
            need = B.prompt_attention_workspace_bytes(p)
            ws = torch.empty(need, dtype=torch.uint8, device=dev) if need else None
        B.prompt_attention(p, None if ws is None else ws.data_ptr(), s)
    if stream is not None:
        _record(stream, q, k, v, starts, key_starts, out, lse)
    return (out, lse) if return_lse else out


class KV4Cache(_Fixed):
    """One layer's key/value cache in 4 bits: n_pages pages of 64 tokens.

    pages uint8 [n_pages, kv_heads, bytes]; fmt "nvfp4" (groups of 16, with
    k_scale and v_scale, one float32 > 0 each on the device, None standing for 1)
    or "mxfp4" (groups of 32).  With track=True the cache also keeps, for eviction,
    weights float32 and positions int32 [n_pages, kv_heads, 64].

    Sequences are given to each call: table int32 [n, width] names the pages of
    each sequence, lens int32 [n] its tokens, those that come with the call
    included.  Handing out pages is the caller's part.  The constructor waits until
    the pages are zeros (not in a capture, where that is part of the graph).  Calls
    that write the cache (append, evict, attend with accumulate) have to be ordered
    with all others on it; attend and read may run at once.  The cache may be dropped
    while calls are under way, but not while a captured graph is to be replayed."""

    _fixed = frozenset(("fmt", "head_dim", "kv_heads", "n_pages", "device", "pages", "weights", "positions", "k_scale",
                        "v_scale", "_memory", "_streams", "_sizes", "_c", "_ref"))

    def __init__(self, n_pages, kv_heads, head_dim, fmt="nvfp4", k_scale=None, v_scale=None, track=False, device="cuda"):
        _need(fmt in _FORMAT, "unknown format %r" % (fmt,))
        _need(head_dim in HEAD_DIMS, "head_dim must be one of %s" % (HEAD_DIMS,))
        _need(n_pages > 0 and 0 < kv_heads <= B.SC_KV4_MAX_HEADS, "n_pages and kv_heads must be positive, heads at most %d"
              % B.SC_KV4_MAX_HEADS)
        for t, name in ((k_scale, "k_scale"), (v_scale, "v_scale")):
            _need(t is None or fmt == "nvfp4", "only nvfp4 has a global scale")
            _need(t is None or (t.dtype == torch.float32 and t.numel() == 1 and t.is_cuda),
                  "%s must be one float32 on the GPU" % name)
        pages = torch.zeros((n_pages, kv_heads, B.kv4_page_bytes(_FORMAT[fmt], head_dim)), dtype=torch.uint8, device=device)
        dev = pages.device
        weights = positions = None
        if track:
            weights = torch.zeros((n_pages, kv_heads, PAGE), dtype=torch.float32, device=dev)
            positions = torch.zeros((n_pages, kv_heads, PAGE), dtype=torch.int32, device=dev)
        for t, name in ((k_scale, "k_scale"), (v_scale, "v_scale")):
            _need(t is None or t.device == dev, "%s must be with the cache" % name)

        def ptr(t):
            return None if t is None else t.data_ptr()

        # zeros before any stream uses it (in a capture they are nodes of the graph, in its order)
        with torch.cuda.device(dev):
            if not torch.cuda.is_current_stream_capturing():
                torch.cuda.current_stream().synchronize()
        memory = [t.detach() for t in (pages, weights, positions, k_scale, v_scale) if t is not None]
        c = B.sc_kv4_cache(_FORMAT[fmt], head_dim, kv_heads, n_pages, ptr(pages), ptr(weights), ptr(positions),
                           ptr(k_scale), ptr(v_scale))
        self.__dict__.update(fmt=fmt, head_dim=head_dim, kv_heads=kv_heads, n_pages=n_pages, device=dev, pages=pages,
                             weights=weights, positions=positions, k_scale=k_scale, v_scale=v_scale, _memory=memory,
                             _streams={torch.cuda.current_stream(dev).cuda_stream}, _sizes={}, _c=c,
                             _ref=ctypes.byref(c))

    def _used_on(self, s):
        """The cache may be dropped while the current stream (raw: s, not in _streams yet) works on it."""
        _record(torch.cuda.current_stream(self.device), *self._memory)
        self._streams.add(s)

    def _seqs(self, table, lens):
        dev = self.device
        if not (table.dim() == 2 and table.dtype == _INT and table.device == dev and table.shape[1] >= 1
                and (table.shape[1] == 1 or table.stride(1) == 1)):
            raise ValueError("table must be an int32 tensor [sequences, pages] on %s, contiguous along its rows" % dev)
        n, width = table.shape
        _ints(lens, "lens", n, dev)
        ld = table.stride(0) if n > 1 else width
        _need(ld >= width, "table has rows that overlap")
        return B.KV4_SEQS.pack(n, width, ld, table.data_ptr(), lens.data_ptr())

    def _rows(self, k, v, types):
        dev = self.device
        _rows3(k, "k", types, dev)
        _rows3(v, "v", types, dev)
        shape = k.shape
        if not (shape[1] == self.kv_heads and shape[2] == self.head_dim and v.shape == shape and v.dtype == k.dtype):
            raise ValueError("k %s %s and v %s %s do not fit the cache or each other" % (
                tuple(shape), k.dtype, tuple(v.shape), v.dtype))
        ks, vs = k.stride(), v.stride()
        return B.KV4_ROWS.pack(_TYPE[k.dtype], k.data_ptr(), v.data_ptr(), ks[0], ks[1], vs[0], vs[1])

    def _deal(self, tokens, n, starts):
        if starts is not None:
            _ints(starts, "starts", n + 1, self.device)
            return starts.data_ptr()
        if tokens and (n == 0 or tokens % n):
            raise ValueError("%d tokens cannot be dealt out to %d sequences" % (tokens, n))
        return None

    def _four(self, t, name, dtypes):
        if not (t.dim() == 4 and t.dtype in dtypes and t.device == self.device and t.stride(3) == 1):
            raise ValueError("%s must be [sequences, rows, heads, head_dim] of %s on %s, contiguous along head_dim"
                             % (name, dtypes, self.device))

    def append(self, k, v, table, lens, starts=None, positions=None, stream=None):
        """Quantise tokens into the cache: k and v [tokens, kv_heads, head_dim] (float32, bfloat16 or
        float16).  starts int32 [n + 1] packs the sequences' new tokens (None: tokens / n each); they are each
        sequence's last, so the last one goes to place lens - 1.  positions int32 [tokens] are kept for eviction
        (default: the places).  Their weights are 0 until attend has accumulated some: an evict right after a
        prompt keeps its first places, unless attend was given the prompt's last rows (up to 16) with accumulate
        before.  Places the table does not have and pages the cache does not have are not written;
        two tokens must not have one place.  tokens * kv_heads * head_dim is below 2^32, here and in read."""
        seqs = self._seqs(table, lens)
        rows = self._rows(k, v, _TYPE)
        tokens = k.shape[0]
        ps = self._deal(tokens, lens.shape[0], starts)
        if positions is not None:
            _need(self.positions is not None, "the cache keeps no positions")
            _ints(positions, "positions", tokens, self.device)
        with _On(self.device, stream) as s:
            B.kv4_append(self._ref, seqs, rows, tokens, ps, None if positions is None else positions.data_ptr(), s)
            if s not in self._streams:
                self._used_on(s)
        if stream is not None:
            _record(stream, k, v, table, lens, starts, positions)

    def read(self, table, lens, tokens, starts=None, dtype=torch.bfloat16, stream=None):
        """The last tokens of each sequence as the values they stand for: k, v [tokens, kv_heads, head_dim] of
        dtype, packed as in append.  Places or pages that are not there read as NaN; rows outside of the sequences
        are not written."""
        seqs = self._seqs(table, lens)
        _need(dtype in _TYPE, "unsupported type %s" % (dtype,))
        _need(tokens >= 0, "tokens must be >= 0")
        ps = self._deal(tokens, lens.shape[0], starts)
        with _On(self.device, stream) as s:
            heads, dim = self.kv_heads, self.head_dim
            k = torch.empty((tokens, heads, dim), dtype=dtype, device=self.device)
            v = torch.empty((tokens, heads, dim), dtype=dtype, device=self.device)
            rows = B.KV4_ROWS.pack(_TYPE[dtype], k.data_ptr(), v.data_ptr(), heads * dim, dim, heads * dim, dim)
            B.kv4_read(self._ref, seqs, rows, tokens, ps, s)
            if s not in self._streams:
                self._used_on(s)
        if stream is not None:
            _record(stream, table, lens, starts, k, v)
        return k, v

    def attend(self, q, table, lens, scale=None, accumulate=False, out=None, stream=None):
        """Attention of each sequence's last tokens over the cache: q [n, rows, heads, head_dim] (bfloat16 or
        float16; rows up to 16: a token and its drafts; heads a multiple of kv_heads; n * rows * heads up to 2^23;
        any strides but along head_dim).  Row r sees the places below lens - rows + r + 1; a row that sees none gets 0.  With accumulate
        every token's weight grows by its probabilities, summed over the rows and the heads that share its keys;
        sequences of such a call must not share pages.
        Sequences with a length that cannot be give NaN, as do rows that see a page the cache does not have, and all
        that see anything where k_scale is NaN, infinite or negative.  out, if given, must not overlap q (and takes
        no part in a gradient)."""
        if out is None and _wants_grad(q):
            return _ForInference.apply("KV4Cache.attend", lambda: self.attend(
                q, table, lens, scale, accumulate, None, stream), q)
        seqs = self._seqs(table, lens)
        dev = self.device
        self._four(q, "q", _NARROW)
        n, rows, heads, dim = q.shape
        if not (n == lens.shape[0] and dim == self.head_dim):
            raise ValueError("q %s does not fit the cache or the table" % (tuple(q.shape),))
        if not (1 <= rows <= B.SC_KV4_MAX_ROWS and 0 < heads <= B.SC_KV4_MAX_GROUP * self.kv_heads
                and heads % self.kv_heads == 0):
            raise ValueError("rows must be in [1, %d], heads a multiple of kv_heads, up to %d times"
                             % (B.SC_KV4_MAX_ROWS, B.SC_KV4_MAX_GROUP))
        _need(not accumulate or self.weights is not None, "the cache keeps no weights")
        scale = _scale_of(scale, dim)
        # the workspace follows from the sizes
        key = (n, table.shape[1], rows, heads, bool(accumulate))
        need = self._sizes.get(key)
        if need is None:
            if len(self._sizes) > 1000:
                self._sizes.clear()
            need = self._sizes[key] = B.kv4_attention_workspace_bytes(self._ref, seqs, rows, heads, accumulate)
        with _On(dev, stream) as s:
            if out is None:
                out = torch.empty((n, rows, heads, dim), dtype=q.dtype, device=dev)
            else:
                self._four(out, "out", (q.dtype,))
                _need(out.shape == q.shape, "out does not fit q")
                _writable(out, "out")
            ws = torch.empty(need, dtype=torch.uint8, device=dev)
            qs, os = q.stride(), out.stride()
            x = B.KV4_QUERY.pack(_TYPE[q.dtype], rows, heads, scale, q.data_ptr(), out.data_ptr(), qs[0], qs[1], qs[2],
                                 os[0], os[1], os[2])
            B.kv4_attention(self._ref, seqs, x, accumulate, ws.data_ptr(), s)
            if s not in self._streams:
                self._used_on(s)
        if stream is not None:
            _record(stream, q, table, lens, out)
        return out

    def evict(self, table, lens, keep, recent=0, sinks=0, stream=None):
        """Cut every sequence of more than `keep` tokens down to `keep`; returns the new lens.

        Of each head the tokens at positions below sinks or among the last `recent` positions stay before all
        others, then those with the largest weights, equal ones by place.  They keep their places below keep, or move
        into those that became free, so a sequence's tokens are not in order afterwards: give append positions from
        then on.  Sequences that are cut must not share pages; one with a length or page that cannot be stays as it
        is.  Weights are what attend has accumulated (0 for tokens that were only appended).  A call takes up to 2^17 sequences times kv_heads."""
        _need(self.weights is not None, "the cache keeps no weights")
        seqs = self._seqs(table, lens)
        _need(keep >= 1 and recent >= 0 and sinks >= 0 and recent + sinks <= keep,
              "keep must be positive, recent and sinks >= 0 and together at most keep")
        _need(keep < 2 ** 31, "keep is too large")
        with _On(self.device, stream) as s:
            new = torch.empty_like(lens)
            ws = torch.empty(B.kv4_evict_workspace_bytes(self._ref, seqs, keep), dtype=torch.uint8, device=self.device)
            B.kv4_evict(self._ref, seqs, keep, recent, sinks, new.data_ptr(), ws.data_ptr(), s)
            if s not in self._streams:
                self._used_on(s)
        if stream is not None:
            _record(stream, table, lens, new)
        return new
