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


def _rows3(t, name, dtypes, dev=None):
    """[tokens, heads, head_dim] with the last dimension contiguous."""
    _need(t.dim() == 3, "%s must be [tokens, heads, head_dim]" % name)
    _need(t.dtype in dtypes, "%s has type %s" % (name, t.dtype))
    _need(t.is_cuda and (dev is None or t.device == dev), "%s must be on the GPU%s" % (name, "" if dev is None else ", on %s" % dev))
    _need(t.shape[2] in HEAD_DIMS, "%s: head_dim must be one of %s" % (name, HEAD_DIMS))
    _need(t.stride(2) == 1, "%s must be contiguous along head_dim" % name)


def _ints(t, name, shape, dev):
    _need(t.dtype == torch.int32 and tuple(t.shape) == shape and t.device == dev and t.is_contiguous(),
          "%s must be a contiguous int32 tensor of shape %s on %s" % (name, shape, dev))


def _scale_of(scale, dim):
    if scale is None:
        return 1.0 / math.sqrt(dim)
    scale = float(scale)
    _need(0.0 < scale < 3e38, "scale must be positive and finite")
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
    _rows3(q, "q", _NARROW)
    dev = q.device
    for t, name in ((k, "k"), (v, "v")):
        _rows3(t, name, (q.dtype,), dev)
    rows, heads, dim = q.shape
    keys, kv_heads = k.shape[0], k.shape[1]
    _need(k.shape[2] == dim and k.shape == v.shape, "q %s, k %s and v %s do not fit" % (
        tuple(q.shape), tuple(k.shape), tuple(v.shape)))
    _need(kv_heads > 0 and heads > 0 and heads % kv_heads == 0, "heads must be a multiple of kv_heads")
    _need(starts.dim() == 1 and starts.shape[0] >= 1, "starts must be [sequences + 1]")
    n = starts.shape[0] - 1
    _ints(starts, "starts", (n + 1,), dev)
    if key_starts is None:
        _need(keys == rows, "%d rows and %d keys: key_starts are needed" % (rows, keys))
        key_starts = starts
    else:
        _ints(key_starts, "key_starts", (n + 1,), dev)
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
        p = B.sc_prompt(_TYPE[q.dtype], dim, heads, kv_heads, n, rows, keys, scale, q.data_ptr(), k.data_ptr(),
                        v.data_ptr(), out.data_ptr(), None if lse is None else lse.data_ptr(), starts.data_ptr(),
                        key_starts.data_ptr(), (qs[0], qs[1]), (ks[0], ks[1]), (vs[0], vs[1]), (os[0], os[1]))
        ref = ctypes.byref(p)
        need = B.prompt_attention_workspace_bytes(ref)
        ws = torch.empty(need, dtype=torch.uint8, device=dev) if need else None
        B.prompt_attention(ref, None if ws is None else ws.data_ptr(), s)
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
    included.  Handing out pages is the caller's part.  Calls that write the cache
    (append, evict, attend with accumulate) have to be ordered with all others on
    it; attend and read may run at once.  The cache may be dropped while calls are
    under way, but not while a captured graph is to be replayed."""

    _fixed = frozenset(("fmt", "head_dim", "kv_heads", "n_pages", "device", "pages", "weights", "positions", "k_scale",
                        "v_scale", "_memory", "_streams", "_c", "_ref"))

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

        memory = [t.detach() for t in (pages, weights, positions, k_scale, v_scale) if t is not None]
        c = B.sc_kv4_cache(_FORMAT[fmt], head_dim, kv_heads, n_pages, ptr(pages), ptr(weights), ptr(positions),
                           ptr(k_scale), ptr(v_scale))
        self.__dict__.update(fmt=fmt, head_dim=head_dim, kv_heads=kv_heads, n_pages=n_pages, device=dev, pages=pages,
                             weights=weights, positions=positions, k_scale=k_scale, v_scale=v_scale, _memory=memory,
                             _streams={torch.cuda.current_stream(dev).cuda_stream}, _c=c, _ref=ctypes.byref(c))

    def _used_on(self, s):
        """The cache may be dropped while the current stream (raw: s, not in _streams yet) works on it."""
        _record(torch.cuda.current_stream(self.device), *self._memory)
        self._streams.add(s)

    def _seqs(self, table, lens):
        dev = self.device
        _need(table.dim() == 2 and table.dtype == torch.int32 and table.device == dev and table.shape[1] >= 1
              and (table.shape[1] == 1 or table.stride(1) == 1),
              "table must be an int32 tensor [sequences, pages] on %s, contiguous along its rows" % dev)
        n, width = table.shape
        _ints(lens, "lens", (n,), dev)
        ld = table.stride(0) if n > 1 else width
        _need(ld >= width, "table has rows that overlap")
        return B.sc_kv4_seqs(n, width, ld, table.data_ptr(), lens.data_ptr())

    def _rows(self, k, v, types):
        dev = self.device
        for t, name in ((k, "k"), (v, "v")):
            _rows3(t, name, types, dev)
            _need(t.shape[1] == self.kv_heads and t.shape[2] == self.head_dim, "%s does not fit the cache" % name)
        _need(k.shape == v.shape and k.dtype == v.dtype, "k and v differ")
        ks, vs = k.stride(), v.stride()
        return B.sc_kv4_rows(_TYPE[k.dtype], k.data_ptr(), v.data_ptr(), ks[0], ks[1], vs[0], vs[1])

    def _deal(self, tokens, n, starts):
        if starts is not None:
            _ints(starts, "starts", (n + 1,), self.device)
            return starts.data_ptr()
        _need(n > 0 and tokens % n == 0 or tokens == 0, "%d tokens cannot be dealt out to %d sequences" % (tokens, n))
        return None

    def append(self, k, v, table, lens, starts=None, positions=None, stream=None):
        """Quantise tokens into the cache: k and v [tokens, kv_heads, head_dim] (float32, bfloat16 or
        float16).  starts int32 [n + 1] packs the sequences' new tokens (None: tokens / n each); they are each
        sequence's last, so the last one goes to place lens - 1.  positions int32 [tokens] are kept for eviction
        (default: the places).  Places the table does not have and pages the cache does not have are not written;
        two tokens must not have one place."""
        seqs = self._seqs(table, lens)
        rows = self._rows(k, v, _TYPE)
        tokens = k.shape[0]
        ps = self._deal(tokens, lens.shape[0], starts)
        if positions is not None:
            _need(self.positions is not None, "the cache keeps no positions")
            _ints(positions, "positions", (tokens,), self.device)
        with _On(self.device, stream) as s:
            B.kv4_append(self._ref, ctypes.byref(seqs), ctypes.byref(rows), tokens, ps,
                         None if positions is None else positions.data_ptr(), s)
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
            k = torch.empty((tokens, self.kv_heads, self.head_dim), dtype=dtype, device=self.device)
            v = torch.empty_like(k)
            rows = self._rows(k, v, _TYPE)
            B.kv4_read(self._ref, ctypes.byref(seqs), ctypes.byref(rows), tokens, ps, s)
            if s not in self._streams:
                self._used_on(s)
        if stream is not None:
            _record(stream, table, lens, starts, k, v)
        return k, v

    def attend(self, q, table, lens, scale=None, accumulate=False, out=None, stream=None):
        """Attention of each sequence's last tokens over the cache: q [n, rows, heads, head_dim] (bfloat16 or
        float16; rows up to 16: a token and its drafts; heads a multiple of kv_heads; any strides but along
        head_dim).  Row r sees the places below lens - rows + r + 1; a row that sees none gets 0.  With accumulate
        every token's weight grows by its probabilities, summed over the rows and the heads that share its keys.
        Sequences with a length that cannot be give NaN, as do rows that see a page the cache does not have.  out,
        if given, must not overlap q (and takes no part in a gradient)."""
        if out is None and _wants_grad(q):
            return _ForInference.apply("KV4Cache.attend", lambda: self.attend(
                q, table, lens, scale, accumulate, None, stream), q)
        seqs = self._seqs(table, lens)
        dev = self.device

        def four(t, name, dtypes):
            _need(t.dim() == 4 and t.dtype in dtypes and t.device == dev,
                  "%s must be [sequences, rows, heads, head_dim] of %s on %s" % (name, dtypes, dev))
            _need(t.stride(3) == 1, "%s must be contiguous along head_dim" % name)

        four(q, "q", _NARROW)
        n, rows, heads, dim = q.shape
        _need(n == lens.shape[0] and dim == self.head_dim, "q %s does not fit the cache or the table" % (tuple(q.shape),))
        _need(1 <= rows <= B.SC_KV4_MAX_ROWS, "rows must be in [1, %d]" % B.SC_KV4_MAX_ROWS)
        _need(heads > 0 and heads % self.kv_heads == 0 and heads // self.kv_heads <= B.SC_KV4_MAX_GROUP,
              "heads must be a multiple of kv_heads, up to %d times" % B.SC_KV4_MAX_GROUP)
        _need(not accumulate or self.weights is not None, "the cache keeps no weights")
        scale = _scale_of(scale, dim)
        with _On(dev, stream) as s:
            if out is None:
                out = torch.empty((n, rows, heads, dim), dtype=q.dtype, device=dev)
            else:
                four(out, "out", (q.dtype,))
                _need(out.shape == q.shape, "out does not fit q")
                _writable(out, "out")
            sref = ctypes.byref(seqs)
            ws = torch.empty(B.kv4_attention_workspace_bytes(self._ref, sref, rows, heads, accumulate), dtype=torch.uint8,
                             device=dev)
            x = B.sc_kv4_query(_TYPE[q.dtype], rows, heads, scale, q.data_ptr(), out.data_ptr(), q.stride()[:3],
                               out.stride()[:3])
            B.kv4_attention(self._ref, sref, ctypes.byref(x), accumulate, ws.data_ptr(), s)
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
        is."""
        _need(self.weights is not None, "the cache keeps no weights")
        seqs = self._seqs(table, lens)
        _need(keep >= 1 and recent >= 0 and sinks >= 0 and recent + sinks <= keep,
              "keep must be positive, recent and sinks >= 0 and together at most keep")
        _need(keep < 2 ** 31, "keep is too large")
        with _On(self.device, stream) as s:
            new = torch.empty_like(lens)
            sref = ctypes.byref(seqs)
            ws = torch.empty(B.kv4_evict_workspace_bytes(self._ref, sref, keep), dtype=torch.uint8, device=self.device)
            B.kv4_evict(self._ref, sref, keep, recent, sinks, new.data_ptr(), ws.data_ptr(), s)
            if s not in self._streams:
                self._used_on(s)
        if stream is not None:
            _record(stream, table, lens, new)
        return new
