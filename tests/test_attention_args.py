"""Refusals of the attention operators and of the 4-bit key/value cache: wrong
arguments return an error before anything is enqueued (no GPU needed)."""
import ctypes

import pytest

from hbm_expert_slot_amd import binding as B

P = 0x10000     # stands for a device pointer: never followed
R = ctypes.byref


def _fails(f, *args):
    with pytest.raises(B.SlotCacheError) as e:
        f(*args)
    assert e.value.status == B.SC_E_ARG and str(e.value)


def _cache(**kw):
    d = dict(format=B.SC_FP4_NV, head_dim=128, kv_heads=8, n_pages=4, d_pages=P, d_weights=P, d_positions=P,
             d_k_scale=None, d_v_scale=P)
    d.update(kw)
    return B.sc_kv4_cache(*[d[n] for n, _ in B.sc_kv4_cache._fields_])


def _seqs(**kw):
    d = dict(n_seqs=2, width=3, ld_table=3, d_table=P, d_lens=P)
    d.update(kw)
    return B.sc_kv4_seqs(*[d[n] for n, _ in B.sc_kv4_seqs._fields_])


def _rows(**kw):
    d = dict(type=B.SC_DTYPE_BF16, d_k=P, d_v=P, k_token=1024, k_head=128, v_token=1024, v_head=128)
    d.update(kw)
    return B.sc_kv4_rows(*[d[n] for n, _ in B.sc_kv4_rows._fields_])


def _query(**kw):
    d = dict(type=B.SC_DTYPE_BF16, rows=1, q_heads=16, scale=0.1, d_q=P, d_out=P, q_stride=(2048, 2048, 128),
             out_stride=(2048, 2048, 128))
    d.update(kw)
    return B.sc_kv4_query(*[d[n] for n, _ in B.sc_kv4_query._fields_])


BAD_CACHES = [dict(format=2), dict(head_dim=96), dict(head_dim=0), dict(kv_heads=0), dict(kv_heads=1025), dict(n_pages=0),
              dict(d_pages=None), dict(d_pages=P + 8), dict(d_weights=None), dict(d_positions=None), dict(d_weights=P + 4),
              dict(d_k_scale=P + 2), dict(format=B.SC_FP4_MX)]
BAD_SEQS = [dict(n_seqs=-1), dict(n_seqs=65537), dict(width=0), dict(width=(1 << 24) + 1), dict(ld_table=2),
            dict(d_table=None), dict(d_lens=None), dict(d_table=P + 2), dict(d_lens=P + 1)]


def _every_call(c, s):
    return [(B.kv4_append, c, s, R(_rows()), 2, None, None, None), (B.kv4_read, c, s, R(_rows()), 2, None, None),
            (B.kv4_attention, c, s, R(_query()), 0, P, None), (B.kv4_attention_workspace_bytes, c, s, 1, 16, 0),
            (B.kv4_evict, c, s, 10, 0, 0, P, P, None), (B.kv4_evict_workspace_bytes, c, s, 10)]


@pytest.mark.parametrize("change", BAD_CACHES)
def test_caches_that_are_refused(change):
    for call in _every_call(R(_cache(**change)), R(_seqs())):
        _fails(*call)


@pytest.mark.parametrize("change", BAD_SEQS)
def test_sequences_that_are_refused(change):
    for call in _every_call(R(_cache()), R(_seqs(**change))):
        _fails(*call)


def test_null_structures():
    for call in _every_call(None, R(_seqs())) + _every_call(R(_cache()), None):
        _fails(*call)
    c, s = R(_cache()), R(_seqs())
    _fails(B.kv4_append, c, s, None, 2, None, None, None)
    _fails(B.kv4_read, c, s, None, 2, None, None)
    _fails(B.kv4_attention, c, s, None, 0, P, None)
    _fails(B.prompt_attention, None, None, None)


@pytest.mark.parametrize("change,tokens", [
    (dict(type=3), 2), (dict(d_k=None), 2), (dict(d_v=None), 2), (dict(d_k=P + 1), 2), (dict(type=B.SC_DTYPE_F32, d_v=P + 2), 2),
    (dict(k_token=-1), 2), (dict(v_head=-1), 2), (dict(), -1), (dict(), 3), (dict(), 2 ** 31 - 2),
])
def test_rows_that_are_refused(change, tokens):
    c, s, r = R(_cache()), R(_seqs()), R(_rows(**change))
    _fails(B.kv4_append, c, s, r, tokens, None, None, None)
    _fails(B.kv4_read, c, s, r, tokens, None, None)


def test_unaligned_starts_and_positions():
    c, s, r = R(_cache()), R(_seqs()), R(_rows())
    _fails(B.kv4_append, c, s, r, 2, P + 2, None, None)
    _fails(B.kv4_append, c, s, r, 2, P, P + 1, None)
    _fails(B.kv4_read, c, s, r, 2, P + 2, None)


@pytest.mark.parametrize("change", [
    dict(type=B.SC_DTYPE_F32), dict(rows=0), dict(rows=17), dict(q_heads=0), dict(q_heads=12), dict(q_heads=8 * 65),
    dict(scale=0.0), dict(scale=-1.0), dict(scale=float("nan")), dict(scale=float("inf")), dict(d_q=None), dict(d_out=None),
    dict(d_q=P + 1), dict(q_stride=(-1, 0, 0)), dict(out_stride=(0, 0, -128)),
])
def test_queries_that_are_refused(change):
    _fails(B.kv4_attention, R(_cache()), R(_seqs()), R(_query(**change)), 0, P, None)


def test_attention_workspace_and_weights():
    c, s, q = R(_cache()), R(_seqs()), R(_query())
    _fails(B.kv4_attention, c, s, q, 0, None, None)
    _fails(B.kv4_attention, c, s, q, 0, P + 16, None)
    _fails(B.kv4_attention, R(_cache(d_weights=None, d_positions=None)), s, q, 1, P, None)
    n = B.kv4_attention_workspace_bytes(c, s, 1, 16, 0)
    assert B.kv4_attention_workspace_bytes(c, s, 1, 16, 1) > n > 0
    _fails(B.kv4_attention, c, R(_seqs(n_seqs=65536)), R(_query(rows=16)), 0, P, None)     # 2^24 query rows


@pytest.mark.parametrize("keep,recent,sinks", [(0, 0, 0), (-1, 0, 0), (4, 5, 0), (4, 3, 2), (4, -1, 0), (4, 0, -1),
                                               (4, 2 ** 31 - 1, 2 ** 31 - 1)])
def test_evictions_that_are_refused(keep, recent, sinks):
    _fails(B.kv4_evict, R(_cache()), R(_seqs()), keep, recent, sinks, P, P, None)


def test_eviction_needs_weights_and_memory():
    c, s = R(_cache()), R(_seqs())
    _fails(B.kv4_evict, R(_cache(d_weights=None, d_positions=None)), s, 4, 0, 0, P, P, None)
    _fails(B.kv4_evict, c, s, 4, 0, 0, None, P, None)
    _fails(B.kv4_evict, c, s, 4, 0, 0, P, None, None)
    _fails(B.kv4_evict, c, s, 4, 0, 0, P + 2, P, None)
    _fails(B.kv4_evict, c, s, 4, 0, 0, P, P + 2, None)
    assert B.kv4_evict_workspace_bytes(c, s, 64) > B.kv4_evict_workspace_bytes(c, s, 1000) > 0


def test_page_bytes():
    assert B.kv4_page_bytes(B.SC_FP4_NV, 128) == 2 * 64 * (64 + 8)
    assert B.kv4_page_bytes(B.SC_FP4_MX, 256) == 2 * 64 * (128 + 8)
    _fails(B.kv4_page_bytes, 5, 128)
    _fails(B.kv4_page_bytes, B.SC_FP4_NV, 80)


def _prompt(**kw):
    d = dict(type=B.SC_DTYPE_BF16, head_dim=128, q_heads=16, kv_heads=4, n_seqs=2, rows=100, keys=100, scale=0.1, d_q=P,
             d_k=P, d_v=P, d_out=P, d_lse=None, d_starts=P, d_key_starts=P, q_stride=(2048, 128), k_stride=(512, 128),
             v_stride=(512, 128), out_stride=(2048, 128))
    d.update(kw)
    return B.sc_prompt(*[d[n] for n, _ in B.sc_prompt._fields_])


@pytest.mark.parametrize("change", [
    dict(type=B.SC_DTYPE_F32), dict(head_dim=96), dict(q_heads=0), dict(kv_heads=0), dict(kv_heads=3), dict(q_heads=2048),
    dict(n_seqs=-1), dict(n_seqs=65537), dict(rows=-1), dict(rows=(1 << 24) + 1), dict(keys=-1), dict(scale=0.0),
    dict(scale=float("nan")), dict(scale=float("inf")), dict(d_q=None), dict(d_k=None), dict(d_v=None), dict(d_out=None),
    dict(d_q=P + 1), dict(d_lse=P + 2), dict(d_starts=None), dict(d_key_starts=None), dict(d_starts=P + 2),
    dict(rows=1 << 24, q_heads=1024, kv_heads=1), dict(k_stride=((1 << 23) + 1, 0)), dict(v_stride=((1 << 23) + 1, 0)),
    dict(q_stride=(-1, 0)), dict(k_stride=(0, -1)), dict(v_stride=(-1, 0)), dict(out_stride=(-1, 0)),
])
def test_prompts_that_are_refused(change):
    _fails(B.prompt_attention, R(_prompt(**change)), None, None)


def test_prompt_workspace():
    assert B.prompt_attention_workspace_bytes(R(_prompt())) == 0
    few = _prompt(rows=100, keys=20000)
    assert B.prompt_attention_workspace_bytes(R(few)) > 0
    _fails(B.prompt_attention, R(few), None, None)
    _fails(B.prompt_attention, R(few), P + 8, None)
    _fails(B.prompt_attention_workspace_bytes, None)
    _fails(B.prompt_attention_workspace_bytes, R(_prompt(head_dim=80)))


def test_nothing_to_do_is_no_error():
    B.prompt_attention(R(_prompt(rows=0)), None, None)
    B.prompt_attention(R(_prompt(n_seqs=0)), None, None)
    c, none = R(_cache()), R(_seqs(n_seqs=0))
    B.kv4_append(c, none, R(_rows()), 0, None, None, None)
    B.kv4_read(c, R(_seqs()), R(_rows()), 0, None, None)
    B.kv4_attention(c, none, R(_query()), 0, P, None)
    B.kv4_evict(c, none, 4, 0, 0, None, None, None)


def test_the_python_layer_names_what_is_wrong():
    torch = pytest.importorskip("torch")
    from hbm_expert_slot_amd import ops
    q = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="q must be on the GPU"):
        ops.prompt_attention(q, q, q, torch.tensor([0, 4], dtype=torch.int32))
    with pytest.raises(ValueError, match="q must be"):
        ops.prompt_attention(q[0], q, q, torch.tensor([0, 4], dtype=torch.int32))
    with pytest.raises(ValueError, match="q has type"):
        ops.prompt_attention(q.float(), q, q, torch.tensor([0, 4], dtype=torch.int32))
    for kw in (dict(fmt="fp4"), dict(head_dim=80), dict(n_pages=0), dict(kv_heads=0), dict(kv_heads=1025),
               dict(fmt="mxfp4", k_scale=torch.ones(1))):
        with pytest.raises(ValueError):
            ops.KV4Cache(**dict(dict(n_pages=2, kv_heads=2, head_dim=64), **kw))


def test_structures_as_bytes():
    """The packed forms have the layout of the structures."""
    import ctypes as ct
    for packer, cls, flat in ((B.PROMPT, B.sc_prompt, 23), (B.KV4_SEQS, B.sc_kv4_seqs, 5), (B.KV4_ROWS, B.sc_kv4_rows, 7),
                              (B.KV4_QUERY, B.sc_kv4_query, 12)):
        assert packer.size == ct.sizeof(cls)
        got = cls.from_buffer_copy(packer.pack(*range(1, flat + 1)))
        vals = []
        for name, _ in cls._fields_:
            v = getattr(got, name)
            vals += list(v) if isinstance(v, ct.Array) else [v]
        assert vals == list(range(1, flat + 1))


def test_new_lengths_over_the_lengths_are_refused():
    """Blocks of other heads may read a length when its new one is written."""
    c, s = R(_cache()), R(_seqs(d_lens=P, n_seqs=4))
    for new in (P, P + 4, P + 12, P - 12):
        _fails(B.kv4_evict, c, s, 4, 0, 0, new, P + 4096, None)
        assert "overlap" in B.slotcache_last_error()


def _workspace(**kw):
    return B.prompt_attention_workspace_bytes(R(_prompt(**kw)))


@pytest.mark.parametrize("rows,keys,heads,n", [(65536, 16384, 32, 1), (200000, 8192, 32, 1), (1 << 20, 8192, 8, 1),
                                               (1 << 24, 8192, 127, 1), (1 << 24, 1 << 23, 64, 3), (16385, 16384, 16, 1)])
def test_rows_that_see_nothing_need_no_workspace(rows, keys, heads, n):
    """More rows than keys: the first ones are no work that could be uneven."""
    assert _workspace(rows=rows, keys=keys, q_heads=heads, kv_heads=1, n_seqs=n) == 0


def test_prompt_workspace_is_bounded():
    for d in (64, 128, 256):
        most = 0
        for heads in (1, 2, 4, 7, 8, 16, 32, 64, 128):
            for n in (1, 3, 16, 64, 300, 1000, 4000):
                for rows in (1, 16, 127, 1000, 4096, 16384, 70000):
                    for keys in (0, 4095, 4096, 10000, 100000):
                        sizes = dict(rows=rows * n, keys=keys * n, q_heads=heads, kv_heads=1, n_seqs=n, head_dim=d)
                        if rows * n <= 1 << 24 and (rows * n // 128 + n) * heads < 1 << 24:
                            most = max(most, _workspace(**sizes))
        assert 0 < most <= 5120 * 128 * (4 * d + 8)
    # parts that were measured as a gain
    assert _workspace(rows=16384, keys=16384, q_heads=4, kv_heads=4, n_seqs=1) == 2 * 129 * 4 * 128 * (512 + 8)
    assert _workspace(rows=16 * 64, keys=8000 * 64, q_heads=32, kv_heads=8, n_seqs=64) > 0
    assert _workspace(rows=1107, keys=13527, q_heads=16, kv_heads=2, n_seqs=2, head_dim=256) > 0


@pytest.mark.parametrize("heads,dim", [(1, 64), (1, 256), (3, 128), (8, 128), (1024, 256)])
def test_the_most_tokens_of_a_call(heads, dim):
    """tokens * kv_heads * head_dim < 2^32, and no less.  Keys that are NULL are what is wrong with a call that is
    not too large."""
    c, s, r = R(_cache(kv_heads=heads, head_dim=dim)), R(_seqs(n_seqs=1)), R(_rows(d_k=None))
    most = (2 ** 32 - 1) // (heads * dim)
    for tokens, what in ((most, "NULL"), (most + 1, "too many tokens")):
        for f, args in ((B.kv4_append, (P, None, None)), (B.kv4_read, (P, None))):
            with pytest.raises(B.SlotCacheError, match=what):
                f(c, s, r, tokens, *args)


def test_the_most_query_rows_of_a_call():
    c = R(_cache(kv_heads=8))
    for n, rows, heads in ((65536, 16, 8), (65536, 2, 64), (16384, 1, 512)):
        assert B.kv4_attention_workspace_bytes(c, R(_seqs(n_seqs=n)), rows, heads, 1) > 0
    for n, rows, heads in ((65536, 16, 16), (65536, 3, 64), (16385, 1, 512)):
        _fails(B.kv4_attention_workspace_bytes, c, R(_seqs(n_seqs=n)), rows, heads, 1)
        _fails(B.kv4_attention, c, R(_seqs(n_seqs=n)), R(_query(rows=rows, q_heads=heads)), 0, P, None)


def test_the_most_sequences_of_an_eviction():
    for n, heads in ((65536, 2), (16384, 8), (128, 1024)):
        assert B.kv4_evict_workspace_bytes(R(_cache(kv_heads=heads)), R(_seqs(n_seqs=n)), 10) > 0
    for n, heads in ((65536, 3), (16385, 8), (129, 1024)):
        _fails(B.kv4_evict_workspace_bytes, R(_cache(kv_heads=heads)), R(_seqs(n_seqs=n)), 10)
        _fails(B.kv4_evict, R(_cache(kv_heads=heads)), R(_seqs(n_seqs=n)), 10, 0, 0, 16 * P, 2 * P, None)


@pytest.mark.parametrize("first", [
    "import hbm_expert_slot_amd.attention", "from hbm_expert_slot_amd.attention import KV4Cache, prompt_attention",
    "from hbm_expert_slot_amd.ops import KV4Cache, prompt_attention", "from hbm_expert_slot_amd.ops import *; KV4Cache; FP4Weight",
    "import hbm_expert_slot_amd as h; h.ops.prompt_attention; assert 'KV4Cache' in dir(h.ops)",
])
def test_either_module_can_be_imported_first(first):
    pytest.importorskip("torch")
    import os
    import subprocess
    import sys
    check = "; from hbm_expert_slot_amd import attention, ops; assert ops.KV4Cache is attention.KV4Cache and " \
            "ops.prompt_attention is attention.prompt_attention and not hasattr(ops, 'prompt')"
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", first + check], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-1000:]


def test_scales_that_exceed_fp32_in_base_2():
    """Scores are formed in base 2: log2(e) times a scale above 2.358e38 would be infinite, and 0 times that NaN."""
    torch = pytest.importorskip("torch")
    from hbm_expert_slot_amd import attention
    assert torch.tensor(2.3e38) * 1.4426950408889634 < float("inf") and torch.tensor(2.36e38) * 1.4426950408889634 == float("inf")
    for scale in (2.31e38, 2.9e38):
        _fails(B.prompt_attention, R(_prompt(scale=scale)), None, None)
        _fails(B.kv4_attention, R(_cache()), R(_seqs()), R(_query(scale=scale)), 0, P, None)
        with pytest.raises(ValueError, match="scale"):
            attention._scale_of(scale, 64)
    assert attention._scale_of(2.3e38, 64) == 2.3e38
