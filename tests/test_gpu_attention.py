"""Attention over prompts, the 4-bit key/value cache, attention over it and
eviction from it, against float64."""
import numpy as np
import pytest

from oracle import attention as oa

from gpu_util import log, torch_cuda

pytestmark = pytest.mark.gpu

TYPES = {"bf16": "bfloat16", "fp16": "float16", "fp32": "float32"}
EPS = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11, "fp32": 2.0 ** -24}      # half a step
P_EPS = {"nvfp4": (2.0 ** -11, 2.0 ** -39), "mxfp4": (2.0 ** -16, 0.0)}      # of P: relative, of the largest
TINY = {"bf16": 1e-37, "fp16": 2.0 ** -25, "fp32": 1e-37}


def _ops():
    from hbm_expert_slot_amd import ops
    return ops


def _np(t):
    return t.detach().cpu().double().numpy()


def _ints(torch, v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _starts(torch, n):
    return _ints(torch, np.concatenate(([0], np.cumsum(n))).tolist())


def _randn(torch, seed, *shape):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return torch.randn(*shape, generator=g, device="cuda")


def _close(got, want, bound, dtype, what):
    got = _np(got)
    assert np.array_equal(np.isnan(got), np.isnan(want)), (what, "NaN")
    assert np.array_equal(np.isinf(got), np.isinf(want)), (what, "infinities")
    ok = np.isfinite(want)
    over = np.abs(got[ok] - want[ok]) - (bound[ok] * (1 + EPS[dtype]) + EPS[dtype] * np.abs(want[ok]) + TINY[dtype])
    assert over.size == 0 or over.max() <= 0, (what, float(over.max()), int(over.argmax()))


# ---- prompts ---------------------------------------------------------------

def _check_prompt(torch, q, k, v, new, full, dtype, scale=None, lse=True):
    ops = _ops()
    starts, key_starts = _starts(torch, new), _starts(torch, full)
    out, ls = ops.prompt_attention(q, k, v, starts, key_starts, scale=scale, return_lse=True)
    assert out.dtype == q.dtype and out.shape == q.shape
    qn, kn, vn = _np(q), _np(k), _np(v)
    sc = 1.0 / np.sqrt(q.shape[2]) if scale is None else scale
    q0 = k0 = 0
    for i, (n, a) in enumerate(zip(new, full)):
        o, l, _, eo, el, _ = oa.attend(qn[q0:q0 + n], kn[k0:k0 + a], vn[k0:k0 + a], sc, EPS[dtype], 2.0 ** -39 if dtype == "fp16" else 0.0)
        _close(out[q0:q0 + n], o, eo, dtype, ("out", i, n, a))
        _close(ls[q0:q0 + n], l, el, "fp32", ("lse", i, n, a))
        q0, k0 = q0 + n, k0 + a
    return out


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("d,hq,hkv", [(64, 4, 2), (128, 6, 2), (256, 3, 1), (128, 1, 1), (64, 8, 1)])
def test_prompts_of_all_lengths(d, hq, hkv, dtype):
    torch = torch_cuda()
    log("prompts", d, hq, hkv, dtype)
    new = [1, 2, 31, 32, 33, 0, 63, 64, 65, 127, 128, 129, 200]
    T = sum(new)
    dt = getattr(torch, TYPES[dtype])
    q, k, v = (_randn(torch, 3 * d + i, T, h, d).to(dt) for i, h in enumerate((hq, hkv, hkv)))
    _check_prompt(torch, 2 * q, k, v, new, new, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("new,full", [([1, 1], [300, 1]), ([5, 40, 0, 130], [700, 40, 9, 131]), ([64], [1000]),
                                      ([10, 200], [3, 140])])
def test_chunks_of_prompts(new, full, dtype):
    """More keys than rows; and fewer, whose first rows see nothing."""
    torch = torch_cuda()
    log("chunks", new, full, dtype)
    dt = getattr(torch, TYPES[dtype])
    q = _randn(torch, 1, sum(new), 4, 128).to(dt)
    k, v = (_randn(torch, 2 + i, sum(full), 2, 128).to(dt) for i in range(2))
    _check_prompt(torch, q, k, v, new, full, dtype, scale=0.2)


@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("fp16", 64), ("bf16", 256)])
def test_few_rows_over_many_keys(dtype, d):
    """Keys in parts, some of which are behind what a row sees, or of sequences that have no key for a part."""
    torch = torch_cuda()
    log("few rows, many keys", dtype, d)
    dt = getattr(torch, TYPES[dtype])
    for new, full in (([7, 130, 1], [9000, 131, 8000]), ([3, 0, 2], [16500, 10, 1]), ([40], [5000])):
        q = _randn(torch, 1, sum(new), 2, d).to(dt)
        k, v = (_randn(torch, 2 + i, sum(full) + 3, 1, d).to(dt)[3:] for i in range(2))
        assert sum(full) // len(full) >= 4096
        _check_prompt(torch, 2 * q, k, v, new, full, dtype)


def test_prompt_of_a_few_thousand_tokens():
    torch = torch_cuda()
    log("long prompt")
    q, k, v = (_randn(torch, i, 1500, 2, 128).to(torch.bfloat16) for i in range(3))
    k[700:710] *= 8          # the maximum moves late
    _check_prompt(torch, 3 * q, k, v, [1500], [1500], "bf16")


def test_prompt_strides_and_alignment():
    """Views of one projection at odd offsets, heads apart, and an output inside a larger tensor."""
    torch = torch_cuda()
    log("prompt strides")
    new, hq, hkv, d = [70, 33, 129], 4, 2, 64
    T = sum(new)
    x = _randn(torch, 5, T, (hq + 2 * hkv) * d + 3).to(torch.bfloat16)
    q = x[:, 1:1 + hq * d].unflatten(1, (hq, d))
    k = x[:, 1 + hq * d:1 + (hq + hkv) * d].unflatten(1, (hkv, d))
    v = x[:, 1 + (hq + hkv) * d:1 + (hq + 2 * hkv) * d].unflatten(1, (hkv, d))
    want = _check_prompt(torch, q, k, v, new, new, "bf16")
    big = torch.full((T + 2, hq + 1, d + 5), 7.0, dtype=torch.bfloat16, device="cuda")
    out = big[1:T + 1, 1:, 3:3 + d]
    got = _ops().prompt_attention(q, k, v, _starts(torch, new), out=out)
    assert got.data_ptr() == out.data_ptr() and torch.equal(out, want)
    out.fill_(7.0)
    assert bool((big == 7.0).all())
    # heads before tokens
    kt = k.transpose(0, 1).contiguous().transpose(0, 1)
    vt = v.transpose(0, 1).contiguous().transpose(0, 1)
    assert torch.equal(_ops().prompt_attention(q, kt, vt, _starts(torch, new)), want)
    # one head for all by a stride of zero
    one = _ops().prompt_attention(q, k[:, :1], v[:, :1], _starts(torch, new))
    assert torch.equal(_ops().prompt_attention(q, k[:, :1].expand(-1, 4, -1), v[:, :1].expand(-1, 4, -1),
                                               _starts(torch, new)), one)


def test_prompt_rows_outside_of_the_sequences():
    torch = torch_cuda()
    log("rows behind the last sequence")
    q, k, v = (_randn(torch, i, 300, 2, 64).to(torch.float16) for i in range(3))
    out = torch.full_like(q, 9.0)
    k[250:], v[250:] = float("nan"), float("inf")         # of no sequence
    _ops().prompt_attention(q, k, v, _ints(torch, [10, 100, 250]), out=out)
    assert bool((out[:10] == 9.0).all()) and bool((out[250:] == 9.0).all()) and bool(torch.isfinite(out).all())
    want = _ops().prompt_attention(q[10:100].contiguous(), k[10:100].contiguous(), v[10:100].contiguous(),
                                   _ints(torch, [0, 90]))
    assert torch.equal(out[10:100], want)
    # starts that make no sense: nothing is written for that sequence
    for bad in ([0, 400], [50, 20], [-3, 20]):
        out.fill_(9.0)
        _ops().prompt_attention(q, k, v, _ints(torch, bad), out=out)
        assert bool((out == 9.0).all()), bad


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("which", ["k", "v"])
@pytest.mark.parametrize("at", [0, 40, 90, 199])
def test_prompt_values_that_are_not_finite(at, which, bad):
    """Rows before the token do not see it; the others do."""
    torch = torch_cuda()
    log("not finite", at, which, bad)
    q, k, v = (_randn(torch, i, 200, 2, 64).to(torch.bfloat16) for i in range(3))
    sane = _ops().prompt_attention(q, k, v, _ints(torch, [0, 200]))
    (k if which == "k" else v)[at, 0, 5] = bad
    out = _ops().prompt_attention(q, k, v, _ints(torch, [0, 200]))
    assert torch.equal(out[:at], sane[:at]) and torch.equal(out[:, 1], sane[:, 1])
    if which == "v":
        o = out[at:, 0]
        assert not bool(torch.isfinite(o[:, 5]).any()) and torch.equal(torch.cat((o[:, :5], o[:, 6:]), 1),
                                                                       torch.cat((sane[at:, 0, :5], sane[at:, 0, 6:]), 1))
    elif bad != bad:
        assert bool(torch.isnan(out[at:, 0]).all())


# ---- the cache -------------------------------------------------------------

class Filled:
    """A cache with sequences of given lengths on pages in random order, among pages of NaN scales; the float64
    values it holds by place."""

    def __init__(self, torch, fmt, d, hkv, lens, dtype="bf16", track=False, scales=(None, None), seed=0, extra=0, size=1.0):
        rng = np.random.default_rng(seed)
        need = [(n + extra + 63) // 64 for n in lens]
        pages = sum(need) + 3
        self.torch, self.lens, self.hkv, self.d = torch, list(lens), hkv, d
        gs = [None if s is None else torch.tensor([s], device="cuda") for s in scales]
        self.cache = _ops().KV4Cache(pages, hkv, d, fmt, k_scale=gs[0], v_scale=gs[1], track=track)
        self.cache.pages.fill_(255)
        if track:
            self.cache.weights.fill_(float("nan"))
        order = rng.permutation(pages)
        table = np.full((len(lens), max(max(need), 1) + 1), -1, np.int32)
        i = 0
        for b, n in enumerate(need):
            table[b, :n] = order[i:i + n]
            i += n
        self.table, self.d_lens = _ints(torch, table.tolist()), _ints(torch, list(lens))
        T = sum(lens)
        dt = getattr(torch, TYPES[dtype])
        k = (_randn(torch, seed + 1, T, hkv, d) * size).to(dt)
        v = (_randn(torch, seed + 2, T, hkv, d) * size).to(dt)
        self.fmt, self.scales = fmt, scales
        self.k, self.v = self.held(k, 0), self.held(v, 1)
        self.cache.append(k, v, self.table, self.d_lens, _starts(torch, lens))

    def held(self, x, side):
        g = self.scales[side]
        return oa.quantized(_np(x), self.fmt, None if g is None else np.float32(g))

    def of(self, b):
        s = sum(self.lens[:b])
        return self.k[s:s + self.lens[b]], self.v[s:s + self.lens[b]]

    def check_read(self, dtypes=("bf16", "fp32")):
        torch = self.torch
        for dt in dtypes:
            k, v = self.cache.read(self.table, self.d_lens, sum(self.lens), _starts(torch, self.lens),
                                   dtype=getattr(torch, TYPES[dt]))
            for got, want in ((k, self.k), (v, self.v)):
                w = torch.tensor(want).float().to(getattr(torch, TYPES[dt]))
                assert torch.equal(torch.nan_to_num(got.cpu(), nan=777.0), torch.nan_to_num(w, nan=777.0)), dt


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("d,hkv", [(64, 3), (128, 2), (256, 1)])
def test_append_and_read(d, hkv, fmt, dtype):
    torch = torch_cuda()
    log("append", d, hkv, fmt, dtype)
    Filled(torch, fmt, d, hkv, [1, 0, 5, 63, 64, 65, 200], dtype, seed=d).check_read(("bf16", "fp16", "fp32"))
    if fmt == "nvfp4":
        Filled(torch, fmt, d, hkv, [130, 7], dtype, scales=(0.037, 2.0 ** -9), seed=d + 1).check_read()
        # scales that reach the ends of E4M3
        Filled(torch, fmt, d, hkv, [130, 7], dtype, scales=(100.0, 1e-5), seed=d + 2).check_read(("fp32",))


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
def test_append_on_and_beside_borders(dtype):
    """Every bf16 (fp16) number of a few binades against largest elements whose scale is or is not rounded: quotients
    that are borders, and those a step beside; then scales far from 1, subnormal and largest numbers."""
    torch = torch_cuda()
    log("append borders", dtype)
    dt = getattr(torch, TYPES[dtype])
    bits = {"bf16": 7, "fp16": 10, "fp32": 10}[dtype]
    m = np.arange(1 << bits) / (1 << bits) + 1.0
    x = np.concatenate([m * 2.0 ** e for e in range(-4, 3)])
    x = np.concatenate((x, -x))
    tops = [6.0, 6.5, 7.0, 5.5, 4.25, 6.75, 15.75, 3.0 * (1 + 2.0 ** -bits), 448.0 * 6]
    for scales in ((None, None), (0.5, 4.0), (0.037, 1.5)):
        rows = []
        for t in tops:
            y = x[: len(x) // 60 * 60].reshape(-1, 60)
            y = np.concatenate((y[:, :15], np.full((len(y), 1), t), y[:, 15:30], np.full((len(y), 1), -t), y[:, 30:45],
                                np.full((len(y), 1), t), y[:, 45:], np.full((len(y), 1), t)), 1)
            rows.append(y)
        y = np.concatenate(rows)
        if dtype == "fp32":                      # a step of fp32 beside the borders
            y = np.concatenate((y, np.nextafter(y.astype(np.float32), np.float32(0)), np.nextafter(y.astype(np.float32), np.float32(1e9))))
        for size in (1.0, 2.0 ** -12):
            k = torch.tensor(y * size, dtype=torch.float64).to(dt).cuda().view(-1, 1, 64)
            c = Filled(torch, "nvfp4", 64, 1, [k.shape[0]], dtype, scales=scales)
            c.cache.append(k, k, c.table, c.d_lens)
            c.k, c.v = c.held(k, 0), c.held(k, 1)
            c.check_read(("fp32",))
    y = np.concatenate(rows)
    for size in (2.0 ** -14, 2.0 ** -24, 2.0 ** 4):
        k = torch.tensor(y * size, dtype=torch.float64).to(dt).cuda().view(-1, 1, 64)
        for fmt in ("nvfp4", "mxfp4"):
            c = Filled(torch, fmt, 64, 1, [k.shape[0]], dtype)
            c.cache.append(k, k, c.table, c.d_lens)
            c.k, c.v = c.held(k, 0), c.held(k, 1)
            c.check_read(("fp32",))


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
def test_append_what_is_not_finite(fmt):
    torch = torch_cuda()
    log("append nan", fmt)
    c = Filled(torch, fmt, 128, 2, [70], "fp32")
    x = _randn(torch, 9, 3, 2, 128)
    x[0, 0, 5], x[1, 1, 100], x[2, 0, 127] = float("nan"), float("inf"), -float("inf")
    c.cache.append(x, -x, c.table, c.d_lens)
    k, v = c.cache.read(c.table, c.d_lens, 3, dtype=torch.float32)
    g = 16 if fmt == "nvfp4" else 32
    nan = torch.isnan(k)
    assert torch.equal(nan, torch.isnan(v)) and int(nan.sum()) == 3 * g
    assert bool(nan[0, 0, 5]) and bool(nan[1, 1, 100]) and bool(nan[2, 0, 127])


def test_append_in_steps_gives_the_same_cache():
    """Token by token with drafts that are overwritten, and all at once."""
    torch = torch_cuda()
    log("append in steps")
    c = Filled(torch, "nvfp4", 128, 2, [140, 90], track=True)
    n = [140, 90]
    k, v = _randn(torch, 1, 230, 2, 128).to(torch.bfloat16), _randn(torch, 2, 230, 2, 128).to(torch.bfloat16)
    whole = _ops().KV4Cache(c.cache.n_pages, 2, 128, track=True)
    whole.append(k, v, c.table, c.d_lens, _starts(torch, n))
    step = _ops().KV4Cache(c.cache.n_pages, 2, 128, track=True)
    at = [0, 0]
    rng = np.random.default_rng(3)
    while at != n:
        take = [min(int(rng.integers(0, 9)), n[b] - at[b]) for b in range(2)]
        junk = [min(3, n[b] - at[b] - take[b]) for b in range(2)]
        # drafts first, which the next step overwrites
        for extra in (junk, [0, 0]):
            cnt = [take[b] + extra[b] for b in range(2)]
            rows = torch.cat([torch.arange(at[b], at[b] + cnt[b]) + (0 if b == 0 else 140) for b in range(2)]).cuda()
            kk, vv = k[rows], v[rows]
            if extra is junk:
                kk, vv = kk * 3, vv - 1
            step.append(kk, vv, c.table, _ints(torch, [at[b] + cnt[b] for b in range(2)]), _starts(torch, cnt))
        at = [at[b] + take[b] for b in range(2)]
    for p in range(2):
        a = whole.read(c.table, c.d_lens, 230, _starts(torch, n))[p]
        assert torch.equal(a, step.read(c.table, c.d_lens, 230, _starts(torch, n))[p])
    for b in range(2):
        for i in range(n[b]):
            page = int(c.table[b, i // 64])
            assert int(step.positions[page, 1, i % 64]) == i and float(step.weights[page, 0, i % 64]) == 0.0


def test_append_strides_and_given_positions():
    torch = torch_cuda()
    log("append strides")
    c = Filled(torch, "mxfp4", 64, 2, [100], track=True)
    x = _randn(torch, 4, 5, 2 * 2 * 64 + 1).half()
    k, v = x[:, 1:129].unflatten(1, (2, 64)), x[:, 129:].unflatten(1, (2, 64))
    c.cache.append(k, v, c.table, c.d_lens, positions=_ints(torch, [7, 8, 9, 1000, 11]))
    gk, gv = c.cache.read(c.table, c.d_lens, 5, dtype=torch.float32)
    assert np.array_equal(_np(gk), oa.quantized(_np(k), "mxfp4")) and np.array_equal(_np(gv), oa.quantized(_np(v), "mxfp4"))
    page = int(c.table[0, 1])
    assert c.cache.positions[page, 1, 31:36].tolist() == [7, 8, 9, 1000, 11]


def test_append_to_places_that_are_not_there():
    """Nothing is written: places behind the table or before it, pages outside of the cache, tokens of no sequence."""
    torch = torch_cuda()
    log("append nowhere")
    c = Filled(torch, "nvfp4", 64, 1, [64, 64], track=True)
    before = [t.clone() for t in (c.cache.pages, c.cache.weights, c.cache.positions)]
    k = _randn(torch, 1, 6, 1, 64)
    bad = c.table.clone()
    bad[:, 1] = _ints(torch, [-1, c.cache.n_pages])
    c.cache.append(k, k, bad, _ints(torch, [67, 67]))                            # pages -1 and n_pages
    c.cache.append(k, k, c.table[:, :1], _ints(torch, [67, 1000000]))            # behind the table
    c.cache.append(k, k, c.table, _ints(torch, [-5, 0]))                         # before the first place
    c.cache.append(k, k, c.table, _ints(torch, [3, 3]), _ints(torch, [9, 12, 15]))   # of no sequence
    for a, b in zip(before, (c.cache.pages, c.cache.weights, c.cache.positions)):
        assert torch.equal(torch.nan_to_num(a.float(), nan=7.0), torch.nan_to_num(b.float(), nan=7.0))
    k2, v2 = c.cache.read(c.table[:, :1], _ints(torch, [66, 64]), 6, dtype=torch.float32)
    nan = torch.isnan(k2).all(-1).flatten().tolist()
    assert nan == [False, True, True, False, False, False] and torch.equal(torch.isnan(k2), torch.isnan(v2))


# ---- attention over the cache ------------------------------------------------

def _check_attend(torch, c, q, dtype, accumulate=False, scale=None, out=None):
    got = c.cache.attend(q, c.table, c.d_lens, scale=scale, accumulate=accumulate, out=out)
    qn = _np(q)
    sc = 1.0 / np.sqrt(c.d) if scale is None else scale
    sums = []
    for b in range(len(c.lens)):
        k, v = c.of(b)
        o, _, w, eo, _, ew = oa.attend(qn[b], k, v, sc, *P_EPS[c.fmt])
        _close(got[b], o, eo, dtype, ("out", b, c.lens[b]))
        sums.append((w, ew))
    return got, sums


LENS = [1, 2, 15, 16, 17, 63, 64, 65, 127, 128, 129, 0, 700]


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("d,hkv,group,rows", [(64, 2, 1, 1), (64, 1, 7, 3), (128, 2, 8, 1), (128, 2, 6, 4), (128, 1, 5, 16),
                                              (256, 1, 4, 1), (256, 1, 9, 3), (128, 3, 1, 2)])
def test_attend(d, hkv, group, rows, fmt, dtype):
    torch = torch_cuda()
    log("attend", d, hkv, group, rows, fmt, dtype)
    c = Filled(torch, fmt, d, hkv, LENS, seed=d + rows)
    q = (2 * _randn(torch, 7, len(LENS), rows, hkv * group, d)).to(getattr(torch, TYPES[dtype]))
    _check_attend(torch, c, q, dtype)


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
def test_attend_one_long_sequence_and_short_ones(fmt):
    """Parts of the list that hold a head's middle, its end and many whole heads."""
    torch = torch_cuda()
    log("attend long", fmt)
    lens = [5, 9000, 1, 0, 64] + [3] * 70
    c = Filled(torch, fmt, 64, 2, lens, seed=3)
    q = _randn(torch, 8, len(lens), 2, 4, 64).to(torch.bfloat16)
    _check_attend(torch, c, 3 * q, "bf16", scale=0.3)


def test_attend_with_scales_of_all():
    torch = torch_cuda()
    log("attend scales")
    c = Filled(torch, "nvfp4", 128, 2, [77, 300], scales=(0.013, 2.5), seed=4)
    _check_attend(torch, c, _randn(torch, 1, 2, 1, 8, 128).to(torch.float16), "fp16")


@pytest.mark.parametrize("size", [1e-30, 1e-10, 1e4, 1e20])
@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
def test_attend_queries_of_any_size(size, fmt):
    torch = torch_cuda()
    log("attend query size", size, fmt)
    c = Filled(torch, fmt, 128, 1, [200], seed=5)
    q = _randn(torch, 1, 1, 2, 2, 128)
    q[:, :, :, 64:] *= 2.0 ** -20          # small elements beside large ones count
    q = (q * size).to(torch.bfloat16)
    _check_attend(torch, c, q, "bf16", scale=0.5 / size)


def test_attend_mxfp4_of_any_size():
    torch = torch_cuda()
    log("attend mxfp4 sizes")
    for size in (2.0 ** -60, 2.0 ** 50):
        c = Filled(torch, "mxfp4", 64, 1, [150], dtype="fp32", size=size, seed=6)
        q = _randn(torch, 1, 1, 1, 2, 64).to(torch.bfloat16)
        _check_attend(torch, c, q, "bf16", scale=1.0 / size / 8)


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
def test_attend_scores_far_apart(fmt):
    """One key takes everything, early or late, and scores around -1000."""
    torch = torch_cuda()
    log("attend far scores", fmt)
    c = Filled(torch, fmt, 64, 1, [300, 300], seed=7)
    q = 40 * _randn(torch, 1, 2, 1, 2, 64)
    _check_attend(torch, c, q.to(torch.bfloat16), "bf16", scale=1.0)


@pytest.mark.parametrize("fmt,dtype,d,hkv,group,rows", [("nvfp4", "bf16", 128, 2, 8, 1), ("mxfp4", "fp16", 128, 2, 8, 4),
                                                        ("nvfp4", "bf16", 64, 3, 5, 2), ("mxfp4", "bf16", 256, 1, 3, 6),
                                                        ("nvfp4", "fp16", 256, 1, 1, 1)])
def test_attend_keeps_weights(fmt, dtype, d, hkv, group, rows):
    torch = torch_cuda()
    log("attend weights", fmt, dtype, d, hkv, group, rows)
    c = Filled(torch, fmt, d, hkv, LENS, track=True, seed=11)
    start = c.cache.weights.clone()
    q = (2 * _randn(torch, 7, len(LENS), rows, hkv * group, d)).to(getattr(torch, TYPES[dtype]))
    got, sums = _check_attend(torch, c, q, dtype, accumulate=True)
    assert torch.equal(got, c.cache.attend(q, c.table, c.d_lens))
    _check_attend(torch, c, q, dtype, accumulate=True)                     # and adds the same again
    touched = torch.zeros_like(start, dtype=torch.bool)
    for b, (w, ew) in enumerate(sums):
        n = c.lens[b]
        for p in range((n + 63) // 64):
            m = min(64, n - 64 * p)
            page = int(c.table[b, p])
            touched[page, :, :m] = True
            got_w = c.cache.weights[page, :, :m].t()
            rows_w = slice(64 * p, 64 * p + m)
            _close(got_w, 2 * w[rows_w], 2 * ew[rows_w] + 2.0 ** -23 * w[rows_w], "fp32", ("weights", b, p))
    # tokens of no sequence keep what they had
    assert torch.equal(torch.nan_to_num(c.cache.weights[~touched], nan=7.0), torch.nan_to_num(start[~touched], nan=7.0))


def test_attend_lengths_and_pages_that_cannot_be():
    torch = torch_cuda()
    log("attend bad pages")
    c = Filled(torch, "nvfp4", 64, 2, [100, 100, 100, 100], track=True)
    q = _randn(torch, 1, 4, 2, 4, 64).to(torch.bfloat16)
    good = c.cache.attend(q, c.table, c.d_lens)
    bad = c.table.clone()
    bad[1, 1], bad[3, 0] = c.cache.n_pages, -7
    got = c.cache.attend(q, bad, c.d_lens, accumulate=True)
    assert torch.equal(got[0], good[0]) and torch.equal(got[2], good[2])
    assert bool(torch.isnan(got[1]).all()) and bool(torch.isnan(got[3]).all())
    got = c.cache.attend(q, c.table, _ints(torch, [100, -1, 64 * c.table.shape[1] + 1, 100]))
    assert torch.equal(got[0], good[0]) and torch.equal(got[3], good[3]) and bool(torch.isnan(got[1:3]).all())


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("which", ["k", "v"])
def test_attend_values_that_are_not_finite(which, fmt):
    """A token whose group reads as NaN: rows before it are not touched, the others are."""
    torch = torch_cuda()
    log("attend nan", which, fmt)
    for d in (64, 128, 256):
        c = Filled(torch, fmt, d, 2, [130, 90])
        q = _randn(torch, 1, 2, 4, 6, d).to(torch.bfloat16)
        k, v = _randn(torch, 2, 8, 2, d), _randn(torch, 3, 8, 2, d)
        c.cache.append(k, v, c.table, c.d_lens)
        sane = c.cache.attend(q, c.table, c.d_lens)
        (k if which == "k" else v)[2, 1, 35] = float("nan")           # row 2 of the first sequence, head 1
        c.cache.append(k, v, c.table, c.d_lens)
        out = c.cache.attend(q, c.table, c.d_lens)
        assert torch.equal(out[1], sane[1]) and torch.equal(out[0, :2], sane[0, :2]) and torch.equal(out[0, :, :3], sane[0, :, :3])
        nan = torch.isnan(out[0, 2:, 3:])
        if which == "k":
            assert bool(nan.all())
        else:
            g = 16 if fmt == "nvfp4" else 32
            lo = 35 // g * g
            assert bool(nan[..., lo:lo + g].all()) and int(nan.sum()) == nan.shape[0] * nan.shape[1] * g


def test_attend_strides():
    torch = torch_cuda()
    log("attend strides")
    c = Filled(torch, "nvfp4", 64, 2, [70, 5, 129])
    big = _randn(torch, 1, 2, 3, 6 * 64 + 3).to(torch.bfloat16)
    q = big[:, :, 2:2 + 4 * 64].unflatten(2, (4, 64)).transpose(0, 1)          # [3, 2, 4, 64]
    want = c.cache.attend(q.contiguous(), c.table, c.d_lens)
    assert torch.equal(c.cache.attend(q, c.table, c.d_lens), want)
    pool = torch.full((3, 5, 2, 64 + 1), 3.0, dtype=torch.bfloat16, device="cuda")
    out = pool[:, :4, :, 1:].transpose(1, 2)
    c.cache.attend(q, c.table, c.d_lens, out=out)
    assert torch.equal(out, want)
    out.fill_(3.0)
    assert bool((pool == 3.0).all())
    wide = torch.full((3, 9), -1, dtype=torch.int32, device="cuda")
    wide[:, 2:2 + c.table.shape[1]] = c.table
    assert torch.equal(c.cache.attend(q, wide[:, 2:2 + c.table.shape[1]], c.d_lens), want)


def test_attend_does_not_depend_on_the_pages_or_the_batch_beyond_rounding():
    torch = torch_cuda()
    log("attend repeat")
    c = Filled(torch, "nvfp4", 128, 2, [1000, 3, 500])
    q = _randn(torch, 1, 3, 1, 8, 128).to(torch.bfloat16)
    a = c.cache.attend(q, c.table, c.d_lens)
    for _ in range(5):
        assert torch.equal(a, c.cache.attend(q, c.table, c.d_lens))


def test_attend_with_very_many_columns():
    """Sixteen rows of 64 query heads on one key head: chunks of columns, with the weights of all of them."""
    torch = torch_cuda()
    log("attend columns")
    for fmt, d in (("nvfp4", 64), ("mxfp4", 256)):
        c = Filled(torch, fmt, d, 1, [200, 70, 9], track=True)
        q = _randn(torch, 5, 3, 16, 64, d).to(torch.bfloat16)
        _, sums = _check_attend(torch, c, q, "bf16", accumulate=True)
        for b, (w, ew) in enumerate(sums):
            page = int(c.table[b, 0])
            m = min(64, c.lens[b])
            _close(c.cache.weights[page, 0, :m], w[:m, 0], ew[:m, 0] + 2.0 ** -22 * w[:m, 0], "fp32", ("weights", b))


@pytest.mark.parametrize("n", [64, 65, 300])
def test_many_sequences(n):
    """More sequences than a wavefront has lanes, and than a block has threads."""
    torch = torch_cuda()
    log("many sequences", n)
    rng = np.random.default_rng(n)
    lens = [int(x) for x in rng.integers(0, 90, n)]
    lens[n // 2] = 1500
    c = Filled(torch, "nvfp4", 64, 1, lens, track=True, seed=n)
    c.check_read(("bf16",))
    q = _randn(torch, 5, n, 1, 3, 64).to(torch.bfloat16)
    _check_attend(torch, c, q, "bf16", accumulate=True)
    assert c.cache.evict(c.table, c.d_lens, 80, recent=3).tolist() == [min(x, 80) for x in lens]
    T = sum(lens)
    q, k, v = (_randn(torch, i, T, h, 64).to(torch.float16) for i, h in enumerate((2, 1, 1)))
    _check_prompt(torch, q, k, v, lens, lens, "fp16")


def test_a_cache_of_more_than_4_gib():
    """Pages behind 2^32 bytes, and positions and weights of them."""
    torch = torch_cuda()
    log("large cache")
    pages, lens = 62000, [100, 70]
    cache = _ops().KV4Cache(pages, 8, 128, track=True)
    assert cache.pages.numel() > 2 ** 32
    table = _ints(torch, [[pages - 1, 3], [pages - 2, 30000]])
    k, v = (_randn(torch, i, 170, 8, 128).to(torch.bfloat16) for i in range(2))
    d_lens, starts = _ints(torch, lens), _starts(torch, lens)
    cache.append(k, v, table, d_lens, starts)
    small = _ops().KV4Cache(4, 8, 128, track=True)
    table2 = _ints(torch, [[0, 1], [2, 3]])
    small.append(k, v, table2, d_lens, starts)
    q = _randn(torch, 7, 2, 2, 16, 128).to(torch.bfloat16)

    def same():
        for a, b in zip(cache.read(table, d_lens, 170, starts), small.read(table2, d_lens, 170, starts)):
            assert torch.equal(a, b)
        for a, b in ((cache.weights, small.weights), (cache.positions, small.positions)):
            assert torch.equal(a[table.long()], b[table2.long()])

    same()
    assert torch.equal(cache.attend(q, table, d_lens, accumulate=True), small.attend(q, table2, d_lens, accumulate=True))
    same()
    assert torch.equal(cache.evict(table, d_lens, 60, recent=5), small.evict(table2, d_lens, 60, recent=5))
    same()


def test_attend_and_prompts_at_once_on_two_streams():
    """Calls that only read the cache may run at once; each has its own workspace."""
    torch = torch_cuda()
    log("at once")
    c = Filled(torch, "nvfp4", 128, 2, [3000, 2000])
    q = [_randn(torch, i, 2, 2, 8, 128).to(torch.bfloat16) for i in range(2)]
    want = [c.cache.attend(x, c.table, c.d_lens) for x in q]
    pq = [_randn(torch, 9 + i, 40, 2, 128).to(torch.bfloat16) for i in range(2)]
    pk = _randn(torch, 11, 9000, 1, 128).to(torch.bfloat16)
    st, ks = _ints(torch, [0, 40]), _ints(torch, [0, 9000])
    pwant = [_ops().prompt_attention(x, pk, pk, st, ks) for x in pq]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    outs = []
    for _ in range(20):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                outs.append((c.cache.attend(q[i], c.table, c.d_lens), want[i]))
                outs.append((_ops().prompt_attention(pq[i], pk, pk, st, ks), pwant[i]))
    torch.cuda.synchronize()
    for got, w in outs:
        assert torch.equal(got, w)


# ---- eviction ----------------------------------------------------------------

def _check_evict(torch, c, weights, positions, keep, recent, sinks):
    """weights, positions: [tokens, hkv] by place of each sequence."""
    s = 0
    for b, n in enumerate(c.lens):
        for p in range((n + 63) // 64):
            m = min(64, n - 64 * p)
            page = int(c.table[b, p])
            c.cache.weights[page, :, :m] = torch.tensor(weights[s + 64 * p:s + 64 * p + m].T.copy(), device="cuda")
            c.cache.positions[page, :, :m] = torch.tensor(positions[s + 64 * p:s + 64 * p + m].T.copy(), device="cuda")
        s += n
    new = c.cache.evict(c.table, c.d_lens, keep, recent=recent, sinks=sinks)
    want = [min(n, keep) for n in c.lens]
    assert new.tolist() == want
    k, v = c.cache.read(c.table, new, sum(want), _starts(torch, want), dtype=torch.float32)
    k, v = _np(k), _np(v)
    s = o = 0
    for b, n in enumerate(c.lens):
        ck, cv = c.of(b)
        for h in range(c.hkv):
            src = oa.evict(weights[s:s + n, h], positions[s:s + n, h], keep, recent, sinks)
            assert np.array_equal(k[o:o + want[b], h], ck[src, h]), (b, h)
            assert np.array_equal(v[o:o + want[b], h], cv[src, h]), (b, h)
            place = np.arange(want[b])
            page = _np(c.table[b]).astype(int)[place // 64]
            assert np.array_equal(_np(c.cache.positions)[page, h, place % 64], positions[s:s + n, h][src])
            assert np.array_equal(np.nan_to_num(_np(c.cache.weights)[page, h, place % 64], nan=-5.0),
                                  np.nan_to_num(weights[s:s + n, h][src].astype(np.float64), nan=-5.0))
        s += n
        o += want[b]
    return new


@pytest.mark.parametrize("fmt,d,hkv", [("nvfp4", 128, 2), ("mxfp4", 64, 3), ("mxfp4", 256, 1), ("nvfp4", 64, 1),
                                       ("nvfp4", 256, 2), ("mxfp4", 128, 1)])
@pytest.mark.parametrize("keep,recent,sinks", [(1, 0, 0), (1, 1, 0), (64, 10, 4), (100, 100, 0), (129, 0, 129), (700, 5, 5)])
def test_evict(fmt, d, hkv, keep, recent, sinks):
    torch = torch_cuda()
    log("evict", fmt, d, hkv, keep, recent, sinks)
    lens = [0, 1, 64, 65, 130, 500, 1100, 1024]
    c = Filled(torch, fmt, d, hkv, lens, track=True, seed=keep)
    rng = np.random.default_rng(keep)
    T = sum(lens)
    w = np.where(rng.random((T, hkv)) < 0.5, rng.integers(0, 4, (T, hkv)), rng.exponential(1.0, (T, hkv))).astype(np.float32)
    at = np.concatenate([np.tile(np.arange(n)[:, None], (1, hkv)) for n in lens]).astype(np.int32)
    for s, n in zip(np.concatenate(([0], np.cumsum(lens)[:-1])), lens):      # tokens of an earlier eviction: out of order
        for h in range(hkv):
            at[s:s + n, h] = rng.permutation(at[s:s + n, h]) * 3
    _check_evict(torch, c, w, at, keep, recent, sinks)


def test_evict_weights_of_all_kinds():
    torch = torch_cuda()
    log("evict kinds")
    n = 600
    c = Filled(torch, "nvfp4", 64, 1, [n], track=True)
    rng = np.random.default_rng(2)
    w = rng.choice(np.array([0.0, -0.0, 1e-45, 1e-38, 1.0, 1.0000001, np.inf, np.nan, 3e38, -1.0], np.float32), (n, 1))
    at = np.arange(n, dtype=np.int32)[:, None]
    for keep in (500, 300, 100, 20):
        c = Filled(torch, "nvfp4", 64, 1, [n], track=True)
        _check_evict(torch, c, w, at, keep, 3, 2)
    c = Filled(torch, "nvfp4", 64, 1, [n], track=True)
    _check_evict(torch, c, np.zeros((n, 1), np.float32), at, 250, 0, 0)      # all equal: the first places


def test_evict_long_sequences():
    """Around the most places whose keys are held in registers (32768), and far more."""
    torch = torch_cuda()
    log("evict long")
    for n, keep in ((32768, 20000), (32769, 400), (70001, 35000)):
        c = Filled(torch, "mxfp4", 64, 1, [n, 130], track=True, seed=n)
        rng = np.random.default_rng(n)
        w = np.floor(rng.exponential(30.0, (n + 130, 1))).astype(np.float32) / 8
        at = np.concatenate((np.arange(n), np.arange(130))).astype(np.int32)[:, None]
        _check_evict(torch, c, w, at, keep, keep // 10, 3)


def test_evict_leaves_what_it_cannot_do():
    torch = torch_cuda()
    log("evict bad")
    c = Filled(torch, "nvfp4", 64, 2, [200, 200, 200, 100], track=True)
    c.cache.weights.uniform_()
    bad = c.table.clone()
    bad[1, 2] = c.cache.n_pages
    lens = _ints(torch, [200, 200, 64 * bad.shape[1] + 1, 100])
    keep_pages = torch.cat((c.table[1, :2], c.table[2, :4], c.table[3, :2])).long()
    before = [t[keep_pages].clone() for t in (c.cache.pages, c.cache.weights, c.cache.positions)]
    new = c.cache.evict(bad, lens, 100)
    assert new.tolist() == [100, 200, 64 * bad.shape[1] + 1, 100] and lens.tolist()[0] == 200
    for a, t in zip(before, (c.cache.pages, c.cache.weights, c.cache.positions)):
        assert torch.equal(a, t[keep_pages])


def test_evict_twice_and_go_on():
    """Recent tokens are those of the last positions, wherever they are after an eviction."""
    torch = torch_cuda()
    log("evict twice")
    c = Filled(torch, "mxfp4", 128, 2, [300], track=True)
    w = np.random.default_rng(1).random((300, 2)).astype(np.float32)
    at = np.tile(np.arange(300, dtype=np.int32)[:, None], (1, 2))
    lens = _check_evict(torch, c, w, at, 100, 50, 4)
    k = _randn(torch, 1, 20, 2, 128).to(torch.bfloat16)
    c.cache.append(k, k, c.table, _ints(torch, [120]), positions=_ints(torch, list(range(300, 320))))
    lens = c.cache.evict(c.table, _ints(torch, [120]), 72, recent=68, sinks=4)
    assert lens.tolist() == [72]
    for h in range(2):
        got = sorted(int(c.cache.positions[int(c.table[0, i // 64]), h, i % 64]) for i in range(72))
        assert got == list(range(4)) + list(range(252, 320))


# ---- together ----------------------------------------------------------------

def test_prompt_cache_steps_and_eviction_together():
    """A prompt, its keys into the cache, steps with drafts that keep weights, eviction, more steps: as a program does."""
    torch = torch_cuda()
    log("together")
    ops = _ops()
    hq, hkv, d, new = 8, 2, 128, [150, 40]
    T = sum(new)
    starts = _starts(torch, new)
    q, k, v = (_randn(torch, i, T, h, d).to(torch.bfloat16) for i, h in enumerate((hq, hkv, hkv)))
    _check_prompt(torch, q, k, v, new, new, "bf16")
    c = Filled(torch, "nvfp4", d, hkv, new, track=True, extra=200)
    cache, table = c.cache, c.table
    cache.append(k, v, table, _ints(torch, new), starts)
    hk = [c.held(x, i) for i, x in enumerate((k, v))]
    seqs = [[hk[0][:150], hk[1][:150]], [hk[0][150:], hk[1][150:]]]
    sums = [np.zeros((n, hkv)) for n in new]
    lens = _ints(torch, new)
    pos = [150, 40]
    for step in range(4):
        R = 3
        kn, vn = (_randn(torch, 100 + 2 * step + i, 2 * R, hkv, d).to(torch.bfloat16) for i in range(2))
        qn = _randn(torch, 200 + step, 2, R, hq, d).to(torch.bfloat16)
        lens = lens + R
        at = _ints(torch, [p + i for p in pos for i in range(R)])
        cache.append(kn, vn, table, lens, positions=at)
        out = cache.attend(qn, table, lens, accumulate=True)
        hn = [c.held(x, i) for i, x in enumerate((kn, vn))]
        for b in range(2):
            for i in range(2):
                seqs[b][i] = np.concatenate((seqs[b][i], hn[i][b * R:b * R + R]))
            o, _, w, eo, _, ew = oa.attend(_np(qn)[b], seqs[b][0], seqs[b][1], 1 / np.sqrt(d), *P_EPS["nvfp4"])
            _close(out[b], o, eo, "bf16", ("step", step, b))
            sums[b] = np.concatenate((sums[b], np.zeros((R, hkv)))) + w
            pos[b] += R
        if step == 1:
            w_dev = cache.weights.clone()
            lens = cache.evict(table, lens, 100, recent=16, sinks=2)
            assert lens.tolist() == [100, 46]
            n = 156
            place = np.arange(n)
            page = _np(table[0]).astype(int)[place // 64]
            for h in range(hkv):
                wd = _np(w_dev)[page, h, place % 64]
                assert np.allclose(wd, sums[0][:, h], rtol=1e-4, atol=1e-6)
                src = oa.evict(wd.astype(np.float32), place, 100, 16, 2)
                for i in range(2):
                    seqs[0][i][:100, h] = seqs[0][i][src, h]
                sums[0][:100, h] = sums[0][src, h]
            seqs[0] = [x[:100] for x in seqs[0]]
            sums[0] = sums[0][:100]


def test_calls_are_captured_and_replayed():
    torch = torch_cuda()
    log("graph")
    c = Filled(torch, "nvfp4", 128, 2, [300, 70], track=True, extra=64)
    q = _randn(torch, 1, 2, 2, 8, 128).to(torch.bfloat16)
    k, v = (_randn(torch, 2 + i, 4, 2, 128).to(torch.bfloat16) for i in range(2))
    pq, pk, pv = (_randn(torch, 5 + i, 200, h, 128).to(torch.bfloat16) for i, h in enumerate((8, 2, 2)))
    starts = _ints(torch, [0, 77, 200])
    lens = c.d_lens + 2

    def step():
        c.cache.append(k, v, c.table, lens)
        o = c.cache.attend(q, c.table, lens, accumulate=True)
        new = c.cache.evict(c.table, lens, 200, recent=10)
        a, b = c.cache.read(c.table, new, 100)
        return o, new, a, b, _ops().prompt_attention(pq, pk, pv, starts)

    state = [t.clone() for t in (c.cache.pages, c.cache.weights, c.cache.positions)]

    def reset():
        for t, s in zip((c.cache.pages, c.cache.weights, c.cache.positions), state):
            t.copy_(s)

    step()
    reset()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        res = step()
    for i in range(4):
        q.copy_(_randn(torch, 50 + i, 2, 2, 8, 128))
        reset()
        want = [t.clone() for t in step()]
        w = c.cache.weights.clone()
        reset()
        g.replay()
        torch.cuda.synchronize()
        for a, b in zip(res, want):
            assert torch.equal(a, b), i
        assert torch.equal(torch.nan_to_num(w, nan=7.0), torch.nan_to_num(c.cache.weights, nan=7.0))


def test_calls_on_a_given_stream():
    torch = torch_cuda()
    log("streams")
    c = Filled(torch, "mxfp4", 64, 2, [500, 90])
    q = _randn(torch, 1, 2, 1, 8, 64).to(torch.bfloat16)
    want = c.cache.attend(q, c.table, c.d_lens)
    pq = _randn(torch, 2, 300, 2, 64).to(torch.bfloat16)
    st = _ints(torch, [0, 300])
    pwant = _ops().prompt_attention(pq, pq, pq, st)
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    outs = []
    for i in range(20):
        for s in (s1, s2):
            outs.append((c.cache.attend(q.clone() if s is None else q, c.table, c.d_lens, stream=s),
                         _ops().prompt_attention(pq, pq, pq, st, stream=s)))
    torch.cuda.synchronize()
    for a, b in outs:
        assert torch.equal(a, want) and torch.equal(b, pwant)


def test_gradients_are_refused():
    torch = torch_cuda()
    log("gradients")
    ops = _ops()
    q = _randn(torch, 1, 5, 2, 64).to(torch.bfloat16).requires_grad_()
    out = ops.prompt_attention(q, q.detach(), q.detach(), _ints(torch, [0, 5]))
    with pytest.raises(NotImplementedError, match="prompt_attention"):
        out.sum().backward()
    c = Filled(torch, "nvfp4", 64, 1, [30])
    qa = _randn(torch, 1, 1, 1, 2, 64).to(torch.bfloat16).requires_grad_()
    with pytest.raises(NotImplementedError, match="attend"):
        c.cache.attend(qa, c.table, c.d_lens).sum().backward()
    with torch.no_grad():
        c.cache.attend(qa, c.table, c.d_lens)


def test_arguments_that_are_refused():
    torch = torch_cuda()
    log("refusals")
    ops = _ops()
    c = Filled(torch, "nvfp4", 64, 2, [30, 40])
    cache, bf = c.cache, torch.bfloat16
    q = torch.zeros(2, 1, 4, 64, dtype=bf, device="cuda")
    k = torch.zeros(4, 2, 64, dtype=bf, device="cuda")
    table, lens = c.table, c.d_lens
    bad = [
        lambda: cache.attend(q[:1], table, lens), lambda: cache.attend(q.float(), table, lens),
        lambda: cache.attend(q[:, :, :3], table, lens), lambda: cache.attend(q[..., :32], table, lens),
        lambda: cache.attend(q.transpose(2, 3), table, lens), lambda: cache.attend(q.cpu(), table, lens),
        lambda: cache.attend(q.expand(2, 17, 4, 64), table, lens), lambda: cache.attend(q, table.long(), lens),
        lambda: cache.attend(q, table.cpu(), lens), lambda: cache.attend(q, table, lens.long()),
        lambda: cache.attend(q, table, lens[:1]), lambda: cache.attend(q, table, lens, scale=0.0),
        lambda: cache.attend(q, table, lens, scale=float("nan")), lambda: cache.attend(q, table, lens, accumulate=True),
        lambda: cache.attend(q, table, lens, out=q.new_empty(1, 1, 4, 64)),
        lambda: cache.attend(q, table, lens, out=q.new_empty(1, 1, 4, 64).expand(2, 1, 4, 64)),
        lambda: cache.attend(q, table[:, :0], lens), lambda: cache.attend(q, table[:1].expand(2, -1), lens),
        lambda: cache.evict(table, lens, 10), lambda: cache.append(k[:3], k[:3], table, lens),
        lambda: cache.append(k, k[:2], table, lens), lambda: cache.append(k, k.float(), table, lens),
        lambda: cache.append(k[:, :1], k[:, :1], table, lens), lambda: cache.append(k.int(), k.int(), table, lens),
        lambda: cache.append(k, k, table, lens, starts=lens), lambda: cache.append(k, k, table, lens, positions=lens),
        lambda: cache.read(table, lens, 3), lambda: cache.read(table, lens, -2),
        lambda: cache.read(table, lens, 2, dtype=torch.int32),
        lambda: ops.prompt_attention(k, k, k, lens.long()), lambda: ops.prompt_attention(k, k[:3], k[:3], lens),
        lambda: ops.prompt_attention(k, k, k.half(), lens), lambda: ops.prompt_attention(k[:, :1], k, k, lens),
        lambda: ops.prompt_attention(k, k, k, lens, scale=-1.0), lambda: ops.prompt_attention(k, k, k, lens[:0]),
        lambda: ops.prompt_attention(k, k, k, lens, key_starts=lens[:1]),
        lambda: ops.prompt_attention(k, k, k, lens, out=k[:3]),
        lambda: ops.prompt_attention(k, k, k, lens, out=k[:1].clone().expand(4, -1, -1)),
    ]
    for i, f in enumerate(bad):
        with pytest.raises(ValueError):
            f()
            pytest.fail("call %d was taken" % i)
    with pytest.raises(AttributeError):
        cache.pages = cache.pages.clone()
    t = ops.KV4Cache(2, 1, 64, track=True)
    for kw in (dict(keep=0), dict(keep=4, recent=5), dict(keep=4, recent=3, sinks=2), dict(keep=4, recent=-1)):
        with pytest.raises(ValueError):
            t.evict(table, lens, **kw)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("at", [3, 8990])
def test_few_rows_over_many_keys_that_are_not_finite(at, d):
    """A value of the first part, which all rows see, and one of the last, which some do not."""
    torch = torch_cuda()
    log("parts, not finite", at, d)
    q, k, v = (_randn(torch, i, n, 1, d).to(torch.bfloat16) for i, n in enumerate((20, 9000, 9000)))
    starts, keys = _ints(torch, [0, 20]), _ints(torch, [0, 9000])
    sane = _ops().prompt_attention(q, k, v, starts, keys)
    v[at, 0, 7] = float("inf")
    out = _ops().prompt_attention(q, k, v, starts, keys)
    blind = max(0, at - 8980)                   # rows before the token
    assert torch.equal(out[:blind], sane[:blind]) and not bool(torch.isfinite(out[blind:, 0, 7]).any())
    out[blind:, 0, 7] = sane[blind:, 0, 7]
    assert torch.equal(out, sane)


@pytest.mark.parametrize("d", [128, 256])
def test_prompt_values_that_are_not_finite_at_many_places(d):
    """In both LDS buffers, at their ends too, with both ways into LDS."""
    torch = torch_cuda()
    log("not finite, many", d)
    n = 300
    x = _randn(torch, 1, n, 3 * d + 1).to(torch.float16)
    for shift in (0, 1):                        # 16-byte aligned rows, and others
        big = torch.zeros(n, 3 * d + 8, dtype=torch.float16, device="cuda")
        big[:, shift:shift + 3 * d] = x[:, :3 * d]
        q, k, v = (big[:, shift + i * d:shift + (i + 1) * d].unsqueeze(1) for i in range(3))
        sane = _ops().prompt_attention(q, k, v, _ints(torch, [0, n])).clone()
        for at in (0, 31, 32, 63, 64, 127, 128, 255, 256, 299):
            keep = v[at, 0, at % d].clone()
            v[at, 0, at % d] = float("nan")
            out = _ops().prompt_attention(q, k, v, _ints(torch, [0, n]))
            v[at, 0, at % d] = keep
            assert torch.equal(out[:at], sane[:at]) and bool(torch.isnan(out[at:, 0, at % d]).all()), at
            out[at:, 0, at % d] = sane[at:, 0, at % d]
            assert torch.equal(out, sane), at


def test_attend_rows_before_a_page_that_cannot_be():
    """Of two rows only the second sees the token on a page that the cache does not have."""
    torch = torch_cuda()
    log("attend, bad page of the last row")
    c = Filled(torch, "nvfp4", 64, 1, [65])
    q = _randn(torch, 1, 1, 2, 4, 64).to(torch.bfloat16)
    good = c.cache.attend(q, c.table, c.d_lens)
    for bad in (-1, c.cache.n_pages, 2 ** 31 - 1):
        table = c.table.clone()
        table[0, 1] = bad
        got = c.cache.attend(q, table, c.d_lens)
        assert torch.equal(got[0, 0], good[0, 0]) and bool(torch.isnan(got[0, 1]).all())


def test_no_sequences_and_no_tokens():
    torch = torch_cuda()
    log("nothing")
    ops = _ops()
    c = ops.KV4Cache(3, 2, 64, track=True)
    table, lens = torch.zeros(0, 2, dtype=torch.int32, device="cuda"), torch.zeros(0, dtype=torch.int32, device="cuda")
    q = torch.zeros(0, 1, 4, 64, dtype=torch.bfloat16, device="cuda")
    k = torch.zeros(0, 2, 64, dtype=torch.bfloat16, device="cuda")
    assert c.attend(q, table, lens, accumulate=True).shape == (0, 1, 4, 64)
    c.append(k, k, table, lens)
    assert c.read(table, lens, 0)[0].shape == (0, 2, 64) and c.evict(table, lens, 5).shape == (0,)
    one = _ints(torch, [[0, 1]])
    c.append(k, k, one, _ints(torch, [0]))
    out = c.attend(torch.ones(1, 2, 4, 64, dtype=torch.bfloat16, device="cuda"), one, _ints(torch, [0]), accumulate=True)
    assert not bool(out.any()) and c.evict(one, _ints(torch, [0]), 5).tolist() == [0]
    zero = _ints(torch, [0])
    assert ops.prompt_attention(k, k, k, zero).shape == (0, 2, 64)
    rows = torch.ones(4, 2, 64, dtype=torch.bfloat16, device="cuda")
    out, lse = ops.prompt_attention(rows, k, k, _ints(torch, [0, 4]), _ints(torch, [0, 0]), return_lse=True)
    assert not bool(out.any()) and bool((lse == -float("inf")).all())


@pytest.mark.parametrize("dtype,d", [("bf16", 64), ("fp16", 128), ("bf16", 256)])
@pytest.mark.parametrize("rows,keys", [(4200, 4200), (9000, 4200)])
def test_long_prompts_in_two_parts(rows, keys, dtype, d):
    """Eight heads of 4200 rows and more have over 256 blocks, the last of which take twice the average: their keys
    are cut.  With fewer keys than rows the first ones see nothing."""
    torch = torch_cuda()
    log("prompt in two parts", rows, keys, dtype, d)
    dt = getattr(torch, TYPES[dtype])
    q = (2 * _randn(torch, 1, rows, 8, d)).to(dt)
    k, v = (_randn(torch, 2 + i, keys, 1, d).to(dt) for i in range(2))
    out, lse = _ops().prompt_attention(q, k, v, _ints(torch, [0, rows]), _ints(torch, [0, keys]), return_lse=True)
    qn, kn, vn, blind = _np(q), _np(k), _np(v), rows - keys
    assert not bool(out[:blind].any()) and bool((lse[:blind] == -float("inf")).all())
    for i in (0, 1, 127, 128, 2047, 2048, 2111, 2112, 4031, 4095, 4096, 4198, 4199):
        r = blind + i
        o, l, _, eo, el, _ = oa.attend(qn[r:r + 1], kn[:i + 1], vn[:i + 1], 1.0 / np.sqrt(d), EPS[dtype],
                                       2.0 ** -39 if dtype == "fp16" else 0.0)
        _close(out[r:r + 1], o, eo, dtype, ("out", i))
        _close(lse[r:r + 1], l, el, "fp32", ("lse", i))


@pytest.mark.parametrize("bad", [float("nan"), -1.0, float("inf"), -float("inf")])
@pytest.mark.parametrize("d,group,rows", [(64, 3, 2), (128, 8, 4), (256, 1, 1)])
def test_attend_with_a_scale_of_keys_that_cannot_be(d, group, rows, bad):
    """Every row that sees a key is NaN, and so are the weights of all that is seen; with a list of pages (the table
    has over eight) and without."""
    torch = torch_cuda()
    log("attend, bad scale of keys", d, group, rows, bad)
    for lens in ([0, 1, 70, 700], [3, 130]):
        c = Filled(torch, "nvfp4", d, 2, lens, scales=(1.0, 2.0), track=True)
        c.cache.k_scale.fill_(bad)
        start = c.cache.weights.clone()
        q = _randn(torch, 1, len(lens), rows, 2 * group, d).to(torch.bfloat16)
        out = c.cache.attend(q, c.table, c.d_lens)
        assert torch.equal(torch.nan_to_num(out, nan=3.0), torch.nan_to_num(c.cache.attend(
            q, c.table, c.d_lens, accumulate=True), nan=3.0))
        for b, n in enumerate(lens):
            for r in range(rows):
                if n - rows + r + 1 > 0:
                    assert bool(torch.isnan(out[b, r]).all()), (b, r)
                else:
                    assert not bool(out[b, r].any()), (b, r)
            for p in range((n + 63) // 64):
                m = min(64, n - 64 * p)
                page = int(c.table[b, p])
                assert bool(torch.isnan(c.cache.weights[page, :, :m]).all()), (b, p)
                assert torch.equal(torch.nan_to_num(c.cache.weights[page, :, m:], nan=7.0),
                                   torch.nan_to_num(start[page, :, m:], nan=7.0))


def test_append_of_very_many_tokens():
    """One head, 15.1 million tokens: the first, some and the last ones, and nothing behind them."""
    torch = torch_cuda()
    log("many tokens")
    n, d = 15_100_001, 64
    k = _randn(torch, 1, n, 1, d).to(torch.bfloat16)
    pages = (n + 63) // 64
    cache = _ops().KV4Cache(pages + 1, 1, d, "mxfp4")
    table = torch.arange(pages, dtype=torch.int32, device="cuda").unsqueeze(0)
    cache.append(k, k, table, _ints(torch, [n]))
    assert not bool(cache.pages[pages].any())
    whole = cache.read(table, _ints(torch, [n]), n)
    for at in (0, 1, 4095, 2 ** 23, n // 2, 14_961_000, n - 70):
        m = min(70, n - at)
        want = torch.tensor(oa.quantized(_np(k[at:at + m]), "mxfp4")).float().to(torch.bfloat16)
        for got in whole + cache.read(table, _ints(torch, [at + m]), m):
            got = got[at:at + m] if got.shape[0] == n else got
            assert torch.equal(got.cpu(), want), at


def test_a_new_cache_on_another_stream():
    """A cache is zeros before its constructor returns: what another stream appends right away stays."""
    torch = torch_cuda()
    log("new cache, other stream")
    k = _randn(torch, 1, 200, 2, 64).to(torch.bfloat16)
    table, lens = _ints(torch, [[3, 1, 0, 2]]), _ints(torch, [200])
    want = torch.tensor(oa.quantized(_np(k), "mxfp4")).float()
    busy = torch.zeros(1 << 28, device="cuda")
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(3):
        for _ in range(20):                     # several milliseconds on the current stream, before the zeros
            busy.add_(1.0)
        cache = _ops().KV4Cache(4, 2, 64, "mxfp4", track=True)
        cache.append(k, k, table, lens, stream=side)
        torch.cuda.synchronize()
        got = cache.read(table, lens, 200, dtype=torch.float32)
        assert torch.equal(got[0].cpu(), want) and torch.equal(got[1].cpu(), want)
        assert cache.positions[1, 0].tolist() == list(range(64, 128))


def test_a_new_cache_within_a_captured_graph():
    """Its zeros belong to the graph then."""
    torch = torch_cuda()
    log("new cache, captured")
    k = _randn(torch, 1, 100, 1, 64).to(torch.bfloat16)
    q = _randn(torch, 2, 1, 1, 2, 64).to(torch.bfloat16)
    table, lens = _ints(torch, [[0, 1]]), _ints(torch, [100])

    def step():
        cache = _ops().KV4Cache(2, 1, 64, track=True)
        cache.append(k, k, table, lens)
        return cache, cache.attend(q, table, lens, accumulate=True), cache.weights

    want = step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = step()
    for _ in range(3):
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(got[1], want[1]) and torch.equal(got[2], want[2])


def test_the_largest_scale():
    """Scores of zero stay zero under it: every row has the mean of the values that it sees."""
    torch = torch_cuda()
    log("largest scale")
    q = torch.zeros(70, 2, 64, dtype=torch.bfloat16, device="cuda")
    v = _randn(torch, 1, 70, 1, 64).to(torch.bfloat16)
    _check_prompt(torch, q, v, v, [70], [70], "bf16", scale=2.3e38)
    c = Filled(torch, "mxfp4", 64, 1, [70])
    _check_attend(torch, c, q[:3].unsqueeze(0), "bf16", scale=2.3e38)


@pytest.mark.parametrize("scale", [1e-30, 1e-38, 1e-42])
def test_the_smallest_scales(scale):
    """Scores of nearly zero, and masked ones that stay masked."""
    torch = torch_cuda()
    log("smallest scale", scale)
    q, v = _randn(torch, 1, 70, 2, 64).to(torch.bfloat16), _randn(torch, 2, 70, 1, 64).to(torch.bfloat16)
    _check_prompt(torch, q, v, v, [70], [70], "bf16", scale=scale)
    c = Filled(torch, "nvfp4", 64, 1, [70])
    _check_attend(torch, c, q[:3].unsqueeze(0), "bf16", scale=scale)


def _later(torch, stream, dst, src, busy):
    """dst gets src on the stream, behind work of tens of milliseconds."""
    with torch.cuda.stream(stream):
        for _ in range(200):
            busy.add_(1.0)
        dst.copy_(src)


def _behind(stream):
    """Waits for the stream, which has to be busy until now: what came before it on the host was not waited for."""
    assert not stream.query()
    stream.synchronize()


def test_calls_run_on_the_given_stream():
    """Every call's input is written late on the stream that is given, while the current stream is idle: a call that
    ran on the current one would read what was there before.  What the calls leave is read on that stream as well."""
    torch = torch_cuda()
    log("given stream")
    ops = _ops()
    n, d, hkv = [300, 70], 128, 2
    T = sum(n)
    side, busy = torch.cuda.Stream(), torch.zeros(1 << 27, device="cuda")
    table, lens, starts = _ints(torch, [[0, 1, 2, 3, 4], [5, 6, 7, 8, 9]]), _ints(torch, n), _starts(torch, n)
    k1, v1 = (_randn(torch, i, T, hkv, d).to(torch.bfloat16) for i in range(2))
    q1 = _randn(torch, 3, 2, 2, 8, d).to(torch.bfloat16)
    pq1 = _randn(torch, 4, T, 4, d).to(torch.bfloat16)
    w1 = torch.rand(10, hkv, 64, device="cuda")

    def fresh():
        c = ops.KV4Cache(10, hkv, d, track=True)
        c.append(k1, v1, table, lens, starts)
        c.weights.copy_(w1)
        return c

    c = fresh()
    want = dict(prompt=ops.prompt_attention(pq1, k1, v1, starts), attend=c.attend(q1, table, lens),
                read=c.read(table, lens, T, starts))
    c.attend(q1, table, lens, accumulate=True)
    want["weights"] = c.weights.clone()
    want["new"] = c.evict(table, lens, 64, recent=8)
    want["evicted"] = c.read(table, want["new"], 128)
    nothing = torch.zeros_like
    torch.cuda.synchronize()

    # a prompt, whose queries come late
    pq = nothing(pq1)
    torch.cuda.synchronize()
    _later(torch, side, pq, pq1, busy)
    got, lse = ops.prompt_attention(pq, k1, v1, starts, return_lse=True, stream=side)
    _behind(side)
    assert torch.equal(got, want["prompt"])

    # attention, whose queries come late
    c, q = fresh(), nothing(q1)
    torch.cuda.synchronize()
    _later(torch, side, q, q1, busy)
    got = c.attend(q, table, lens, stream=side)
    _behind(side)
    assert torch.equal(got, want["attend"])

    # append, whose keys come late, and read behind it
    c, k = ops.KV4Cache(10, hkv, d, track=True), nothing(k1)
    torch.cuda.synchronize()
    _later(torch, side, k, k1, busy)
    c.append(k, v1, table, lens, starts, stream=side)
    got = c.read(table, lens, T, starts, stream=side)
    _behind(side)
    assert all(torch.equal(a, b) for a, b in zip(got, want["read"]))

    # weights that come late, what attention adds to them, and the eviction that goes by them
    c = fresh()
    c.weights.zero_()
    torch.cuda.synchronize()
    _later(torch, side, c.weights, w1, busy)
    c.attend(q1, table, lens, accumulate=True, stream=side)
    with torch.cuda.stream(side):
        w = c.weights.clone()
    new = c.evict(table, lens, 64, recent=8, stream=side)
    got = c.read(table, new, 128, stream=side)
    _behind(side)
    assert torch.equal(w, want["weights"]) and torch.equal(new, want["new"])
    assert all(torch.equal(a, b) for a, b in zip(got, want["evicted"]))


def test_what_calls_on_a_stream_use_may_be_dropped():
    """Inputs, caches and results that are dropped while a stream has the call still before it: their memory is not
    given out to the current stream before."""
    torch = torch_cuda()
    log("dropped")
    ops = _ops()
    side, busy = torch.cuda.Stream(), torch.zeros(1 << 27, device="cuda")
    n, d, hkv = 640, 128, 2
    table, lens, starts = torch.arange(10, dtype=torch.int32, device="cuda").unsqueeze(0), _ints(torch, [n]), _ints(torch, [0, n])
    k1, v1 = (_randn(torch, i, n, hkv, d).to(torch.bfloat16) for i in range(2))
    q1 = _randn(torch, 3, 1, 1, 8, d).to(torch.bfloat16)
    scale1 = torch.tensor([0.5], device="cuda")
    first = ops.KV4Cache(10, hkv, d, k_scale=scale1)
    first.append(k1, v1, table, lens)
    want, pwant = first.attend(q1, table, lens), ops.prompt_attention(k1, k1, v1, starts)
    for _ in range(3):
        c = ops.KV4Cache(10, hkv, d, k_scale=scale1.clone())
        c.append(k1, v1, table, lens)
        q, k, v, t, ln, st = q1.clone(), k1.clone(), v1.clone(), table.clone(), lens.clone(), starts.clone()
        torch.cuda.synchronize()
        sizes = [x.numel() * x.element_size() for x in (c.pages, q, k, v, t, ln, st)]
        with torch.cuda.stream(side):
            for _ in range(200):
                busy.add_(1.0)
        got = c.attend(q, t, ln, stream=side)
        pgot = ops.prompt_attention(k, k, v, st, stream=side)
        del c, q, k, v, t, ln, st
        junk = [torch.full((s,), 255, dtype=torch.uint8, device="cuda") for s in sizes for _ in range(4)]
        torch.cuda.current_stream().synchronize()
        _behind(side)
        assert torch.equal(got, want) and torch.equal(pgot, pwant)
        del junk


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
def test_attend_on_other_pages_and_in_other_batches(fmt):
    """On other pages: the same bits.  Alone or in another batch, whose list is cut elsewhere: the same but for the
    order of the sums, whose bounds hold for each."""
    torch = torch_cuda()
    log("other pages, other batches", fmt)
    lens = [1000, 3, 500, 64, 2500]
    c = Filled(torch, fmt, 128, 2, lens)
    q = _randn(torch, 1, 5, 2, 8, 128).to(torch.bfloat16)
    want, _ = _check_attend(torch, c, q, "bf16")
    k, v = c.cache.read(c.table, c.d_lens, sum(lens), _starts(torch, lens), dtype=torch.float32)
    perm = torch.randperm(c.cache.n_pages, device="cuda").to(torch.int32)
    other = _ops().KV4Cache(c.cache.n_pages, 2, 128, fmt)
    table = torch.where(c.table >= 0, perm[c.table.clamp(min=0).long()], c.table)
    assert not torch.equal(table, c.table)
    other.append(k, v, table, c.d_lens, _starts(torch, lens))          # representable: the same codes
    assert torch.equal(other.attend(q, table, c.d_lens), want)
    sc = 1.0 / np.sqrt(128)
    for some in ([0], [4], [2, 0], [4, 3, 1, 0], [0, 0, 0]):
        got = c.cache.attend(q[some], c.table[some], c.d_lens[some])
        for i, b in enumerate(some):
            o, _, _, eo, _, _ = oa.attend(_np(q)[b], *c.of(b), sc, *P_EPS[fmt])
            _close(got[i], o, eo, "bf16", (some, b))


def test_a_prompt_whose_last_rows_leave_weights_before_eviction():
    """append leaves weights of 0; the last rows of the prompt, attended to again with accumulate, give the tokens
    theirs, and eviction goes by them."""
    torch = torch_cuda()
    log("weights of a prompt")
    ops = _ops()
    hq, hkv, d, n = 8, 2, 128, [300, 150]
    T, R, keep = sum(n), 16, 100
    starts, lens = _starts(torch, n), _ints(torch, n)
    q, k, v = (2 * _randn(torch, i, T, h, d) for i, h in enumerate((hq, hkv, hkv)))
    q, k, v = q.to(torch.bfloat16), k.to(torch.bfloat16), v.to(torch.bfloat16)
    ops.prompt_attention(q, k, v, starts)
    c = Filled(torch, "nvfp4", d, hkv, n, track=True)
    c.cache.append(k, v, c.table, lens, starts)
    c.k, c.v = c.held(k, 0), c.held(v, 1)
    last = torch.cat([torch.arange(int(e) - R, int(e)) for e in np.cumsum(n)]).cuda()
    c.cache.attend(q[last].view(2, R, hq, d), c.table, lens, accumulate=True)
    got = c.cache.weights.clone()
    new = c.cache.evict(c.table, lens, keep, recent=8, sinks=2)
    assert new.tolist() == [keep, keep]
    gk, _ = c.cache.read(c.table, new, 2 * keep, dtype=torch.float32)
    for b in range(2):
        ck, cv = c.of(b)
        _, _, w, _, _, ew = oa.attend(_np(q[last].view(2, R, hq, d))[b], ck, cv, 1.0 / np.sqrt(d), *P_EPS["nvfp4"])
        place = np.arange(n[b])
        page = _np(c.table[b]).astype(int)[place // 64]
        for h in range(hkv):
            wd = _np(got)[page, h, place % 64]
            assert (np.abs(wd - w[:, h]) <= ew[:, h] + 2.0 ** -23 * w[:, h]).all()
            src = oa.evict(wd.astype(np.float32), place, keep, 8, 2)
            assert not np.array_equal(src, np.arange(keep))
            assert np.array_equal(_np(gk)[b * keep:(b + 1) * keep, h], ck[src, h])


def test_as_many_sequences_as_a_call_takes():
    """65536 of them: lists, searches and grids at their limits."""
    torch = torch_cuda()
    log("65536 sequences")
    ops, n = _ops(), 65536
    cache = ops.KV4Cache(n, 2, 64, "mxfp4", track=True)
    lens = torch.arange(n, dtype=torch.int32, device="cuda") % 7            # 0 .. 6 tokens
    T = int(lens.sum())
    starts = torch.zeros(n + 1, dtype=torch.int32, device="cuda")
    starts[1:] = torch.cumsum(lens, 0)
    k, v = (_randn(torch, i, T, 2, 64).to(torch.bfloat16) for i in range(2))
    for width in (1, 9):                                                    # without a list of pages, and with one
        table = torch.full((n, width), -1, dtype=torch.int32, device="cuda")
        table[:, 0] = torch.randperm(n, device="cuda")
        cache.append(k, v, table, lens, starts)
        rk, rv = (_np(x) for x in cache.read(table, lens, T, starts, dtype=torch.float32))
        assert np.array_equal(rk, oa.quantized(_np(k), "mxfp4"))
        q = _randn(torch, 5, n, 1, 4, 64).to(torch.bfloat16)
        out = cache.attend(q, table, lens, accumulate=True)
        new = cache.evict(table, lens, 4)
        assert torch.equal(new, lens.clamp(max=4))
        assert not bool(out[lens == 0].any())
        for b in (1, 6, 6999, 32768 + 5, 65500, n - 1):
            s, m = int(starts[b]), int(lens[b])
            o, _, w, eo, _, ew = oa.attend(_np(q[b]), rk[s:s + m], rv[s:s + m], 0.125, *P_EPS["mxfp4"])
            _close(out[b], o, eo, "bf16", (width, b))
    q = _randn(torch, 6, T, 2, 64).to(torch.bfloat16)
    out, lse = ops.prompt_attention(q, k, v, starts, return_lse=True)
    for b in (1, 6, 6999, 32768 + 5, 65500, n - 1):
        s, m = int(starts[b]), int(lens[b])
        o, l, _, eo, el, _ = oa.attend(_np(q[s:s + m]), _np(k[s:s + m]), _np(v[s:s + m]), 0.125, EPS["bf16"])
        _close(out[s:s + m], o, eo, "bf16", b)
        _close(lse[s:s + m], l, el, "fp32", b)
