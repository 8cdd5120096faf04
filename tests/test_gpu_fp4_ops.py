"""4-bit weights on the GPU: quantising and reading back (whole numbers equal the
float64 oracle's), and products against float64."""
import numpy as np
import pytest

from oracle import fp4

from gpu_util import log, torch_cuda

pytestmark = pytest.mark.gpu

TYPES = {"bf16": "bfloat16", "fp16": "float16", "fp32": "float32"}


def _ops():
    from hbm_expert_slot_amd import ops
    return ops


def _np64(t):
    return t.detach().cpu().double().numpy()


def _weights(torch, rows, cols, dtype, seed, scale=0.02):
    rng = np.random.default_rng(seed)
    w = rng.standard_normal((rows, cols)) * scale * np.exp(0.5 * rng.standard_normal((rows, 1)))
    return torch.tensor(w, dtype=getattr(torch, TYPES[dtype])).cuda()


def _check_quant(torch, w, q, fmt, given=None):
    codes, sb, gs = fp4.quantize(_np64(w), fmt, given)
    assert np.array_equal(q.scales.cpu().numpy(), sb)
    assert np.array_equal(fp4.unpack(q.codes.cpu().numpy()), codes)
    if fmt == "nvfp4":
        assert np.float32(q.global_scale.item()) == gs
    v = fp4.values(codes, sb, fmt, gs)
    for dt in TYPES.values():
        got = _ops().fp4_dequantize(q, getattr(torch, dt))
        want = torch.tensor(v).float().to(getattr(torch, dt))
        assert torch.equal(torch.nan_to_num(got.cpu(), nan=777.0), torch.nan_to_num(want, nan=777.0)), dt


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("fmt,rows,cols", [("nvfp4", 1, 16), ("nvfp4", 3, 48), ("nvfp4", 257, 1040),
                                           ("nvfp4", 64, 6144), ("mxfp4", 1, 32), ("mxfp4", 5, 96),
                                           ("mxfp4", 130, 2080)])
def test_quantize(fmt, rows, cols, dtype):
    torch = torch_cuda()
    log("quantize", fmt, rows, cols, dtype)
    w = _weights(torch, rows, cols, dtype, rows * 7 + cols)
    _check_quant(torch, w, _ops().fp4_quantize(w, fmt), fmt)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("g", [2.0 ** -13, 0.00123, 2.0 ** -7])
def test_quantize_with_a_given_scale(g, dtype):
    """Powers of two make ties common; the large one saturates scales at 0, the small one at 448."""
    torch = torch_cuda()
    log("given scale", g, dtype)
    w = _weights(torch, 96, 512, dtype, 5, scale=0.05)
    w[0] = torch.round(w[0] * 512) / 512
    w[1, :16] = torch.tensor([6, .25, .75, 1.25, 1.75, 2.5, 3.5, 5, -.25, -.75, -1.25, -1.75, -2.5, -3.5, -5, 0]) * g
    w[2] *= 1e4
    w[3] *= 1e-6
    gs = torch.tensor([g], dtype=torch.float32).cuda()
    _check_quant(torch, w, _ops().fp4_quantize(w, "nvfp4", global_scale=gs), "nvfp4", np.float32(g))


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
def test_quantize_next_to_borders(fmt):
    """fp32 weights one step beside a rounding border take the side they are on."""
    torch = torch_cuda()
    rng = np.random.default_rng(3)
    base = np.float32(rng.uniform(0.5, 2, (64, 1)))
    mid = np.array([.25, .75, 1.25, 1.75, 2.5, 3.5, 5.0], np.float32)
    w = np.zeros((64, 64), np.float32)
    w[:, 0::16] = 6 * base                      # every group's max: the scale is about base
    for i in range(7):
        b = (base * mid[i]).astype(np.float32)[:, 0]
        w[:, 2 * i + 1] = np.nextafter(b, np.float32(0))
        w[:, 2 * i + 2] = -np.nextafter(b, np.float32(9))
        w[:, 16 + 2 * i + 1] = b
    t = torch.tensor(w).cuda()
    for g in ([np.float32(2.0 ** -9), np.float32(0.0017)] if fmt == "nvfp4" else [None]):
        gs = None if g is None else torch.tensor([g]).cuda()
        _check_quant(torch, t, _ops().fp4_quantize(t, fmt, global_scale=gs), fmt, g)


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
def test_quantize_edges(fmt):
    """Zeros, infinities, NaN, denormals and the type's extremes; each spoils its own group only."""
    torch = torch_cuda()
    w = _weights(torch, 12, 64, "fp32", 9)
    w[0] = 0
    w[1, 5] = float("nan")
    w[2, 40] = float("inf")
    w[3, 63] = -float("inf")
    w[4] = 1e-42
    w[5, :32] = -0.0
    _check_quant(torch, w, _ops().fp4_quantize(w, fmt), fmt)
    z = torch.zeros(3, 64, device="cuda")
    _check_quant(torch, z, _ops().fp4_quantize(z, fmt), fmt)
    big = torch.full((2, 64), 3e38, device="cuda")
    big[1] = 1.0
    if fmt == "mxfp4":
        _check_quant(torch, big, _ops().fp4_quantize(big, fmt), fmt)
    else:
        q = _ops().fp4_quantize(big, fmt)
        codes, sb, gs = fp4.quantize(_np64(big), fmt)
        assert np.array_equal(q.scales.cpu().numpy(), sb) and np.float32(q.global_scale.item()) == gs


def test_quantize_strides_and_views():
    torch = torch_cuda()
    big = _weights(torch, 40, 300, "bf16", 11)
    for off, cols in ((0, 288), (1, 288), (8, 96)):
        w = big[3:33, off:off + cols]
        _check_quant(torch, w, _ops().fp4_quantize(w, "nvfp4"), "nvfp4")
    q = _ops().FP4Weight.empty(30, 96)
    out = torch.full((30, 120), 7.0, device="cuda")
    _ops().fp4_quantize(w, out=q)
    _ops().fp4_dequantize(q, out=out[:, 3:99])
    assert torch.equal(out[:, 3:99], _ops().fp4_dequantize(q)) and (out[:, :3] == 7).all() and (out[:, 99:] == 7).all()


def test_no_rows():
    torch = torch_cuda()
    ops = _ops()
    q = ops.fp4_quantize(torch.empty(0, 64, device="cuda", dtype=torch.bfloat16))
    assert q.shape == (0, 64) and ops.fp4_dequantize(q).shape == (0, 64)
    x = torch.ones(3, 64, device="cuda", dtype=torch.bfloat16)
    assert ops.fp4_linear(x, q).shape == (3, 0)
    w = ops.fp4_quantize(torch.ones(5, 64, device="cuda"))
    assert ops.fp4_linear(x[:0], w).shape == (0, 5)


# ---- products -------------------------------------------------------------------

def _random_fp4(torch, rows, cols, fmt, seed):
    rng = np.random.default_rng(seed)
    codes = rng.integers(0, 16, (rows, cols)).astype(np.uint8)
    g = fp4.GROUP[fmt]
    if fmt == "nvfp4":
        sb = rng.integers(0x20, 0x7F, (rows, cols // g)).astype(np.uint8)
        gs = np.float32(rng.uniform(0.001, 0.002))
    else:
        sb = rng.integers(110, 130, (rows, cols // g)).astype(np.uint8)
        gs = None
    q = _ops().FP4Weight(torch.tensor(fp4.pack(codes)).cuda(), torch.tensor(sb).cuda(),
                         None if gs is None else torch.tensor([gs]).cuda(), fmt)
    return q, fp4.values(codes, sb, fmt, gs)


def _bound(x, w, dtype, torch, terms):
    """Rounding of `terms` fp32 additions against the sum of magnitudes (each adds half a step of a
    partial sum no larger than that), and of the result to its type."""
    mag = np.abs(x) @ np.abs(w).T
    want = x @ w.T
    return terms * 2.0 ** -24 * mag + torch.finfo(dtype).eps / 2 * np.abs(want) * 1.01 + 1e-37


# one chain of fp32 additions: 16 or 32 products of a group, one addition per group of a lane,
# the sums over lanes and wavefronts; the bias and the scale of the matrix add three roundings
def _terms(K):
    return 32 + 2 * (K // 512 + 1) + 12 + 3


LINEAR = [
    (1, 1, 16, "nvfp4"), (1, 5, 32, "mxfp4"), (1, 64, 512, "nvfp4"), (1, 130, 2064, "nvfp4"), (1, 77, 6144, "nvfp4"),
    (2, 33, 48, "nvfp4"), (3, 40, 1056, "mxfp4"), (4, 130, 2064, "nvfp4"), (5, 19, 544, "mxfp4"),
    (7, 65, 1040, "nvfp4"), (8, 256, 4096, "nvfp4"), (9, 31, 528, "nvfp4"), (13, 67, 2064, "nvfp4"),
    (16, 128, 6144, "mxfp4"), (17, 96, 1040, "nvfp4"), (33, 100, 512, "nvfp4"), (64, 129, 800, "mxfp4"),
    (100, 64, 16400, "nvfp4"), (1, 70, 17424, "nvfp4"),
]


@pytest.mark.parametrize("x_type", ["bf16", "fp16"])
@pytest.mark.parametrize("M,N,K,fmt", LINEAR)
def test_linear(M, N, K, fmt, x_type):
    torch = torch_cuda()
    ops = _ops()
    log("linear", M, N, K, fmt, x_type)
    q, w = _random_fp4(torch, N, K, fmt, M * 1000 + N)
    rng = np.random.default_rng(K)
    x = torch.tensor(rng.standard_normal((M, K)), dtype=getattr(torch, TYPES[x_type])).cuda()
    bias = torch.tensor(rng.standard_normal(N), dtype=torch.float32).cuda()
    x64, b64 = _np64(x), _np64(bias)
    for out, b in ((torch.float32, bias), (x.dtype, None)):
        y = _np64(ops.fp4_linear(x, q, bias=b, out_dtype=out))
        want = x64 @ w.T + (0 if b is None else b64)
        tol = _bound(x64, w, out, torch, _terms(K)) + (0 if b is None else 2.0 ** -22 * np.abs(b64))
        assert (np.abs(y - want) <= tol).all(), (out, np.abs((y - want) / tol).max())


# each shape lies in another of the ranges that choose a tile size
TILED = [(5, 4096, 144), (16, 4200, 1040), (20, 5000, 208), (64, 2050, 2064), (128, 2100, 1040), (30, 8300, 96),
         (130, 4100, 272), (300, 6600, 144), (1100, 14500, 48)]


@pytest.mark.parametrize("x_type", ["bf16", "fp16"])
@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("M,N,K", TILED)
def test_linear_tiles(M, N, K, fmt, x_type):
    torch = torch_cuda()
    ops = _ops()
    if fmt == "mxfp4":
        K = (K + 31) // 32 * 32
    log("linear tiles", M, N, K, fmt, x_type)
    q, w = _random_fp4(torch, N, K, fmt, M + N)
    g = torch.Generator().manual_seed(K)
    big = torch.randn(M + 1, K + 8, generator=g).to(getattr(torch, TYPES[x_type]))
    x = big[1:, 3:3 + K]                         # rows that start at odd elements
    y = ops.fp4_linear(big.cuda()[1:, 3:3 + K], q, out_dtype=torch.float32).double().cpu()
    wt = torch.tensor(w).t()
    want, mag = x.double() @ wt, x.double().abs() @ wt.abs()
    # a matrix instruction adds 32 products to a sum, the groups of a block add 8; the scale of the matrix
    tol = (32 + K / 32 + 8 + 1) * 2.0 ** -24 * mag + 1e-37
    assert ((y - want).abs() <= tol).all(), ((y - want).abs() / tol).max()


@pytest.mark.parametrize("M", [1, 4, 5, 40])
def test_linear_mx_smallest_and_largest_scales(M):
    """Weights down to 2^-128, below the smallest normal bf16 and fp32, and up to 6 * 2^125."""
    torch = torch_cuda()
    ops = _ops()
    rng = np.random.default_rng(M)
    N, K = 48, 256
    codes = rng.integers(0, 16, (N, K)).astype(np.uint8)
    for byte, size in ((0, 2.0 ** 100), (1, 2.0 ** 100), (252, 2.0 ** -60)):
        sb = np.full((N, K // 32), byte, np.uint8)
        q = ops.FP4Weight(torch.tensor(fp4.pack(codes)).cuda(), torch.tensor(sb).cuda(), None, "mxfp4")
        x = torch.tensor(rng.standard_normal((M, K)) * size, dtype=torch.bfloat16).cuda()
        w = fp4.values(codes, sb, "mxfp4", None)
        y = _np64(ops.fp4_linear(x, q, out_dtype=torch.float32))
        want, tol = _np64(x) @ w.T, _bound(_np64(x), w, torch.float32, torch, _terms(K))
        assert (np.abs(y - want) <= tol).all(), byte


@pytest.mark.parametrize("M", [1, 4, 13, 40])
def test_linear_strides_and_rows_beside_the_output(M):
    torch = torch_cuda()
    ops = _ops()
    q, _ = _random_fp4(torch, 37, 1040, "nvfp4", 3)
    rng = np.random.default_rng(M)
    big = torch.tensor(rng.standard_normal((M + 2, 1100)), dtype=torch.bfloat16).cuda()
    for off in (0, 1, 8):
        x = big[1:M + 1, off:off + 1040]
        out = torch.full((M + 2, 64), 9.0, device="cuda")
        ops.fp4_linear(x, q, out=out[1:M + 1, 5:42])
        dense = ops.fp4_linear(x.contiguous(), q, out_dtype=torch.float32)
        assert torch.equal(out[1:M + 1, 5:42], dense)
        out[1:M + 1, 5:42] = 9.0
        assert (out == 9.0).all()


@pytest.mark.parametrize("M", [1, 3, 9, 40])
@pytest.mark.parametrize("fmt,K", [("nvfp4", 1040), ("nvfp4", 1024), ("mxfp4", 1056)])
def test_linear_nan_stays_where_it_is(M, fmt, K):
    """A NaN scale reaches its output column only, a NaN or infinity in x its row only."""
    torch = torch_cuda()
    ops = _ops()
    q, _ = _random_fp4(torch, 70, K, fmt, 8)
    x = torch.randn(M, K, device="cuda").to(torch.bfloat16)
    clean = ops.fp4_linear(x, q, out_dtype=torch.float32)
    keep = q.scales.clone()
    q.scales[33, q.scales.shape[1] - 1] = 0x7F if fmt == "nvfp4" else 0xFF
    y = ops.fp4_linear(x, q, out_dtype=torch.float32)
    assert torch.isnan(y[:, 33]).all()
    y[:, 33] = clean[:, 33]
    assert torch.equal(y, clean)
    q.scales.copy_(keep)
    for bad in (float("nan"), float("inf")):
        xb = x.clone()
        xb[M // 2, K - 1] = bad
        y = ops.fp4_linear(xb, q, out_dtype=torch.float32)
        assert not torch.isfinite(y[M // 2]).any()
        y[M // 2] = clean[M // 2]
        assert torch.equal(y, clean)


def test_linear_on_another_stream_and_replayed():
    torch = torch_cuda()
    ops = _ops()
    q, _ = _random_fp4(torch, 96, 2048, "nvfp4", 4)
    x = torch.randn(4, 2048, device="cuda").to(torch.bfloat16)
    want = ops.fp4_linear(x, q)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y = ops.fp4_linear(x, q, stream=side)
    side.synchronize()
    assert torch.equal(y, want)
    out = torch.empty_like(want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        ops.fp4_linear(x, q, out=out)
    for i in range(4):
        x.copy_(torch.randn(4, 2048, device="cuda").to(torch.bfloat16))
        eager = ops.fp4_linear(x, q)
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, eager), i


def test_quantize_replayed():
    torch = torch_cuda()
    ops = _ops()
    w = _weights(torch, 64, 512, "bf16", 2)
    q = ops.FP4Weight.empty(64, 512)
    ops.fp4_quantize(w, out=q)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        ops.fp4_quantize(w, out=q)
    for i in range(3):
        w.copy_(_weights(torch, 64, 512, "bf16", 20 + i))
        g.replay()
        torch.cuda.synchronize()
        _check_quant(torch, w, q, "nvfp4")


def test_a_weight_keeps_its_memory():
    """Tensors whose storage is exchanged, or that are dropped, after the weight was made."""
    torch = torch_cuda()
    ops = _ops()
    q, w = _random_fp4(torch, 96, 2048, "nvfp4", 6)
    x = torch.randn(3, 2048, device="cuda").to(torch.bfloat16)
    want, values = ops.fp4_linear(x, q), ops.fp4_dequantize(q)
    for t in (q.codes, q.scales, q.global_scale):
        t.data = torch.zeros_like(t)
    filler = [torch.full((n,), 0x7F, dtype=torch.uint8, device="cuda") for n in (96 * 1024, 96 * 128, 4) for _ in range(4)]
    assert torch.equal(ops.fp4_linear(x, q), want) and torch.equal(ops.fp4_dequantize(q), values)
    del filler


def _busy(torch, stream, ms=40):
    """Keeps a stream busy for about `ms` (a matrix product of 0.1 ms and more, many times)."""
    a = torch.zeros(4096, 4096, dtype=torch.bfloat16, device="cuda")
    torch.mm(a, a)
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        for _ in range(10 * ms):
            torch.mm(a, a)
    a.record_stream(stream)


@pytest.mark.parametrize("op", ["quantize", "dequantize", "linear"])
def test_tensors_dropped_while_another_stream_needs_them(op):
    """Operands, weights and outputs of a call on a busy stream are not given out again until it is done."""
    torch = torch_cuda()
    ops = _ops()
    side = torch.cuda.Stream()
    q0, _ = _random_fp4(torch, 512, 1024, "nvfp4", 12)
    x0 = torch.randn(512, 1024, device="cuda").to(torch.bfloat16)
    bias0 = torch.randn(512, device="cuda")
    want = {"quantize": lambda: ops.fp4_dequantize(ops.fp4_quantize(x0)), "dequantize": lambda: ops.fp4_dequantize(q0),
            "linear": lambda: ops.fp4_linear(x0, q0, bias=bias0)}[op]()
    torch.cuda.synchronize()
    _busy(torch, side)
    mine = [x0.clone(), bias0.clone(), q0.codes.clone(), q0.scales.clone(), q0.global_scale.clone()]
    sizes = [t.numel() * t.element_size() for t in mine]
    x, bias, q = mine[0], mine[1], ops.FP4Weight(*mine[2:])
    side.wait_stream(torch.cuda.current_stream())
    if op == "quantize":
        kept = ops.fp4_quantize(x, stream=side)
    elif op == "dequantize":
        kept = ops.fp4_dequantize(q, stream=side)
    else:
        kept = ops.fp4_linear(x, q, bias=bias, stream=side)
    used = {"quantize": mine[:1], "dequantize": mine[2:], "linear": mine}[op]
    used = [t.data_ptr() for t in used]
    del x, bias, q, mine
    new = [torch.full((n,), 0x7F, dtype=torch.uint8, device="cuda") for n in sizes for _ in range(4)]
    assert not side.query(), "the stream was not busy long enough to tell"
    assert not {t.data_ptr() for t in new} & set(used)
    torch.cuda.synchronize()
    assert torch.equal(ops.fp4_dequantize(kept) if op == "quantize" else kept, want)


def test_no_rows_on_a_given_stream():
    torch = torch_cuda()
    ops = _ops()
    side = torch.cuda.Stream()
    q = ops.fp4_quantize(torch.empty(0, 64, device="cuda"), stream=side)
    assert ops.fp4_dequantize(q, stream=side).shape == (0, 64)
    assert ops.fp4_linear(torch.empty(2, 64, device="cuda", dtype=torch.bfloat16), q, stream=side).shape == (2, 0)
    side.synchronize()


def test_linear_has_no_gradient_and_says_so():
    """Not a result that looks like one of constants: a layer in front of it would silently not be trained."""
    torch = torch_cuda()
    ops = _ops()
    q, _ = _random_fp4(torch, 40, 256, "nvfp4", 2)
    x, bias = torch.randn(3, 256, device="cuda").to(torch.bfloat16), torch.randn(40, device="cuda")
    want = ops.fp4_linear(x, q, bias=bias, out_dtype=torch.float32)
    for a, b in ((x.clone().requires_grad_(), bias), (x, bias.clone().requires_grad_())):
        y = ops.fp4_linear(a, q, bias=b, out_dtype=torch.float32)
        assert torch.equal(y, want) and y.requires_grad
        with pytest.raises(NotImplementedError):
            y.sum().backward()
        with torch.no_grad():
            assert not ops.fp4_linear(a, q, bias=b).requires_grad
        assert torch.equal(ops.fp4_linear(a, q, bias=b, out=torch.empty_like(want)), want)
    assert not want.requires_grad


# nb blocks of weight rows, a multiple of eight, that each meet several blocks of operand rows; every tile size
BLOCKS = [(20, 1024), (48, 2048), (128, 2048), (128, 4096), (256, 6144), (520, 6144), (1040, 12288)]


@pytest.mark.parametrize("x_type,fmt", [("bf16", "nvfp4"), ("fp16", "mxfp4"), ("fp16", "nvfp4")])
@pytest.mark.parametrize("M,N", BLOCKS)
def test_linear_blocks_that_share_weight_rows(M, N, x_type, fmt):
    """Every tile of the output is written, and by the rows it belongs to."""
    torch = torch_cuda()
    K = 144 if fmt == "nvfp4" else 160
    log("linear blocks", M, N, K, fmt, x_type)
    q, w = _random_fp4(torch, N, K, fmt, M + N)
    x = torch.randn(M, K, generator=torch.Generator().manual_seed(K)).to(getattr(torch, TYPES[x_type]))
    out = torch.full((M, N), float("nan"), device="cuda")
    _ops().fp4_linear(x.cuda(), q, out=out)
    wt = torch.tensor(w).t()
    want, mag = x.double() @ wt, x.double().abs() @ wt.abs()
    # as above: 32 products of an instruction, the chunks, eight groups, the scale of the matrix
    tol = (32 + K / 32 + 8 + 1) * 2.0 ** -24 * mag + 1e-37
    err = (out.double().cpu() - want).abs()
    assert bool((err <= tol).all()), float((err / tol).max())


# more groups than the threads of the grid, and more bytes than its blocks take at once; odd row counts
@pytest.mark.parametrize("fmt,rows,cols,dtype", [("nvfp4", 1409, 4112, "bf16"), ("nvfp4", 2579, 2080, "fp32"),
                                                 ("mxfp4", 2579, 2080, "fp32"), ("mxfp4", 1409, 4128, "fp16")])
@pytest.mark.parametrize("strided", [False, True])
def test_quantize_more_groups_than_threads(fmt, rows, cols, dtype, strided):
    torch = torch_cuda()
    log("quantize", fmt, rows, cols, dtype, strided)
    big = _weights(torch, rows, cols + 24, dtype, rows)
    w = big[:, 5:5 + cols] if strided else big[:, :cols].contiguous()
    w[rows - 1, cols - 1] = 9.0                # the matrix's largest
    w[rows - 2, cols - 40] = float("nan")
    w[rows - 1, 3] = float("inf")
    _check_quant(torch, w, _ops().fp4_quantize(w, fmt), fmt)


# ---- more threads than one launch has (2^32) ----------------------------------------

def _rows_of(q, a, b):
    return _ops().FP4Weight(q.codes[a:b], q.scales[a:b], q.global_scale, q.fmt)


def _large_fp4(torch, rows, cols, fmt):
    q = _ops().FP4Weight.empty(rows, cols, fmt)
    for a in range(0, rows, 1 << 24):
        q.codes[a:a + (1 << 24)].random_(0, 256)
        q.scales[a:a + (1 << 24)].random_(0x28, 0x70)
    return q


def test_dequantize_a_matrix_of_more_than_2_to_34_elements():
    """64 GiB of fp32 values."""
    torch = torch_cuda()
    rows, cols = (1 << 14) + 3, 1 << 20
    log("dequantize", rows, cols)
    q = _large_fp4(torch, rows, cols, "mxfp4")
    out = torch.empty(rows, cols, device="cuda")
    out[-4:] = float("nan")
    out[:4] = float("nan")
    _ops().fp4_dequantize(q, out=out)
    for a in range(0, rows, 1024):
        b = min(rows, a + 1024)
        assert torch.equal(out[a:b], _ops().fp4_dequantize(_rows_of(q, a, b))), a


@pytest.mark.parametrize("M,N", [(1, (1 << 29) + 40), (5, (1 << 27) + 40)])
def test_linear_with_very_many_weight_rows(M, N):
    torch = torch_cuda()
    log("linear", M, N)
    q = _large_fp4(torch, N, 16, "nvfp4")
    x = torch.randn(M, 16, device="cuda").to(torch.bfloat16)
    bias = torch.randn(N, device="cuda")
    out = torch.full((M, N), float("nan"), device="cuda")
    _ops().fp4_linear(x, q, bias=bias, out=out)
    for a in range(0, N, 1 << 24):
        b = min(N, a + (1 << 24))
        part = _ops().fp4_linear(x, _rows_of(q, a, b), bias=bias[a:b], out_dtype=torch.float32)
        assert torch.equal(out[:, a:b], part), a


def test_linear_with_very_many_operand_rows():
    """2^30 rows and some: 64 GiB of x."""
    torch = torch_cuda()
    M, K = (1 << 30) + 70, 32
    log("linear", M)
    q = _large_fp4(torch, 2, K, "mxfp4")
    x = torch.empty(M, K, dtype=torch.float16, device="cuda")
    for a in range(0, M, 1 << 26):
        x[a:a + (1 << 26)].normal_()
    out = torch.full((M, 2), float("nan"), dtype=torch.float16, device="cuda")
    _ops().fp4_linear(x, q, out=out)
    for a in range(0, M, 1 << 26):
        b = min(M, a + (1 << 26))
        part = _ops().fp4_linear(x[a:b], q)
        if b - a > 1000:
            assert torch.equal(out[a:b], part), a
        else:                                  # few rows: another order of the 32 products
            assert torch.allclose(out[a:b].float(), part.float(), rtol=2e-3, atol=1e-3), a
