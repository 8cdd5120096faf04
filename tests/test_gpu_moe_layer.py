"""The whole mixture-of-experts layer against float64: picks equal, weights and outputs within the rounding
of fp32 sums."""
import numpy as np
import pytest

from oracle import moe as om
from synth.gen import bf16_bits_from_f32, e4m3_bits_rne
from oracle.formats import decode_bf16

from gpu_util import log, torch_cuda

pytestmark = pytest.mark.gpu


def _blob(rng, H, I):
    n = 27 * H * I // 16
    b = rng.integers(0, 256, n, dtype=np.uint8)
    a, s, c = I * H, I * H // 8, H * I // 2
    for lo, hi in ((a, a + s), (a + s + c, n)):
        b[lo:hi] = e4m3_bits_rne(100 + 80 * np.abs(rng.standard_normal(hi - lo)))
    return b


class Case:
    def __init__(self, M, H, I, E, k, Is=0, score="softmax", scale=1.0, seed=0, max_rows=16):
        import torch
        from hbm_expert_slot_amd.ops import MoELayer
        rng = np.random.default_rng([seed, M, H, I, E, k])
        self.M, self.H, self.I, self.E, self.k, self.Is, self.score, self.scale = M, H, I, E, k, Is, score, scale
        self.x = decode_bf16(bf16_bits_from_f32(rng.standard_normal((M, H)).astype(np.float32)))
        self.router = decode_bf16(bf16_bits_from_f32((rng.standard_normal((E, H)) * 1.5 / np.sqrt(H)).astype(np.float32)))
        self.blobs = np.stack([_blob(rng, H, I) for _ in range(E)])
        self.gs = (rng.uniform(0.5, 1.5, (E, 2)) / 480 / np.sqrt([H, I])).astype(np.float32)
        self.bias = rng.standard_normal(E).astype(np.float32) * np.float32(0.05) if score == "sigmoid" else None
        self.shared = _blob(rng, H, Is) if Is else None
        self.sgs = (rng.uniform(0.5, 1.5, 2) / 480 / np.sqrt([H, max(Is, 1)])).astype(np.float32) if Is else None
        self.torch = torch
        cu = lambda v: None if v is None else torch.tensor(v).cuda()
        self.tx = torch.tensor(self.x, dtype=torch.bfloat16).cuda()
        self.args = dict(router=torch.tensor(self.router, dtype=torch.bfloat16).cuda(), blobs=cu(self.blobs),
                         global_scales=cu(self.gs), shared_blob=cu(self.shared), shared_global_scales=cu(self.sgs),
                         score=score, score_bias=cu(self.bias), routed_scale=scale, max_rows=max_rows)
        self.layer = MoELayer(H, I, k, **self.args)

    def want(self, x=None):
        x = self.x if x is None else x
        ids, w, gap = om.route_layer(x, self.router, self.k, self.score,
                                     None if self.bias is None else self.bias.astype(np.float64), self.scale)
        y, mag = om.moe_layer(x, ids, w, lambda e: self.blobs[e], self.gs, self.H, self.I, self.shared, self.sgs, self.Is)
        return ids, w, gap, y, mag

    def run(self, x=None, dtype=None, **kw):
        t = self.torch
        x = self.tx if x is None else x
        ids = t.full((x.shape[0], self.k), -1, dtype=t.int32, device="cuda")
        w = t.full((x.shape[0], self.k), float("nan"), device="cuda")
        y = self.layer.forward(x, out_dtype=dtype or t.float32, ids=ids, weights=w, **kw)
        return y, ids, w

    def check(self, y, ids, w, want=None):
        t = self.torch
        ids64, w64, gap, y64, mag = want or self.want()
        # scores: fp32 sums of H products in chains of at most H / 256 (8 lanes-wide steps of a wavefront) + 8 levels
        znorm = (np.abs(self.x) @ np.abs(self.router).T).max()
        assert (gap > (self.H / 256 + 16) * 2.0 ** -23 * max(znorm, 1)).all(), "draw other inputs: scores too close"
        assert np.array_equal(ids.cpu().numpy(), ids64)
        wtol = (self.H / 256 + 16) * 2.0 ** -23 * max(znorm, 1) + 2.0 ** -18
        assert np.abs(w.cpu().numpy() - w64).max() <= wtol * self.scale
        # sums: group of 16, steps of 512, lanes; twice (gate/up and down), h in 24 bits, SiLU to a few ulps, the
        # weights, picks added in fp32
        terms = 2 * (16 + (self.H + max(self.I, self.Is)) // 256 + 12) + 8 + self.k
        got = y.double().cpu().numpy()
        eps = t.finfo(y.dtype).eps / 2 if y.dtype != t.float32 else 0.0
        tol = (terms * 2.0 ** -24 + wtol) * mag + eps * np.abs(y64) * 1.01
        assert (np.abs(got - y64) <= tol).all(), np.abs((got - y64) / tol).max()
        rel = np.linalg.norm(got - y64) / np.linalg.norm(y64)
        assert rel <= (2e-5 if y.dtype == t.float32 else 2.0 ** -8), rel
        return rel


CASES = [
    dict(M=1, H=256, I=128, E=16, k=2), dict(M=1, H=64, I=64, E=1, k=1), dict(M=1, H=64, I=64, E=5, k=5, Is=64),
    dict(M=1, H=1088, I=320, E=33, k=8, Is=320, score="sigmoid", scale=2.5),
    dict(M=2, H=512, I=192, E=12, k=3), dict(M=3, H=704, I=64, E=20, k=4, Is=128, score="sigmoid"),
    dict(M=4, H=256, I=576, E=9, k=2, Is=64), dict(M=5, H=576, I=128, E=40, k=6),
    dict(M=8, H=1024, I=256, E=24, k=8, Is=256), dict(M=11, H=320, I=192, E=7, k=7, score="sigmoid"),
    dict(M=16, H=512, I=128, E=3, k=2, Is=192), dict(M=16, H=2112, I=1088, E=4, k=1),
    dict(M=16, H=64, I=64, E=300, k=32), dict(M=16, H=128, I=64, E=1024, k=8, score="sigmoid"),
    dict(M=7, H=128, I=64, E=600, k=3), dict(M=4, H=8256, I=64, E=6, k=2), dict(M=16, H=64, I=4160, E=2, k=2),
]


@pytest.mark.parametrize("c", CASES, ids=lambda c: "-".join("%s%s" % (k, v) for k, v in c.items()))
def test_layer(c):
    torch = torch_cuda()
    log("moe layer", c)
    case = Case(**c)
    want = case.want()
    for dt in (torch.float32, torch.bfloat16):
        rel = case.check(*case.run(dtype=dt), want=want)
        log("  rel L2", dt, "%.2e" % rel)
    a, b = case.run()[0], case.run()[0]
    assert torch.equal(a, b)


# one row: many picks, h longer than LDS holds at a time, ragged steps, shared and routed sizes far apart
ONE = [
    dict(M=1, H=256, I=2048, E=40, k=32), dict(M=1, H=192, I=1088, E=33, k=32, Is=64, score="sigmoid"),
    dict(M=1, H=64, I=64, E=1024, k=32), dict(M=1, H=8256, I=64, E=6, k=2, Is=4160), dict(M=1, H=32768, I=64, E=2, k=2),
    dict(M=1, H=64, I=32768, E=2, k=1), dict(M=1, H=64, I=64, E=2, k=1, Is=32768), dict(M=1, H=576, I=576, E=1000, k=1),
    dict(M=1, H=4160, I=1600, E=10, k=9, Is=576, score="sigmoid", scale=0.5),
]


@pytest.mark.parametrize("c", ONE, ids=lambda c: "-".join("%s%s" % (k, v) for k, v in c.items()))
def test_one_row(c):
    torch = torch_cuda()
    log("moe layer, one row", c)
    case = Case(**c, max_rows=2)
    want = case.want()
    log("  rel L2 %.2e" % case.check(*case.run(), want=want))
    case.check(*case.run(dtype=torch.bfloat16), want=want)
    a = case.run()[0]
    for _ in range(3):
        assert torch.equal(case.run()[0], a)


# so many tiles that a task takes two or four of an expert's, and numbers that these do not divide
MANY = [
    dict(M=16, H=4160, I=64, E=40, k=8), dict(M=12, H=8256, I=64, E=40, k=8, Is=64), dict(M=16, H=64, I=2048, E=40, k=8),
    dict(M=9, H=128, I=4160, E=36, k=6, Is=128, score="sigmoid"), dict(M=4, H=12352, I=64, E=30, k=6),
]


@pytest.mark.parametrize("c", MANY, ids=lambda c: "-".join("%s%s" % (k, v) for k, v in c.items()))
def test_many_tiles(c):
    torch_cuda()
    log("moe layer, many tiles", c)
    case = Case(**c)
    log("  rel L2 %.2e" % case.check(*case.run()))


def test_one_row_beside_the_output_and_with_nan():
    torch = torch_cuda()
    case = Case(1, 576, 192, 20, 3, Is=64)
    want, ids0, _ = case.run()
    out = torch.full((3, 600), 9.0, device="cuda")
    case.layer.forward(case.tx, out=out[1:2, 5:581])
    assert torch.equal(out[1:2, 5:581], want)
    out[1:2, 5:581] = 9.0
    assert (out == 9.0).all()
    for bad in (float("nan"), float("inf")):
        x = case.tx.clone()
        x[0, 3] = bad
        y, ids, _ = case.run(x)
        assert not torch.isfinite(y).any()
        assert len(set(ids[0].tolist())) == 3 and int(ids.min()) >= 0 and int(ids.max()) < 20
    y, ids, _ = case.run()
    assert torch.equal(y, want) and torch.equal(ids, ids0)


def test_one_row_gives_up_a_wait_that_does_not_end():
    """A share marked as taken that nobody computes (as a call that shares its workspace could leave it): every block
    leaves after its bounded wait, the result is NaN, and the workspace serves the next call."""
    torch = torch_cuda()
    case = Case(1, 576, 192, 20, 3, Is=64)
    want = case.run()[0]
    torch.cuda.synchronize()
    claims = 5 * 16 * 32 + 2 * 32 + (513 + 32) // 32 * 32 + 1024 + 513 * 32     # words of the kernel for more rows
    case.layer.workspace.view(torch.int32)[claims] = 1
    log("a share that nobody computes")
    y = case.layer.forward(case.tx)
    torch.cuda.synchronize()
    assert torch.isnan(y).all()
    assert torch.equal(case.run()[0], want)


@pytest.mark.parametrize("M", [1, 2, 16])
def test_replayed(M):
    """Two graphs of one layer, replayed in turn with eager calls of other row counts between them."""
    torch = torch_cuda()
    case = Case(M, 512, 576, 40, 8, Is=192)
    case.layer.forward(case.tx)
    graphs, outs, xs = [], [], []
    for i in range(2):
        xs.append(torch.empty_like(case.tx))
        outs.append(torch.empty(M, 512, device="cuda"))
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[i]):
            case.layer.forward(xs[i], out=outs[i])
    other = torch.randn(3, 512, device="cuda").to(torch.bfloat16)
    for r in range(4):
        for i in range(2):
            xs[i].copy_(torch.randn(M, 512, device="cuda").to(torch.bfloat16))
            eager = case.layer.forward(xs[i])
            case.layer.forward(other[:1 + (r + i) % 3])
            outs[i].zero_()
            graphs[i].replay()
        torch.cuda.synchronize()
        for i in range(2):
            assert torch.equal(outs[i], case.layer.forward(xs[i])), (r, i)


def test_layers_of_one_row_and_of_many_at_once():
    """Layers with workspaces of their own on three streams: none waits for blocks that another keeps out."""
    torch = torch_cuda()
    cases = [Case(1, 2048, 1024, 16, 8, Is=512, seed=1), Case(1, 2048, 1024, 16, 8, Is=512, seed=2),
             Case(16, 1024, 512, 16, 4, seed=3)]
    want = [c.run()[0] for c in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    outs = [[], [], []]
    for _ in range(20):
        for i, (c, s) in enumerate(zip(cases, streams)):
            outs[i].append(c.layer.forward(c.tx, stream=s))
    torch.cuda.synchronize()
    for i in range(3):
        for y in outs[i]:
            assert torch.equal(y, want[i]), i


def test_sizes_of_the_configurations():
    """One row and sixteen rows at the inner sizes of the GLM-shaped layer, few experts."""
    torch_cuda()
    for c in (dict(M=1, H=6144, I=2048, E=12, k=8, Is=2048, score="sigmoid", scale=2.5),
              dict(M=16, H=4096, I=2048, E=10, k=3)):
        log("moe layer", c)
        case = Case(**c)
        log("  rel L2 %.2e" % case.check(*case.run()))


def test_rows_of_a_layer_in_turn():
    """One layer object serves calls of every row count, smaller after larger."""
    torch = torch_cuda()
    case = Case(16, 512, 192, 24, 4, Is=128)
    full = case.run()[0]
    for M in (16, 1, 4, 2, 9, 3, 16, 5, 0, 1):
        y = case.layer.forward(case.tx[:M])
        assert y.shape == (M, 512)
        if M:
            assert float((y - full[:M]).norm() / full[:M].norm()) < 1e-6, M
    assert torch.equal(case.run()[0], full)


def test_strides_and_rows_beside_the_output():
    torch = torch_cuda()
    case = Case(5, 320, 128, 10, 3)
    want = case.run()[0]
    for off in (0, 1, 8):
        big = torch.zeros(8, 400, dtype=torch.bfloat16, device="cuda")
        big[2:7, off:off + 320] = case.tx
        out = torch.full((8, 400), 9.0, device="cuda")
        case.layer.forward(big[2:7, off:off + 320], out=out[2:7, 3:323])
        assert torch.equal(out[2:7, 3:323], want)
        out[2:7, 3:323] = 9.0
        assert (out == 9.0).all()


def test_ties_go_to_the_lower_expert():
    torch = torch_cuda()
    case = Case(3, 128, 64, 40, 6)
    case.args["router"].zero_()
    ids = case.run()[1].cpu().numpy()
    assert (ids == np.arange(6)).all()
    w = case.run()[2]
    assert torch.allclose(w, torch.full_like(w, 1 / 6), rtol=1e-6)


def test_a_nan_row_stays_alone():
    torch = torch_cuda()
    case = Case(6, 256, 128, 12, 3, Is=64)
    clean = case.run()[0]
    for bad in (float("nan"), float("inf")):
        x = case.tx.clone()
        x[2, 100] = bad
        y, ids, w = case.run(x)
        assert not torch.isfinite(y[2]).any()
        # the other rows: the same picks; experts may meet other row counts, so not the same bits
        keep = [0, 1, 3, 4, 5]
        assert float((y[keep] - clean[keep]).norm() / clean[keep].norm()) < 1e-6
        i2 = ids[2].cpu().numpy()
        assert len(set(i2.tolist())) == 3 and (i2 >= 0).all() and (i2 < 12).all()
    assert torch.equal(case.run()[0], clean)


def test_an_experts_nan_scale_reaches_its_rows_only():
    torch = torch_cuda()
    case = Case(8, 256, 128, 12, 2)
    y0, ids, _ = case.run()
    e = int(ids[0, 0])
    case.args["blobs"][e, 128 * 256 + 5] = 0x7F
    y = case.run()[0]
    hit = (ids == e).any(1)
    assert torch.isnan(y[hit]).any(1).all() and torch.equal(y[~hit], y0[~hit])


def test_replayed_and_eager_in_turn():
    torch = torch_cuda()
    case = Case(4, 512, 192, 24, 4, Is=64, score="sigmoid")
    x = case.tx.clone()
    out = torch.empty(4, 512, device="cuda")
    case.layer.forward(x, out=out)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        case.layer.forward(x, out=out)
    for i in range(4):
        x.copy_(torch.randn(4, 512, device="cuda").to(torch.bfloat16))
        eager = case.layer.forward(x)
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, eager), i


def test_two_layers_on_two_streams():
    """Layers with workspaces of their own may run at once."""
    torch = torch_cuda()
    cases = [Case(4, 1024, 512, 16, 4, Is=256, seed=s) for s in (1, 2)]
    want = [c.run()[0] for c in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    outs = [[], []]
    for _ in range(20):
        for i, (c, s) in enumerate(zip(cases, streams)):
            outs[i].append(c.layer.forward(c.tx, stream=s))
    torch.cuda.synchronize()
    for i in range(2):
        for y in outs[i]:
            assert torch.equal(y, want[i])


def test_quantised_weights_through_the_layer():
    """Experts quantised on the device into blobs, then run: the whole set together.  The result is that of the
    dequantised matrices, and near that of the weights they came from."""
    torch = torch_cuda()
    from hbm_expert_slot_amd import ops
    H, I, E, k, M = 256, 192, 6, 2, 3
    g = torch.Generator(device="cuda")
    g.manual_seed(4)
    w13 = torch.randn(E, 2 * I, H, device="cuda", generator=g) / H ** 0.5
    w2 = torch.randn(E, H, I, device="cuda", generator=g) / I ** 0.5
    blobs = torch.zeros(E, ops.blob_bytes(H, I), dtype=torch.uint8, device="cuda")
    gs = torch.zeros(E, 2, device="cuda")
    for e in range(E):
        q13, q2 = ops.expert_matrices(blobs[e], H, I, gs[e])
        ops.fp4_quantize(w13[e], out=q13)
        ops.fp4_quantize(w2[e], out=q2)
    router = (torch.randn(E, H, device="cuda", generator=g) / H ** 0.5).to(torch.bfloat16)
    x = torch.randn(M, H, device="cuda", generator=g).to(torch.bfloat16)
    layer = ops.MoELayer(H, I, k, router, blobs, gs)
    ids = torch.empty(M, k, dtype=torch.int32, device="cuda")
    wt = torch.empty(M, k, device="cuda")
    y = layer.forward(x, ids=ids, weights=wt)
    for m in range(M):
        want = torch.zeros(H, device="cuda", dtype=torch.float64)
        for j in range(k):
            q13, q2 = ops.expert_matrices(blobs[int(ids[m, j])], H, I, gs[int(ids[m, j])])
            gu = ops.fp4_linear(x[m:m + 1], q13, out_dtype=torch.float32)[0].double()
            h = gu[:I] / (1 + torch.exp(-gu[:I])) * gu[I:]
            want += wt[m, j].double() * (ops.fp4_dequantize(q2).double() @ h)
        # w13's products and w2's: fp32 sums of at most 40 terms each, twice
        assert float((y[m].double() - want).norm() / want.norm()) < 1e-5


# ---- sigmoid scores near their ends ------------------------------------------------

def _scored(M, z, bias, k, scale=1.0):
    """Picks and weights of a layer whose logits are exactly z [E] for every row (x is 1 in three places, where the
    router holds three bf16 parts of z)."""
    import torch
    from hbm_expert_slot_amd.ops import MoELayer
    E, H, I = len(z), 64, 64
    rng = np.random.default_rng(E)
    router = np.zeros((E, H), np.float32)
    for i in range(3):
        router[:, i] = decode_bf16(bf16_bits_from_f32((z - router.sum(1, dtype=np.float64)).astype(np.float32)))
    assert np.array_equal(router.sum(1, dtype=np.float64), z)
    x = torch.zeros(M, H, dtype=torch.bfloat16, device="cuda")
    x[:, :3] = 1
    cu = lambda v: None if v is None else torch.tensor(v).cuda()
    layer = MoELayer(H, I, k, torch.tensor(router, dtype=torch.bfloat16).cuda(),
                     cu(np.stack([_blob(rng, H, I) for _ in range(E)])),
                     cu(np.full((E, 2), 1e-4, np.float32)), score="sigmoid", score_bias=cu(bias), routed_scale=scale)
    ids = torch.full((M, k), -1, dtype=torch.int32, device="cuda")
    w = torch.full((M, k), float("nan"), device="cuda")
    layer.forward(x, ids=ids, weights=w)
    return ids.cpu().numpy(), w.double().cpu().numpy()


def _steps(E, base, seed):
    """E different logits from base on, 2^-12 apart, in any order."""
    return base + np.random.default_rng(seed).permutation(E) * 2.0 ** -12


# the kernels for one row, for up to four and for more; experts per lane that are sorted, and that are not
ROWS_AND_EXPERTS = [(1, 40), (3, 40), (7, 40), (1, 700), (6, 700)]


@pytest.mark.parametrize("base", [10.0, 20.0, 100.0, -20.0, -100.0])
@pytest.mark.parametrize("M,E", ROWS_AND_EXPERTS)
def test_sigmoid_scores_that_fp32_cannot_tell_apart(M, E, base):
    """Without a bias the order is that of the logits: near 1 sigmoids of different logits are one fp32 number."""
    torch_cuda()
    z = _steps(E, base, M)
    ids, _ = _scored(M, z, None, 6)
    assert (ids == np.argsort(-z)[:6]).all()


@pytest.mark.parametrize("base", [0.0, 10.0, 20.0, -20.0])
@pytest.mark.parametrize("M,E", ROWS_AND_EXPERTS)
def test_sigmoid_scores_with_one_bias_for_all(M, E, base):
    """The same bias for all leaves that order; at 20 the neighbours' sums differ by 5e-13."""
    torch_cuda()
    z = _steps(E, base, M + 1)
    for b in (0.0, 0.25, -0.75):
        ids, _ = _scored(M, z, np.full(E, b, np.float32), 6)
        assert (ids == np.argsort(-z)[:6]).all(), b


@pytest.mark.parametrize("M,E", ROWS_AND_EXPERTS)
def test_sigmoid_scores_and_biases_that_nearly_balance(M, E):
    """Sums apart by less than fp32 holds next to 1."""
    torch_cuda()
    rng = np.random.default_rng(M * E)
    z = 10.0 + rng.integers(0, 4096, E) * 2.0 ** -12
    bias = (rng.standard_normal(E) * 1e-6).astype(np.float32)
    by = 1.0 / (1.0 + np.exp(-z)) + bias.astype(np.float64)
    order = np.argsort(-by, kind="stable")
    # sigmoid's distance to 1 is 4.5e-5 and known to 16 steps of fp32
    assert (-np.diff(by[order[:7]])).min() > 4.5e-5 * 16 * 2.0 ** -24, "draw other inputs: scores too close"
    ids, _ = _scored(M, z, bias, 6)
    assert (ids == order[:6]).all()


def test_sigmoid_ties_go_to_the_lower_expert():
    torch_cuda()
    for z in (0.0, 12.0, 90.0, -90.0):
        for bias in (None, np.full(300, 0.5, np.float32)):
            ids, w = _scored(2, np.full(300, z), bias, 5)
            assert (ids == np.arange(5)).all() and np.abs(w - 0.2).max() < 1e-6


@pytest.mark.parametrize("M,E", ROWS_AND_EXPERTS)
@pytest.mark.parametrize("base", [-20.0, -86.0, -88.0, -95.0, -120.0])
def test_sigmoid_weights_far_below_zero(M, E, base):
    """Sigmoids that are denormal in fp32, or below it, have weights in their own proportion."""
    torch_cuda()
    rng = np.random.default_rng(E)
    z = base - rng.permutation(E) * 0.25
    ids, w = _scored(M, z, None, 6, scale=2.0)
    assert (ids == np.argsort(-z)[:6]).all()
    top = np.sort(z)[::-1][:6]
    v = np.exp(top - top.max()) / (1.0 + np.exp(top))
    # exponentials of exact differences, a reciprocal, a sum of six and a division, a few steps each
    assert np.abs(w - 2.0 * v / v.sum()).max() <= 2.0 * 16 * 2.0 ** -24


@pytest.mark.parametrize("given", [True, False])
@pytest.mark.parametrize("M", [1, 5])
def test_a_layer_dropped_while_another_stream_works_on_it(M, given):
    """Its workspace and weights, and the call's operand, are not given out again until the stream is done."""
    torch = torch_cuda()
    case = Case(M, 512, 192, 24, 4, Is=128)
    want = case.run()[0]
    side = torch.cuda.Stream()
    a = torch.zeros(4096, 4096, dtype=torch.bfloat16, device="cuda")
    torch.mm(a, a)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        for _ in range(400):
            torch.mm(a, a)
    x = case.tx
    mine = [v for v in case.args.values() if torch.is_tensor(v)] + [case.layer.workspace] + ([x] if given else [])
    mine = [(t.data_ptr(), t.numel() * t.element_size()) for t in mine]
    if given:
        y = case.layer.forward(x, stream=side)
        del x
    else:
        with torch.cuda.stream(side):
            y = case.layer.forward(x)
    del case
    new = [torch.full((n,), 0x7F, dtype=torch.uint8, device="cuda") for _, n in mine for _ in range(4)]
    assert not side.query(), "the stream was not busy long enough to tell"
    assert not {t.data_ptr() for t in new} & {p for p, _ in mine}
    torch.cuda.synchronize()
    assert torch.equal(y, want)


@pytest.mark.parametrize("M", [1, 3, 9])
def test_prepare_makes_a_workspace_ready(M):
    torch = torch_cuda()
    case = Case(M, 320, 192, 20, 3, Is=64)
    want = case.run()[0]
    for fill in (0x00, 0x5A, 0xFF):
        case.layer.workspace.fill_(fill)
        case.layer.prepare()
        assert torch.equal(case.run()[0], want)


def test_a_layer_has_no_gradient_and_says_so():
    torch = torch_cuda()
    from hbm_expert_slot_amd.ops import MoELayer
    case = Case(3, 320, 192, 20, 3, Is=64)
    want, want_ids, _ = case.run()
    assert not want.requires_grad
    y, ids, _ = case.run(case.tx.clone().requires_grad_())
    assert torch.equal(y, want) and torch.equal(ids, want_ids)
    with pytest.raises(NotImplementedError):
        y.sum().backward()
    args = dict(case.args, router=torch.nn.Parameter(case.args["router"]))
    layer = MoELayer(320, 192, 3, **args)
    y = layer.forward(case.tx)
    assert torch.equal(y, want)
    with pytest.raises(NotImplementedError):
        y.sum().backward()
    with torch.no_grad():
        assert not layer.forward(case.tx).requires_grad


def test_captured_on_a_given_stream_and_dropped():
    """The whole path on the stream that captures, first calls of a layer among them; tensors dropped while it
    captures and after it."""
    torch = torch_cuda()
    from hbm_expert_slot_amd import ops
    case = Case(2, 512, 192, 24, 4, Is=64)
    w = torch.randn(256, 512, device="cuda")
    side = torch.cuda.Stream()
    x = case.tx.clone()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        q = ops.fp4_quantize(w, stream=side)
        y = case.layer.forward(x, out_dtype=torch.bfloat16, stream=side)
        z = ops.fp4_linear(y, q, out_dtype=torch.float32, stream=side)
        values = ops.fp4_dequantize(q, stream=side)
        del y
    for i in range(4):
        x.copy_(torch.randn(2, 512, device="cuda").to(torch.bfloat16))
        eager_q = ops.fp4_quantize(w)
        want = ops.fp4_linear(case.layer.forward(x, out_dtype=torch.bfloat16), eager_q, out_dtype=torch.float32)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(z, want) and torch.equal(values, ops.fp4_dequantize(eager_q)), i
    del g, case, x, w, q, z, values
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    again = Case(2, 512, 192, 24, 4, Is=64)
    again.check(*again.run())


H_DONE = 5 * 16 * 32 + 2 * 32      # control word: gate/up tiles of the first expert that are done


@pytest.mark.parametrize("M", [4, 9])
def test_rows_give_up_a_wait_that_does_not_end(M):
    """An expert whose h is never counted complete: every block leaves after its bounded wait, the result is NaN, and
    the workspace serves the next call."""
    torch = torch_cuda()
    case = Case(M, 576, 192, 20, 3, Is=64)
    want = case.run()[0]
    torch.cuda.synchronize()
    case.layer.workspace.view(torch.int32)[H_DONE] = -1000
    log("an expert that is never complete", M)
    y = case.layer.forward(case.tx)
    torch.cuda.synchronize()
    assert torch.isnan(y).all()
    assert torch.equal(case.run()[0], want)
