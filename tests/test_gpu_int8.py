"""The int8 (W8A8) layer on the GPU: packing and quantization bit for bit against the oracle, the product
against the exact integer sum, at the sizes where it can go wrong."""
import numpy as np
import pytest
import torch

from helpers import require_gpu
from oracle import int8 as O

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
U = 2.0 ** -24                                     # half a step of binary32, relative


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def _lib():
    from w4a4_rank_absorbed_b200 import svdq as C
    return C


def _dev(a, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(a)).cuda()
    return t if dtype is None else t.to(dtype)


def _host(t):
    return t.double().cpu().numpy()


def output_bound(xq, sx, wq, sw, bias, kind):
    """Largest |Y - exact|, element by element.  float32 steps of the epilogue: the conversion of the sum, its
    product with sx (each at most U relative to the product p), then one fused multiply-add with sw and the
    bias (U of the result): (2 U + U^2) |p| + U |y|; 2.5 U |p| + U |y| covers it.  Then the rounding to the
    output type: half its step, relative 2^-8 (bf16) or 2^-11 (fp16), absolute 2^-25 for fp16's subnormals."""
    p = O.linear(xq, sx, wq, sw)
    y = p if bias is None else p + bias.astype(np.float64)[None, :]
    e = 2.5 * U * np.abs(p) + U * np.abs(y) + 2.0 ** -149
    half = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11, "fp32": 0.0}[kind]
    return y, e + half * (np.abs(y) + e) + (2.0 ** -25 if kind == "fp16" else 0.0)


def _codes(r, rows, K):
    q = r.integers(-127, 128, (rows, K)).astype(np.int8)
    return q, r.uniform(1e-3, 2e-2, rows).astype(np.float32)


def _linear(C, xq, sx, wq, sw, bias, kind, pad=0):
    M, K = xq.shape
    N = wq.shape[0]
    full = torch.full((M, N + pad), 7.0, dtype=TYPES[kind], device="cuda")
    Y = full[:, :N]
    C.svdq_linear_i8(_dev(xq), _dev(sx), _dev(wq), _dev(sw), None if bias is None else _dev(bias), Y, M, N, K)
    torch.cuda.synchronize()
    assert C.svdq_get_device_error() == (0, 0)
    assert bool((full[:, N:] == 7.0).all())
    return _host(Y)


# one token to several tiles; sizes just below, at and above the tile edges 16, 32, 64, 128, 256; K of one
# 16-byte chunk, of a partial 128-byte chunk, of many
SHAPES = [(1, 16, 16), (1, 1, 16), (2, 17, 32), (1, 4096, 4096), (3, 130, 144), (15, 257, 272), (16, 128, 128),
          (17, 127, 400), (31, 1000, 1040), (33, 640, 1296), (64, 256, 512), (65, 255, 528), (77, 1288, 2048),
          (127, 129, 256), (128, 384, 1024), (129, 100, 112), (200, 3, 2064), (255, 512, 640), (257, 513, 656),
          (300, 1024, 12288), (513, 768, 128), (1000, 1001, 1040), (1024, 2048, 512), (2049, 300, 272), (4608, 33, 64), (700, 160, 256), (2304, 320, 320), (5000, 224, 128), (9500, 480, 96)]


@pytest.mark.parametrize("M,N,K", SHAPES)
@pytest.mark.parametrize("kind", ["bf16", "fp16", "fp32"])
def test_linear(M, N, K, kind):
    C = _lib()
    r = np.random.default_rng(M * 7919 + N * 31 + K)
    (xq, sx), (wq, sw) = _codes(r, M, K), _codes(r, N, K)
    bias = None if (M + N) % 3 == 0 else r.normal(size=N).astype(np.float32)
    if kind == "fp16":
        sx = (sx * np.float32(2.0 ** -6)).astype(np.float32)      # stay inside fp16's range
    y, bound = output_bound(xq, sx, wq, sw, bias, kind)
    got = _linear(C, xq, sx, wq, sw, bias, kind)
    assert np.all(np.abs(got - y) <= bound), float(np.max(np.abs(got - y) / bound))


@pytest.mark.parametrize("M,N,K", [(1, 100, 64), (20, 130, 256), (150, 65, 144), (700, 511, 128), (4097, 514, 64)])
@pytest.mark.parametrize("pad", [1, 8, 16])
def test_linear_into_a_wider_matrix(M, N, K, pad):
    """Y's rows at a pitch that leaves them at any alignment; the columns past N stay as they were."""
    C = _lib()
    r = np.random.default_rng(pad)
    (xq, sx), (wq, sw) = _codes(r, M, K), _codes(r, N, K)
    for kind in TYPES:
        s = sx if kind != "fp16" else (sx * np.float32(2.0 ** -6)).astype(np.float32)
        y, bound = output_bound(xq, s, wq, sw, None, kind)
        assert np.all(np.abs(_linear(C, xq, s, wq, sw, None, kind, pad) - y) <= bound)


@pytest.mark.parametrize("M", [1, 40, 300, 600])
def test_extreme_codes_and_longest_sum(M):
    """-128 is a code too; K just below the limit brings the sum next to 2^31 without overflow."""
    C = _lib()
    K, N = (1 << 17) - 16, 32
    xq = np.full((M, K), -128, dtype=np.int8)
    wq = np.full((N, K), -128, dtype=np.int8)
    wq[1::2] = 127
    sx, sw = np.full(M, 2.0 ** -20, np.float32), np.full(N, 0.5, np.float32)
    y, bound = output_bound(xq[:1], sx[:1], wq, sw, None, "fp32")
    assert np.all(np.abs(_linear(C, xq, sx, wq, sw, None, "fp32") - y) <= bound)


@pytest.mark.parametrize("M", [5, 500])
def test_scales_zero_nan_and_infinite(M):
    C = _lib()
    r = np.random.default_rng(5)
    (xq, sx), (wq, sw) = _codes(r, M, 64), _codes(r, 48, 64)
    xq[1], sx[1] = 0, 0.0
    xq[3], sx[3] = 0, np.nan
    wq[7], sw[7] = 0, np.nan
    bias = r.normal(size=48).astype(np.float32)
    got = _linear(C, xq, sx, wq, sw, bias, "fp32")
    ok = np.ones(48, bool)
    ok[7] = False
    assert np.array_equal(got[1, ok], bias[ok].astype(np.float64))
    assert np.isnan(got[3]).all() and np.isnan(got[:, 7]).all()
    rows = [m for m in range(M) if m not in (1, 3)]
    y, bound = output_bound(xq[rows], sx[rows], wq[ok], sw[ok], bias[ok], "fp32")
    assert np.all(np.abs(got[np.ix_(rows, np.where(ok)[0])] - y) <= bound)


@pytest.mark.parametrize("M,K", [(1, 16), (1, 4096), (3, 1040), (7, 48), (40, 2064), (129, 640), (257, 1280), (2, 12288),
                                 (5, 65536 + 16), (1000, 320)])
@pytest.mark.parametrize("kind", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("smooth", [True, False])
def test_quantize_is_bit_exact(M, K, kind, smooth):
    C = _lib()
    r = np.random.default_rng(M + K)
    x = r.normal(size=(M, K)).astype(np.float32)
    x[:, r.integers(0, K, max(1, K // 100))] *= 40
    inv_s = r.uniform(0.1, 3.0, K).astype(np.float32) if smooth else None
    if M > 2:
        x[1] = 0.0
        x[2] *= 2.0 ** -110 if kind != "fp16" else 0.0
    X = torch.full((M, K + 8), 3.0, dtype=TYPES[kind], device="cuda")[:, :K]       # a pitch wider than the row
    X.copy_(_dev(x))
    Xq = torch.empty((M, K), dtype=torch.int8, device="cuda")
    sx = torch.empty(M, dtype=torch.float32, device="cuda")
    C.svdq_quantize_act_i8(X, M, K, None if inv_s is None else _dev(inv_s), Xq, sx)
    q, s = O.quantize_rows(O.smooth(X.float().cpu().numpy(), inv_s))
    assert np.array_equal(sx.cpu().numpy(), s)
    assert np.array_equal(Xq.cpu().numpy(), q)


@pytest.mark.parametrize("K", [64, 1024, 4096])
def test_quantize_non_finite_and_smallest_rows(K):
    C = _lib()
    x = np.random.default_rng(6).normal(size=(8, K)).astype(np.float32)
    x[0, 3], x[1, 0], x[2, K - 1] = np.nan, np.inf, -np.inf
    x[3] = 0
    x[4] *= 2.0 ** -120
    x[5] = 0
    x[5, 1] = 2.0 ** -100
    x[6] = 3.0e38 * np.sign(x[6])
    Xq = torch.empty((8, K), dtype=torch.int8, device="cuda")
    sx = torch.empty(8, dtype=torch.float32, device="cuda")
    C.svdq_quantize_act_i8(_dev(x), 8, K, None, Xq, sx)
    q, s = O.quantize_rows(x)
    assert np.array_equal(sx.cpu().numpy(), s, equal_nan=True) and np.isnan(s[:3]).all()
    assert np.array_equal(Xq.cpu().numpy(), q)


@pytest.mark.parametrize("K,N", [(16, 1), (64, 33), (144, 31), (512, 96), (1040, 100), (4096, 32)])
def test_pack_weight_is_bit_exact(K, N):
    C = _lib()
    r = np.random.default_rng(K + N)
    w = r.normal(size=(K, N)).astype(np.float32)
    if N > 30:
        w[:, 5] = 0
        w[2, 9] = np.inf
        w[:, 11] *= 2.0 ** -115
    Wq = torch.empty((N, K), dtype=torch.int8, device="cuda")
    sw = torch.empty(N, dtype=torch.float32, device="cuda")
    C.svdq_pack_weight_i8(_dev(w), K, N, Wq, sw)
    q, s = O.quantize_rows(np.ascontiguousarray(w.T))
    assert np.array_equal(sw.cpu().numpy(), s, equal_nan=True)
    assert np.array_equal(Wq.cpu().numpy(), q)


def _layer(K, N, seed, bias=True):
    from w4a4_rank_absorbed_b200.calib import calibrate_w8a8
    from w4a4_rank_absorbed_b200.layer import W8A8Linear
    r = np.random.default_rng(seed)
    X = r.normal(size=(64, K))
    X[:, ::37] *= 30
    W = r.normal(0, 0.05, (K, N))
    data = calibrate_w8a8(X, W, bias=r.normal(size=N) if bias else None)
    return data, W8A8Linear(data)


@pytest.mark.parametrize("M,K,N", [(1, 64, 16), (1, 1280, 5120), (9, 2048, 130), (120, 272, 333), (700, 512, 640)])
@pytest.mark.parametrize("kind", ["bf16", "fp16", "fp32"])
def test_layer_is_quantize_then_linear(M, K, N, kind):
    """One call gives what the two give, bit for bit, and the exact sum within the output's bound."""
    data, L = _layer(K, N, M)
    x = np.random.default_rng(M).normal(size=(M, K)).astype(np.float32)
    X = _dev(x, TYPES[kind])
    Y = L(X)
    assert Y.dtype == TYPES[kind] and tuple(Y.shape) == (M, N)
    Xq, sx = L.quantize(X)
    Y2 = L.gemm(Xq, sx, torch.empty_like(Y))
    assert torch.equal(Y, Y2)
    q, s = O.quantize_rows(O.smooth(X.float().cpu().numpy(), data.inv_s.numpy()))
    wq, sw = O.quantize_rows(np.ascontiguousarray(data.W_hat.numpy().T))
    y, bound = output_bound(q, s, wq, sw, data.bias.numpy(), kind)
    assert np.all(np.abs(_host(Y) - y) <= bound)
    Y32 = L.forward(X.reshape(1, M, K), dtype=torch.float32)
    assert tuple(Y32.shape) == (1, M, N)


def test_layer_checkpoint_and_empty_batch():
    from w4a4_rank_absorbed_b200.layer import W8A8Linear
    _, L = _layer(256, 96, 3, bias=False)
    X = torch.randn(5, 256, device="cuda", dtype=torch.bfloat16)
    L2 = W8A8Linear.from_state_dict(L.state_dict())
    assert torch.equal(L(X), L2(X))
    assert tuple(L(X[:0]).shape) == (0, 96)
    with pytest.raises(ValueError):
        L(X.cpu())
    with pytest.raises(ValueError):
        L(X, out=torch.empty(5, 95, device="cuda", dtype=torch.bfloat16))


def test_layer_on_streams_and_in_graphs():
    """Calls on two streams at once, and two captured graphs replayed at once, keep to their own buffers."""
    _, L = _layer(1024, 512, 4)
    g = torch.Generator(device="cuda").manual_seed(1)
    Xs = [torch.randn(n, 1024, device="cuda", generator=g).to(torch.bfloat16) for n in (1, 37, 300, 1)]
    want = [L(X) for X in Xs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in Xs]
    for _ in range(20):
        got = [L.forward(X, stream=s) for X, s in zip(Xs, streams)]
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graphs, outs = [], []
    for X in Xs[:2]:
        G = torch.cuda.CUDAGraph()
        with torch.cuda.graph(G):
            outs.append(L(X))
        graphs.append(G)
    for _ in range(20):
        for G, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                G.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(outs, want))


def test_work_queued_before_and_after_the_layer_is_ordered():
    """The input is written just before the call and overwritten just after it, the weight too: each call sees
    what the stream held at its place."""
    C = _lib()
    M, N, K = 4, 2048, 4096
    g = torch.Generator(device="cuda").manual_seed(2)
    Xa = torch.randn(M, K, device="cuda", generator=g).to(torch.bfloat16)
    Wa = torch.randint(-127, 128, (N, K), device="cuda", generator=g, dtype=torch.int8)
    Wb = torch.randint(-127, 128, (N, K), device="cuda", generator=g, dtype=torch.int8)
    sw = torch.rand(N, device="cuda", generator=g)
    ws = torch.empty(C.svdq_forward_i8_workspace_bytes(M, K), dtype=torch.uint8, device="cuda")

    def call(X, W):
        Y = torch.empty(M, N, device="cuda", dtype=torch.float32)
        C.svdq_forward_i8(X, M, K, None, W, sw, None, Y, N, ws)
        return Y

    want = [call(Xa, Wa).clone(), call(-Xa, Wb).clone()]
    torch.cuda.synchronize()
    X, W = Xa.clone(), Wa.clone()
    for _ in range(30):
        X.copy_(Xa)
        W.copy_(Wa)
        y0 = call(X, W)
        W.copy_(Wb)
        X.neg_()
        y1 = call(X, W)
        assert torch.equal(y0, want[0]) and torch.equal(y1, want[1])


@pytest.mark.parametrize("M,N,K,pad,smooth", [
    (1, 5, 16, 0, True), (1, 128, 144, 8, False), (1, 5120, 1280, 0, True), (2, 1001, 2064, 16, True),
    (1, 4096, 4096, 0, False), (3, 320, 4096, 0, True), (1, 1288, 12288, 0, True), (1, 12288, 4096, 0, True),
    (4, 256, 1280, 8, True), (7, 640, 640, 0, False), (8, 129, 1040, 0, True), (9, 64, 320, 0, True),
    (10, 1280, 320, 0, True), (16, 1280, 256, 0, True), (16, 1280, 320, 0, True), (16, 2048, 1040, 0, True), (17, 320, 320, 0, True), (1, 64, 20480, 0, True)])
@pytest.mark.parametrize("kind", TYPES)
def test_few_tokens_give_the_bits_of_the_two_calls(M, N, K, pad, smooth, kind):
    """The one-call form may quantize inside its GEMM; integers are exact, so its results are the same bits.
    Rows of zeros, of tiny values and (with more than two) one infinity and one NaN are among them."""
    C = _lib()
    g = torch.Generator(device="cuda").manual_seed(M * 1000 + K)
    full = (torch.randn(M, K + pad, device="cuda", generator=g) * 4).to(TYPES[kind])
    X = full[:, :K]
    if M > 2:
        X[1] = 0.0
        X[2, K - 1] = float("inf")
    if M > 3:
        X[3, K // 2] = float("nan")
        X[3, 0] = float("-inf")
    if M > 4:
        X[4] = 2.0 ** -120 if kind != "fp16" else 2.0 ** -24
    inv_s = torch.rand(K, device="cuda", generator=g) + 0.5 if smooth else None
    W = torch.randint(-127, 128, (N, K), device="cuda", generator=g, dtype=torch.int8)
    sw = torch.rand(N, device="cuda", generator=g)
    bias = torch.randn(N, device="cuda", generator=g) if smooth else None
    q = torch.empty(M, K, dtype=torch.int8, device="cuda")
    sx = torch.empty(M, device="cuda")
    want = torch.empty(M, N, device="cuda")
    C.svdq_quantize_act_i8(X, M, K, inv_s, q, sx)
    C.svdq_linear_i8(q, sx, W, sw, bias, want, M, N, K)
    ws = torch.empty(C.svdq_forward_i8_workspace_bytes(M, K), dtype=torch.uint8, device="cuda")
    for ypad in (0, 3):
        out = torch.full((M, N + ypad), 7.0, device="cuda")
        for _ in range(2):
            C.svdq_forward_i8(X, M, K, inv_s, W, sw, bias, out[:, :N], N, ws)
        torch.cuda.synchronize()
        assert C.svdq_get_device_error() == (0, 0)
        assert torch.equal(out[:, :N].nan_to_num(1e30), want.nan_to_num(1e30))
        assert torch.equal(out[:, :N].isnan(), want.isnan())
        assert bool((out[:, N:] == 7.0).all())


def test_output_over_the_input():
    """Y on X's memory: X is read whole before Y is written."""
    C = _lib()
    K = 1280
    g = torch.Generator(device="cuda").manual_seed(5)
    X = torch.randn(2, K, device="cuda", generator=g).to(torch.bfloat16)
    W = torch.randint(-127, 128, (K, K), device="cuda", generator=g, dtype=torch.int8)
    sw = torch.rand(K, device="cuda", generator=g)
    ws = torch.empty(C.svdq_forward_i8_workspace_bytes(2, K), dtype=torch.uint8, device="cuda")
    want = torch.empty_like(X)
    C.svdq_forward_i8(X, 2, K, None, W, sw, None, want, K, ws)
    for _ in range(20):
        Y = X.clone()
        C.svdq_forward_i8(Y, 2, K, None, W, sw, None, Y, K, ws)
        assert torch.equal(Y, want)


def test_rows_that_graphs_and_neighbours_share_with_few_tokens():
    """A chain of one-token layers, each reading the row that the launch before it wrote, in a replayed graph."""
    C = _lib()
    K = 1024
    g = torch.Generator(device="cuda").manual_seed(6)
    W = [torch.randint(-127, 128, (K, K), device="cuda", generator=g, dtype=torch.int8) for _ in range(6)]
    sw = torch.full((K,), 1.0 / (73.0 * 32.0), device="cuda")
    ws = torch.empty(C.svdq_forward_i8_workspace_bytes(1, K), dtype=torch.uint8, device="cuda")
    X = torch.randn(1, K, device="cuda", generator=g).to(torch.bfloat16)
    bufs = [torch.empty(1, K, device="cuda", dtype=torch.bfloat16) for _ in W]

    def chain(sync):
        x = X
        for w, y in zip(W, bufs):
            C.svdq_forward_i8(x, 1, K, None, w, sw, None, y, K, ws)
            if sync:
                torch.cuda.synchronize()
            x = y
        return x

    want = chain(True).clone()
    G = torch.cuda.CUDAGraph()
    with torch.cuda.graph(G):
        chain(False)
    for _ in range(50):
        for b in bufs:
            b.zero_()
        G.replay()
        assert torch.equal(bufs[-1], want)
        assert torch.equal(chain(False), want)


@pytest.mark.parametrize("M", [1, 4, 40, 600])
def test_two_buffers_passed_to_and_fro(M):
    """Layers that write one another's input, launch after launch: each reads what the launch just before it wrote where
    earlier ones had read and written other values."""
    C = _lib()
    K = 1024
    g = torch.Generator(device="cuda").manual_seed(7)
    W = [torch.randint(-127, 128, (K, K), device="cuda", generator=g, dtype=torch.int8) for _ in range(3)]
    sw = torch.full((K,), 1.0 / (73.0 * 32.0), device="cuda")
    ws = torch.empty(C.svdq_forward_i8_workspace_bytes(M, K), dtype=torch.uint8, device="cuda")
    X = torch.randn(M, K, device="cuda", generator=g).to(torch.bfloat16)
    pair = [X.clone(), torch.empty_like(X)]

    def run(sync):
        pair[0].copy_(X)
        for i in range(24):
            C.svdq_forward_i8(pair[i % 2], M, K, None, W[i % 3], sw, None, pair[(i + 1) % 2], K, ws)
            if sync:
                torch.cuda.synchronize()
        return pair[0].clone()

    want = run(True)
    assert bool(want.isfinite().all()) and float(want.abs().max()) > 0
    for _ in range(20):
        assert torch.equal(run(False), want)
    G = torch.cuda.CUDAGraph()
    with torch.cuda.graph(G):
        run(False)
    for _ in range(20):
        G.replay()
        assert torch.equal(pair[0], want)


@pytest.mark.parametrize("M,N,K", [(12964, 390, 1552), (19264, 256, 1072), (12729, 270, 1856), (6169, 494, 1696),
                                   (16384, 1280, 1280), (18999, 1001, 272)])
def test_last_rounds_in_strips(M, N, K):
    """Many tiles with few left for the last round.  Every step is exact or one rounding of binary32, so results are bits:
    the sums are whole numbers below 2^53, and the product of two float32 numbers is exact in float64."""
    C = _lib()
    g = torch.Generator(device="cuda").manual_seed(M)
    q = torch.randint(-127, 128, (M, K), device="cuda", generator=g, dtype=torch.int8)
    W = torch.randint(-127, 128, (N, K), device="cuda", generator=g, dtype=torch.int8)
    sx, sw = torch.rand(M, device="cuda", generator=g), torch.rand(N, device="cuda", generator=g)
    full = torch.full((M, N + 8), 7.0, device="cuda")
    C.svdq_linear_i8(q, sx, W, sw, None, full[:, :N], M, N, K)
    torch.cuda.synchronize()
    assert C.svdq_get_device_error() == (0, 0)
    acc = (q.double() @ W.double().T).float()
    want = ((acc * sx[:, None]).double() * sw.double()[None, :]).float()
    assert torch.equal(full[:, :N], want)
    assert bool((full[:, N:] == 7.0).all())
