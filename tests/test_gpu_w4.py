"""GPU parity of the products with 4-bit weights (moe_w4_matvec, fused_moe_w4)
against the fp64 oracle (oracle/w4.py).

Two gates.  Exact: whole activations of at most 8, scales that are powers of
two; every sum is a whole multiple of a power of two below 2^24, so the result
is the exact one, rounded once.  Random: each element within 6 standard
deviations of the oracle's error model plus the type's half step; and the whole
within the half step in the 2-norm (a rounding is off by 0.58 of it at most on
average, the fp32 sums by far less).
"""

import numpy as np
import pytest
import torch

import mixture_experts_ffn_moe_amd as moe
from oracle import w4

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16}
TINY = {"bf16": 2.0 ** -134, "f16": 2.0 ** -25}
FORMATS = [("int4", 32, False), ("int4", 32, True), ("int4", 64, True), ("int4", 128, False),
           ("int4", 128, True), ("int4", 0, True), ("mx", 32, False)]
FMT_IDS = [f"{f}-g{g}{'-z' if z else ''}" for f, g, z in FORMATS]


def weights(fmt, group, zeros, E, N, K, elem, rng, exact=False):
    """(codes, scales, zeros) on the host as numpy, and on the GPU."""
    w = rng.integers(0, 256, (E, N, K // 2), dtype=np.uint8)
    n = K // group if group else 1
    if fmt == "mx":
        s = rng.integers(119, 124, (E, N, n), dtype=np.uint8)
        dev = torch.from_numpy(s).cuda()
    else:
        v = 2.0 ** rng.integers(-7, -4, (E, N, n)) if exact else rng.uniform(0.3, 1.5, (E, N, n)) / (5 * K ** 0.5)
        dev = torch.from_numpy(v).to(TYPES[elem]).cuda()
        s = dev.double().cpu().numpy()
    z = rng.integers(0, 16, (E, N, n), dtype=np.uint8) if zeros else None
    return (w, s, z), (torch.from_numpy(w).cuda(), dev, None if z is None else torch.from_numpy(z).cuda())


def activations(shape, elem, rng, exact=False):
    v = rng.integers(-8, 9, shape).astype(np.float64) if exact else rng.normal(size=shape)
    t = torch.from_numpy(v).to(TYPES[elem]).cuda()
    return t.double().cpu().numpy(), t


def parts(elem):
    return 1 if elem == "bf16" else 2


def reference(fmt, W, group, x, ids, swiglu, elem, per_route):
    """(y, sigma) of every route."""
    T, k = ids.shape
    E, N = W[0].shape[:2]
    K = x.shape[-1]
    n = N // 2 if swiglu else N
    y, s = np.zeros((T, k, n)), np.zeros((T, k, n))
    for t in range(T):
        for j in range(k):
            e = int(ids[t, j])
            if 0 <= e < E:
                one = [None if v is None else v[e] for v in W]
                a, b = w4.product(fmt, *one, group or K, x[t, j] if per_route else x[t], parts(elem))
                if swiglu:
                    a, b = w4.silu_mul((a[:n], b[:n]), (a[n:], b[n:]))
                y[t, j], s[t, j] = a, b
    return y, s


def rounded(v, elem):
    return torch.from_numpy(v).to(TYPES[elem]).double().numpy()


def check(got, ref, sigma, elem, what):
    got = got.double().cpu().numpy()
    u = torch.finfo(TYPES[elem]).eps / 2
    dev = 6 * sigma
    bad = ~(np.abs(got - ref) <= dev + u * (np.abs(ref) + dev) + TINY[elem])
    assert not bad.any(), (what, int(bad.sum()), float(np.nanmax(np.abs(got - ref))))
    norm = np.linalg.norm(ref)
    if elem == "bf16" or norm > 0.1 * np.sqrt(ref.size):
        assert np.linalg.norm(got - ref) <= u * norm + TINY[elem] * np.sqrt(ref.size), what


# T, K, N, E, top_k; E past the routes and below them; odd N, short and ragged K
SHAPES = [(1, 128, 16, 1, 1), (1, 4096, 48, 9, 6), (3, 384, 33, 4, 2), (7, 1152, 20, 2, 2),
          (40, 256, 18, 3, 2), (2, 2176, 1, 5, 3)]


@pytest.mark.parametrize("elem", list(TYPES))
@pytest.mark.parametrize("fmt,group,zeros", FORMATS, ids=FMT_IDS)
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_matvec(shape, fmt, group, zeros, elem):
    T, K, N, E, k = shape
    rng = np.random.default_rng(T * K + N)
    W, D = weights(fmt, group, zeros, E, N, K, elem, rng)
    # some routes elsewhere, some experts twice in a token
    ids = rng.integers(-1, E + 1, (T, k)).astype(np.int32)
    x, X = activations((T, K), elem, rng)
    out = torch.full((T, k, N), float("nan"), dtype=TYPES[elem], device="cuda")
    got = moe.moe_w4_matvec(fmt, X, *D, torch.from_numpy(ids).cuda(), group, out=out)
    y, s = reference(fmt, W, group, x, ids, False, elem, False)
    check(got, y, s, elem, "product")
    xr, XR = activations((T, k, K), elem, rng)
    got = moe.moe_w4_matvec(fmt, XR, *D, torch.from_numpy(ids).cuda(), group)
    y, s = reference(fmt, W, group, xr, ids, False, elem, True)
    check(got, y, s, elem, "product, a vector per route")


@pytest.mark.parametrize("elem", list(TYPES))
@pytest.mark.parametrize("fmt,group,zeros", FORMATS, ids=FMT_IDS)
@pytest.mark.parametrize("shape", [(1, 128, 2, 1, 1), (5, 640, 70, 6, 2), (19, 2048, 34, 2, 1)], ids=str)
def test_matvec_swiglu(shape, fmt, group, zeros, elem):
    T, K, N, E, k = shape
    rng = np.random.default_rng(T + K)
    W, D = weights(fmt, group, zeros, E, N, K, elem, rng)
    ids = rng.integers(0, E + 1, (T, k)).astype(np.int32)
    x, X = activations((T, K), elem, rng)
    out = torch.full((T, k, N // 2), float("nan"), dtype=TYPES[elem], device="cuda")
    got = moe.moe_w4_matvec(fmt, X, *D, torch.from_numpy(ids).cuda(), group, swiglu=True, out=out)
    y, s = reference(fmt, W, group, x, ids, True, elem, False)
    check(got, y, s, elem, "swiglu")


@pytest.mark.parametrize("elem", list(TYPES))
@pytest.mark.parametrize("fmt,group,zeros", FORMATS, ids=FMT_IDS)
@pytest.mark.parametrize("T,K,N", [(1, 128, 16), (4, 3200, 40), (16, 1024, 31), (17, 4224, 16), (37, 256, 100)])
def test_linear_exact(T, K, N, fmt, group, zeros, elem):
    """No routing, and exact arithmetic: the result is the exact one rounded."""
    rng = np.random.default_rng(T + K + N)
    W, D = weights(fmt, group, zeros, 1, N, K, elem, rng, exact=True)
    x, X = activations((T, K), elem, rng, exact=True)
    got = moe.moe_w4_matvec(fmt, X, *D, None, group).double().cpu().numpy()
    d = w4.dequant(fmt, *[None if v is None else v[0] for v in W], group or K)
    assert np.array_equal(got, rounded(x @ d.T, elem))


@pytest.mark.parametrize("K", [32, 96, 160, 1056, 4128])
@pytest.mark.parametrize("fmt,group", [("int4", 32), ("mx", 32)])
def test_ragged_contraction(K, fmt, group):
    """A contraction that ends inside a step; what lies behind a row (the next
    row's codes and scales, NaN scales among them) is not seen."""
    rng = np.random.default_rng(K)
    N = 24
    W, D = weights(fmt, group, fmt == "int4", 2, N, K, "bf16", rng, exact=True)
    if fmt == "mx":
        W[1][1], D[1][1] = 255, 255
    else:
        D[1][1] = float("nan")
    x, X = activations((3, K), "bf16", rng, exact=True)
    ids = torch.zeros(3, 1, dtype=torch.int32, device="cuda")
    got = moe.moe_w4_matvec(fmt, X, *D, ids, group).double().cpu().numpy()
    d = w4.dequant(fmt, *[None if v is None else v[0] for v in W], group)
    assert np.array_equal(got[:, 0], rounded(x @ d.T, "bf16"))
    # every other row with NaN scales: each row sees its own
    for row in (0, N - 1):
        D2 = [None if v is None else v.clone() for v in D]
        D2[1][0, row] = 255 if fmt == "mx" else float("nan")
        alone = moe.moe_w4_matvec(fmt, X, *D2, ids, group).double().cpu().numpy()
        assert np.isnan(alone[:, 0, row]).all()
        keep = np.arange(N) != row
        assert np.array_equal(alone[:, 0, keep], got[:, 0, keep])


def test_scale_range():
    """e8m0 scales over their range, fp16 activations: no overflow on the way."""
    K, N = 64, 16
    codes = torch.full((1, N, K // 2), 0x22, dtype=torch.uint8)        # every weight 1
    scale = torch.zeros(1, N, 2, dtype=torch.uint8)
    exps = [0, 1, 2, 60, 100, 126, 127, 128, 140, 200, 240, 250, 252, 253, 126, 125]
    scale[0, :, 0] = torch.tensor(exps, dtype=torch.uint8)
    x = torch.zeros(1, K, dtype=torch.float16)
    x[0, 3] = 1.0
    got = moe.moe_w4_matvec("mx", x.bfloat16().cuda(), codes.cuda(), scale.cuda(), None, None, 32)
    want = torch.tensor([2.0 ** (e - 127) for e in exps], dtype=torch.float64)
    normal = want >= 2.0 ** -126                 # the accumulator's smallest normal
    assert torch.equal(got[0].double().cpu()[normal], want[normal])
    assert bool((got[0].double().cpu()[~normal] <= 2.0 ** -126).all())
    got = moe.moe_w4_matvec("mx", x.cuda(), codes.cuda(), scale.cuda(), None, None, 32)
    assert torch.equal(got[0].cpu(), want.to(torch.float16))
    scale[0, 0, 0] = 255
    got = moe.moe_w4_matvec("mx", x.bfloat16().cuda(), codes.cuda(), scale.cuda(), None, None, 32)
    assert bool(got[0, 0].isnan()) and bool(got[0, 1:].isfinite().all())


def test_one_token_is_not_another():
    """A NaN token leaves the others alone; a route elsewhere is zeros."""
    rng = np.random.default_rng(8)
    W, D = weights("int4", 128, True, 2, 40, 512, "bf16", rng)
    x, X = activations((20, 512), "bf16", rng)
    ids = torch.zeros(20, 1, dtype=torch.int32, device="cuda")
    ids[5] = 7
    clean = moe.moe_w4_matvec("int4", X, *D, ids, 128)
    X[3, 100], X[9, 7] = float("nan"), float("inf")
    got = moe.moe_w4_matvec("int4", X, *D, ids, 128)
    assert bool(got[3].isnan().all()) and not bool(got[9].isfinite().any())
    keep = [t for t in range(20) if t not in (3, 9)]
    assert torch.equal(got[keep], clean[keep]) and not bool(got[5].any())


FFN = [(1, 128, 128, 4, 1), (1, 512, 256, 16, 6), (6, 640, 128, 4, 3), (33, 256, 384, 3, 2)]


@pytest.mark.parametrize("elem", list(TYPES))
@pytest.mark.parametrize("fmt,group,zeros", FORMATS, ids=FMT_IDS)
@pytest.mark.parametrize("shape", FFN, ids=str)
def test_ffn(shape, fmt, group, zeros, elem):
    T, K, I, E, k = shape
    rng = np.random.default_rng(T + K + I)
    W1, D1 = weights(fmt, group, zeros, E, 2 * I, K, elem, rng)
    W2, D2 = weights(fmt, group, zeros, E, K, I, elem, rng)
    x, X = activations((T, K), elem, rng)
    ids = rng.integers(0, E + 1, (T, k)).astype(np.int32)
    ids[0, 0] = 0
    w = rng.random((T, k)).astype(np.float32)
    w[ids == E] = np.nan                     # behind a route elsewhere: not seen
    out = torch.full((T, K), float("nan"), dtype=TYPES[elem], device="cuda")
    ws = torch.full((moe.moe_w4_workspace_size(T, K, 2 * I, k),), 0xFF, dtype=torch.uint8, device="cuda")
    got = moe.fused_moe_w4(fmt, X, *D1, *D2, torch.from_numpy(ids).cuda(), torch.from_numpy(w).cuda(), group,
                           out=out, workspace=ws)
    ref, sigma = w4.ffn(fmt, W1, W2, group, x, ids, w, parts(elem))
    check(got, ref, sigma, elem, "ffn")
    again = moe.fused_moe_w4(fmt, X, *D1, *D2, torch.from_numpy(ids).cuda(), torch.from_numpy(w).cuda(), group)
    assert torch.equal(got, again)


def test_empty():
    for elem in TYPES.values():
        W = [torch.zeros(2, 64, 64, dtype=torch.uint8, device="cuda"),
             torch.ones(2, 64, 1, dtype=elem, device="cuda"), None]
        x = torch.empty(0, 128, dtype=elem, device="cuda")
        ids = torch.empty(0, 3, dtype=torch.int32, device="cuda")
        assert moe.moe_w4_matvec("int4", x, *W, ids, 0).shape == (0, 3, 64)
    W1 = [torch.zeros(2, 256, 64, dtype=torch.uint8, device="cuda"),
          torch.ones(2, 256, 1, dtype=torch.float16, device="cuda"), None]
    W2 = [torch.zeros(2, 128, 64, dtype=torch.uint8, device="cuda"),
          torch.ones(2, 128, 1, dtype=torch.float16, device="cuda"), None]
    assert moe.fused_moe_w4("int4", x, *W1, *W2, ids, torch.empty(0, 3, device="cuda"), 128).shape == (0, 128)


def test_most_routes():
    """4,096 routes in one call: the most it takes, many passes per expert."""
    rng = np.random.default_rng(9)
    T, k, K, N, E = 1024, 4, 128, 16, 3
    W, D = weights("int4", 128, True, E, N, K, "bf16", rng, exact=True)
    x, X = activations((T, K), "bf16", rng, exact=True)
    ids = rng.integers(-1, E + 1, (T, k)).astype(np.int32)
    got = moe.moe_w4_matvec("int4", X, *D, torch.from_numpy(ids).cuda(), 128).double().cpu().numpy()
    d = np.stack([w4.dequant("int4", *[v[e] for v in W], 128) for e in range(E)])
    want = np.einsum("tk,enk->ten", x, d)
    for e in range(-1, E + 1):
        t, j = np.nonzero(ids == e)
        ref = rounded(want[t, e], "bf16") if 0 <= e < E else np.zeros((len(t), N))
        assert np.array_equal(got[t, j], ref)


def test_decode_run_with_the_router():
    """A decode step as it is served: the router's ids and weights go straight
    into the FFN; the parts alone (products in route order, the weighted sum)
    give the same up to the rounding of the rows."""
    rng = np.random.default_rng(10)
    T, K, I, E, k = 5, 256, 128, 16, 4
    W1, D1 = weights("int4", 64, True, E, 2 * I, K, "bf16", rng)
    W2, D2 = weights("int4", 64, True, E, K, I, "bf16", rng)
    x, X = activations((T, K), "bf16", rng)
    logits = torch.from_numpy(rng.normal(size=(T, E)).astype(np.float32)).cuda()
    ids, w, *_ = moe.moe_route_align(logits, k, 16)
    out = moe.fused_moe_w4("int4", X, *D1, *D2, ids, w, 64)
    ref, sigma = w4.ffn("int4", W1, W2, 64, x, ids.cpu().numpy(), w.double().cpu().numpy(), 1)
    check(out, ref, sigma, "bf16", "router and ffn")
    h = moe.moe_w4_matvec("int4", X, *D1, ids, 64, swiglu=True)
    y = moe.moe_w4_matvec("int4", h, *D2, ids, 64)
    parts_out = moe.moe_unpermute(y.reshape(T * k, K), None, w, k)
    # h, the rows and the sum are rounded to bf16 here: three half steps, each
    # of a value or of a sum of terms no larger than the rows' magnitudes
    size = (w[:, :, None] * y.float().abs()).sum(1).double().cpu().numpy()
    err = np.abs(parts_out.double().cpu().numpy() - ref)
    rms = np.sqrt((ref ** 2).mean())
    assert (err <= 6 * sigma + 2.0 ** -8 * (2 * size + 8 * rms)).all()


def test_graph_and_streams():
    """Captured and replayed with new tokens and routing, and on a stream."""
    rng = np.random.default_rng(11)
    T, K, I, E, k = 3, 512, 128, 8, 2
    _, D1 = weights("mx", 32, False, E, 2 * I, K, "bf16", rng)
    _, D2 = weights("mx", 32, False, E, K, I, "bf16", rng)
    x = torch.zeros(T, K, dtype=torch.bfloat16, device="cuda")
    ids = torch.zeros(T, k, dtype=torch.int32, device="cuda")
    w = torch.full((T, k), 0.5, device="cuda")
    out = torch.empty(T, K, dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(moe.moe_w4_workspace_size(T, K, 2 * I, k), dtype=torch.uint8, device="cuda")

    def step(stream=None):
        return moe.fused_moe_w4("mx", x, *D1, *D2, ids, w, 32, out=out, workspace=ws, stream=stream)

    def fill(seed):
        g = torch.Generator().manual_seed(seed)
        x.copy_(torch.randn(T, K, generator=g))
        ids.copy_(torch.randint(-1, E, (T, k), generator=g))

    fill(0)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    step(side)
    torch.cuda.synchronize()
    first = out.clone()
    assert torch.equal(step(), first)
    fresh = moe.fused_moe_w4("mx", x, *D1, *D2, ids, w, 32, stream=side)   # its own buffers
    torch.cuda.synchronize()
    assert torch.equal(fresh, first)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for seed in (1, 2, 3):
        fill(seed)
        eager = step().clone()
        out.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, eager), seed
