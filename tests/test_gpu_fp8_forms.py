"""Every kernel of the 8-bit linear layers and of their weights' gradient, at sizes
that reach it: each number of rows and of weight rows a workgroup, each size of
tile, dense and over a plan, and the workgroups that stay with more tiles than
CUs, ten steps a tile, whole lines and ragged ones.

Which kernel a case reaches is read from the profiler (test_cases_reach_their_kernels),
so that a changed rule cannot drop one.  Results are exact where values are whole and
scales powers of two (sums are multiples of 2^-2 below 2^14), else within 6 standard
deviations of the oracle's error model and half a step of the output's type."""

import re
import zlib

import pytest
import torch

import mixture_experts_ffn_moe_amd as moe
from oracle.fp8 import KAPPA, U

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16}
HALF = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11}
TINY = {"bf16": 2.0 ** -134, "f16": 2.0 ** -25}
KINDS = ("f32", "e8m0")
F8, I32 = torch.float8_e4m3fn, torch.int32
MARK = 1234.0


def up(n, to=128):
    return -(-n // to)


# Dense layers: rows, K, N -> kernel.  rows<NT, MW, KW>: 16 NT rows by 16 MW weight
# rows; tile<BM, BN, TM, KG, D>; stay.
DENSE = [
    (9, 400, 300, "rows<1, 1, 8>"), (16, 400, 16400, "rows<1, 2, 8>"), (5, 272, 32801, "rows<1, 4, 8>"),
    (100, 1168, 500, "rows<1, 1, 8>"),
    (20, 400, 4100, "rows<2, 1, 8>"), (32, 400, 16410, "rows<2, 2, 8>"), (17, 272, 32768, "rows<2, 4, 4>"),
    (200, 1168, 520, "tile<64, 64, 16, 2, 3>"), (1100, 1168, 1701, "tile<64, 128, 32, 2, 3>"),
    (1900, 1168, 2100, "tile<128, 128, 64, 2, 2>"), (2500, 1168, 3000, "tile<128, 128, 32, 1, 2>"),
    (4608, 1280, 4608, "stay"), (4500, 1168, 4600, "stay"), (4609, 1168, 4601, "stay"), (256, 1040, 70000, "stay"),
]
# Over a plan: blocks' experts drawn from E (one elsewhere), block_m, K, N.
PLAN = [
    (5, 3, 16, 400, 300, "rows<1, 1, 8>"), (33, 6, 16, 400, 520, "rows<1, 2, 8>"), (65, 9, 16, 400, 500, "rows<1, 4, 8>"),
    (5, 3, 32, 400, 300, "rows<2, 1, 8>"), (33, 6, 32, 400, 520, "rows<2, 2, 8>"), (65, 9, 32, 272, 500, "rows<2, 4, 4>"),
    (7, 3, 64, 1168, 520, "tile<64, 64, 16, 2, 3>"), (40, 3, 64, 400, 700, "tile<64, 128, 32, 2, 3>"),
    (60, 5, 64, 1168, 777, "tile<64, 128, 32, 1, 2>"),
    (4, 2, 128, 1168, 520, "tile<64, 64, 16, 2, 3>"), (9, 3, 128, 400, 1600, "tile<64, 128, 32, 2, 3>"),
    (20, 3, 128, 1168, 1500, "tile<128, 128, 64, 2, 2>"), (24, 3, 128, 1168, 2600, "tile<128, 128, 32, 1, 2>"),
    (45, 4, 128, 1280, 4608, "stay"), (45, 4, 128, 1168, 4601, "stay"), (700, 9, 128, 1168, 264, "stay"), (2100, 9, 128, 656, 264, "stay"),
    (2, 2, 256, 1168, 520, "tile<64, 64, 16, 2, 3>"), (5, 3, 256, 400, 1800, "tile<64, 128, 32, 2, 3>"),
    (10, 3, 256, 1168, 1600, "tile<128, 128, 64, 2, 2>"), (12, 3, 256, 1168, 2400, "tile<128, 128, 32, 1, 2>"),
    (22, 4, 256, 1280, 4608, "stay"), (22, 4, 256, 1168, 4601, "stay"),
]
# Weights' gradients: rows, N, K -> kernel.
DW = [
    (1280, 500, 520, "tile<64, 64, 16, 2, 3>"), (1280, 1100, 1701, "tile<64, 128, 32, 2, 3>"),
    (1280, 1900, 2100, "tile<128, 128, 64, 2, 2>"), (1280, 2500, 3000, "tile<128, 128, 32, 1, 2>"),
    (1280, 4608, 4608, "stay"), (1152, 4500, 4600, "stay"), (1280, 4609, 4601, "stay"),
]
# Over a plan: blocks, experts, block_m, N, K.
DW_PLAN = [
    (20, 3, 128, 300, 400, "tile<64, 64, 16, 2, 3>"), (20, 3, 128, 500, 1200, "tile<64, 128, 32, 2, 3>"),
    (20, 3, 128, 900, 1200, "tile<128, 128, 64, 2, 2>"), (20, 3, 128, 1500, 1500, "tile<128, 128, 32, 1, 2>"),
    (40, 4, 128, 2304, 2304, "stay"), (40, 4, 128, 2300, 2305, "stay"), (15, 3, 256, 2500, 2504, "stay"),
    (30, 40, 128, 700, 1000, "stay"), (300, 1024, 128, 32, 48, "stay"),
]


def seed(*parts):
    g = torch.Generator(device="cuda")
    g.manual_seed(zlib.crc32(repr(parts).encode()))
    return g


def operand(shape, scales, kind, g, exact):
    """(codes, scales, fp64 values of the scales)."""
    if exact:
        q = torch.randint(-2, 3, shape, generator=g, device="cuda").float()
        e = torch.randint(-1, 2, scales, generator=g, device="cuda")
    else:
        q = (torch.randn(shape, generator=g, device="cuda") * 100).clamp(-448, 448)
        e = torch.randint(-9, -6, scales, generator=g, device="cuda")
    v = torch.exp2(e.double())
    if kind == "f32" and not exact:
        v = (v * (1 + torch.rand(scales, generator=g, device="cuda").double())).float().double()
    return q.to(F8), v.float() if kind == "f32" else (e + 127).to(torch.uint8), v


def rows_of(q, v):
    """Values of rows with a scale for each 128."""
    return q.double() * v.repeat_interleave(128, -1)[..., :q.shape[-1]]


def blocks_of(q, v):
    return q.double() * v.repeat_interleave(128, -2)[..., :q.shape[-2], :].repeat_interleave(128, -1)[..., :q.shape[-1]]


def close(out, x, w, elem, exact):
    """out against x @ w.T of fp64 values."""
    y = x @ w.T.contiguous()
    if exact:
        assert float(y.abs().max()) < 2 ** 14
        assert torch.equal(out, y.to(TYPES[elem]))
        return
    norm2 = (x * x) @ (w * w).T.contiguous()
    add = U * (up(x.shape[1]) + 2) ** 0.5 * (y.abs() + 3 * norm2.sqrt())
    sigma = (KAPPA ** 2 * norm2 + add * add).sqrt()
    off = (out.double() - y).abs()
    assert bool((off <= HALF[elem] * y.abs() + TINY[elem] + 6 * sigma * (1 + HALF[elem])).all())
    assert float(off.norm()) <= HALF[elem] * float(y.norm())


# ---- the calls: inputs, the call itself, and its comparison -------------------------

def dense(case, kind, elem, exact):
    M, K, N, _ = case
    g = seed("dense", *case[:3], kind, exact)
    x, w = operand((M, K), (M, up(K)), kind, g, exact), operand((N, K), (up(N), up(K)), kind, g, exact)
    out = torch.full((M, N), MARK, dtype=TYPES[elem], device="cuda")

    def call():
        moe.moe_fp8_linear(x[0], x[1], w[0][None], w[1][None], out=out)

    def compare():
        close(out, rows_of(x[0], x[2]), blocks_of(w[0], w[2]), elem, exact)
    return call, compare


def block_experts(n, E, g):
    """Experts of n blocks in runs, as the planner lays them out; the first run is elsewhere."""
    cut = torch.randint(1, n + 1, (E,), generator=g, device="cuda").sort()[0]
    return (torch.searchsorted(cut, torch.arange(n, device="cuda"), right=True) - 1).to(I32)


def plan(case, kind, elem, exact):
    n, E, bm, K, N, _ = case
    g = seed("plan", *case[:5], kind, exact)
    ids, M = block_experts(n, E, g), n * bm
    used = M - bm // 2 + 3 if bm >= 64 else M - 5
    ntp = torch.tensor([used], dtype=I32, device="cuda")
    x, w = operand((M, K), (M, up(K)), kind, g, exact), operand((E, N, K), (E, up(N), up(K)), kind, g, exact)
    x[0].view(torch.uint8)[used:] = 0x7F  # NaN: neither read nor written
    out = torch.full((M, N), MARK, dtype=TYPES[elem], device="cuda")

    def call():
        moe.moe_fp8_linear(x[0], x[1], w[0], w[1], ids, ntp, bm, out=out)

    def compare():
        assert bool((out[used:] == MARK).all())
        of, values = ids.repeat_interleave(bm)[:used], rows_of(x[0], x[2])
        for e in range(-1, E):
            at = (of == e).nonzero()[:, 0]
            if not len(at):
                continue
            if e < 0:
                assert not out[at].any()
            else:
                close(out[at], values[at], blocks_of(w[0][e], w[2][e]), elem, exact)
    return call, compare


def dw(case, kind, elem, exact):
    M, N, K, _ = case
    g = seed("dw", *case[:3], kind, exact)
    dy, x = operand((N, M), (N, M // 128), kind, g, exact), operand((K, M), (K, M // 128), kind, g, exact)
    out = torch.full((1, N, K), MARK, dtype=TYPES[elem], device="cuda")

    def call():
        moe.moe_fp8_linear_dw(dy[0], dy[1], x[0], x[1], out=out)

    def compare():
        close(out[0], rows_of(dy[0], dy[2]), rows_of(x[0], x[2]), elem, exact)
    return call, compare


def dw_plan(case, kind, elem, exact):
    n, E, bm, N, K, _ = case
    g = seed("dw_plan", *case[:5], kind, exact)
    ids, M = block_experts(n, E, g), n * bm
    used = M - bm  # the last block is not in use
    ntp = torch.tensor([used], dtype=I32, device="cuda")
    dy, x = operand((N, M), (N, M // 128), kind, g, exact), operand((K, M), (K, M // 128), kind, g, exact)
    dy[0].view(torch.uint8)[:, used:] = 0x7F  # NaN: not read
    x[0].view(torch.uint8)[:, used:] = 0x7F
    out = torch.full((E, N, K), MARK, dtype=TYPES[elem], device="cuda")

    def call():
        moe.moe_fp8_linear_dw(dy[0], dy[1], x[0], x[1], E, ids, ntp, bm, out=out)

    def compare():
        a, b, of = rows_of(dy[0], dy[2]), rows_of(x[0], x[2]), ids.repeat_interleave(bm)[:used]
        for e in range(E):
            at = (of == e).nonzero()[:, 0]
            if len(at):
                close(out[e], a[:, at], b[:, at], elem, exact)
            else:
                assert not out[e].any()
    return call, compare


ALL = [(f, c) for f, cases in ((dense, DENSE), (plan, PLAN), (dw, DW), (dw_plan, DW_PLAN)) for c in cases]


def name_of(p):
    return "-".join(str(v) for v in (p[0].__name__, *p[1][:-1], re.sub("[ ,]+", ".", p[1][-1])))


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("what", ALL, ids=name_of)
def test_results(what, kind):
    make, case = what
    for elem, exact in (("bf16", True), ("f16", True), ("bf16", False)):
        call, compare = make(case, kind, elem, exact)
        call()
        compare()


def test_cases_reach_their_kernels():
    from torch.profiler import ProfilerActivity, profile

    calls = [(make(case, "f32", "bf16", True)[0], make, case) for make, case in ALL]
    torch.cuda.synchronize()
    with profile(activities=[ProfilerActivity.CUDA]) as p:
        for call, _, _ in calls:
            call()
        torch.cuda.synchronize()
    ran = [e for e in p.events() if "k_fp8_" in e.name]
    if not p.events():
        pytest.skip("the profiler sees no kernels here")
    ran.sort(key=lambda e: e.time_range.start)
    assert len(ran) == len(calls)
    for e, (_, make, case) in zip(ran, calls):
        form, args = re.search(r"k_fp8_(\w+)<([^>]*)>", e.name).groups()
        args = args.split(", ")[2:]  # behind the output's and the scales' types
        if form != "rows":
            kinds = {dense: ["false", "false"], plan: ["false", "true"], dw: ["true", "false"], dw_plan: ["true", "true"]}
            assert args[:2] == kinds[make], (name_of((make, case)), e.name)
            args = args[2:]
        assert (f"{form}<{', '.join(args)}>" if args else form) == case[-1], (name_of((make, case)), e.name)
