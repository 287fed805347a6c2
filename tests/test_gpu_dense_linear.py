"""The dense linear (bias, activation, residual in the epilogue) and its backward against the fp64 oracle,
within first-order rounding bounds (block_bounds.py)."""
import pytest
import torch

import block_bounds as BB
from oracle import block as OB
from tolerances import assert_within_bound

pytestmark = pytest.mark.gpu
BF, F32, F64 = torch.bfloat16, torch.float32, torch.float64
ACTS = ("none", "relu", "gelu", "gelu_tanh", "silu")

# (M, N, K): one row, every tile width of the split kernel, its contraction splits, ragged edges in each
# direction, contractions shorter than one block, more tiles than SMs
SHAPES = [(1, 8, 8), (1, 4096, 4096), (1, 72, 2056), (1, 1000, 264), (1, 264, 8200), (2, 576, 1536), (16, 136, 72), (17, 1536, 576), (33, 640, 2048), (64, 128, 64),
          (65, 264, 520), (127, 1000, 136), (128, 128, 128), (129, 136, 1032), (333, 1536, 576), (300, 64, 8),
          (200, 2304, 8200), (1000, 1160, 328), (2100, 2048, 200), (4000, 16, 72)]
# with the shapes above, every tile and split of both forms, in the forward and in each gradient (148 SMs)
TILES = [(2177, 2136, 8), (17, 920, 2400), (1341, 4792, 16), (34, 3944, 1008), (2680, 1032, 1968), (795, 8, 672),
         (522, 8, 3936), (1051, 8, 2832), (2643, 8, 2928), (335, 2392, 784), (97, 1456, 4768), (265, 2480, 4792)]


def _inputs(M, N, K, seed=0):
    g = torch.Generator().manual_seed(M + 3 * N + 7 * K + seed)

    def n(*s, std=1.0):
        return (std * torch.randn(*s, generator=g)).to(BF).cuda()
    return {"x": n(M, K), "w": n(N, K, std=0.5 * K ** -0.5), "b": n(N, std=0.3), "res": n(M, N), "dy": n(M, N),
            "z": n(M, N, std=1.5)}


def _check(got, ref_bound, what, rel=5e-3):
    ref, bound = ref_bound
    assert_within_bound(got.double().cpu(), ref.cpu(), bound.cpu() + 2.0 ** -126, rel=rel, what=what)


def _d(t):
    return None if t is None else t.double()


@pytest.mark.parametrize("M,N,K", SHAPES + TILES)
def test_forward(lsq, M, N, K):
    t = _inputs(M, N, K)
    for i, (bias, res, keep) in enumerate([(True, True, True), (False, False, False), (True, False, True),
                                           (False, True, False), (True, True, False)]):
        kind = ACTS[(i + M) % 5]
        b, r = t["b"] if bias else None, t["res"] if res else None
        y = torch.empty(M, N, dtype=BF, device="cuda")
        z = torch.empty_like(y) if keep else None
        lsq.lsq_linear_fwd(t["x"], t["w"], b, ACTS.index(kind), r, z, y, M, N, K)
        want = BB.linear_fwd(_d(t["x"]), _d(t["w"]), _d(b), kind, _d(r))
        _check(y, want["y"], f"linear y {kind}")
        if keep:
            _check(z, want["z"], f"linear z {kind}")


@pytest.mark.parametrize("kind", ACTS)
def test_forward_in_place_residual_and_repeat(lsq, kind):
    M, N, K = 150, 328, 712
    t = _inputs(M, N, K, 1)
    y = torch.empty(M, N, dtype=BF, device="cuda")
    lsq.lsq_linear_fwd(t["x"], t["w"], t["b"], ACTS.index(kind), t["res"], None, y, M, N, K)
    h = t["res"].clone()
    lsq.lsq_linear_fwd(t["x"], t["w"], t["b"], ACTS.index(kind), h, None, h, M, N, K)
    assert torch.equal(h, y)


@pytest.mark.parametrize("M,N,K", SHAPES + TILES)
def test_backward(lsq, M, N, K):
    t = _inputs(M, N, K, 2)
    for i in range(2):
        kind = ACTS[(i * 2 + N // 8 + M) % 5]
        act = ACTS.index(kind)
        z = t["z"] if kind != "none" else None
        ws = torch.empty(lsq.lsq_linear_bwd_workspace_size(M, N, K, act), dtype=torch.uint8, device="cuda")
        dx = torch.empty(M, K, dtype=BF, device="cuda")
        dw = torch.empty(N, K, dtype=F32 if i else BF, device="cuda")
        db = torch.empty(N, dtype=F32, device="cuda")
        lsq.lsq_linear_bwd(t["dy"], t["x"], t["w"], z, act, dx, dw, i, db, 0, M, N, K, ws)
        want = BB.linear_bwd(_d(t["dy"]), _d(t["x"]), _d(t["w"]), _d(t["z"]), kind, M + 32, dw_f32=bool(i))
        # dz is rounded once before the two products: with few terms that alone is up to 2^-8 of the result,
        # and the result's own rounding another 2^-8
        for name, got in (("dx", dx), ("dw", dw), ("db", db)):
            _check(got, want[name], f"linear {name} {kind}", rel=8e-3)


@pytest.mark.parametrize("kind", ACTS)
def test_backward_parts_and_accumulation(lsq, kind):
    """Each gradient alone equals the whole call's, bit for bit; fp32 gradients accumulate."""
    M, N, K = 90, 200, 456
    act = ACTS.index(kind)
    t = _inputs(M, N, K, 3)
    z = t["z"] if kind != "none" else None
    ws = torch.empty(lsq.lsq_linear_bwd_workspace_size(M, N, K, act), dtype=torch.uint8, device="cuda")
    dx, dw, db = (torch.empty(M, K, dtype=BF, device="cuda"), torch.empty(N, K, dtype=F32, device="cuda"),
                  torch.empty(N, dtype=F32, device="cuda"))
    lsq.lsq_linear_bwd(t["dy"], t["x"], t["w"], z, act, dx, dw, 1, db, 0, M, N, K, ws)
    dx1, dw1, db1 = torch.empty_like(dx), torch.full_like(dw, 0.5), torch.full_like(db, 0.5)
    none_ws = None if kind == "none" else ws
    lsq.lsq_linear_bwd(t["dy"], None, t["w"], z, act, dx1, None, 0, None, 0, M, N, K, none_ws)
    lsq.lsq_linear_bwd(t["dy"], t["x"], None, z, act, None, dw1, 1, None, 1, M, N, K, none_ws)
    lsq.lsq_linear_bwd(t["dy"], None, None, z, act, None, None, 0, db1, 1, M, N, K, ws)
    assert torch.equal(dx, dx1) and torch.equal(dw + 0.5, dw1) and torch.equal(db + 0.5, db1)
    dwb = torch.empty(N, K, dtype=BF, device="cuda")
    lsq.lsq_linear_bwd(t["dy"], t["x"], None, z, act, None, dwb, 0, None, 0, M, N, K, none_ws)
    assert torch.equal(dwb, dw.to(BF))     # the same sums, rounded once


@pytest.mark.parametrize("M,N,K", [(70, 2048, 4096), (2177, 2136, 264), (700, 72, 136)])
def test_fp32_weight_gradient_accumulates_in_either_form(lsq, M, N, K):
    """Two accumulating calls on top of a start: one fp32 addition an element and call, in the calls' order."""
    t, u = _inputs(M, N, K, 6), _inputs(M, N, K, 7)
    one, two = (torch.empty(N, K, dtype=F32, device="cuda") for _ in range(2))
    lsq.lsq_linear_bwd(t["dy"], t["x"], None, None, 0, None, one, 1, None, 0, M, N, K, None)
    lsq.lsq_linear_bwd(u["dy"], u["x"], None, None, 0, None, two, 1, None, 0, M, N, K, None)
    start = torch.randn(N, K, generator=torch.Generator().manual_seed(1)).cuda()
    acc = start.clone()
    for v in (t, u):
        lsq.lsq_linear_bwd(v["dy"], v["x"], None, None, 0, None, acc, 1, None, 1, M, N, K, None)
    assert torch.equal(acc, (start + one) + two)


@pytest.mark.parametrize("kind", ACTS)
def test_extreme_pre_activations(lsq, kind):
    """act and act' at magnitudes where their parts over- and underflow, infinities and NaN among them: the
    product is exact (w = 1, K = 8 with one nonzero), so z is the chosen value."""
    vals = torch.tensor([0.0, -0.0, 1e-30, -1e-30, 5.0, -5.0, 12.0, -12.0, 40.0, -40.0, 90.0, -90.0, 2e4, -2e4, 1e20,
                         -1e20, 3e38, -3e38, float("inf"), float("-inf"), float("nan")]).to(BF)
    M, N, K = len(vals), 8, 8
    x = torch.zeros(M, K, dtype=BF)
    x[:, 0] = vals
    w = torch.zeros(N, K, dtype=BF)
    w[:, 0] = 1.0
    fin = vals.isfinite()
    x[~fin, 0] = 0.0
    bias = torch.zeros(N, dtype=BF)
    y = torch.empty(M, N, dtype=BF, device="cuda")
    lsq.lsq_linear_fwd(x.cuda(), w.cuda(), bias.cuda(), ACTS.index(kind), None, None, y, M, N, K)
    want = OB.act(vals.double(), kind)
    got = y.double().cpu()[:, 0]
    err, tol = (got - want).abs(), 2.0 ** -8 * want.abs() + 2.0 ** -20 * vals.double().abs().clamp(max=1)
    assert (err <= tol)[fin].all(), (kind, vals[fin][~(err <= tol)[fin]])
    # act' at all of them, the non-finite too, through the bias gradient of one row each
    db = torch.empty(8, dtype=F32, device="cuda")
    zz = vals.double().clone().requires_grad_(True)
    (ref,) = torch.autograd.grad(OB.act(zz, kind).sum(), zz)
    limit = {float("inf"): 1.0, float("-inf"): 0.0}
    ws = torch.empty(lsq.lsq_linear_bwd_workspace_size(1, 8, 8, ACTS.index(kind)), dtype=torch.uint8, device="cuda")
    one = torch.ones(1, 8, dtype=BF, device="cuda")
    if kind == "none":
        return
    for v, r in zip(vals.tolist(), ref.tolist()):
        z = torch.full((1, 8), v, dtype=BF, device="cuda")
        lsq.lsq_linear_bwd(one, None, None, z, ACTS.index(kind), None, None, 0, db, 0, 1, 8, 8, ws)
        if v != v:
            assert db.isnan().all()
            continue
        if abs(v) > 1e3:
            r = 1.0 if v > 0 else 0.0      # the definition's limits (fp64's own formula overflows there)
        r = limit.get(v, r)
        assert (db.double() - r).abs().max().item() <= 2.0 ** -18 * (1 + min(abs(v), 8)), (kind, v)


def test_nan_and_inf_stay_in_their_rows(lsq):
    M, N, K = 40, 136, 264
    t = _inputs(M, N, K, 4)
    x = t["x"].clone()
    x[3, 5] = float("nan")
    x[8, 7] = float("inf")
    y, clean = (torch.empty(M, N, dtype=BF, device="cuda") for _ in range(2))
    lsq.lsq_linear_fwd(x, t["w"], t["b"], 0, None, None, y, M, N, K)
    lsq.lsq_linear_fwd(t["x"], t["w"], t["b"], 0, None, None, clean, M, N, K)
    keep = torch.ones(M, dtype=torch.bool)
    keep[[3, 8]] = False
    assert torch.equal(y[keep], clean[keep]) and y[3].isnan().all() and not y[8].isfinite().any()


def test_rows_behind_the_last_are_left_alone(lsq):
    M, N, K = 70, 136, 72
    t = _inputs(M + 4, N, K, 5)
    y, z = (torch.full((M + 4, N), 7.0, dtype=BF, device="cuda") for _ in range(2))
    lsq.lsq_linear_fwd(t["x"], t["w"], t["b"], 2, t["res"], z, y, M, N, K)
    dx = torch.full((M + 4, K), 7.0, dtype=BF, device="cuda")
    dw = torch.full((N + 4, K), 7.0, dtype=F32, device="cuda")
    db = torch.full((N + 4,), 7.0, dtype=F32, device="cuda")
    ws = torch.empty(lsq.lsq_linear_bwd_workspace_size(M, N, K, 2), dtype=torch.uint8, device="cuda")
    lsq.lsq_linear_bwd(t["dy"], t["x"], t["w"], z, 2, dx, dw, 1, db, 0, M, N, K, ws)
    for u, n in ((y, M), (z, M), (dx, M), (dw, N), (db, N)):
        assert (u[n:] == 7).all() and not (u[:n] == 7).all()


def test_after_copies_and_joins_in_a_graph(lsq):
    """Calls captured behind a copy, a fill and the join of another stream, which are no kernels of this library:
    each waits for all of them, in the graph's replays as in the eager run."""
    M, N, K = 96, 264, 520
    g = torch.Generator(device="cuda").manual_seed(5)
    src = [torch.randn(M, K, device="cuda", generator=g).to(torch.bfloat16) for _ in range(2)]
    w = torch.randn(N, K, device="cuda", generator=g).to(torch.bfloat16)
    big = torch.randn(64, 1 << 20, device="cuda", generator=g)      # keeps the other stream busy for a while
    x = torch.empty(M, K, dtype=torch.bfloat16, device="cuda")
    y, y2, dw = (torch.empty(s, dtype=t, device="cuda") for s, t in
                 (((M, N), torch.bfloat16), ((M, N), torch.bfloat16), ((N, K), torch.float32)))
    staged = torch.empty_like(src[0])
    side = torch.cuda.Stream()

    def run():
        cur = torch.cuda.current_stream()
        x.copy_(staged)                                              # a copy node, then a kernel that reads it
        lsq.lsq_linear_fwd(x, w, None, 0, None, None, y, M, N, K)
        dw.zero_()                                                   # a fill, then a kernel that adds to it
        lsq.lsq_linear_bwd(y, x, w, None, 0, None, dw, 1, None, 1, M, N, K, None)
        side.wait_stream(cur)
        with torch.cuda.stream(side):
            big.mul_(1.0)
            x.mul_(2.0)
        cur.wait_stream(side)                                        # the join, then a kernel that reads it
        lsq.lsq_linear_fwd(x, w, None, 0, None, None, y2, M, N, K)

    want = []
    for s in src:
        staged.copy_(s)
        run()
        torch.cuda.synchronize()
        want.append([t.clone() for t in (y, dw, y2)])
    cap = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=cap):
        run()
    for _ in range(3):
        for s, w0 in zip(src, want):
            staged.copy_(s)
            torch.cuda.synchronize()
            graph.replay()
            torch.cuda.synchronize()
            for got, ref in zip((y, dw, y2), w0):
                assert torch.equal(got, ref)
    for s, (y0, dw0, y20) in zip(src, want):                         # and the eager results are the products
        ref = s.double() @ w.double().t()
        assert (y0.double() - ref).norm() <= 2 ** -8 * ref.norm()
        assert (y20.double() - 2 * ref).norm() <= 2 ** -8 * (2 * ref).norm()
        ref = y0.double().t() @ s.double()
        assert (dw0.double() - ref).norm() <= 2e-5 * ref.norm()


# both products in one launch: every pair of tile widths, equal and unequal splits, clusters that tiles do not fill
# (148 SMs); the last three take separate launches
TOGETHER = [(1, 8, 8), (194, 8, 8), (65, 264, 8), (1, 520, 8), (25, 384, 2480), (17, 328, 2640), (70, 536, 784),
            (1, 456, 1056), (66, 8, 2936), (281, 72, 264), (187, 776, 8), (196, 536, 8), (475, 264, 264),
            (1043, 1488, 8), (501, 2864, 8), (1670, 8, 136), (162, 8, 2400), (490, 2200, 8), (258, 784, 8),
            (129, 136, 2080), (521, 72, 552), (971, 2056, 8), (289, 1296, 8), (314, 72, 2416), (430, 672, 864),
            (2091, 400, 8), (449, 1560, 312), (278, 72, 2840), (585, 80, 848), (72, 792, 1152), (652, 2312, 8),
            (479, 1920, 8), (8, 576, 1536), (33, 4096, 1024), (2048, 576, 1536)]


@pytest.mark.parametrize("M,N,K", TOGETHER)
def test_both_gradients_together_and_alone(lsq, M, N, K):
    """dx and dW of one call: within the bounds, and bit for bit what each alone gives, in both output types."""
    act = ACTS.index("silu")
    t = _inputs(M, N, K, 11)
    ws = torch.empty(lsq.lsq_linear_bwd_workspace_size(M, N, K, act), dtype=torch.uint8, device="cuda")
    for f32 in (0, 1):
        dx, dx1 = (torch.empty(M, K, dtype=BF, device="cuda") for _ in range(2))
        dw, dw1 = (torch.full((N, K), 0.25, dtype=F32 if f32 else BF, device="cuda") for _ in range(2))
        lsq.lsq_linear_bwd(t["dy"], t["x"], t["w"], t["z"], act, dx, dw, f32, None, f32, M, N, K, ws)
        lsq.lsq_linear_bwd(t["dy"], None, t["w"], t["z"], act, dx1, None, 0, None, 0, M, N, K, ws)
        lsq.lsq_linear_bwd(t["dy"], t["x"], None, t["z"], act, None, dw1, f32, None, f32, M, N, K, ws)
        assert torch.equal(dx, dx1) and torch.equal(dw, dw1)
        if not f32:
            want = BB.linear_bwd(_d(t["dy"]), _d(t["x"]), _d(t["w"]), _d(t["z"]), "silu", M + 32, dw_f32=False)
            _check(dx, want["dx"], "dx together", rel=8e-3)
            _check(dw, want["dw"], "dw together", rel=8e-3)
