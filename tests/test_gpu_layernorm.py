"""LayerNorm forward and backward against the fp64 oracle, within first-order rounding bounds (block_bounds.py)."""
import pytest
import torch

import block_bounds as BB
from oracle import block as OB
from tolerances import assert_within_bound

pytestmark = pytest.mark.gpu
BF, F32, F64 = torch.bfloat16, torch.float32, torch.float64

SHAPES = [(1, 8), (1, 4096), (3, 16384), (130, 576), (37, 1000), (9, 264), (1, 1024), (5, 1032), (600, 4096),
          (700, 5120), (300, 8200), (5000, 64), (2, 12288), (1200, 512), (311, 2048), (1, 16384), (400, 16376)]


def _inputs(rows, d, seed=0, offset=0.0):
    g = torch.Generator().manual_seed(1000 * rows + d + seed)

    def n(*s):
        return torch.randn(*s, generator=g)
    x = n(rows, d) * (1 + 30 * (torch.rand(d, generator=g) < 0.01)) + offset
    return {"x": x.to(BF).cuda(), "g": (1 + 0.2 * n(d)).to(BF).cuda(), "b": (0.1 * n(d)).to(BF).cuda(),
            "dy": n(rows, d).to(BF).cuda(), "res": n(rows, d).to(BF).cuda()}


def _check(got, ref_bound, what, rel=5e-3):
    ref, bound = ref_bound
    # an absolute floor of fp32's smallest normal: exact zeros in the bound stay comparable
    assert_within_bound(got.double().cpu(), ref.cpu(), bound.cpu() + 2.0 ** -126, rel=rel, what=what)


def _stats(x, eps):
    x = x.double()
    return x.mean(1).float(), ((x.var(1, unbiased=False) + eps) ** -0.5).float()


@pytest.mark.parametrize("rows,d", SHAPES)
@pytest.mark.parametrize("bias", [True, False])
def test_forward(lsq, rows, d, bias):
    t = _inputs(rows, d)
    b = t["b"] if bias else None
    y = torch.empty(rows, d, dtype=BF, device="cuda")
    mean, rstd = (torch.empty(rows, dtype=F32, device="cuda") for _ in range(2))
    lsq.lsq_layernorm_fwd(t["x"], t["g"], b, y, mean, rstd, rows, d, 1e-5)
    want = BB.layernorm_fwd(t["x"].double(), t["g"].double(), b.double() if bias else None, 1e-5)
    for name, got in (("y", y), ("mean", mean), ("rstd", rstd)):
        _check(got, want[name], f"layernorm {name}", rel=1.0 if name == "mean" else 5e-3)
    y2 = torch.empty_like(y)
    lsq.lsq_layernorm_fwd(t["x"], t["g"], b, y2, None, None, rows, d, 1e-5)
    assert torch.equal(y, y2)


def test_forward_far_mean_and_constant_rows(lsq):
    """Rows whose mean is far above their spread, rows without any spread, and rows of zeros."""
    rows, d = 64, 1536
    t = _inputs(rows, d, offset=100.0)
    x = t["x"].clone()
    x[5] = 3.0
    x[6] = 0.0
    y = torch.empty_like(x)
    mean, rstd = (torch.empty(rows, dtype=F32, device="cuda") for _ in range(2))
    lsq.lsq_layernorm_fwd(x, t["g"], t["b"], y, mean, rstd, rows, d, 1e-5)
    want = BB.layernorm_fwd(x.double(), t["g"].double(), t["b"].double(), 1e-5)
    for name, got in (("y", y), ("mean", mean), ("rstd", rstd)):
        _check(got, want[name], f"layernorm far mean {name}")


@pytest.mark.parametrize("rows,d", SHAPES)
@pytest.mark.parametrize("res", [True, False])
def test_backward(lsq, rows, d, res):
    t = _inputs(rows, d, seed=1)
    mean, rstd = _stats(t["x"], 1e-5)
    out = torch.empty(rows, d, dtype=BF, device="cuda")
    dg, db = (torch.empty(d, dtype=F32, device="cuda") for _ in range(2))
    ws = torch.empty(lsq.lsq_layernorm_bwd_workspace_size(rows, d), dtype=torch.uint8, device="cuda")
    args = (t["dy"], t["x"], t["g"], mean, rstd)
    lsq.lsq_layernorm_bwd(*args, t["res"] if res else None, out, dg, db, 0, rows, d, ws)
    want = BB.layernorm_bwd(*(v.double() for v in args), t["res"].double() if res else None, rows + 64)
    for name, got in (("dx", out), ("dg", dg), ("db", db)):
        _check(got, want[name], f"layernorm {name}")
    # frozen gain and bias, one of the two, in place over the residual gradient: the same numbers
    out2 = t["res"].clone() if res else torch.empty_like(out)
    lsq.lsq_layernorm_bwd(*args, out2 if res else None, out2, None, None, 0, rows, d, None)
    assert torch.equal(out, out2)
    db2 = torch.full_like(db, 0.25)
    lsq.lsq_layernorm_bwd(*args, t["res"] if res else None, out2, None, db2, 1, rows, d, ws)
    assert torch.equal(db2, db + 0.25)
    dg2 = torch.full_like(dg, -2.0)
    lsq.lsq_layernorm_bwd(*args, t["res"] if res else None, out2, dg2, None, 1, rows, d, ws)
    assert torch.equal(dg2, dg - 2.0)


def test_backward_matches_autograd_and_differences(lsq):
    """Through the library's own forward statistics: against autograd of the oracle's forward, and the
    directional derivative of the fp64 forward."""
    rows, d, eps = 24, 320, 1e-5
    t = _inputs(rows, d, seed=2)
    y = torch.empty(rows, d, dtype=BF, device="cuda")
    mean, rstd = (torch.empty(rows, dtype=F32, device="cuda") for _ in range(2))
    lsq.lsq_layernorm_fwd(t["x"], t["g"], t["b"], y, mean, rstd, rows, d, eps)
    dx = torch.empty_like(y)
    dg, db = (torch.empty(d, dtype=F32, device="cuda") for _ in range(2))
    ws = torch.empty(lsq.lsq_layernorm_bwd_workspace_size(rows, d), dtype=torch.uint8, device="cuda")
    lsq.lsq_layernorm_bwd(t["dy"], t["x"], t["g"], mean, rstd, None, dx, dg, db, 0, rows, d, ws)
    xs = [t[k].double().requires_grad_(True) for k in ("x", "g", "b")]
    ref = torch.autograd.grad(OB.layernorm(*xs, eps), xs, grad_outputs=t["dy"].double())
    for name, got, want, tol in (("dx", dx, ref[0], 2.0 ** -8), ("dg", dg, ref[1], 1e-5), ("db", db, ref[2], 1e-5)):
        assert (got.double() - want).norm() <= tol * want.norm(), name
    g = torch.Generator().manual_seed(5)
    h = 1e-6
    for k, grad in (("x", dx), ("g", dg), ("b", db)):
        v = torch.randn(t[k].shape, generator=g).double().cuda()
        args = {n: t[n].double() for n in ("x", "g", "b")}
        up, dn = ({**args, k: args[k] + s * h * v} for s in (1, -1))
        fd = ((OB.layernorm(up["x"], up["g"], up["b"], eps) - OB.layernorm(dn["x"], dn["g"], dn["b"], eps))
              * t["dy"].double()).sum() / (2 * h)
        # the directional derivative carries the gradient's rounding: 2^-8 of each component it sums
        assert abs(fd - (grad.double() * v).sum()) <= 2.0 ** -8 * (grad.double() * v).norm() * 4 + 1e-6, k


def test_non_finite_rows_stay_in_their_rows(lsq):
    rows, d = 40, 640
    t = _inputs(rows, d, seed=3)
    x = t["x"].clone()
    x[7, 100], x[9, 3] = float("nan"), float("inf")
    y, clean = torch.empty_like(x), torch.empty_like(x)
    lsq.lsq_layernorm_fwd(x, t["g"], t["b"], y, None, None, rows, d, 1e-5)
    lsq.lsq_layernorm_fwd(t["x"], t["g"], t["b"], clean, None, None, rows, d, 1e-5)
    keep = torch.ones(rows, dtype=torch.bool)
    keep[[7, 9]] = False
    assert torch.equal(y[keep], clean[keep]) and y[[7, 9]].isnan().all()


def test_rows_behind_the_last_are_left_alone_and_runs_repeat(lsq):
    rows, d = 77, 1160
    t = _inputs(rows + 3, d, seed=4)
    mean, rstd = _stats(t["x"], 1e-5)
    ws = torch.empty(lsq.lsq_layernorm_bwd_workspace_size(rows, d), dtype=torch.uint8, device="cuda")
    runs = []
    for _ in range(2):
        y, out = (torch.full((rows + 3, d), 7.0, dtype=BF, device="cuda") for _ in range(2))
        dg, db = (torch.empty(d, dtype=F32, device="cuda") for _ in range(2))
        lsq.lsq_layernorm_fwd(t["x"], t["g"], t["b"], y, None, None, rows, d, 1e-5)
        lsq.lsq_layernorm_bwd(t["dy"], t["x"], t["g"], mean, rstd, t["res"], out, dg, db, 0, rows, d, ws)
        assert (y[rows:] == 7).all() and (out[rows:] == 7).all()
        runs.append((y, out, dg, db))
    for a, b in zip(*runs):
        assert torch.equal(a, b)


@pytest.mark.parametrize("rows,d", [(700, 5120), (77, 1160), (1200, 512), (3, 16384)])
def test_in_place(lsq, rows, d):
    """y over x, and the gradient over dy or x, give what separate outputs give."""
    t = _inputs(rows, d, seed=8)
    mean, rstd = _stats(t["x"], 1e-5)
    y = torch.empty_like(t["x"])
    lsq.lsq_layernorm_fwd(t["x"], t["g"], t["b"], y, None, None, rows, d, 1e-5)
    x = t["x"].clone()
    lsq.lsq_layernorm_fwd(x, t["g"], t["b"], x, None, None, rows, d, 1e-5)
    assert torch.equal(x, y)
    ws = torch.empty(lsq.lsq_layernorm_bwd_workspace_size(rows, d), dtype=torch.uint8, device="cuda")

    def bwd(dy, x, out):
        dg, db = (torch.empty(d, dtype=F32, device="cuda") for _ in range(2))
        lsq.lsq_layernorm_bwd(dy, x, t["g"], mean, rstd, t["res"], out, dg, db, 0, rows, d, ws)
        return out, dg, db
    want = bwd(t["dy"], t["x"], torch.empty_like(y))
    a = t["dy"].clone()
    b = t["x"].clone()
    for got in (bwd(a, t["x"], a), bwd(t["dy"], b, b)):
        assert all(torch.equal(p, q) for p, q in zip(got, want))


@pytest.mark.parametrize("rows,d", [(1300, 2056), (1185, 2048), (1184, 2048), (2000, 2304)])
@pytest.mark.parametrize("bias", [True, False])
def test_forward_of_more_rows_than_run_at_once(lsq, rows, d, bias):
    """Two words a thread (the other widths are among the shapes above), and both sides of where it begins."""
    test_forward(lsq, rows, d, bias)


# the walkers with their second kernel, by warps and by blocks of each width, and both sides of where they begin
MANY = [(1025, 504), (1024, 504), (1100, 64), (1537, 512), (1536, 512), (1540, 264), (2000, 576), (1700, 768),
        (1540, 1032), (2100, 2304), (1600, 5128), (1700, 4096), (600, 16384), (512, 16384), (513, 16384)]


@pytest.mark.parametrize("rows,d", MANY)
@pytest.mark.parametrize("res", [True, False])
def test_backward_of_many_rows(lsq, rows, d, res):
    test_backward(lsq, rows, d, res)


@pytest.mark.parametrize("rows,d", [(2000, 520), (1540, 1160), (600, 16384), (1536, 512), (1024, 64), (1, 8), (33, 8200)])
def test_in_place_at_other_sizes(lsq, rows, d):
    test_in_place(lsq, rows, d)


def test_few_rows_captured_in_place(lsq):
    """In place over dy the sums are a launch of their own, before the rows': captured, replayed twice."""
    rows, d = 200, 1000
    t = _inputs(rows, d, seed=9)
    mean, rstd = _stats(t["x"], 1e-5)
    ws = torch.empty(lsq.lsq_layernorm_bwd_workspace_size(rows, d), dtype=torch.uint8, device="cuda")
    want = [torch.empty_like(t["dy"]), *(torch.empty(d, dtype=F32, device="cuda") for _ in range(2))]
    lsq.lsq_layernorm_bwd(t["dy"], t["x"], t["g"], mean, rstd, t["res"], *want, 0, rows, d, ws)
    dy, dg, db = torch.empty_like(t["dy"]), torch.empty_like(want[1]), torch.empty_like(want[2])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        dy.copy_(t["dy"])
        lsq.lsq_layernorm_bwd(dy, t["x"], t["g"], mean, rstd, t["res"], dy, dg, db, 0, rows, d, ws)
    for _ in range(2):
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip((dy, dg, db), want))


@pytest.mark.parametrize("rows,d", [(592, 576), (591, 576), (700, 1024), (592, 264), (148, 16384), (149, 16384)])
def test_forward_where_the_fetch_ahead_ends(lsq, rows, d):
    test_forward(lsq, rows, d, True)
    test_forward(lsq, rows, d, False)
