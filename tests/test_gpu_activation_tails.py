"""The activations of the dense linear where their results are small, in relative terms, and at infinities and NaN.

z is exact (one product by 1, the others 0), over every bf16 from -128 to -2^-10.  The kernels take the logistic
function, and the normal distribution's tail, through exp2 of an argument of at most 126 in size, made with up to
four fp32 roundings: 126 ln 2 * 4 * 2^-24 = 2.1e-5 of the result; the fit of the normal tail adds 1e-4 and the few
other operations 2^-20.  The sum, 1.3e-4, is held to 2^-12; the output's rounding to bf16 adds 2^-8.  Below 2^-126
exp2 and the reciprocal give 0: up to 230 * 2^-126 is lost there (tanh-GELU's derivative at -10: z u' = 230).
"""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu
BF, F32, F64 = torch.bfloat16, torch.float32, torch.float64
ACTS = ("none", "relu", "gelu", "gelu_tanh", "silu")
REL, LOST = 2.0 ** -12, 2.0 ** -118


def _ref(z, kind):
    """In forms without cancellation for negative z."""
    if kind == "gelu":
        return 0.5 * z * torch.erfc(-z / math.sqrt(2.0))
    if kind == "gelu_tanh":
        return z * torch.sigmoid(2.0 * math.sqrt(2.0 / math.pi) * (z + 0.044715 * z ** 3))
    return z * torch.sigmoid(z)


def _negative():
    """Every bf16 in [-128, -2^-10], the count a multiple of 8."""
    lo, hi = (int(torch.tensor(v, dtype=BF).view(torch.int16)) & 0x7fff for v in (2.0 ** -10, 128.0))
    bits = torch.arange(lo, hi + 1, dtype=torch.int32) - 0x8000
    v = bits.to(torch.int16).view(BF)
    return torch.cat([v, v[-1:].expand(-len(v) % 8)])


def _forward(lsq, vals, kind, form):
    """act of each value, by one row of many columns or by many rows of N columns."""
    n = len(vals)
    if form == "row":
        M, N, K = 1, n, 8
        x, w = torch.zeros(1, K, dtype=BF), torch.zeros(N, K, dtype=BF)
        x[0, 0], w[:, 0] = 1.0, vals
    else:
        M, N, K = n, {"tiles": 8, "pairs": 2136}[form], 8
        x, w = torch.zeros(M, K, dtype=BF), torch.zeros(N, K, dtype=BF)
        x[:, 0], w[:, 0] = vals, 1.0
    y = torch.empty(M, N, dtype=BF, device="cuda")
    lsq.lsq_linear_fwd(x.cuda(), w.cuda(), None, ACTS.index(kind), None, None, y, M, N, K)
    if form != "row":
        assert torch.equal(y.view(torch.int16), y[:, :1].expand(M, N).contiguous().view(torch.int16))
        y = y[:, 0]
    return y.reshape(-1).double().cpu()


@pytest.mark.parametrize("form", ["row", "tiles", "pairs"])
@pytest.mark.parametrize("kind", ["gelu", "gelu_tanh", "silu"])
def test_negative_values_keep_their_relative_accuracy(lsq, kind, form):
    vals = _negative()
    got, want = _forward(lsq, vals, kind, form), _ref(vals.double(), kind)
    err = (got - want).abs() - LOST
    worst = (err / want.abs().clamp(min=1e-300)).argmax()
    assert (err <= (2.0 ** -8 + REL) * want.abs()).all(), (kind, vals[worst].item(), got[worst].item(),
                                                           want[worst].item())


@pytest.mark.parametrize("kind", ["gelu", "gelu_tanh", "silu"])
def test_negative_derivatives_keep_their_relative_accuracy(lsq, kind):
    """From z = -2 down, beyond the derivatives' zero (at -0.75 to -1.28), where their terms no longer cancel: act' is
    then at least 0.43 of its larger term (SiLU at -2), so the terms' 2^-12 is at most 2^-11 of it here.  Read in fp32 from the bias gradient of one row."""
    vals = _negative()
    n = len(vals)
    z = vals.double().requires_grad_(True)
    (want,) = torch.autograd.grad(_ref(z, kind).sum(), z)
    ws = torch.empty(lsq.lsq_linear_bwd_workspace_size(1, n, 8, ACTS.index(kind)), dtype=torch.uint8, device="cuda")
    db, one = torch.empty(n, dtype=F32, device="cuda"), torch.ones(1, n, dtype=BF, device="cuda")
    lsq.lsq_linear_bwd(one, None, None, vals.view(1, n).cuda(), ACTS.index(kind), None, None, 0, db, 0, 1, n, 8, ws)
    got, far = db.double().cpu(), vals.double() <= -2.0
    err = (got - want).abs() - LOST
    worst = torch.where(far, err / want.abs().clamp(min=1e-300), err - err).argmax()
    assert (err <= 2 * REL * want.abs())[far].all(), (kind, vals[worst].item(), got[worst].item(), want[worst].item())


@pytest.mark.parametrize("form", ["row", "tiles", "pairs"])
@pytest.mark.parametrize("kind", ACTS)
def test_infinities_and_nan_in_the_forward(lsq, kind, form):
    """The limits: +inf at +inf, 0 at -inf (-inf without an activation), NaN at NaN; the largest finite values too."""
    inf, nan = float("inf"), float("nan")
    big = torch.finfo(BF).max
    vals = torch.tensor([inf, -inf, nan, big, -big, 1.0, -1.0, 0.0] * 40, dtype=BF)
    got = _forward(lsq, vals, kind, form)
    low = {"none": (-inf, -big)}.get(kind, (0.0, 0.0))
    want = torch.tensor([inf, low[0], nan, big, low[1]] * 40, dtype=F64)
    got = got.view(-1, 8)[:, :5].reshape(-1)
    same = (got == want) | (got.isnan() & want.isnan())
    assert same.all(), (kind, got[:5], want[:5])
