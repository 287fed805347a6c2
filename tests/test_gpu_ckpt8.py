"""8-bit checkpoints: codes and restored values bit for bit against the oracle's integer arithmetic, and the
RMSNorm passes that write and read them against the library's own RMSNorm on the same rows."""
import numpy as np
import pytest
import torch

from oracle import block as OB
from oracle import decoder as D
from tolerances import assert_close_ew

pytestmark = pytest.mark.gpu
BF, F32, F64 = torch.bfloat16, torch.float32, torch.float64

SHAPES = [(1, 8), (1, 64), (3, 72), (5, 576), (2, 1000), (1, 1032), (33, 1024), (700, 64), (3, 2056), (2, 4096),
          (1, 8200), (1, 16384), (400, 1160), (400, 2304), (320, 4104)]


def _x(rows, d, seed=0):
    g = torch.Generator().manual_seed(77 * rows + d + seed)
    x = torch.randn(rows, d, generator=g) * torch.exp(2 * torch.randn(rows, d, generator=g))
    x[rows // 2, : d // 2] = 0.0
    return x.to(BF)


def _split(ckpt, rows, d):
    """the documented layout: codes, then from the next multiple of 16 bytes the block maxima"""
    c = ckpt.cpu().numpy()
    off, nb = -(-rows * d // 16) * 16, -(-d // 64)
    return (c[:rows * d].view(np.int8).reshape(rows, d),
            c[off:off + rows * nb * 2].view(np.uint16).reshape(rows, nb))


def _roundtrip(lsq, x):
    rows, d = x.shape
    ckpt = torch.empty(lsq.lsq_ckpt8_size(rows, d), dtype=torch.uint8, device="cuda")
    back = torch.empty(rows, d, dtype=BF, device="cuda")
    lsq.lsq_ckpt8_pack(x.cuda(), ckpt, rows, d)
    lsq.lsq_ckpt8_unpack(ckpt, back, rows, d)
    return ckpt, back


def _bits(t):
    return t.cpu().contiguous().view(torch.int16)


@pytest.mark.parametrize("rows,d", SHAPES)
def test_bit_exact(lsq, rows, d):
    x = _x(rows, d)
    ckpt, back = _roundtrip(lsq, x)
    take = slice(0, 12)              # the integer oracle is slow: the first rows, and the middle one below
    for sl in (take, slice(rows // 2, rows // 2 + 1), slice(rows - 1, rows)):
        codes, amax = OB.ckpt8_pack(x[sl])
        got_c, got_a = _split(ckpt, rows, d)
        assert np.array_equal(got_c[sl], codes) and np.array_equal(got_a[sl], amax)
        assert torch.equal(_bits(back[sl]), _bits(OB.ckpt8_unpack(codes, amax)))


def test_every_pair_of_significands(lsq):
    """All 128 significands of a block's maximum against every smaller magnitude down to where codes are 0:
    each tie and near-tie of the rounding, both signs."""
    mags = torch.arange(0x3F80 - 9 * 128, 0x4000, dtype=torch.int32)     # 2^-9 .. just below 2
    rows = []
    for m in range(128):
        top = 0x3F80 + m
        small = mags[mags <= top]
        pad = -len(small) % 63
        body = torch.cat([small, small.new_zeros(pad)]).view(-1, 63)
        sign = torch.where(torch.arange(63) % 2 == 1, 0x8000, 0).to(torch.int32)
        body = body | sign
        rows.append(torch.cat([torch.full((len(body), 1), top, dtype=torch.int32), body], dim=1))
    bits = torch.cat(rows)
    bits = torch.where(bits >= 0x8000, bits - 0x10000, bits).to(torch.int16)
    x = bits.view(BF)
    ckpt, back = _roundtrip(lsq, x)
    # the definition in float64, exact here: 254 |x| + amax and its quotient's floor (no quotient but a true
    # tie lies within 1e-5 of an integer)
    v = x.double()
    top = v[:, :1]
    q = (torch.sign(v) * torch.floor((254 * v.abs() + top) / (2 * top))).to(torch.int8).double()   # no -0 code
    got_c, got_a = _split(ckpt, *x.shape)
    assert np.array_equal(got_c, q.numpy())
    assert np.array_equal(got_a[:, 0], _bits(x[:, 0]).numpy().view(np.uint16))
    assert torch.equal(_bits(back), _bits((q * top / 127).float().to(BF)))
    probe = torch.arange(0, x.shape[0], 211)
    codes, amax = OB.ckpt8_pack(x[probe])
    assert np.array_equal(got_c[probe.numpy()], codes)


def test_extremes_and_non_finite_blocks(lsq):
    tops = [2.0 ** -133, 2.0 ** -119, 2.0 ** -118, 2.0 ** -100, 1.0, 3.3e38, float("inf"), float("nan"), 0.0]
    x = torch.zeros(len(tops), 136, dtype=BF)
    for r, t in enumerate(tops):
        x[r, 0::2], x[r, 1::2] = t, -t * 0.4
        x[r, 128:] = 1.0             # the short last block of the row is its own
    _, back = _roundtrip(lsq, x)
    want = OB.ckpt8_roundtrip(x)
    assert torch.equal(back.cpu().isnan(), want.isnan())
    ok = ~want.isnan()
    assert torch.equal(back.cpu().float()[ok], want.float()[ok])


@pytest.mark.parametrize("rows,d", SHAPES)
def test_fused_passes_equal_their_parts(lsq, rows, d):
    """pack + RMSNorm, unpack + RMSNorm and RMSNorm's backward on the restored rows: the checkpoint bit for
    bit, the norm's values within the elementwise tolerance of the oracle on the rows they read."""
    eps = 1e-5
    x = _x(rows, d, 1).cuda()
    gen = torch.Generator().manual_seed(d)
    g = (1 + 0.2 * torch.randn(d, generator=gen)).to(BF).cuda()
    dy, res = (torch.randn(rows, d, generator=gen).to(BF).cuda() for _ in range(2))
    ckpt, back = _roundtrip(lsq, x)
    size = lsq.lsq_ckpt8_size(rows, d)
    c2 = torch.zeros(size, dtype=torch.uint8, device="cuda")
    y, x2, y2, out, out0 = (torch.empty(rows, d, dtype=BF, device="cuda") for _ in range(5))
    rs, rs2 = (torch.empty(rows, dtype=F32, device="cuda") for _ in range(2))
    lsq.lsq_rmsnorm_fwd_pack8(x, g, y, rs, c2, rows, d, eps)
    for a, b in zip(_split(ckpt, rows, d), _split(c2, rows, d)):
        assert np.array_equal(a, b)
    lsq.lsq_rmsnorm_fwd_unpack8(c2, g, x2, y2, rs2, rows, d, eps)
    assert torch.equal(_bits(x2), _bits(back))
    lsq.lsq_rmsnorm_bwd_unpack8(dy, c2, g, rs2, res, out, rows, d)
    lsq.lsq_rmsnorm_bwd_unpack8(dy, c2, g, rs2, None, out0, rows, d)
    for name, got, gr, src in (("y", y, rs, x), ("y restored", y2, rs2, x2)):
        ref = D.rmsnorm(src.cpu().to(F64), g.cpu().to(F64), eps)
        assert_close_ew(got.double().cpu().numpy(), ref.numpy(), what=name)
        want = (src.cpu().to(F64).square().mean(1) + eps) ** -0.5
        assert torch.all((gr.cpu().to(F64) - want).abs() <= 1e-5 * want)
    xs = x2.cpu().to(F64).requires_grad_(True)
    (dx,) = torch.autograd.grad(D.rmsnorm(xs, g.cpu().to(F64), eps), xs, grad_outputs=dy.cpu().to(F64))
    assert_close_ew(out0.double().cpu().numpy(), dx.numpy(), what="dx restored")
    assert_close_ew(out.double().cpu().numpy(), (dx + res.cpu().to(F64)).numpy(), what="dx restored + res")
    inplace = res.clone()
    lsq.lsq_rmsnorm_bwd_unpack8(dy, c2, g, rs2, inplace, inplace, rows, d)
    assert torch.equal(inplace, out)


def test_size_is_what_is_written(lsq):
    """Bytes behind the checkpoint stay as they were, for a length that ends inside a 16-byte group."""
    rows, d = 3, 72
    size = lsq.lsq_ckpt8_size(rows, d)
    buf = torch.full((size + 64,), 0xA5, dtype=torch.uint8, device="cuda")
    lsq.lsq_ckpt8_pack(_x(rows, d).cuda(), buf, rows, d)
    used = -(-rows * d // 16) * 16 + rows * 2 * 2
    assert used <= size and (buf[used:] == 0xA5).all()


@pytest.mark.parametrize("rows,d", [(1000, 4104), (1580, 2048), (1578, 2048), (400, 8200), (390, 8328)])
def test_more_rows_than_run_at_once(lsq, rows, d):
    """Two and four words a thread, and both sides of where they begin."""
    test_bit_exact(lsq, rows, d)
    test_fused_passes_equal_their_parts(lsq, rows, d)


@pytest.mark.parametrize("rows,d", [(592, 776), (591, 1024), (592, 264), (148, 16384), (149, 8328)])
def test_where_the_fetch_ahead_ends(lsq, rows, d):
    test_fused_passes_equal_their_parts(lsq, rows, d)
