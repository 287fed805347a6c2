"""Refusals of the LayerNorm, dense-linear and 8-bit checkpoint calls: made on the host before anything is
enqueued, so they are tested without a GPU (raw addresses stand in for device pointers and are never read)."""
import pytest
import torch

from nf4_layer_streamed_blockwise_b200 import lib as L

P = 1 << 20          # a 256-byte aligned address; the arguments lie 1 MB apart
S = 0                # the default stream's handle
EINVAL, EUNSUPPORTED = 1, 6


def _refused(status, fn, *args, **kw):
    with pytest.raises(L.LsqError) as e:
        fn(*args, stream=S, **kw)
    assert e.value.status == status, e.value


def _at(n):
    return [P * (k + 1) for k in range(n)]


# call, arguments, the ones that must be given, the ones that must be aligned, where rows and d stand, pairs of
# which the second is written while the first is read (not even the same place where marked True)
CASES = {
    "ln_fwd": (L.lsq_layernorm_fwd, [*_at(6), 4, 64, 1e-5], (0, 1, 3), (0, 1, 2, 3), 6, [(0, 3, False)]),
    "pack": (L.lsq_ckpt8_pack, [*_at(2), 4, 64], (0, 1), (0, 1), 2, [(0, 1, True)]),
    "unpack": (L.lsq_ckpt8_unpack, [*_at(2), 4, 64], (0, 1), (0, 1), 2, [(0, 1, True)]),
    "fwd_pack8": (L.lsq_rmsnorm_fwd_pack8, [*_at(5), 4, 64, 1e-5], (0, 1, 2, 4), (0, 1, 2, 4), 5,
                  [(0, 2, False), (0, 4, True), (2, 4, True)]),
    "fwd_unpack8": (L.lsq_rmsnorm_fwd_unpack8, [*_at(5), 4, 64, 1e-5], (0, 1, 2, 3), (0, 1, 2, 3), 5,
                    [(0, 2, True), (0, 3, True), (2, 3, True)]),
    "bwd_unpack8": (L.lsq_rmsnorm_bwd_unpack8, [*_at(6), 4, 64], (0, 1, 2, 3, 5), (0, 1, 2, 4, 5), 6,
                    [(0, 5, False), (4, 5, False), (1, 5, True)]),
}


@pytest.mark.parametrize("name", sorted(CASES))
def test_row_passes_refuse(name):
    fn, args, required, aligned, rows_at, apart = CASES[name]
    for a, b, never in apart:
        _refused(EINVAL, fn, *[args[a] + 128 if k == b else v for k, v in enumerate(args)])
        if never:
            _refused(EINVAL, fn, *[args[a] if k == b else v for k, v in enumerate(args)])
    for i in required:
        _refused(EINVAL, fn, *[None if k == i else a for k, a in enumerate(args)])
    for i in aligned:
        _refused(EINVAL, fn, *[P + 8 if k == i else a for k, a in enumerate(args)])
    for rows, d, status in ((0, 64, EINVAL), (-1, 64, EINVAL), (1 << 31, 64, EINVAL), (4, 0, EINVAL), (4, 60, EINVAL),
                            (4, -8, EINVAL), (4, 16392, EUNSUPPORTED)):
        _refused(status, fn, *args[:rows_at], rows, d, *args[rows_at + 2:])


def test_layernorm_backward_refuses():
    ws = torch.empty(0, dtype=torch.uint8)

    def call(status, **kw):
        a = dict(zip(("dy", "x", "g", "mean", "rstd", "dres_in", "dres_out", "dg", "db"), _at(9)), accumulate=0,
                 rows=4, d=64, workspace=None)
        a.update(kw)
        _refused(status, L.lsq_layernorm_bwd, *a.values())
    for k in ("dy", "x", "g", "mean", "rstd", "dres_out"):
        call(EINVAL, **{k: None})
    for k in ("dy", "x", "g", "dres_in", "dres_out", "dg", "db"):
        call(EINVAL, **{k: P + 8})
    call(EINVAL)                                 # gradients wanted, no workspace
    for k in (1, 2, 6):                          # dres_out 128 bytes into dy, x, dres_in
        call(EINVAL, dg=None, db=None, dres_out=P * k + 128)
    call(EINVAL, rows=0)
    call(EINVAL, d=12)
    call(EUNSUPPORTED, d=16392)
    call(EINVAL, workspace=ws)                   # a CPU tensor


def test_linear_forward_refuses():
    def call(status, **kw):
        a = dict(x=P, w=2 * P, bias=3 * P, act=0, residual=4 * P, z=5 * P, y=6 * P, M=4, N=64, K=64)
        a.update(kw)
        _refused(status, L.lsq_linear_fwd, *a.values())
    for k in ("x", "w", "y"):
        call(EINVAL, **{k: None})
    for k in ("x", "w", "bias", "residual", "z", "y"):
        call(EINVAL, **{k: 9 * P + 8})
    for k, v in (("M", 0), ("M", (1 << 30) + 1), ("N", 0), ("N", 60), ("K", 4), ("K", 0), ("K", -8), ("act", -1),
                 ("act", 5)):
        call(EINVAL, **{k: v})
    for out in ("y", "z"):                       # an output on x, w, bias, or a few bytes into them
        for k in (1, 2, 3):
            call(EINVAL, **{out: k * P})
            call(EINVAL, **{out: k * P + 64})
    call(EINVAL, z=6 * P)                        # z on y, z on the residual, y a few rows into the residual
    call(EINVAL, z=4 * P + 128)
    call(EINVAL, y=4 * P + 128)


def test_linear_backward_refuses():
    def call(status, **kw):
        a = dict(dy=P, x=2 * P, w=3 * P, z=4 * P, act=2, dx=5 * P, dw=6 * P, dw_f32=1, dbias=7 * P, accumulate=0,
                 M=4, N=64, K=64, workspace=None)
        a.update(kw)
        _refused(status, L.lsq_linear_bwd, *a.values())
    call(EINVAL, dy=None)
    call(EINVAL, x=None)
    call(EINVAL, w=None)
    call(EINVAL, z=None)
    call(EINVAL, dx=None, dw=None, dbias=None)
    call(EINVAL, accumulate=1, dw_f32=0)
    call(EINVAL)                                 # no workspace
    call(EINVAL, act=0)                          # no workspace for dbias
    call(EINVAL, act=9)
    call(EINVAL, N=20)
    for k in ("dy", "x", "w", "z", "dx", "dw", "dbias"):
        call(EINVAL, **{k: 9 * P + 4})
    for k in ("dx", "dw"):                       # no activation, no dbias: no workspace, so these reach the check
        for at in (1, 2, 3):
            call(EINVAL, act=0, dbias=None, **{k: at * P + 128})
    call(EINVAL, act=0, dbias=None, dx=6 * P)


def test_tensor_arguments_are_checked():
    """The binding checks what an address cannot carry: type, size, density and device."""
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    for bad in (x.float(), x[:, :32], x[:2], x.t(), x):        # type, size, size, density, not on a GPU
        _refused(EINVAL, L.lsq_ckpt8_pack, bad, P, 4, 64)
    short = torch.zeros(100, dtype=torch.uint8)
    _refused(EINVAL, L.lsq_ckpt8_pack, P, short, 4, 64)


def test_sizes():
    assert L.lsq_ckpt8_size(3, 72) == 256 and L.lsq_ckpt8_size(2048, 4096) == 2048 * 4096 + 2048 * 64 * 2
    assert L.lsq_layernorm_bwd_workspace_size(1, 64) % 256 == 0
    assert L.lsq_linear_bwd_workspace_size(128, 256, 64, 0) < L.lsq_linear_bwd_workspace_size(128, 256, 64, 1)


# the row passes' other overlaps: call, arguments, pairs of an output and the argument whose place it is given
OVERLAPS = {
    "ln_fwd": (L.lsq_layernorm_fwd, [*_at(6), 4, 64, 1e-5],
               [(3, 1), (3, 2), (4, 0), (4, 1), (4, 2), (4, 3), (5, 0), (5, 3), (5, 4)]),
    "fwd_pack8": (L.lsq_rmsnorm_fwd_pack8, [*_at(5), 4, 64, 1e-5], [(2, 1), (3, 0), (3, 1), (3, 2), (3, 4), (4, 1)]),
    "fwd_unpack8": (L.lsq_rmsnorm_fwd_unpack8, [*_at(5), 4, 64, 1e-5], [(2, 1), (3, 1), (4, 0), (4, 1), (4, 2), (4, 3)]),
    "bwd_unpack8": (L.lsq_rmsnorm_bwd_unpack8, [*_at(6), 4, 64], [(5, 2), (5, 3)]),
}


@pytest.mark.parametrize("name", sorted(OVERLAPS))
def test_row_passes_refuse_every_overlap(name):
    fn, args, pairs = OVERLAPS[name]
    for out, other in pairs:
        _refused(EINVAL, fn, *[args[other] if k == out else v for k, v in enumerate(args)])


def test_statistics_are_aligned():
    for name, at in (("ln_fwd", 4), ("ln_fwd", 5), ("fwd_pack8", 3), ("fwd_unpack8", 4), ("bwd_unpack8", 3)):
        fn, args, _ = OVERLAPS[name]
        _refused(EINVAL, fn, *[v + 2 if k == at else v for k, v in enumerate(args)])


def test_layernorm_backward_refuses_every_overlap():
    """dy x g mean rstd dres_in dres_out dg db, then the workspace."""
    fn, need = L._fn("lsq_layernorm_bwd"), L.lsq_layernorm_bwd_workspace_size(4, 64)
    a = _at(10)
    for out, others in ((6, (2, 3, 4)), (7, (0, 1, 2, 3, 4, 5, 6)), (8, (0, 1, 2, 3, 4, 5, 6, 7)), (9, range(9))):
        for other in others:
            v = list(a)
            v[out] = v[other]
            assert fn(*v[:9], 0, 4, 64, v[9], need, S) == EINVAL, (out, other)
    for k in (3, 4):
        v = list(a)
        v[k] += 2
        assert fn(*v[:9], 0, 4, 64, v[9], need, S) == EINVAL, k


def test_linear_backward_refuses_every_overlap():
    """dy x w z dx dw dbias, then the workspace."""
    fn, need = L._fn("lsq_linear_bwd"), L.lsq_linear_bwd_workspace_size(4, 64, 64, 2)
    a = _at(8)
    for out, others in ((4, (0, 1, 2, 3)), (5, (0, 1, 2, 3, 4)), (6, (0, 1, 2, 3, 4, 5)), (7, range(7))):
        for other in others:
            v = list(a)
            v[out] = v[other]
            assert fn(*v[:4], 2, v[4], v[5], 1, v[6], 0, 4, 64, 64, v[7], need, S) == EINVAL, (out, other)


@pytest.mark.parametrize("act", [0, 2])
def test_a_workspace_for_more_rows_serves_fewer(act):
    """Sized once for the largest batch, as a ragged run does it."""
    for N in (8, 576, 1000, 4096, 40000):
        sizes = [L.lsq_linear_bwd_workspace_size(M, N, 64, act) for M in (*range(1, 1200), *range(4700, 4800), 9000)]
        assert sizes == sorted(sizes), N
    for d in (8, 64, 576, 2048, 5120, 16384):
        sizes = [L.lsq_layernorm_bwd_workspace_size(r, d) for r in (*range(1, 3100), 5000, 9000)]
        assert sizes == sorted(sizes), d
