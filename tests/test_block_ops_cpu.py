"""Refusals of the LayerNorm, dense-linear and 8-bit checkpoint calls: made on the host before anything is
enqueued, so they are tested without a GPU (raw addresses stand in for device pointers and are never read)."""
import pytest
import torch

from nf4_layer_streamed_blockwise_b200 import lib as L

P = 1 << 20          # a 256-byte aligned address
S = 0                # the default stream's handle
EINVAL, EUNSUPPORTED = 1, 6


def _refused(status, fn, *args, **kw):
    with pytest.raises(L.LsqError) as e:
        fn(*args, stream=S, **kw)
    assert e.value.status == status, e.value


CASES = {
    "ln_fwd": (L.lsq_layernorm_fwd, [P, P, P, P, P, P, 4, 64, 1e-5], (0, 1, 3), (0, 1, 2, 3), 6),
    "pack": (L.lsq_ckpt8_pack, [P, P, 4, 64], (0, 1), (0, 1), 2),
    "unpack": (L.lsq_ckpt8_unpack, [P, P, 4, 64], (0, 1), (0, 1), 2),
    "fwd_pack8": (L.lsq_rmsnorm_fwd_pack8, [P, P, P, P, P, 4, 64, 1e-5], (0, 1, 2, 4), (0, 1, 2, 4), 5),
    "fwd_unpack8": (L.lsq_rmsnorm_fwd_unpack8, [P, P, P, P, P, 4, 64, 1e-5], (0, 1, 2, 3), (0, 1, 2, 3), 5),
    "bwd_unpack8": (L.lsq_rmsnorm_bwd_unpack8, [P, P, P, P, P, P, 4, 64], (0, 1, 2, 3, 5), (0, 1, 2, 4, 5), 6),
}


@pytest.mark.parametrize("name", sorted(CASES))
def test_row_passes_refuse(name):
    fn, args, required, aligned, rows_at = CASES[name]
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
        a = dict(dy=P, x=P, g=P, mean=P, rstd=P, dres_in=P, dres_out=P, dg=P, db=P, accumulate=0, rows=4, d=64,
                 workspace=None)
        a.update(kw)
        _refused(status, L.lsq_layernorm_bwd, *a.values())
    for k in ("dy", "x", "g", "mean", "rstd", "dres_out"):
        call(EINVAL, **{k: None})
    for k in ("dy", "x", "g", "dres_in", "dres_out", "dg", "db"):
        call(EINVAL, **{k: P + 8})
    call(EINVAL)                                 # gradients wanted, no workspace
    call(EINVAL, rows=0)
    call(EINVAL, d=12)
    call(EUNSUPPORTED, d=16392)
    call(EINVAL, workspace=ws)                   # a CPU tensor


def test_linear_forward_refuses():
    def call(status, **kw):
        a = dict(x=P, w=P, bias=P, act=0, residual=P, z=2 * P, y=P, M=4, N=64, K=64)
        a.update(kw)
        _refused(status, L.lsq_linear_fwd, *a.values())
    for k in ("x", "w", "y"):
        call(EINVAL, **{k: None})
    for k in ("x", "w", "bias", "residual", "z", "y"):
        call(EINVAL, **{k: 4 * P + 8})
    for k, v in (("M", 0), ("M", (1 << 30) + 1), ("N", 0), ("N", 60), ("K", 4), ("K", 0), ("K", -8), ("act", -1),
                 ("act", 5)):
        call(EINVAL, **{k: v})
    call(EINVAL, z=P)                            # z on top of y
    call(EINVAL, y=3 * P, z=P)                   # z on top of the residual


def test_linear_backward_refuses():
    def call(status, **kw):
        a = dict(dy=P, x=P, w=P, z=P, act=2, dx=P, dw=P, dw_f32=1, dbias=P, accumulate=0, M=4, N=64, K=64,
                 workspace=None)
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
        call(EINVAL, **{k: P + 4})


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
