"""Every tensor argument of the layers outside the quantised base, wrong in one property at a time, through the calls:
refused on the host, nothing enqueued."""
import pytest
import torch

pytestmark = pytest.mark.gpu
BF, F32, U8 = torch.bfloat16, torch.float32, torch.uint8
R, D, N = 6, 64, 72


def _calls(lsq):
    """name -> call, its arguments by name (a tensor, or a plain value), the tensors' exact needs."""
    def bf(*s):
        return torch.zeros(*s, dtype=BF, device="cuda")

    def f32(*s):
        return torch.zeros(*s, dtype=F32, device="cuda")

    def ckpt():
        return torch.zeros(lsq._ckpt8_used(R, D), dtype=U8, device="cuda")
    ws = torch.zeros(1 << 16, dtype=U8, device="cuda")
    return {
        "layernorm_fwd": (lsq.lsq_layernorm_fwd, [bf(R, D), bf(D), bf(D), bf(R, D), f32(R), f32(R), R, D, 1e-5]),
        "layernorm_bwd": (lsq.lsq_layernorm_bwd, [bf(R, D), bf(R, D), bf(D), f32(R), f32(R), bf(R, D), bf(R, D), f32(D),
                                                  f32(D), 0, R, D, ws]),
        "pack": (lsq.lsq_ckpt8_pack, [bf(R, D), ckpt(), R, D]),
        "unpack": (lsq.lsq_ckpt8_unpack, [ckpt(), bf(R, D), R, D]),
        "fwd_pack8": (lsq.lsq_rmsnorm_fwd_pack8, [bf(R, D), bf(D), bf(R, D), f32(R), ckpt(), R, D, 1e-5]),
        "fwd_unpack8": (lsq.lsq_rmsnorm_fwd_unpack8, [ckpt(), bf(D), bf(R, D), bf(R, D), f32(R), R, D, 1e-5]),
        "bwd_unpack8": (lsq.lsq_rmsnorm_bwd_unpack8, [bf(R, D), ckpt(), bf(D), f32(R), bf(R, D), bf(R, D), R, D]),
        "linear_fwd": (lsq.lsq_linear_fwd, [bf(R, D), bf(N, D), bf(N), 1, bf(R, N), bf(R, N), bf(R, N), R, N, D]),
        "linear_bwd": (lsq.lsq_linear_bwd, [bf(R, N), bf(R, D), bf(N, D), bf(R, N), 1, bf(R, D), f32(N, D), 1, f32(N), 0,
                                            R, N, D, ws]),
    }


NAMES = ("layernorm_fwd", "layernorm_bwd", "pack", "unpack", "fwd_pack8", "fwd_unpack8", "bwd_unpack8", "linear_fwd",
         "linear_bwd")


@pytest.mark.parametrize("name", NAMES)
def test_each_wrong_tensor_is_refused(lsq, name):
    fn, args = _calls(lsq)[name]
    fn(*args)                                             # as it stands it runs
    before = lsq.lsq_launch_count()
    for i, a in enumerate(args):
        if not torch.is_tensor(a):
            continue
        wrong = []
        if a.dtype != U8:                                 # checkpoints and workspaces go by bytes
            wrong.append(("must be torch", a.to(torch.float16)))
        if a.numel() != 1 << 16:                          # the workspace's size is the library's to check
            wrong.append(("needs", a.flatten()[:-1]))
        wrong.append(("must be contiguous", torch.zeros(a.numel(), 2, dtype=a.dtype, device="cuda")[:, 0]))
        wrong.append(("must be on the current CUDA device", a.cpu()))
        for why, t in wrong:
            with pytest.raises(lsq.LsqError, match=why) as e:
                fn(*args[:i], t, *args[i + 1:])
            assert e.value.status == 1, (name, i, why)
    assert lsq.lsq_launch_count() == before
