"""What the binding checks of a tensor that an address cannot carry, one property wrong at a time (CPU tensors stand in:
their device index is -1)."""
import pytest
import torch

from nf4_layer_streamed_blockwise_b200 import lib as L

BF, F32, U8 = torch.bfloat16, torch.float32, torch.uint8
CPU = -1


def _refused(why, t, dtype, n, dev=CPU):
    with pytest.raises(L.LsqError, match=why) as e:
        L._t("lsq_some_call", "arg", t, dtype, n, dev)
    assert e.value.status == 1 and "lsq_some_call" in str(e.value) and "arg" in str(e.value)


def test_a_good_tensor_passes():
    x = torch.zeros(4, 64, dtype=BF)
    assert L._t("f", "x", x, BF, 256, CPU) == x.data_ptr()
    assert L._t("f", "x", x, BF, 200, CPU) == x.data_ptr()             # longer than needed
    assert L._t("f", "x", x[1:], BF, 192, CPU) == x.data_ptr() + 128   # a dense part
    b = torch.zeros(100, dtype=U8)
    assert L._t("f", "ckpt", b, None, 100, CPU) == b.data_ptr()
    assert L._t("f", "ckpt", x, None, 512, CPU) == x.data_ptr()        # any type, by bytes
    assert L._t("f", "x", None, BF, 8, CPU) is None and L._t("f", "x", 4096, BF, 8, CPU) == 4096


def test_type():
    x = torch.zeros(4, 64, dtype=BF)
    for t in (x.float(), x.half(), x.view(torch.int16), x.double()):
        _refused("must be torch.bfloat16", t, BF, 256)
    _refused("must be torch.float32", x, F32, 256)


def test_length():
    x = torch.zeros(4, 64, dtype=BF)
    _refused("needs 257", x, BF, 257)
    _refused("needs 256", x[:3], BF, 256)
    _refused("needs 513 bytes", x, None, 513)
    _refused("needs 101 bytes", torch.zeros(100, dtype=U8), None, 101)


def test_density():
    x = torch.zeros(8, 64, dtype=BF)
    for t in (x[:, :32], x.t(), x[::2], x[:4, :1].expand(4, 64)):
        assert t.numel() >= 256
        _refused("must be contiguous", t, BF, 256)
        _refused("must be contiguous", t, None, 512)


def test_device():
    x = torch.zeros(4, 64, dtype=BF)
    for dev in (0, 1, -2):                                             # -2: CUDA is not up
        _refused("current CUDA device, got cpu", x, BF, 256, dev)
        _refused("current CUDA device, got cpu", x, None, 512, dev)
