"""Pins of the fp64 oracle for LayerNorm, the dense linear's activations and the 8-bit checkpoint: closed
forms, finite differences, and the checkpoint's definition evaluated another way."""
import math

import numpy as np
import pytest
import torch

from oracle import block as K

F64 = torch.float64


def test_layernorm_closed_form_and_invariances():
    x = torch.tensor([[1.0, -1.0, 1.0, -1.0]], dtype=F64)
    g, b = torch.full((4,), 2.0, dtype=F64), torch.full((4,), 0.5, dtype=F64)
    y = K.layernorm(x, g, b, 0.0)
    assert torch.allclose(y, torch.tensor([[2.5, -1.5, 2.5, -1.5]], dtype=F64), atol=1e-15)
    assert torch.allclose(K.layernorm(3 * x + 7, g, b, 0.0), y, atol=1e-14)   # shift and scale drop out


@pytest.mark.parametrize("kind,at_one", [("relu", 1.0), ("gelu", 0.8413447460685429),
                                         ("gelu_tanh", 0.8411919906082768), ("silu", 0.7310585786300049),
                                         ("none", 1.0)])
def test_activation_values_and_gradients(kind, at_one):
    assert abs(K.act(torch.tensor(1.0, dtype=F64), kind).item() - at_one) < 1e-14
    z = torch.tensor([-3.0, -0.7, 0.3, 2.1], dtype=F64).requires_grad_(True)
    (dz,) = torch.autograd.grad(K.act(z, kind).sum(), z)
    h = 1e-6
    fd = (K.act(z.detach() + h, kind) - K.act(z.detach() - h, kind)) / (2 * h)
    assert torch.allclose(dz, fd, atol=1e-8)


def test_checkpoint_block_by_hand():
    x = torch.zeros(1, 64, dtype=torch.bfloat16)
    x[0, :5] = torch.tensor([127.0, 63.5, -63.5, 0.5, 0.49])
    codes, amax = K.ckpt8_pack(x)
    # amax = 127, so a code is the value rounded, halves away from zero
    assert amax[0, 0] == 0x42FE and list(codes[0, :5]) == [127, 64, -64, 1, 0]
    assert K.ckpt8_unpack(codes, amax)[0, :5].tolist() == [127.0, 64.0, -64.0, 1.0, 0.0]


def test_checkpoint_error_bound_and_fixed_points():
    g = np.random.default_rng(3)
    x = torch.from_numpy(g.standard_normal((6, 200)).astype(np.float32)).to(torch.bfloat16)
    back = K.ckpt8_roundtrip(x)
    top = torch.stack([c.double().abs().amax(1) for c in x.split(64, dim=1)], 1).repeat_interleave(64, 1)[:, :200]
    # half a code step, plus one bf16 rounding of the restored value
    assert torch.all((back.double() - x.double()).abs() <= top / 254 + back.double().abs() * 2.0 ** -8)
    hit = x.double().abs() == top
    assert torch.equal(back[hit], x[hit])                  # the largest magnitude is exact
    assert torch.equal(K.ckpt8_roundtrip(back), back)      # what was restored is kept as it is


def test_checkpoint_special_blocks():
    x = torch.ones(1, 64 * 4 + 8, dtype=torch.bfloat16)
    x[0, 3] = float("inf")
    x[0, 64 + 5] = float("nan")
    x[0, 128:192] = 2.0 ** -119
    x[0, 192:256] = 0.0
    back = K.ckpt8_roundtrip(x)[0].float()
    assert back[:128].isnan().all() and (back[128:256] == 0).all() and (back[256:] == 1).all()
    assert math.isclose(K.ckpt8_roundtrip(torch.full((1, 8), 2.0 ** -118, dtype=torch.bfloat16))[0, 0].item(),
                        2.0 ** -118)
