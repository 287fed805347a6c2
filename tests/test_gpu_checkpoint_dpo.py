"""DPO with 8-bit activation checkpoints: the adapter-off reference and the policy go through the same arithmetic."""
import dataclasses
import math

import numpy as np
import pytest
import torch

import synthetic as S

pytestmark = pytest.mark.gpu
BETA = 0.1


def _run(shape, B, Sq, checkpoint):
    from nf4_layer_streamed_blockwise_b200.trainer import StreamedLoraTrainer
    tr = StreamedLoraTrainer(shape, B, Sq, n_slots=2, init="device", checkpoint=checkpoint)
    for l in range(shape.n_layers):
        for n in S.LINEARS:
            tr.lora.view(tr.lora.op, l, n, "B").zero_()
    out = []
    for step in range(3):
        tr.set_ids(S.tokens(shape, B, Sq, step=step).cuda())
        tr.forward_backward_dpo(BETA)
        torch.cuda.synchronize()
        out.append([t.double().cpu() for t in (tr.pi_logp, tr.ref_logp, tr.loss_dev, tr.dseq)])
    tr.close()
    return out


@pytest.mark.parametrize("checkpoint", ["bf16", "int8"])
@pytest.mark.parametrize("shape,B,Sq", [(S.TINY, 4, 64), (S.TINY_UNTIED, 2, 96),
                                        (dataclasses.replace(S.SMOL, n_layers=4), 8, 512)])
def test_zero_b_policy_is_reference_bitwise(lsq, shape, B, Sq, checkpoint):
    """With every LoRA B zero the sequence log-probabilities are equal bit for bit, the loss log 2 and its gradient
    +-beta / (2 P), with either kind of checkpoint.  Two norms that add a row's squares in another order give an output
    of another rounding about twice in a million: the last case has ten million in each pass."""
    for pi, ref, loss, dseq in _run(shape, B, Sq, checkpoint):
        assert torch.equal(pi, ref), (pi - ref).abs().max()
        assert abs(loss.item() - math.log(2.0)) < 1e-6
        want = np.array([-BETA / 2 / (B // 2), BETA / 2 / (B // 2)] * (B // 2))
        np.testing.assert_allclose(dseq.numpy(), want, rtol=1e-6)
