"""Training steps with 8-bit activation checkpoints, and the operators outside the quantised base run together.

The gradients of a trainer with checkpoint="int8" are held to the fp64 oracle's true gradients within twice
the error of a CPU model that stores activations in bf16 (bf16_model.py) and takes each layer's backward at the
restored input (the oracle's 8-bit checkpoint): the stated cost of the 8 bits, nothing beyond it."""
import dataclasses

import pytest
import torch

import bf16_model as BM
import synthetic as S
from oracle import block as OB
from oracle import decoder as D
from oracle import train as OT
from tolerances import check_model_grads, rel_fro

pytestmark = pytest.mark.gpu
BF, F32, F64 = torch.bfloat16, torch.float32, torch.float64


def _restored(h):
    flat = h.detach().to(BF).reshape(-1, h.shape[-1])
    return OB.ckpt8_roundtrip(flat).to(F64).reshape(h.shape)


def _model(shape, B, Sq, ids):
    """LoRA gradients with bf16 storage and each layer's backward at its restored input."""
    layers = [OT.dequantized_layer(S.layer_weights(shape, l)) for l in range(shape.n_layers)]
    emb = {k: v.to(F64) for k, v in S.embeddings(shape).items()}
    ops = [{n: {ab: OT.operand(t[ab]) for ab in ("A", "B")} for n, t in per.items()} for per in S.lora_init(shape)]
    hs = [emb["embed"][ids.long()]]
    with torch.no_grad():
        for l, W in enumerate(layers):
            hs.append(BM._layer(hs[-1], W, ops[l], shape, shape.s))
    top = hs[-1].clone().requires_grad_(True)
    hn = BM._st(D.rmsnorm(top, emb["final_norm"], shape.eps))
    loss = D.cross_entropy_next_token(BM._st(hn @ emb["lm_head"].T, fwd=False), ids)
    (dh,) = torch.autograd.grad(loss, top)
    grads = [None] * shape.n_layers
    for l in reversed(range(shape.n_layers)):
        leaves = BM._leaves([ops[l]])[0]
        hin = _restored(hs[l]).requires_grad_(True)
        flat = [leaves[n][ab] for n in leaves for ab in ("A", "B")]
        got = torch.autograd.grad(BM._layer(hin, layers[l], leaves, shape, shape.s), [hin] + flat, grad_outputs=dh)
        dh, it = got[0], iter(got[1:])
        grads[l] = {n: {"A": next(it), "B": next(it)} for n in leaves}
    return grads


def _trainer(shape, B, Sq, n_slots=2, init="host", **kw):
    from nf4_layer_streamed_blockwise_b200.trainer import StreamedLoraTrainer
    return StreamedLoraTrainer(shape, B, Sq, n_slots=n_slots, init=init, **kw)


def _step(tr, ids):
    tr.set_ids(ids.cuda())
    tr.forward_backward()
    torch.cuda.synchronize()
    return tr.loss_dev.item(), tr.lora.grad.clone()


@pytest.mark.parametrize("shape,B,Sq", [(S.TINY, 2, 128), (S.TINY_UNTIED, 1, 200)])
def test_gradients_match_the_oracle(lsq, shape, B, Sq):
    ids = S.tokens(shape, B, Sq, step=0)
    layers = [S.layer_weights(shape, l) for l in range(shape.n_layers)]
    lora = [{n: {ab: t[ab] for ab in ("A", "B")} for n, t in per.items()} for per in S.lora_init(shape)]
    ol, og, _ = OT.train(shape, layers, S.embeddings(shape), lora, [ids])
    tr = _trainer(shape, B, Sq, checkpoint="int8")
    loss, g = _step(tr, ids)
    assert abs(loss - ol[0]) <= 1e-3 * abs(ol[0])
    check_model_grads(tr.lora, g, og, shape, BM.tolerance(og, _model(shape, B, Sq, ids)), what="int8 checkpoints")
    tr.close()


def test_equals_bf16_checkpoints_that_went_through_eight_bits(lsq):
    """The same step with bf16 checkpoints, each replaced by its restored values before its layer's recompute:
    only the norm's summation order differs, so every gradient agrees to a fraction of its bf16 noise."""
    from nf4_layer_streamed_blockwise_b200.trainer import StreamedLoraTrainer

    class RoundTrip(StreamedLoraTrainer):
        def _layer_fwd(self, l, W, save, hin=None, hout=None, adapter=True):
            if save:
                M, d = self.h[l].shape
                ck = torch.empty(lsq.lsq_ckpt8_size(M, d), dtype=torch.uint8, device="cuda")
                lsq.lsq_ckpt8_pack(self.h[l], ck, M, d)
                lsq.lsq_ckpt8_unpack(ck, self.h[l], M, d)
            super()._layer_fwd(l, W, save, hin, hout, adapter)

    shape, B, Sq = S.TINY_UNTIED, 2, 128
    ids = S.tokens(shape, B, Sq, step=0)
    a = RoundTrip(shape, B, Sq, n_slots=2, init="host")
    la, ga = _step(a, ids)
    b = _trainer(shape, B, Sq, checkpoint="int8")
    lb, gb = _step(b, ids)
    assert abs(la - lb) <= 1e-4 * abs(la)
    for l in range(shape.n_layers):
        for n in S.LINEARS:
            for ab in ("A", "B"):
                x, y = (t.lora.view(g, l, n, ab).double().cpu().numpy() for t, g in ((a, ga), (b, gb)))
                assert rel_fro(y, x) <= 1e-2, (l, n, ab)
    a.close()
    b.close()


@pytest.mark.parametrize("kind", ["sft", "dpo"])
def test_streamed_resident_and_replayed_agree_bitwise(lsq, kind):
    shape, B, Sq = dataclasses.replace(S.TINY_UNTIED, n_layers=4), 2, 128
    runs = []
    with torch.cuda.stream(torch.cuda.Stream()):
        for n_slots, graph in ((2, False), (None, False), (2, True)):
            tr = _trainer(shape, B, Sq, n_slots=n_slots, init="device", graph=graph, checkpoint="int8")
            out = []
            for t in range(4):
                tr.set_ids(S.tokens(shape, B, Sq, step=t).cuda())
                tr.forward_backward_dpo(0.1) if kind == "dpo" else tr.forward_backward()
                torch.cuda.synchronize()
                out += [tr.loss_dev.clone(), tr.lora.grad.clone()]
                tr.optimizer_step()
            runs.append(out)
            tr.close()
    for other in runs[1:]:
        for x, y in zip(runs[0], other):
            assert torch.equal(x, y)


def test_without_the_rank_state(lsq):
    """The recompute then runs the down projection too and rebuilds the rank-r operands."""
    shape, B, Sq = S.TINY, 1, 96
    ids = S.tokens(shape, B, Sq, step=0)
    a, b = (_trainer(shape, B, Sq, checkpoint="int8") for _ in range(2))
    b.keep_rank_state = False
    (la, ga), (lb, gb) = _step(a, ids), _step(b, ids)
    assert abs(la - lb) <= 1e-4 * abs(la)
    # s U of the forward against s U of the restored inputs: the 8-bit error itself, about half a percent
    assert (ga - gb).norm() <= 3e-2 * ga.norm()
    a.close()
    b.close()


def test_checkpoints_take_half_the_memory(lsq):
    shape, B, Sq = S.TINY_UNTIED, 2, 256
    a, b = _trainer(shape, B, Sq), _trainer(shape, B, Sq, checkpoint="int8")
    bf16 = a.h.numel() * 2 - B * Sq * shape.d * 2          # one of its entries is the stack's output
    assert b.ckpt.numel() <= 0.52 * bf16
    a.close()
    b.close()
    with pytest.raises(ValueError):
        _trainer(shape, B, Sq, checkpoint="fp8")


# ---------------------------------------------------------------- the operators together
class Block:
    """y = x + W2 gelu(W1 LN(x) + b1) + b2 with x kept as an 8-bit checkpoint and every gradient wanted."""

    def __init__(self, lsq, M, d, f, seed=0):
        g = torch.Generator().manual_seed(seed)
        self.L, self.M, self.d, self.f = lsq, M, d, f

        def n(*s, std=1.0, at=0.0):
            return (at + std * torch.randn(*s, generator=g)).to(BF).cuda()
        self.x, self.dy = n(M, d), n(M, d)
        self.g, self.b = n(d, std=0.2, at=1.0), n(d, std=0.1)
        self.w1, self.b1 = n(f, d, std=d ** -0.5), n(f, std=0.1)
        self.w2, self.b2 = n(d, f, std=f ** -0.5), n(d, std=0.1)

        def e(*s, dt=BF):
            return torch.empty(*s, dtype=dt, device="cuda")
        self.ck = e(lsq.lsq_ckpt8_size(M, d), dt=torch.uint8)
        self.xr, self.h, self.y, self.dx, self.dh = (e(M, d) for _ in range(5))
        self.z, self.m, self.dm = (e(M, f) for _ in range(3))
        self.mean, self.rstd = e(M, dt=F32), e(M, dt=F32)
        self.grads = {"dg": e(d, dt=F32), "db": e(d, dt=F32), "dw1": e(f, d, dt=F32), "db1": e(f, dt=F32),
                      "dw2": e(d, f), "db2": e(d, dt=F32)}
        self.ws = e(max(lsq.lsq_linear_bwd_workspace_size(M, f, d, lsq.ACT_GELU),
                        lsq.lsq_linear_bwd_workspace_size(M, d, f, lsq.ACT_NONE),
                        lsq.lsq_layernorm_bwd_workspace_size(M, d)), dt=torch.uint8)

    def _mlp(self, x, y):
        L, M, d, f = self.L, self.M, self.d, self.f
        L.lsq_layernorm_fwd(x, self.g, self.b, self.h, self.mean, self.rstd, M, d, 1e-5)
        L.lsq_linear_fwd(self.h, self.w1, self.b1, L.ACT_GELU, None, self.z, self.m, M, f, d)
        if y is not None:
            L.lsq_linear_fwd(self.m, self.w2, self.b2, L.ACT_NONE, x, None, y, M, d, f)

    def run(self):
        L, M, d, f, G = self.L, self.M, self.d, self.f, self.grads
        L.lsq_ckpt8_pack(self.x, self.ck, M, d)
        self._mlp(self.x, self.y)
        L.lsq_ckpt8_unpack(self.ck, self.xr, M, d)     # the recompute starts here
        self._mlp(self.xr, None)
        L.lsq_linear_bwd(self.dy, self.m, self.w2, None, L.ACT_NONE, self.dm, G["dw2"], 0, G["db2"], 0, M, d, f,
                         self.ws)
        L.lsq_linear_bwd(self.dm, self.h, self.w1, self.z, L.ACT_GELU, self.dh, G["dw1"], 1, G["db1"], 0, M, f, d,
                         self.ws)
        L.lsq_layernorm_bwd(self.dh, self.xr, self.g, self.mean, self.rstd, self.dy, self.dx, G["dg"], G["db"], 0, M,
                            d, self.ws)

    def outputs(self):
        return {"y": self.y, "dx": self.dx, "xr": self.xr, **self.grads}

    def reference(self):
        names = ("x", "g", "b", "w1", "b1", "w2", "b2")

        def f(x, g, b, w1, b1, w2, b2):
            _, m = OB.linear(OB.layernorm(x, g, b, 1e-5), w1, b1, "gelu")
            return OB.linear(m, w2, b2, "none", x)[1]
        vals = {n: getattr(self, n).double().cpu() for n in names}
        y = f(**vals)
        xr = OB.ckpt8_roundtrip(self.x.cpu()).double()
        leaves = [t.clone().requires_grad_(True) for t in (xr, *(vals[n] for n in names[1:]))]
        gr = torch.autograd.grad(f(*leaves), leaves, grad_outputs=self.dy.double().cpu())
        return {"y": y, "xr": xr, **dict(zip(("dx", "dg", "db", "dw1", "db1", "dw2", "db2"), gr))}


@pytest.mark.parametrize("M,d,f", [(1, 64, 256), (100, 264, 1000), (333, 576, 1536), (2048, 512, 2048)])
def test_block_under_a_checkpoint(lsq, M, d, f):
    b = Block(lsq, M, d, f)
    b.run()
    ref = b.reference()
    for name, got in b.outputs().items():
        # seven bf16 roundings lie between the restored input and the farthest gradient (h, z, m, dm, dz, dh and
        # the result), each 2^-8 / sqrt(6) of its value in RMS (uniform over half a step): 1.2e-2 if all aligned
        err = rel_fro(got.double().cpu().numpy(), ref[name].numpy())
        assert err <= (0.0 if name == "xr" else 1.2e-2), (name, err)


def test_block_captured_replayed_and_on_other_streams(lsq):
    """Captured once and replayed on new inputs, and run on two streams at once (own workspaces): the eager
    results, bit for bit."""
    shapes = (260, 320, 1096)
    want = []
    for seed in (1, 2):
        b = Block(lsq, *shapes, seed=seed)
        b.run()
        torch.cuda.synchronize()
        want.append({k: v.clone() for k, v in b.outputs().items()})
    b = Block(lsq, *shapes, seed=1)
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            b.run()
    other = Block(lsq, *shapes, seed=2)
    for w, src in ((want[0], b), (want[1], other)):
        for n in ("x", "dy", "g", "b", "w1", "b1", "w2", "b2"):
            getattr(b, n).copy_(getattr(src, n))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for k, v in b.outputs().items():
            assert torch.equal(v, w[k]), k
    blocks = [Block(lsq, *shapes, seed=k) for k in (1, 2)]
    streams = [torch.cuda.Stream() for _ in blocks]
    torch.cuda.synchronize()
    for _ in range(3):
        for blk, st in zip(blocks, streams):
            with torch.cuda.stream(st):
                blk.run()
    torch.cuda.synchronize()
    for blk, w in zip(blocks, want):
        for k, v in blk.outputs().items():
            assert torch.equal(v, w[k]), k
