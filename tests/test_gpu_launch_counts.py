"""The launch counter against the kernel nodes of a captured graph, for the calls that choose between one kernel and
several by their sizes and arguments."""
import ctypes

import pytest
import torch

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def _kernel_nodes(graph):
    cu = ctypes.CDLL("libcuda.so.1")
    raw, n = ctypes.c_void_p(graph.raw_cuda_graph()), ctypes.c_size_t(0)
    assert cu.cuGraphGetNodes(raw, None, ctypes.byref(n)) == 0
    nodes = (ctypes.c_void_p * max(n.value, 1))()
    assert cu.cuGraphGetNodes(raw, nodes, ctypes.byref(n)) == 0
    kernels = 0
    for node in nodes[:n.value]:
        kind = ctypes.c_int(-1)
        assert cu.cuGraphNodeGetType(ctypes.c_void_p(node), ctypes.byref(kind)) == 0
        kernels += kind.value == 0
    return kernels


def _bf(*shape):
    return torch.randn(*shape, device="cuda").to(BF)


def _layernorm(rows, d, grads, in_place):
    def make(lsq):
        x, dy, g = _bf(rows, d), _bf(rows, d), _bf(d)
        mean, rstd = torch.zeros(rows, device="cuda"), torch.ones(rows, device="cuda")
        dg, db = (torch.empty(d, device="cuda") if grads else None for _ in range(2))
        out = dy if in_place else torch.empty_like(x)
        ws = torch.empty(lsq.lsq_layernorm_bwd_workspace_size(rows, d), dtype=torch.uint8, device="cuda")
        return lambda: lsq.lsq_layernorm_bwd(dy, x, g, mean, rstd, None, out, dg, db, 0, rows, d, ws)
    return make


def _linear(M, N, K, act, dx, dw, db):
    def make(lsq):
        dy, x, w, z = _bf(M, N), _bf(M, K), _bf(N, K), _bf(M, N)
        gx, gw = torch.empty_like(x) if dx else None, torch.empty_like(w) if dw else None
        gb = torch.empty(N, device="cuda") if db else None
        ws = torch.empty(lsq.lsq_linear_bwd_workspace_size(M, N, K, act), dtype=torch.uint8, device="cuda")
        return lambda: lsq.lsq_linear_bwd(dy, x, w, z if act else None, act, gx, gw, 0, gb, 0, M, N, K, ws)
    return make


def _forwards(lsq):
    M, N, K = 40, 64, 128
    x, w, y, h = _bf(M, K), _bf(N, K), _bf(M, N), _bf(M, K)
    rstd, g = torch.empty(M, device="cuda"), _bf(K)
    ck = torch.empty(lsq.lsq_ckpt8_size(M, K), dtype=torch.uint8, device="cuda")

    def run():
        lsq.lsq_layernorm_fwd(x, g, None, h, None, None, M, K, 1e-5)
        lsq.lsq_rmsnorm_fwd(x, g, h, rstd, M, K, 1e-5)          # counted on the binding's side
        lsq.lsq_rmsnorm_fwd_pack8(x, g, h, rstd, ck, M, K, 1e-5)
        lsq.lsq_rmsnorm_fwd_unpack8(ck, g, x, h, rstd, M, K, 1e-5)
        lsq.lsq_rmsnorm_bwd_unpack8(h, ck, g, rstd, None, h, M, K)
        lsq.lsq_ckpt8_pack(x, ck, M, K)
        lsq.lsq_ckpt8_unpack(ck, x, M, K)
        lsq.lsq_linear_fwd(x, w, None, 2, None, None, y, M, N, K)
        lsq.lsq_linear_fwd(x, w, None, 2, None, None, y, 1, N, K)
    return run


# calls, and their kernels on 148 SMs where the case is there for that number
CASES = {
    "forwards": (_forwards, 9),
    "ln few": (_layernorm(100, 576, True, False), 1),
    "ln few frozen": (_layernorm(100, 576, False, False), 1),
    "ln few in place": (_layernorm(100, 576, True, True), 2),     # the sums read dy before the rows overwrite it
    "ln few in place frozen": (_layernorm(100, 576, False, True), 1),
    "ln rings": (_layernorm(2000, 1024, True, False), 2),
    "ln rings frozen": (_layernorm(2000, 1024, False, True), 1),
    "ln short rows": (_layernorm(1200, 64, True, False), 2),
    "linear dbias joined": (_linear(100, 256, 64, 0, False, False, True), 1),
    "linear dbias in two": (_linear(4000, 256, 64, 0, False, False, True), 2),
    "linear all, together": (_linear(130, 576, 1536, 2, True, True, True), 2),
    "linear all, apart": (_linear(3000, 2048, 1024, 2, True, True, True), None),
    "linear dx": (_linear(130, 576, 1536, 0, True, False, False), 1),
    "linear dw of an activation": (_linear(130, 576, 1536, 3, False, True, False), 2),
}


@pytest.mark.parametrize("name", sorted(CASES))
def test_counter_equals_the_graphs_kernels(lsq, name):
    make, expected = CASES[name]
    run = make(lsq)
    run()                                               # set-up of the kernels' attributes outside the capture
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph(keep_graph=True)
    before = lsq.LAUNCHES[0]
    with torch.cuda.graph(graph):
        run()
    counted = lsq.LAUNCHES[0] - before
    assert counted == _kernel_nodes(graph)
    assert expected is None or counted == expected


def test_the_counter_is_set_and_added_to(lsq):
    """As a benchmark resets it, and a replayed graph adds its kernels."""
    run = _layernorm(100, 576, True, True)(lsq)
    lsq.LAUNCHES[0] = 0
    run()
    assert lsq.LAUNCHES[0] == 2
    lsq.LAUNCHES[0] += 5
    run()
    assert lsq.LAUNCHES[0] == 9
