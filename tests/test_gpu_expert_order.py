"""The backward's three launches overlap: each reads what the call's own
quantizer wrote, whatever the workspace held before."""

import pytest
import torch

pytestmark = pytest.mark.gpu


def _bsmm():
    import block_scaled_precision_gemm_gb300 as bsmm
    return bsmm


def inputs(seed, S, E, N, K, dtype=torch.bfloat16):
    g = torch.Generator("cuda").manual_seed(seed)

    def rnd(*s):
        return torch.randn(*s, device="cuda", generator=g).to(dtype)

    cuts = torch.sort(torch.randint(0, S + 1, (E - 1,), device="cuda", generator=g)).values
    offsets = torch.cat([cuts.new_zeros(1), cuts, cuts.new_full((1,), S)]).to(torch.int32)
    return rnd(S, N), rnd(E, N, K), rnd(S // 2, K), offsets, \
        torch.randint(0, S // 2, (S,), device="cuda", generator=g, dtype=torch.int32)


@pytest.mark.parametrize("S,E,N,K", [(4096, 8, 1024, 1024), (700, 20, 288, 544), (6000, 3, 2048, 512)])
def test_graphs_that_share_a_workspace(S, E, N, K):
    """Two captured calls replayed in turn and eager ones between them, dW's tiles
    more than a wave, give the bits of each call alone."""
    bsmm = _bsmm()
    sets = [inputs(i, S, E, N, K) for i in range(3)]
    alone = []
    for dY, W, X, off, rows in sets:
        alone.append([t.clone() for t in bsmm.expert_backward(dY, W, X, off, rows=rows)])
        torch.cuda.synchronize()
    ws = torch.full((bsmm.expert_backward_workspace_size(S, E, N, K),), 0xFF, dtype=torch.uint8, device="cuda")

    def call(i):
        dY, W, X, off, rows = sets[i]
        return bsmm.expert_backward(dY, W, X, off, rows=rows, workspace=ws)

    graphs = []
    for i in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = call(i)
        graphs.append((graph, out))
    for n in range(12):
        graph, out = graphs[n % 2]
        graph.replay()
        got = [(n % 2, [t.clone() for t in out])]
        if n % 3 == 0:
            got.append((2, call(2)))
        for i, pair in got:
            assert torch.equal(pair[0], alone[i][0]) and torch.equal(pair[1], alone[i][1]), n
    assert bsmm.check_device_status()[0] == 0
