"""The workspace of a prepared layer on the device: its size, and graphs that
captured one which was outgrown since."""
import pytest
import torch

from test_gpu_linear_act import Layer

pytestmark = pytest.mark.gpu
N_IN, N_OUT = 1024, 512


@pytest.fixture(scope="module")
def B(cuda_lib):
    from rotated_w4_linear_b200 import binding
    yield binding
    assert binding.paro_fault_status() == 0


def test_no_more_memory_than_the_largest_batch_needs(B):
    L = Layer(B, 4096, N_IN, N_OUT, seed=1)
    layer = B.ParoLinear(L.rot, *L.packed, N_IN, N_OUT)
    y = torch.empty(4096, N_OUT, dtype=torch.float16, device="cuda")
    torch.cuda.synchronize()
    before = torch.cuda.memory_allocated()
    for T in (17, 2047, 2048, 4095, 4096, 5):
        layer(L.x[:T], y[:T])
    need = B.paro_linear_workspace_size(4096, N_IN, N_OUT)
    assert torch.cuda.memory_allocated() - before <= need + 512


@pytest.mark.parametrize("explicit", [False, True])
def test_graphs_of_growing_batches_keep_their_workspaces(B, explicit):
    """Calls captured at three batch sizes, each before the layer grew, with the
    capture's stream given or not; replays after all of it, and memory asked
    for in between, give the eager calls' bits."""
    L = Layer(B, 300, N_IN, N_OUT, seed=2)
    layer = B.ParoLinear(L.rot, *L.packed, N_IN, N_OUT, act="silu")
    graphs, outs, junk = [], [], []
    for T in (9, 40, 300):
        x = L.x[:T].clone()
        layer(x)
        y = torch.empty(T, N_OUT, dtype=torch.float16, device="cuda")
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            layer(x, y, stream=torch.cuda.current_stream() if explicit else None)
        graphs.append(graph)
        outs.append((x, y))
    for T in (20, 41, 299, 300):
        layer(L.x[:T])
        junk.append([torch.full((n,), 255, dtype=torch.uint8, device="cuda")
                     for n in (2 * 9 * N_IN, 2 * 40 * N_IN, 2 * 300 * N_IN)])
    for graph, (x, y) in zip(graphs, outs):
        for _ in range(3):
            y.zero_()
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(y, B.paro_linear_act(L.rot, x, *L.packed, N_OUT, act="silu"))
    torch.cuda.synchronize()
    assert all(bool((j == 255).all()) for js in junk for j in js)
