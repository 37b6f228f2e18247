"""Clipped steps of a ScapeState that do not run on the current stream: the
norms and their workspace are there before the first of them, so nothing that
the current stream still has to do reaches them."""
import math

import pytest
import torch

import synth

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def sc():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import sparse_communication_adam_amd as sc
    sc.lib()
    yield sc
    torch.cuda.empty_cache()


def _state(sc, interleaved, offload=False):
    from sparse_communication_adam_amd.state import ScapeState
    wl = synth.ragged()
    return ScapeState(sc.ScapeConfig(layer_numel=wl.layer_sizes, workers=wl.W, keep_num=1, keep_den=5), interleaved=interleaved,
                      offload=offload)


def _grads(state, interleaved, seed):
    """int16 gradients, zeros behind each layer; worker 1 holds an infinity."""
    W, lay = state.cfg.workers, state.layout
    g = torch.Generator().manual_seed(seed)
    flat = torch.zeros(W, lay.n_pad, dtype=torch.bfloat16)
    for off, n in zip(lay.layer_offset, state.cfg.layer_numel):
        flat[:, off:off + n] = torch.randn(W, n, generator=g).to(torch.bfloat16)
    flat[1, lay.layer_offset[0]] = math.inf
    flat = flat.view(torch.int16).cuda()
    if interleaved:
        return flat.view(W, -1, 64).transpose(0, 1).reshape(-1).contiguous()
    return [f.contiguous() for f in flat]


def _bits(grads):
    return [grads] if isinstance(grads, torch.Tensor) else grads


def _same(a, b):
    assert torch.equal(a.grad_norm.view(torch.int32), b.grad_norm.view(torch.int32))
    assert torch.equal(a.x, b.x) and torch.equal(a.m, b.m) and torch.equal(a.v, b.v)
    for i in range(a.cfg.workers):
        assert torch.equal(a.residual(i).cpu(), b.residual(i).cpu())


@pytest.mark.parametrize("interleaved,offload", [(False, False), (True, False), (False, True)])
def test_first_clipped_step_on_another_stream(sc, interleaved, offload):
    want, got = _state(sc, interleaved), _state(sc, interleaved, offload)
    mine, theirs = _grads(want, interleaved, 3), _grads(want, interleaved, 3)
    want.step(mine, max_norm=0.5)
    a = torch.randn(4096, 4096, device="cuda")
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    assert math.isinf(float(want.grad_norm[1])) and float(want.grad_norm[0]) > 0.5
    s.wait_stream(torch.cuda.current_stream())
    for _ in range(40):  # work of the current stream that is still to come when the step runs on s
        a = torch.tanh(a @ a)
    got.step(theirs, max_norm=0.5, stream=s)
    s.synchronize()
    norm = got.grad_norm.clone()
    torch.cuda.synchronize()
    assert torch.equal(got.grad_norm.view(torch.int32), norm.view(torch.int32))
    _same(got, want)
    for x, y in zip(_bits(theirs), _bits(mine)):
        assert torch.equal(x, y)


@pytest.mark.parametrize("interleaved", [False, True])
def test_first_clipped_step_in_the_callers_graph(sc, interleaved):
    """The norms do not lie in the graph's own memory: they outlive it."""
    want, got = _state(sc, interleaved), _state(sc, interleaved)
    mine, theirs = _grads(want, interleaved, 5), _grads(want, interleaved, 5)
    at = got.grad_norm.data_ptr()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got.step(theirs, max_norm=0.5)
    assert got.grad_norm.data_ptr() == at
    want.step(mine, max_norm=0.5)
    graph.replay()
    torch.cuda.synchronize()
    _same(got, want)
    del graph
    torch.cuda.empty_cache()
    again, same = _grads(want, interleaved, 6), _grads(want, interleaved, 6)
    want.step(again, max_norm=0.5)
    got.step(same, max_norm=0.5)
    torch.cuda.synchronize()
    _same(got, want)
