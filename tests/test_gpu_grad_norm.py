"""Gradient norms and clipping in a context's layout, against float64.

Squares of bf16 values are exact in float64 and their sums are off by at most
n 2^-53, so a norm is off by its own rounding and that of a square root taken
of such a sum: 2 u, u = 2^-24.  A clipped value has its factor's rounding (a
float32 quotient, 2 u with the norm's own) and its own, half a step of 8 bits.
"""
import math
import zlib

import numpy as np
import pytest
import torch

import synth

pytestmark = pytest.mark.gpu

U, HALF = 2.0 ** -24, 2.0 ** -8
NAN, INF = math.nan, math.inf


@pytest.fixture(scope="module", autouse=True)
def sc():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import sparse_communication_adam_amd as sc
    sc.lib()
    yield sc
    torch.cuda.empty_cache()


LAYERS = {
    "ragged": [1000, 37, 1, 64, 4097, 33 * 65, 70000],
    "empty layers": [0, 5, 0, 0, 129, 0],
    "tiles": [32768, 32769, 65535, 7, 8, 9, 131072],
    "one": [1],
    "nothing": [0, 0],
}


class Grads:
    """W workers' gradients in both layouts, NaN between the layers."""

    def __init__(self, sc, sizes, W, key="", spread=True):
        g = torch.Generator().manual_seed(zlib.crc32(f"{sizes}{W}{key}".encode()))
        self.W, self.sizes = W, sizes
        self.ctx = sc.Context(sc.ScapeConfig(layer_numel=sizes, workers=W, keep_num=1, keep_den=10))
        lay = self.ctx.layout
        self.off, n = lay.layer_offset, lay.n_pad
        self.flat = torch.full((W, n), NAN, dtype=torch.bfloat16)
        self.inside = torch.zeros(n, dtype=torch.bool)
        for o, m in zip(self.off, sizes):
            s = 10.0 ** -float(torch.randint(0, 5, (1,), generator=g)) if spread else 1.0
            self.flat[:, o:o + m] = (torch.randn(W, m, generator=g) * s * (1 + torch.arange(W)[:, None])).to(torch.bfloat16)
            self.inside[o:o + m] = True

    def given(self, interleaved):
        if not interleaved:
            return [f.contiguous().cuda() for f in self.flat]
        return self.flat.view(self.W, -1, 64).transpose(0, 1).contiguous().view(-1).cuda()

    def back(self, t, interleaved):
        """[W, n_pad] of a call's output, on the host."""
        if not interleaved:
            return torch.stack([x.cpu() for x in t])
        return t.view(-1, self.W, 64).transpose(0, 1).reshape(self.W, -1).cpu()

    def exact(self):
        x = self.flat.double()
        layer = torch.stack([torch.sqrt((x[:, o:o + m] ** 2).sum(1)) for o, m in zip(self.off, self.sizes)], 1)
        norm = torch.sqrt((layer ** 2).sum(1))
        return torch.cat([norm, torch.sqrt((norm ** 2).mean())[None]]), layer


def _norms(sc, g, t, interleaved, layers=True, stream=None):
    L = len(g.sizes)
    norm = torch.full((g.W + 4,), 7.0, device="cuda")
    layer = torch.full((g.W * L + 3,), 7.0, device="cuda") if layers else None
    ws = torch.full((sc.scape_grad_norm_workspace_bytes(g.ctx),), 0xA5, dtype=torch.uint8, device="cuda")
    call = sc.scape_grad_norm_interleaved if interleaved else sc.scape_grad_norm
    call(g.ctx, t, norm, layer, workspace=ws, stream=stream)
    torch.cuda.synchronize()
    assert bool((norm[g.W + 1:] == 7).all())
    if layers:
        assert bool((layer[g.W * L:] == 7).all())
        layer = layer[:g.W * L].view(g.W, L).cpu()
    return norm[:g.W + 1], layer


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("W", [1, 2, 3, 5, 8, 32])
@pytest.mark.parametrize("name", list(LAYERS))
def test_norms_and_clipping(sc, name, W, interleaved):
    g = Grads(sc, LAYERS[name], W)
    t = g.given(interleaved)
    if not g.flat.numel():
        t = torch.empty(0, dtype=torch.bfloat16, device="cuda") if interleaved else t
    norm, layer = _norms(sc, g, t, interleaved)
    want, want_layer = g.exact()
    assert bool(((norm.cpu().double() - want).abs() <= 2 * U * want).all())
    assert bool(((layer.double() - want_layer).abs() <= 2 * U * want_layer).all())
    again, none = _norms(sc, g, t, interleaved, layers=False)
    assert none is None and torch.equal(again, norm)
    if not g.flat.numel():
        return
    clip = sc.scape_grad_clip_interleaved if interleaved else sc.scape_grad_clip
    for shared in (False, True):
        for max_norm in (float(want[:W].median()) * 0.5, float(want[:W].max()), float(want.max()) * 2):
            out = Grads.given(g, interleaved)
            for o in ([out] if interleaved else out):
                o.fill_(3.0)
            clip(g.ctx, t, norm, max_norm, out=out, shared=shared)
            torch.cuda.synchronize()
            got = g.back(out, interleaved)
            by = (norm[W:].expand(W) if shared else norm[:W]).cpu().double()
            top = float(np.float32(max_norm))
            f = torch.where(by > top, top / by, torch.ones_like(by))[:, None]
            x = g.flat.double()[:, g.inside]
            err = (got[:, g.inside].double() - x * f).abs()
            assert bool((err <= (HALF + 4 * U) * (x * f).abs() + 2.0 ** -126).all())
            whole = (f == 1).squeeze(1)
            assert torch.equal(got[whole][:, g.inside], g.flat[whole][:, g.inside])
            assert bool((got[:, ~g.inside] == 3).all())  # between the layers: as it was
            # in place gives the same, and leaves what lies between the layers alone
            own = Grads.given(g, interleaved)
            clip(g.ctx, own, norm, max_norm, shared=shared)
            torch.cuda.synchronize()
            mine = g.back(own, interleaved)
            assert torch.equal(mine[:, g.inside], got[:, g.inside]) and bool(mine[:, ~g.inside].isnan().all())


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("bad", [NAN, INF, -INF])
def test_norms_that_are_not_finite(sc, bad, interleaved):
    """The worker's gradient becomes 0 (all workers' where the norm is shared), the others' do not change."""
    g = Grads(sc, LAYERS["ragged"], 3)
    g.flat[1, g.off[4] + 4096] = bad
    t = g.given(interleaved)
    norm, layer = _norms(sc, g, t, interleaved)
    n = norm.cpu()
    assert bool(n[[0, 2]].isfinite().all()) and not bool(n[1].isfinite()) and not bool(n[3].isfinite())
    assert layer.isfinite().sum() == layer.numel() - 1 and not bool(layer[1, 4].isfinite())
    clip = sc.scape_grad_clip_interleaved if interleaved else sc.scape_grad_clip
    for shared in (False, True):
        own = g.given(interleaved)
        clip(g.ctx, own, norm, 1e30, shared=shared)
        torch.cuda.synchronize()
        got = g.back(own, interleaved)
        zero = [0, 1, 2] if shared else [1]
        assert bool((got[zero][:, g.inside].view(torch.int16) == 0).all())
        if not shared:
            assert torch.equal(got[[0, 2]][:, g.inside], g.flat[[0, 2]][:, g.inside])


def test_extreme_values(sc):
    """The largest bf16 values do not overflow the sum, the smallest do not vanish from it."""
    for value in (3.0e38, 1.0e-38, 1e-40):
        g = Grads(sc, [5000, 77], 2)
        for o, m in zip(g.off, g.sizes):
            g.flat[:, o:o + m] = value
        g.flat[:, g.off[0] + 1:g.off[0] + 5000] = 0
        g.flat[:, g.off[1] + 1:g.off[1] + 77] = 0
        norm, layer = _norms(sc, g, g.given(False), False)
        v = float(g.flat[0, 0].double())
        assert torch.equal(layer.double(), torch.full((2, 2), v, dtype=torch.float64))
        want = float(torch.tensor(v * math.sqrt(2.0)))
        if math.isfinite(want):
            assert abs(float(norm[0]) - want) <= 2 * U * want + 2.0 ** -149


def test_zero_gradients(sc):
    g = Grads(sc, LAYERS["ragged"], 2)
    g.flat[:, g.inside] = 0
    norm, layer = _norms(sc, g, g.given(True), True)
    assert not bool(norm.any()) and not bool(layer.any())
    own = g.given(True)
    sc.scape_grad_clip_interleaved(g.ctx, own, norm, 1.0)
    torch.cuda.synchronize()
    assert not bool(g.back(own, True)[:, g.inside].any())


def test_gradients_as_bits(sc):
    """int16 views, as the step takes them."""
    g = Grads(sc, LAYERS["ragged"], 3)
    t = g.given(False)
    norm, _ = _norms(sc, g, t, False)
    bits = [x.view(torch.int16) for x in g.given(False)]
    again, _ = _norms(sc, g, bits, False)
    assert torch.equal(norm, again)
    sc.scape_grad_clip(g.ctx, bits, norm, 0.25)
    sc.scape_grad_clip(g.ctx, t, norm, 0.25)
    torch.cuda.synchronize()
    for a, b in zip(bits, t):
        assert torch.equal(a, b.view(torch.int16))


def test_refusals_with_a_context(sc):
    g = Grads(sc, LAYERS["ragged"], 3)
    t, il = g.given(False), g.given(True)
    norm, ws = torch.zeros(4, device="cuda"), torch.zeros(sc.scape_grad_norm_workspace_bytes(g.ctx), dtype=torch.uint8, device="cuda")
    for kind, call in [
        (ValueError, lambda: sc.scape_grad_norm(g.ctx, t[:2], norm, workspace=ws)),
        (ValueError, lambda: sc.scape_grad_norm(g.ctx, il, norm, workspace=ws)),
        (ValueError, lambda: sc.scape_grad_norm(g.ctx, t, norm[:3], workspace=ws)),
        (ValueError, lambda: sc.scape_grad_norm(g.ctx, t, norm)),
        (ValueError, lambda: sc.scape_grad_norm(g.ctx, [x.cpu() for x in t], norm, workspace=ws)),
        (ValueError, lambda: sc.scape_grad_norm(g.ctx, t, norm, torch.zeros(20, device="cuda"), workspace=ws)),
        (TypeError, lambda: sc.scape_grad_norm(g.ctx, [x.float() for x in t], norm, workspace=ws)),
        (sc.ScapeError, lambda: sc.scape_grad_norm(g.ctx, t, norm, workspace=ws[:64])),
        (ValueError, lambda: sc.scape_grad_norm_interleaved(g.ctx, il[64:], norm, workspace=ws)),
        (sc.ScapeError, lambda: sc.scape_grad_norm_interleaved(g.ctx, torch.cat([il, il])[1:], norm, workspace=ws)),
        (sc.ScapeError, lambda: sc.scape_grad_clip(g.ctx, t, norm, 0.0)),
        (sc.ScapeError, lambda: sc.scape_grad_clip(g.ctx, t, norm, -1.0)),
        (sc.ScapeError, lambda: sc.scape_grad_clip(g.ctx, t, norm, NAN)),
        (sc.ScapeError, lambda: sc.scape_grad_clip(g.ctx, t, norm, INF)),
        (ValueError, lambda: sc.scape_grad_clip(g.ctx, t, norm, 1.0, out=t[:2])),
        (ValueError, lambda: sc.scape_grad_clip_interleaved(g.ctx, il, norm[:3], 1.0)),
    ]:
        with pytest.raises(kind):
            call()
    assert sc.lib().scape_grad_clip_interleaved(g.ctx.handle, il.data_ptr(), norm.data_ptr(), 1.0, 2, il.data_ptr(), None) == -1


def test_gradients_that_overlap(sc):
    """One buffer for two workers is read by both, and never written by both."""
    g = Grads(sc, LAYERS["ragged"], 3)
    t, il = g.given(False), g.given(True)
    n = g.ctx.layout.n_pad
    norm = torch.full((4,), 2.0, device="cuda")
    both, wide = torch.zeros(n + 64, dtype=t[0].dtype, device="cuda"), torch.zeros(3 * n + 64, dtype=t[0].dtype, device="cuda")
    for call in [
        lambda: sc.scape_grad_clip(g.ctx, [t[0], t[1], t[0]], norm, 1.0),
        lambda: sc.scape_grad_clip(g.ctx, t, norm, 1.0, out=[t[1], t[0], t[2]]),
        lambda: sc.scape_grad_clip(g.ctx, t, norm, 1.0, out=[both[:n], both[64:], t[2]]),
        lambda: sc.scape_grad_clip(g.ctx, [both[:n], t[1], t[2]], norm, 1.0, out=[both[64:], t[1], t[2]]),
        lambda: sc.scape_grad_clip_interleaved(g.ctx, wide[:3 * n], norm, 1.0, out=wide[64:]),
    ]:
        with pytest.raises(sc.ScapeError):
            call()
    before = [x.clone() for x in t]
    out = [torch.zeros_like(x) for x in t]
    sc.scape_grad_clip(g.ctx, [t[0], t[1], t[0]], norm, 1.0, out=out)  # read twice
    torch.cuda.synchronize()
    assert torch.equal(out[0], out[2]) and all(torch.equal(x.view(torch.int16), y.view(torch.int16)) for x, y in zip(t, before))
    sc.scape_grad_clip_interleaved(g.ctx, il, norm, 1.0, out=wide[:3 * n])


@pytest.mark.parametrize("interleaved", [False, True])
def test_a_clipped_step(sc, interleaved):
    """ScapeState.step(max_norm=) is the step on gradients clipped beforehand, eager and from graphs."""
    from sparse_communication_adam_amd.state import ScapeState
    wl = synth.ragged()
    cfg = sc.ScapeConfig(layer_numel=wl.layer_sizes, workers=wl.W, keep_num=1, keep_den=5)
    states = [ScapeState(cfg, interleaved=interleaved) for _ in range(3)]
    grads = [Grads(sc, wl.layer_sizes, wl.W, key=k) for k in range(5)]
    for gr in grads:
        gr.flat[:, ~gr.inside] = 0
    buf = grads[0].given(interleaved)
    states[2].step(buf, max_norm=0.3, shared_norm=True)  # what the graphs' first step sees as its past
    for s in states[:2]:
        s.step(grads[0].given(interleaved), max_norm=0.3, shared_norm=True)
    states[2].capture(buf, max_norm=0.3, shared_norm=True)
    clip = sc.scape_grad_clip_interleaved if interleaved else sc.scape_grad_clip
    for gr in grads[1:]:
        states[0].step(gr.given(interleaved), max_norm=0.3, shared_norm=True)
        t = gr.given(interleaved)
        norm, _ = _norms(sc, gr, t, interleaved)
        clip(gr.ctx, t, norm, 0.3, shared=True)
        states[1].step(t)
        fresh = gr.given(interleaved)
        for a, b in zip([buf] if interleaved else buf, [fresh] if interleaved else fresh):
            a.copy_(b)
        states[2].step_graph()
        torch.cuda.synchronize()
        assert torch.equal(states[0].grad_norm, norm) and torch.equal(states[2].grad_norm, norm)
        for s in states[1:]:
            assert torch.equal(s.x, states[0].x) and torch.equal(s.m, states[0].m) and torch.equal(s.v, states[0].v)
            for i in range(wl.W):
                assert torch.equal(s.residual(i), states[0].residual(i))
    assert float(states[0].grad_norm[-1]) > 0.3  # they were clipped


def test_largest_offsets(sc):
    """A layer that ends 2^31 elements into the flat buffer, gradients behind 2^32 bytes."""
    sizes = [2 ** 30, 2 ** 30 - 2 ** 20, 2 ** 20 - 200, 100]
    ctx = sc.Context(sc.ScapeConfig(layer_numel=sizes, workers=1, keep_num=1, keep_den=1000))
    n = ctx.layout.n_pad
    g = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    marks = {0: 3.0, 2 ** 30 - 1: 4.0, 2 ** 31 - 2 ** 20 - 1: 12.0, ctx.layout.layer_offset[3] + 99: 84.0}
    for at, v in marks.items():
        g[at] = v
    norm, layer = torch.zeros(2, device="cuda"), torch.zeros(4, device="cuda")
    ws = torch.zeros(sc.scape_grad_norm_workspace_bytes(ctx), dtype=torch.uint8, device="cuda")
    sc.scape_grad_norm(ctx, [g], norm, layer, workspace=ws)
    assert layer.tolist() == [5.0, 12.0, 0.0, 84.0] and norm.tolist() == [85.0, 85.0]
    sc.scape_grad_clip(ctx, [g], norm, 42.5)
    torch.cuda.synchronize()
    for at, v in marks.items():
        assert float(g[at]) == v / 2
    assert int((g != 0).sum()) == 4
    ctx.destroy()
