"""From hidden states to the optimizer's step: a router's choice, tokens to their
experts and back, the vocabulary loss, every gradient, the workers' norms and a
clipped step, as a program strings them together.  The parameters' gradients are
compared with float64 autograd over the same choices.

Tolerance, in norm: the hidden states, P, dh, the head's gradient and the flat
gradients are rounded to bf16, half a step (2^-8) each at most; the hidden states' rounding
moves a logit, and with it the exponent of a probability: roundings of either sign
add up to less than 2^-8 of the largest logit, twice that in P with its sum.  So
(5 + 2 max|z|) 2^-8; what float32 adds is far below.
"""
import zlib

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def sc():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import sparse_communication_adam_amd as sc
    sc.lib()
    yield sc
    torch.cuda.empty_cache()


def _bytes(n):
    return torch.full((max(n, 1),), 0xA5, dtype=torch.uint8, device="cuda")


def _forward_backward(sc, x, label, head, router, experts, k):
    """One worker's loss and gradients (head, router, experts), and what the reference needs."""
    T, h = x.shape
    V, E = head.shape[0], router.shape[0]
    f32 = dict(device="cuda", dtype=torch.float32)
    r = x @ router.t()
    val, idx = torch.empty(T, k, **f32), torch.empty(T, k, device="cuda", dtype=torch.int32)
    sc.scape_topk_rows(r, k, val, idx)
    gate = torch.softmax(val, 1)
    off, row = torch.empty(E + 1, device="cuda", dtype=torch.int32), torch.empty(T, k, device="cuda", dtype=torch.int32)
    sc.scape_expert_sort(idx, E, off, row, workspace=_bytes(sc.scape_expert_sort_workspace_bytes(idx, E)))
    y0 = torch.empty(T * k, h, **f32)
    sc.scape_expert_gather(x, row, y0)
    cut = off.tolist()
    y1 = torch.cat([y0[a:b] @ experts[e].t() for e, (a, b) in enumerate(zip(cut[:-1], cut[1:]))])
    out = torch.empty(T, h, **f32)
    sc.scape_expert_combine(y1, row, out, weight=gate)
    hid, w = (x + out).to(torch.bfloat16), head.to(torch.bfloat16)
    weight = torch.full((T,), 1.0 / T, **f32)
    loss, lse = torch.empty(T, **f32), torch.empty(T, **f32)
    ws = _bytes(max(sc.scape_vocab_loss_workspace_bytes(hid, w), sc.scape_vocab_loss_workspace_bytes(hid, w, grad=True)))
    sc.scape_vocab_loss_forward(hid, w, label, loss, lse, weight=weight, workspace=ws)
    dh, dhead = torch.empty_like(hid), torch.empty_like(w)
    sc.scape_vocab_loss_backward(hid, w, label, lse, dh, dhead, weight=weight, workspace=ws)
    dhid = dh.float()
    dy1, dgate = torch.empty_like(y1), torch.empty_like(gate)
    sc.scape_expert_combine_backward(y1, row, dhid, dy1, weight=gate, dweight=dgate)
    dexp = torch.stack([dy1[a:b].t() @ y0[a:b] for a, b in zip(cut[:-1], cut[1:])])
    dval = gate * (dgate - (gate * dgate).sum(1, keepdim=True))
    dr = torch.zeros_like(r).scatter_(1, idx.long(), dval)
    # the tokens' own gradient: gather's gradient is the combination without weights
    dy0 = torch.cat([dy1[a:b] @ experts[e] for e, (a, b) in enumerate(zip(cut[:-1], cut[1:]))])
    dx = torch.empty_like(x)
    sc.scape_expert_combine(dy0, row, dx)
    dx += dhid + dr @ router
    return loss.sum(), (dhead, dr.t() @ x, dexp), dx, idx


def _reference(x, label, head, router, experts, idx):
    x, head, router, experts = (t.double().requires_grad_() for t in (x, head.to(torch.bfloat16), router, experts))
    gate = torch.softmax((x @ router.t()).gather(1, idx.long()), 1)
    y = torch.stack([x @ e.t() for e in experts.unbind(0)], 1)
    out = (gate[:, :, None] * y.gather(1, idx.long()[:, :, None].expand(-1, -1, x.shape[1]))).sum(1)
    z = (x + out) @ head.t()
    on = (label >= 0) & (label < head.shape[0])
    at = torch.where(on, label, 0).long()
    loss = (torch.where(on, torch.logsumexp(z, 1) - z.gather(1, at[:, None])[:, 0], 0.0)).sum() / x.shape[0]
    loss.backward()
    return float(loss.detach()), (head.grad, router.grad, experts.grad), x.grad, float(z.detach().abs().max())


@pytest.mark.parametrize("interleaved", [False, True])
def test_hidden_states_to_step(sc, interleaved):
    from sparse_communication_adam_amd.state import ScapeState
    g = torch.Generator().manual_seed(zlib.crc32(b"chain"))
    h, V, E, T, k, W = 64, 1000, 5, 130, 2, 2
    sizes = [V * h, E * h, E * h * h]
    state = ScapeState(sc.ScapeConfig(layer_numel=sizes, workers=W, keep_num=1, keep_den=10), interleaved=interleaved)
    off = state.layout.layer_offset
    state.set_params((torch.randn(state.layout.n_pad, generator=g) * 0.1).cuda())
    for step in range(3):
        part = [state.x[o:o + n].clone() for o, n in zip(off, sizes)]
        head, router, experts = part[0].view(V, h), part[1].view(E, h), part[2].view(E, h, h)
        flats = []
        for _ in range(W):
            x = torch.randn(T, h, generator=g).cuda()
            label = torch.randint(0, V, (T,), generator=g).int()
            label[:7] = -100
            label = label.cuda()
            loss, grads, dx, idx = _forward_backward(sc, x, label, head, router, experts, k)
            want, exact, exact_x, top = _reference(x, label, head, router, experts, idx)
            tol = (5 + 2 * top) * 2.0 ** -8
            assert abs(float(loss) - want) <= tol * abs(want)
            for got, ref in zip(grads + (dx,), exact + (exact_x,)):
                assert float((got.double() - ref).norm() / ref.norm()) <= tol
            flat = torch.zeros(state.layout.n_pad, dtype=torch.bfloat16, device="cuda")
            for o, t in zip(off, grads):
                flat[o:o + t.numel()] = t.flatten().to(torch.bfloat16)
            flats.append(flat)
        norms = torch.stack([f.double().norm() for f in flats])
        bound = float(norms.mean()) * 0.5
        both = torch.stack(flats)
        given = both.view(W, -1, 64).transpose(0, 1).contiguous().view(-1) if interleaved else flats
        before = state.x.clone()
        state.step(given, max_norm=bound, shared_norm=True)
        torch.cuda.synchronize()
        rms = float((norms ** 2).mean().sqrt())
        assert abs(float(state.grad_norm[W]) - rms) <= 2.0 ** -22 * rms
        after = given.view(-1, W, 64).transpose(0, 1).reshape(W, -1) if interleaved else torch.stack(given)
        assert float((after.double() - both.double() * (bound / rms)).norm()) <= 2.0 ** -8 * bound * W ** 0.5
        moved = int((state.x != before).sum())
        assert (moved == 0) == (step == 0)  # the first step's mask is empty
        assert moved <= state.layout.k_total
    state.destroy()


def test_captured_chain(sc):
    """Sort, gather, combine, loss, gradients, norms and clip in one graph, replayed on new data."""
    g = torch.Generator().manual_seed(zlib.crc32(b"captured chain"))
    h, V, E, T, k = 64, 700, 6, 90, 2
    bf, dev = torch.bfloat16, dict(device="cuda")
    ctx = sc.Context(sc.ScapeConfig(layer_numel=[V * h], workers=1, keep_num=1, keep_den=10))

    def buffers():
        b = dict(x=torch.zeros(T, h, dtype=bf, **dev), idx=torch.zeros(T, k, dtype=torch.int32, **dev),
                 gate=torch.zeros(T, k, **dev), label=torch.zeros(T, dtype=torch.int32, **dev), w=torch.zeros(V, h, dtype=bf, **dev),
                 off=torch.zeros(E + 1, dtype=torch.int32, **dev), row=torch.zeros(T, k, dtype=torch.int32, **dev),
                 y=torch.zeros(T * k, h, dtype=bf, **dev), hid=torch.zeros(T, h, dtype=bf, **dev), loss=torch.zeros(T, **dev),
                 lse=torch.zeros(T, **dev), dh=torch.zeros(T, h, dtype=bf, **dev), dw=torch.zeros(V * h, dtype=bf, **dev),
                 dy=torch.zeros(T * k, h, dtype=bf, **dev), dgate=torch.zeros(T, k, **dev), norm=torch.zeros(2, **dev))
        b["ws"] = _bytes(max(sc.scape_vocab_loss_workspace_bytes(b["hid"], b["w"], grad=True),
                             sc.scape_vocab_loss_workspace_bytes(b["hid"], b["w"]), sc.scape_grad_norm_workspace_bytes(ctx),
                             sc.scape_expert_sort_workspace_bytes(b["idx"], E)))
        return b

    def run(b):
        sc.scape_expert_sort(b["idx"], E, b["off"], b["row"], workspace=b["ws"])
        sc.scape_expert_gather(b["x"], b["row"], b["y"])
        sc.scape_expert_combine(b["y"], b["row"], b["hid"], weight=b["gate"])
        sc.scape_vocab_loss_forward(b["hid"], b["w"], b["label"], b["loss"], b["lse"], workspace=b["ws"])
        sc.scape_vocab_loss_backward(b["hid"], b["w"], b["label"], b["lse"], b["dh"], b["dw"].view(V, h), workspace=b["ws"])
        sc.scape_expert_combine_backward(b["y"], b["row"], b["dh"], b["dy"], weight=b["gate"], dweight=b["dgate"])
        sc.scape_grad_norm(ctx, [b["dw"]], b["norm"], workspace=b["ws"])
        sc.scape_grad_clip(ctx, [b["dw"]], b["norm"], 1.0)

    cap = buffers()
    run(cap)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run(cap)
    for n in range(4):
        new = buffers()
        new["x"].copy_(torch.randn(T, h, generator=g))
        new["idx"].copy_(torch.randint(-1, E, (T, k), generator=g))
        new["gate"].copy_(torch.rand(T, k, generator=g))
        new["label"].copy_(torch.randint(-3, V, (T,), generator=g))
        new["w"].copy_(torch.randn(V, h, generator=g) * 0.2)
        for t in cap.values():
            t.fill_(3)
        for name in ("x", "idx", "gate", "label", "w"):
            cap[name].copy_(new[name])
        for b in (cap, new):  # rows of y and dy that no place names keep what they had
            b["y"].zero_()
            b["dy"].zero_()
        run(new)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for name in new:
            if name != "ws":
                assert torch.equal(new[name], cap[name]), (n, name)
    ctx.destroy()
