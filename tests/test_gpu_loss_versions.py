"""The loss operators' outputs and autograd: a call that writes a tensor counts
as an in-place change of it, so a backward pass that needs what was there says
so instead of taking the gradient for it."""
import pytest
import torch

from test_gpu_losses import _bytes, sc  # noqa: F401

pytestmark = pytest.mark.gpu


def _teacher(rows, k):
    val = torch.randn(rows, k, device="cuda")
    idx = torch.arange(k, device="cuda", dtype=torch.int32).repeat(rows, 1) * 3
    return val, idx


def test_gradient_over_saved_logits_is_an_error(sc):
    rows, cols, k = 5, 400, 4
    val, idx = _teacher(rows, k)
    loss, stats = torch.empty(rows, device="cuda"), torch.empty(rows, 2, device="cuda")
    a = torch.randn(rows, cols, device="cuda", requires_grad=True)
    for call in range(2):
        z = torch.tanh(a)  # its backward pass needs z
        sc.scape_distill_forward(z, val, idx, loss, stats, dz=z if call == 0 else None)
        if call == 1:
            sc.scape_distill_backward(z, val, idx, stats, z)
        with pytest.raises(RuntimeError, match="inplace"):
            z.backward(z.detach())
    counts, n_tok = torch.ones(1, cols, dtype=torch.int32, device="cuda"), torch.full((1,), 5, dtype=torch.int32, device="cuda")
    r = torch.tanh(a)
    sc.scape_balance_backward(r, counts, n_tok, None, r, k=2)
    with pytest.raises(RuntimeError, match="inplace"):
        r.backward(r.detach())


def test_gradient_over_logits_that_nothing_needs(sc):
    """A matrix product's backward pass needs its inputs only, so the gradient
    may lie over its output: the same weight gradient as from its own tensor."""
    rows, cols, k = 5, 400, 4
    val, idx = _teacher(rows, k)
    loss, stats = torch.empty(rows, device="cuda"), torch.empty(rows, 2, device="cuda")
    x = torch.randn(rows, 16, device="cuda")
    grads = []
    for over in (True, False):
        w = torch.linspace(-1, 1, 16 * cols, device="cuda").view(16, cols).requires_grad_()
        z = x @ w
        dz = z if over else torch.empty_like(z)
        sc.scape_distill_forward(z, val, idx, loss, stats, dz=dz)
        z.backward(dz.detach())
        grads.append(w.grad)
    assert torch.equal(*grads)


def test_every_output_counts_as_written(sc):
    rows, cols, k = 3, 64, 4
    z = torch.randn(rows, cols, device="cuda")
    f = lambda *s: torch.empty(*s, device="cuda")  # noqa: E731
    i = lambda *s: torch.empty(*s, dtype=torch.int32, device="cuda")  # noqa: E731
    val, idx, lse, loss, stats, dz = f(rows, k), i(rows, k), f(rows), f(rows), f(rows, 2), f(rows, cols)
    counts, psum, n_tok, bloss = i(1, cols), f(1, cols), i(1), f(1)

    def written(call, *outs):
        before = [t._version for t in (z, *outs)]
        call()
        after = [t._version for t in (z, *outs)]
        assert after[0] == before[0] and all(b > a for a, b in zip(before[1:], after[1:]))

    written(lambda: sc.scape_topk_rows(z, k, val, idx, lse), val, idx, lse)
    written(lambda: sc.scape_topk_rows(z, k, val, idx), val, idx)
    written(lambda: sc.scape_distill_forward(z, val, idx, loss, stats, t_lse=lse, dz=dz), loss, stats, dz)
    written(lambda: sc.scape_distill_forward(z, val, idx, loss, stats), loss, stats)
    written(lambda: sc.scape_distill_backward(z, val, idx, stats, dz), dz)
    ws = _bytes(sc.scape_balance_workspace_bytes(z))
    written(lambda: sc.scape_balance_forward(z, idx, counts, psum, n_tok, bloss, workspace=ws), counts, psum, n_tok, bloss)
    written(lambda: sc.scape_balance_loss(counts, psum, n_tok, bloss, k), bloss)
    written(lambda: sc.scape_balance_backward(z, counts, n_tok, None, dz, k=k), dz)
    with torch.inference_mode():  # tensors without a version
        out = torch.empty(rows, cols, device="cuda")
        sc.scape_distill_backward(z, val, idx, stats, out)
    torch.cuda.synchronize()
    assert torch.equal(out, _again(sc, z, val, idx, stats))


def _again(sc, z, val, idx, stats):
    dz = torch.empty_like(z)
    sc.scape_distill_backward(z, val, idx, stats, dz)
    return dz
