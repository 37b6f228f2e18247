"""The distillation gradient where the student holds almost nothing outside
the teacher's entries, for instance where all other columns are masked with a
finite value: the tail's gradient is the teacher's mass outside, spread as the
student spreads its own, however far below the entries that lies.

With tail logits that span X e-folds the exponents are off by 6 u X at most
and a sum by (32 + cols / 256 + 9) u, u = 2^-24, plus 8 roundings; log p_T
itself does not enter."""
import pytest
import torch

from test_gpu_losses import HALF, INF, TINY, U, Case, sc  # noqa: F401

pytestmark = pytest.mark.gpu

# the spread of the tail's logits, each row of which has another depth
SPREAD = 8.0


def _case(rows, cols, dtype, scale, k=20):
    c = Case(rows, cols, k, dtype, True, scale, key="faint")
    at = c.idx.long()
    low = torch.finfo(dtype).min
    c.x = torch.rand(rows, cols, generator=torch.Generator().manual_seed(cols)) * SPREAD
    deep = -1e9 if dtype != torch.float16 else -6e4
    c.x[0] = deep
    c.x[1] = low
    c.x[2] -= 10016.0                  # steps of 2^-10 (f32), 8 (f16), 64 (bf16)
    c.x[3] = -INF
    c.x[3, [cols - 1, 0, cols // 2]] = -500.0
    c.x[4] -= 60.0 / scale             # just past what float32 can do from log p_T
    c.x[5] = -INF                      # no tail at all
    c.x[6] = deep
    top = torch.rand(rows, k, generator=torch.Generator().manual_seed(k)) * 4 + 27
    for r in range(rows):
        c.x[r, at[r]] = top[r]
    c.val = (top - 3.0 + torch.rand(rows, k, generator=torch.Generator().manual_seed(7))).float()
    c.lse = (torch.logsumexp(c.val.double() * scale, 1) + 0.7).float()  # half of the teacher's mass outside
    c.lse[6] -= 2.0                    # the teacher holds nothing outside either
    return c


def _reference(c):
    """loss, L and dz in float64, from differences of logits: beside a logit of
    the type's lowest value not even float64 has room for a logarithm."""
    w, x, at = c.weight.double(), c.h * c.scale, c.idx.long()
    q = (c.val.double() * c.scale - c.lse.double()[:, None]).exp()
    known = torch.zeros_like(x, dtype=torch.bool).scatter_(1, at, True)
    tail = x.masked_fill(known, -INF)
    qt = torch.where((tail > -INF).any(1), (1 - q.sum(1)).clamp(min=0), 0.0)
    top, low = x.amax(1), tail.amax(1)
    low = torch.where(low > -INF, low, 0.0)
    log_sum, log_tail = torch.logsumexp(x - top[:, None], 1), torch.logsumexp(tail - low[:, None], 1)
    logp = x.gather(1, at) - top[:, None] - log_sum[:, None]
    loss = (q * (q.log() - logp)).sum(1)
    lpt = low - top + log_tail - log_sum
    loss = loss + torch.where(qt > 0, qt * (qt.log() - lpt), 0.0)
    dz = torch.softmax(x, 1) * (q.sum(1) + qt)[:, None]
    dz = dz - torch.softmax(tail, 1).nan_to_num(0.0) * qt[:, None]
    dz.scatter_add_(1, at, -q)
    return w * loss, top + log_sum, dz * (c.scale * w)[:, None]


def _check(c, dz, ulps_of_lse):
    w = c.weight.double()
    _, lse, rd = _reference(c)
    at = c.idx.long()
    d = dz.cpu().double()
    rows, cols = d.shape
    rel = (32 + cols // 256 + 9 + 8) * U + 6 * U * c.scale * (SPREAD + 64)  # 64: a step of the coarsest type
    p = torch.softmax(c.h * c.scale, 1).nan_to_num(0.0)
    # an entry's q_j and p_j, each with its own error; p's includes that of the statistics where it is made from them
    part = rd.abs().clone()
    q = (c.val.double() * c.scale - c.lse.double()[:, None]).exp()
    part.scatter_add_(1, at, q * c.scale * w[:, None])
    part += 2 * p * c.scale * w[:, None]
    tol = part * (rel + ulps_of_lse * U * lse[:, None].abs()) + HALF[c.dtype] * rd.abs() * 1.001 + TINY[c.dtype]
    worst = (d - rd).abs() - tol
    assert bool((worst <= 0).all()), [(r, float(worst[r].max())) for r in range(min(rows, 7))]


@pytest.mark.parametrize("scale", [1.0, 0.5])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16], ids=str)
@pytest.mark.parametrize("rows,cols", [(600, 2000), (7, 50304), (12, 131075), (7, 262144)], ids=str)
def test_gradient_of_the_forward_call(sc, rows, cols, dtype, scale):
    c = _case(rows, cols, dtype, scale).put()
    loss, stats, dz = c.call(sc)
    rl, lse, _ = _reference(c)
    # L, log p_T and the loss are made of a few terms, each to float32
    assert bool(((stats[:, 0].cpu().double() - lse).abs() <= 64 * U * (1 + lse.abs())).all())
    assert bool(((loss.cpu().double() - rl).abs() <= 64 * U * (1 + rl.abs())).all())
    assert stats[5, 1] == -INF
    _check(c, dz, 0)
    keep = c.z.clone()
    c.call(sc, dz=c.z)
    assert torch.equal(c.z, dz)  # over the logits
    c.z.copy_(keep)


@pytest.mark.parametrize("scale", [1.0, 0.5])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16], ids=str)
@pytest.mark.parametrize("rows,cols", [(600, 2000), (7, 50304), (12, 131075), (7, 262144)], ids=str)
def test_gradient_from_the_statistics(sc, rows, cols, dtype, scale):
    c = _case(rows, cols, dtype, scale).put()
    _, stats, _ = c.call(sc, grad=False)
    back = torch.full_like(c.z, 5.0)
    sc.scape_distill_backward(c.z, c.dev[0], c.dev[1], stats, back, t_lse=c.dev[2], scale=scale, weight=c.dev[3])
    torch.cuda.synchronize()
    _check(c, back, 2)
    sc.scape_distill_backward(c.z, c.dev[0], c.dev[1], stats, c.z, t_lse=c.dev[2], scale=scale, weight=c.dev[3])
    torch.cuda.synchronize()
    assert torch.equal(c.z, back)  # over the logits
