"""Sigmoid scores of tokens whose logits are all very negative: the scores are
s_e / sum_j s_j all the same, which is close to a softmax there, and the slope
1 - s is 1.  Only a token whose logits are all -inf has none."""
import pytest
import torch
import torch.nn.functional as F

from test_gpu_losses import HALF, INF, TINY, U, _bytes, _place, _router, sc  # noqa: F401

pytestmark = pytest.mark.gpu


def _scores(x):
    """p and 1 - s in float64, from logarithms; a token of -inf has 0."""
    return torch.softmax(F.logsigmoid(x), 1).nan_to_num(0.0), torch.sigmoid(-x)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16], ids=str)
@pytest.mark.parametrize("tokens,experts", [(400, 24), (9000, 24), (300, 3), (700, 256), (5000, 61), (90, 1024)])
def test_low_tokens_keep_their_scores(sc, tokens, experts, dtype):
    k = 2
    x, idx, mask = _router(tokens, experts, k, dtype, "low")
    low = torch.finfo(dtype).min
    for i, depth in enumerate([-30.0, -50.0, -70.0, -86.0, -88.0, -95.0, -120.0, -1000.0]):
        x[i::16] += depth
    x[8::16] = low                       # all alike
    x[9::16, ::2] = low                  # some masked, the rest far below
    x[9::16, 1::2] -= 200.0
    x[10::16] = -INF                     # no score
    x[11::16, 1:] = -INF
    x[11::16, 0] = -300.0                # one expert left
    x[12::16, :1] += 90.0                # far above
    mask[8:12] = 1
    z = _place(x, dtype, 0, 1)
    h = z.cpu().double()
    on = mask != 0
    p, slope = _scores(h)
    counts = torch.empty(1, experts, dtype=torch.int32, device="cuda")
    psum, loss = torch.empty(1, experts, device="cuda"), torch.empty(1, device="cuda")
    n_tok = torch.empty(1, dtype=torch.int32, device="cuda")
    sc.scape_balance_forward(z, idx.cuda(), counts, psum, n_tok, loss, alpha=0.01, mask=mask.cuda(), score="sigmoid",
                             workspace=_bytes(sc.scape_balance_workspace_bytes(z)))
    up = torch.full((1,), 1.0 if dtype != torch.float16 else 1024.0 * tokens, device="cuda")
    dz = torch.full_like(z, 5.0)
    sc.scape_balance_backward(z, counts, n_tok, up, dz, k=k, alpha=0.01, mask=mask.cuda(), score="sigmoid")
    torch.cuda.synchronize()
    # every token's scores sum to 1 but for those of -inf
    there = on & (h > -INF).any(1)
    assert int(n_tok) == int(on.sum())
    assert abs(float(psum.double().sum()) - int(there.sum())) <= int(there.sum()) * 64 * U + experts * U * tokens
    # a score: exponents down to -160 rounded once (below that there is nothing left of a score, or differences are
    # taken first), a sum over 16 experts a lane and 6 steps, divisions; sums as in the other balance tests
    rel = U * (2 * 160 + 16 + 6 + 8)
    total = p[on].sum(0)
    seq = max(tokens / 4096 + 8, 64) + 15
    assert bool(((psum[0].cpu().double() - total).abs() <= total * (rel + U * seq) + 1e-37).all())
    c, n = counts[0].cpu().double(), int(n_tok)
    ref = 0.01 * experts / (k * n * n) * float((c * total).sum())
    assert abs(float(loss) - ref) <= ref * (rel + U * (seq + 1))
    G = float(up) * 0.01 * experts / (k * n * n)
    rd = torch.where(on[:, None], G * p * slope * (c - (p * c).sum(1, keepdim=True)), 0.0)
    tol = G * p * (c + (p * c).sum(1, keepdim=True)) * (3 * rel + U * 32) + HALF[dtype] * rd.abs() * 1.001 + TINY[dtype]
    # logits past 2^-126 below the row's best have a score of 0 in float32
    tol = tol + G * (c + (p * c).sum(1, keepdim=True)) * 2.0 ** -120
    assert bool(((dz.cpu().double() - rd).abs() <= tol).all())
    assert bool(dz[8].any()) and not bool(dz[10].any())
