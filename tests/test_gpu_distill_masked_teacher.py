"""Distillation where a teacher's records hold masked entries and the student
is masked with -inf: an entry counts by its own probability, whichever wave of
the workgroup holds its slot (64 slots a wave)."""
import pytest
import torch

from test_gpu_losses import INF, Case, _check_distill, sc  # noqa: F401

pytestmark = pytest.mark.gpu

FORMS = pytest.mark.parametrize("rows,cols", [(8, 2000), (8, 50304), (8, 262144)],
                                ids=["rows in registers", "long rows", "split rows"])


class MaskedCase(Case):
    """The teacher renormalised over entries of the lowest value only: float64
    has no bit left for the logarithm of their number beside the value, so the
    reference takes them relative to the row's largest, which changes nothing
    in the definition."""

    def reference(self, factor):
        keep = self.val
        if not self.tail:
            self.val = self.val.double() - self.val.double().amax(1, keepdim=True)
        try:
            return super().reference(factor)
        finally:
            self.val = keep


def _all_forms(sc, c):
    """Loss alone, loss with gradient, and the gradient from the statistics,
    each against float64."""
    w = c.weight.double()
    loss, stats, _ = c.call(sc, grad=False)
    _check_distill(c, w, loss, stats)
    loss2, stats2, dz = c.call(sc)
    assert torch.equal(loss, loss2) and torch.equal(stats, stats2)
    _check_distill(c, w, dz=dz)
    back = torch.full_like(c.z, 5.0)
    sc.scape_distill_backward(c.z, c.dev[0], c.dev[1], stats, back, t_lse=c.dev[2], scale=c.scale, weight=c.dev[3])
    torch.cuda.synchronize()
    _check_distill(c, w, dz=back)
    return loss


@FORMS
@pytest.mark.parametrize("tail", [True, False], ids=["tail", "renormalised"])
@pytest.mark.parametrize("k", [60, 70, 100, 300, 1024])
@pytest.mark.parametrize("low", [-1e4, -65504.0, -1e9, torch.finfo(torch.float32).min])
def test_masked_entries_in_slots_of_their_own_wave(sc, rows, cols, k, tail, low):
    c = MaskedCase(rows, cols, k, torch.float32, tail, key=f"masked {low}")
    at = c.idx.long()
    last = slice(max(64, k - 6) if k > 64 else k - 6, k)  # of a wave that has no other entry up to k = 70
    # no mass at a column that the student masks: a finite loss
    c.val[0, last] = low
    c.x[0, at[0, last]] = -INF
    # the same in whole waves, all but the first 64
    c.val[1, 64:] = low
    c.x[1, at[1, 64:]] = -INF
    # an entry of every wave but the first keeps its mass, masked ones among them
    c.val[2, 65::3] = low
    c.x[2, at[2, 65::3]] = -INF
    # mass at a masked column: inf, from the first wave and from the last
    c.x[3, at[3, 5]] = -INF
    c.x[4, at[4, k - 1]] = -INF
    c.val[4, last][:-1] = low
    # the heavy entries in the last slots, the masked ones in the first wave
    c.val[5, :min(64, k // 2)] = low
    c.x[5, at[5, :min(64, k // 2)]] = -INF
    # nothing but masked entries
    c.val[6] = low
    c.put()
    loss = _all_forms(sc, c)
    assert bool(loss[[0, 1, 2, 5, 6]].isfinite().all()) and loss[3] == INF and loss[4] == INF


@FORMS
@pytest.mark.parametrize("k", [20, 130])
def test_a_probability_below_float64_is_none(sc, rows, cols, k):
    """A column of -inf under an entry 1400 e-folds below the best, whose
    probability is 0 in float64, beside one 700 below, whose is not: alike in
    the slots of the first wave and in those of another."""
    c = MaskedCase(rows, cols, k, torch.float32, False, key="faint")
    at = c.idx.long()
    n = 64 if k > 64 else k - 10
    c.val[0, n:] -= 700.0
    c.val[0, n + 3] = c.val[0, 0] - 1400.0
    c.x[0, at[0, n + 3]] = -INF
    c.val[1, n:] -= 700.0
    c.x[1, at[1, n + 3]] = -INF  # exp(-700) is a number
    c.put()
    loss = _all_forms(sc, c)
    assert bool(loss[0].isfinite()) and loss[1] == INF
