"""float16 gradients of the head where the rows' factors (weight * dloss * scale)
lie far apart: a word that only rows of small factors move has their precision.

dw is a sum of P h over the rows, P = g (p - onehot).  A term of it is off by
  - half a step of 11 bits of P (HALF), or where |p - onehot| < 2^-28 by 2^-39 of
    the row's factor;
  - the logit's own error in p (Z below) and 8u for the exponential and the factor;
  - h, which dw takes times one power of two a row, so that the largest
    |factor h| of all rows lies in [2^14, 2^15).  It is exact down to 2^-14
    there, and off by 2^-25 at most below: 2^-38 of the largest |factor h|, times
    |p - onehot|;
and the float32 sum by a step of u a term.  dw itself is rounded once (HALF, or
half of the smallest float16, 2^-25).  A logit is a float32 sum of dim exact
products, off by (dim + 2) u of the sum of their magnitudes, and 4u |z|.
"""
import math
import zlib

import pytest
import torch

pytestmark = pytest.mark.gpu

U, HALF, TINY = 2.0 ** -24, 2.0 ** -11, 2.0 ** -25


@pytest.fixture(scope="module", autouse=True)
def sc():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import sparse_communication_adam_amd as sc
    sc.lib()
    yield sc
    torch.cuda.empty_cache()


class Spread:
    """Row 0 is sure of word 0 and has the largest factor; the others, 2^-apart of
    it, are about the other words, which row 0 gives next to nothing."""

    def __init__(self, rows, cols, dim, apart, size=1.0, top=8192.0):
        g = torch.Generator(device="cuda").manual_seed(zlib.crc32(f"{rows}/{cols}/{dim}/{apart}/{size}".encode()))
        new = dict(device="cuda", generator=g)
        h = torch.randn(rows, dim, **new)
        w = torch.randn(cols, dim, **new) / math.sqrt(dim)
        h[:, 0], w[:, 0] = 0.0, 0.0
        h[0, 0], w[0, 0] = 6.0, 8.0  # 48 above the other words, whose p is below 2^-60
        label = torch.randint(1, cols, (rows,), **new)
        label[0] = 0
        self.factor = torch.full((rows,), top * 2.0 ** -apart, device="cuda") * (0.5 + torch.rand(rows, **new))
        self.factor[0] = top
        self.scale = 1.0 / size
        self.h, self.w, self.label = (h * size).half(), w.half(), label.to(torch.int32)

    def exact(self):
        """lse, dw and its tolerance in float64 (from the float32 lse)."""
        h, w, f = self.h.double(), self.w.double(), self.factor.double() * self.scale
        z = (h @ w.t()) * self.scale
        lse = torch.logsumexp(z, 1).float()
        off = (h.shape[1] + 2) * U * (h.abs() @ w.abs().t()).amax(1) * self.scale + 4 * U * z.abs().amax(1)
        p = torch.exp(z - lse.double()[:, None])
        d = p.clone()
        d[torch.arange(len(f), device="cuda"), self.label.long()] -= 1.0
        dP = f[:, None] * (p * (off[:, None] * 1.01 + 8 * U) + d.abs() * HALF + 2.0 ** -39)
        P = d * f[:, None]
        dw = P.t() @ h
        top = float((f[:, None] * h.abs()).max())
        tol = dP.t() @ h.abs() + (len(f) + 4) * U * (P.abs().t() @ h.abs()) + 2.0 ** -38 * top * d.abs().sum(0)[:, None]
        return lse, dw, tol * (1 + HALF) + HALF * dw.abs() + TINY


def _equal(a, b):
    """The same numbers, NaN where there is NaN."""
    return torch.equal(a.isnan(), b.isnan()) and torch.equal(a.masked_fill(a.isnan(), 0), b.masked_fill(b.isnan(), 0))


def _dw(sc, c, lse):
    dw, dh = torch.empty_like(c.w), torch.empty_like(c.h)
    n = sc.scape_vocab_loss_workspace_bytes(c.h, c.w, grad=True)
    ws = torch.full((n,), 0xA5, dtype=torch.uint8, device="cuda")
    sc.scape_vocab_loss_backward(c.h, c.w, c.label, lse, dh, dw, scale=c.scale, dloss=c.factor, workspace=ws)
    alone = torch.empty_like(c.w)
    ws.fill_(0x5A)
    sc.scape_vocab_loss_backward(c.h, c.w, c.label, lse, None, alone, scale=c.scale, dloss=c.factor, workspace=ws)
    torch.cuda.synchronize()
    assert _equal(dw, alone)
    return dw


@pytest.mark.parametrize("apart", [0, 12, 16, 20, 24])
@pytest.mark.parametrize("rows,cols,dim", [(6, 40, 64), (40, 300, 136), (150, 400, 64), (300, 700, 72), (1030, 600, 264)])
def test_words_of_small_factors(sc, rows, cols, dim, apart):
    c = Spread(rows, cols, dim, apart, top=8192.0 if apart else 1024.0)
    lse, dw, tol = c.exact()
    got = _dw(sc, c, lse).double()
    assert bool(((got - dw).abs() <= tol).all()), float(((got - dw).abs() / tol).max())
    assert float((tol[1:].norm(dim=1) / dw[1:].norm(dim=1)).max()) < 2.0 ** -5  # no tolerance hides a word


@pytest.mark.parametrize("size", [2.0 ** -12, 2.0 ** -6, 256.0, 8192.0])
def test_small_and_large_hidden_states(sc, size):
    """Hidden states near both ends of float16: the copy uses its whole range, and nothing in it overflows."""
    for rows, top in ((30, 2.0 ** 13), (300, 2.0 ** 20), (300, 2.0 ** -10)):
        c = Spread(rows, 200, 64, 16, size=size, top=top * min(1.0, size) if size < 1 else top)
        lse, dw, tol = c.exact()
        got = _dw(sc, c, lse).double()
        fits = dw.abs() + tol < 65504
        assert bool((((got - dw).abs() <= tol) | ~fits).all())


def test_rows_of_zeros_and_of_no_number(sc):
    """Hidden states that are 0 do not set the scale; an infinity or a NaN in a row that counts shows in dw, in one
    that does not count nowhere."""
    for rows in (20, 600):
        c = Spread(rows, 300, 64, 20)
        c.h[0] = 0
        lse, dw, tol = c.exact()
        clean = _dw(sc, c, lse)
        assert bool(((clean.double() - dw).abs() <= tol).all())
        c.h[3, 7], c.h[4, 9] = math.inf, math.nan
        bad = _dw(sc, c, lse)
        assert bool((~torch.isfinite(bad[:, 7])).all()) and bool(bad[:, 9].isnan().all())
        c.label[3] = c.label[4] = -100
        c.factor[5] = 0.0
        c.h[5] = math.nan
        off = _dw(sc, c, lse)
        c.h[3:6] = 0
        assert torch.equal(_dw(sc, c, lse), off) and bool(torch.isfinite(off).all())
        c.h.zero_()
        assert not bool(_dw(sc, c, lse).any())


@pytest.mark.parametrize("rows", [20, 600])
def test_a_row_of_zeros_with_a_huge_factor(sc, rows):
    """Zeros have no part in the scale and stay zeros under it, whatever their factor (2^120 above the others here)."""
    c = Spread(rows, 100, 64, 10)
    c.h[0] = 0
    c.factor[1:] = 2.0 ** -20
    c.factor[0] = 2.0 ** 100
    lse = c.exact()[0]
    got = _dw(sc, c, lse)
    c.label[0] = -1
    want = _dw(sc, c, lse)
    assert bool(want.any()) and torch.equal(got, want)


@pytest.mark.parametrize("bad", [math.inf, math.nan])
def test_a_factor_that_is_no_number(sc, bad):
    """It shows in dw, and the scale is that of the others."""
    c = Spread(20, 100, 64, 10)
    lse = c.exact()[0]
    clean = _dw(sc, c, lse)
    c.factor[7] = bad
    got = _dw(sc, c, lse)
    assert not bool(torch.isfinite(got[int(c.label[7])]).any())
    c.label[7] = -1
    c2 = c.factor.clone()
    c.factor[7] = 1.0
    want = _dw(sc, c, lse)
    c.factor.copy_(c2)
    assert torch.equal(_dw(sc, c, lse), want) and bool(torch.isfinite(want).all()) and bool(torch.isfinite(clean).all())


def test_captured_and_replayed(sc):
    """The largest exponent is found anew at every replay."""
    c = Spread(40, 300, 64, 18)
    lse = c.exact()[0]
    dw, dh = torch.empty_like(c.w), torch.empty_like(c.h)
    ws = torch.empty(sc.scape_vocab_loss_workspace_bytes(c.h, c.w, grad=True), dtype=torch.uint8, device="cuda")
    run = lambda: sc.scape_vocab_loss_backward(c.h, c.w, c.label, lse, dh, dw, scale=c.scale, dloss=c.factor, workspace=ws)  # noqa: E731
    run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    for k in range(4):
        c.factor.mul_(2.0 ** (-7 if k % 2 else 3))
        if k == 2:
            c.h.mul_(0.5)
        want = _dw(sc, c, lse)
        dw.fill_(9)
        ws.fill_(k)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(dw, want)
