"""The vocabulary loss and its gradients on a GPU against the definition in
float64.

Tolerances count roundings.  u = 2^-24 and HALF[dtype] are half a step of
float32 and of the 16-bit type, relative to the value.

A logit is a float32 sum of `dim` exact products in any order: off by at most
dim u of the sum of their magnitudes.  With that for the worst column of a row
(Z), the loss' terms 2^x have exponents rounded once and a reference that is a
float32, and their sum has at most 64 terms a lane, 6 joins and a tile's
partial sum for each 256 words: (96 + cols / 256) 2u, and 4u of the largest
|z| for the constant scale*log2(e), the reference and the exponents.

P is off by Z and the same 4u |z| (from the float32 lse that is given), by
HALF of its own rounding, and in float16 by an underflow of 2^-39 of the row's
factor.  The gradients are float32 sums of its products, at most a step a term
off (cols u, rows u), rounded once.
"""
import math
import zlib

import pytest
import torch

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
HALF = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
TINY = {torch.bfloat16: 2.0 ** -126, torch.float16: 2.0 ** -25}
DTYPES = [torch.bfloat16, torch.float16]
NAN, INF = math.nan, math.inf


@pytest.fixture(scope="module", autouse=True)
def sc():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import sparse_communication_adam_amd as sc
    sc.lib()
    yield sc
    torch.cuda.empty_cache()


def _gen(*key):
    return torch.Generator(device="cuda").manual_seed(zlib.crc32("/".join(map(str, key)).encode()))


def _place(x, dtype, pad=0, shift=0):
    """x in rows `pad` elements apart, `shift` elements into a buffer of NaN."""
    rows, cols = x.shape
    buf = torch.full((rows * (cols + pad) + shift + 16,), NAN, dtype=dtype, device="cuda")
    v = buf[shift:shift + rows * (cols + pad)].view(rows, cols + pad)[:, :cols]
    v.copy_(x.to(dtype))
    return v


class Case:
    def __init__(self, rows, cols, dim, dtype, pad=0, shift=0, scale=1.0, spread=1.0, key=""):
        g = _gen("vocab", rows, cols, dim, dtype, key)
        new = dict(device="cuda", generator=g)
        self.dtype, self.scale = dtype, scale
        h = torch.randn(rows, dim, **new)
        w = torch.randn(cols, dim, **new) * (spread / math.sqrt(dim))
        label = torch.randint(0, cols, (rows,), **new)
        h += w[label] * (8 * torch.rand(rows, 1, **new) / scale)
        odd = torch.rand(rows, **new)
        label = torch.where(odd < 0.1, -100, torch.where(odd < 0.15, cols, torch.where(odd < 0.2, 2 ** 31 - 1, label)))
        self.weight = (0.5 + torch.rand(rows, **new)) / rows
        self.weight[torch.rand(rows, **new) < 0.1] = 0.0
        self.dloss = torch.randn(rows, **new) * (1000.0 if dtype == torch.float16 else 1.0)
        self.dloss[torch.rand(rows, **new) < 0.1] = 0.0
        self.h, self.w, self.label = _place(h, dtype, pad, shift), _place(w, dtype, pad, shift), label.to(torch.int32)

    def on(self):
        c = self.w.shape[0]
        return (self.label >= 0) & (self.label < c) & (self.weight != 0)

    def exact(self):
        """z, lse and loss in float64, and the tolerance of a logit (per row)."""
        h, w = self.h.double(), self.w.double()
        z = (h @ w.t()) * self.scale
        mag = (h.abs() @ w.abs().t()).amax(1) * self.scale
        lse = torch.logsumexp(z, 1)
        at = torch.where(self.on(), self.label, 0).long()
        loss = torch.where(self.on(), self.weight.double() * (lse - z.gather(1, at[:, None])[:, 0]), 0.0)
        d = h.shape[1]
        off = (d + 2) * U * mag + 4 * U * z.abs().amax(1)
        return z, lse, loss, off


def _bytes(n):
    return torch.full((max(n, 1),), 0xA5, dtype=torch.uint8, device="cuda")


def _forward(sc, c, weight=True, stream=None):
    n = c.h.shape[0]
    loss, lse = torch.full((n + 3,), 7.0, device="cuda"), torch.full((n + 3,), 7.0, device="cuda")
    ws = _bytes(sc.scape_vocab_loss_workspace_bytes(c.h, c.w))
    sc.scape_vocab_loss_forward(c.h, c.w, c.label, loss, lse, scale=c.scale, weight=c.weight if weight else None,
                                workspace=ws, stream=stream)
    torch.cuda.synchronize()
    assert bool((loss[n:] == 7).all()) and bool((lse[n:] == 7).all())
    return loss[:n], lse[:n]


def _check_forward(sc, c):
    loss, lse = _forward(sc, c)
    z, want_lse, want, off = c.exact()
    cols = c.w.shape[0]
    tol = off + (96 + cols / 256) * 2 * U + U * want_lse.abs()
    assert bool(((lse.double() - want_lse).abs() <= tol).all())
    tol = c.weight.double().abs() * (tol + off) + U * want.abs()
    assert bool(((loss.double() - want).abs() <= tol).all())
    assert bool((loss[~c.on()] == 0).all())


def _exact_grad(c, lse, dloss):
    """dh and dw in float64 from the lse that is given, and their tolerances."""
    z, _, _, off = c.exact()
    h, w = c.h.double(), c.w.double()
    n, cols = z.shape
    g = c.weight.double() * c.scale * (1.0 if dloss is None else dloss.double())
    g = torch.where(c.on(), g, 0.0)
    p = torch.exp(z - lse.double()[:, None])
    y = torch.zeros_like(p).scatter_(1, torch.where(c.on(), c.label, 0).long()[:, None], 1.0)
    P = (p - y) * g[:, None]
    half, tiny = HALF[c.dtype], TINY[c.dtype]
    # + 8u: the exponential and the factor's own roundings
    dP = g.abs()[:, None] * (p * (off[:, None] * 1.01 + 8 * U) + (p - y).abs() * half +
                             (2.0 ** -39 if c.dtype == torch.float16 else 0.0)) + 2 * U * P.abs()
    hh = torch.where((g != 0)[:, None], h, 0.0)
    dh, dw = P @ w, P.t() @ hh
    tol_h = dP @ w.abs() + (cols + 4) * U * (P.abs() @ w.abs())
    tol_w = dP.t() @ hh.abs() + (n + 4) * U * (P.abs().t() @ hh.abs())
    if c.dtype == torch.float16:  # the copy of h, against the largest factor
        tol_w = tol_w + n * float(g.abs().max()) * 2.0 ** -24
    return (dh, tol_h * (1 + half) + half * dh.abs() + tiny), (dw, tol_w * (1 + half) + half * dw.abs() + tiny), P


def _backward(sc, c, lse, dloss, want_h=True, want_w=True, pad=0, shift=0, stream=None):
    n, d = c.h.shape
    dh = _place(torch.full((n, d), NAN), c.dtype, pad, shift) if want_h else None
    dw = _place(torch.full((c.w.shape[0], d), NAN), c.dtype, pad, shift) if want_w else None
    ws = _bytes(sc.scape_vocab_loss_workspace_bytes(c.h, c.w, grad=True))
    sc.scape_vocab_loss_backward(c.h, c.w, c.label, lse, dh, dw, scale=c.scale, weight=c.weight, dloss=dloss, workspace=ws,
                                 stream=stream)
    torch.cuda.synchronize()
    for t in (dh, dw):  # nothing between the rows or behind them
        if t is not None:
            whole = t._base
            assert int(whole.isnan().sum()) == whole.numel() - t.numel() + int(t.isnan().sum())
    return dh, dw


def _check_backward(sc, c, dloss=True, pad=0, shift=0):
    lse = c.exact()[1].float()
    dloss = c.dloss if dloss else None
    (dh, tol_h), (dw, tol_w), _ = _exact_grad(c, lse, dloss)
    got_h, got_w = _backward(sc, c, lse, dloss, pad=pad, shift=shift)
    assert bool(((got_h.double() - dh).abs() <= tol_h).all()), float(((got_h.double() - dh).abs() / tol_h).max())
    assert bool(((got_w.double() - dw).abs() <= tol_w).all()), float(((got_w.double() - dw).abs() / tol_w).max())


SHAPES = [  # rows, cols, dim, pad, shift
    (1, 1, 8, 0, 0), (1, 1000, 64, 0, 0), (2, 37, 72, 8, 8), (7, 255, 136, 0, 0), (16, 256, 128, 16, 0), (17, 257, 64, 0, 8),
    (33, 5000, 520, 0, 0), (64, 511, 1032, 0, 0), (65, 513, 256, 24, 0), (128, 1025, 192, 0, 0), (129, 300, 328, 0, 0),
    (256, 2049, 64, 0, 0), (300, 777, 88, 8, 0), (333, 3001, 400, 0, 0), (520, 1280, 264, 0, 0), (1100, 600, 48, 0, 0),
]


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
@pytest.mark.parametrize("rows,cols,dim,pad,shift", SHAPES)
def test_loss(sc, rows, cols, dim, pad, shift, dtype):
    _check_forward(sc, Case(rows, cols, dim, dtype, pad, shift, scale=0.5 if rows % 2 else 1.0))


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
@pytest.mark.parametrize("rows,cols,dim,pad,shift", SHAPES)
def test_gradients(sc, rows, cols, dim, pad, shift, dtype):
    _check_backward(sc, Case(rows, cols, dim, dtype, pad, shift, scale=0.5 if rows % 2 else 1.0), pad=pad, shift=shift)


@pytest.mark.parametrize("rows,cols,dim", [(16400, 9000, 24), (5, 20000, 64), (70, 50257, 72), (4000, 17001, 40)])
def test_several_pieces_and_splits(sc, rows, cols, dim):
    """More words than a piece holds, few rows over many words, odd ends of both."""
    for dtype in DTYPES:
        c = Case(rows, cols, dim, dtype, key="pieces")
        _check_forward(sc, c)
        _check_backward(sc, c, dloss=dtype == torch.bfloat16)


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
def test_large_logits(sc, dtype):
    """Rows whose largest logit holds all the mass, logits in the thousands."""
    c = Case(40, 700, 64, dtype, spread=200.0, key="large")
    _check_forward(sc, c)
    _check_backward(sc, c)


@pytest.mark.parametrize("rows", [3, 20, 60, 100, 200, 300])
@pytest.mark.parametrize("dtype", DTYPES, ids=str)
def test_logits_far_below_zero(sc, dtype, rows):
    """Every logit near -400: what lies behind the last word of a tile counts for nothing there, too."""
    c = Case(rows, 100, 64, dtype, key="low")
    c.h[:, 0] = 20
    c.w[:, 0] = -20
    _check_forward(sc, c)
    _check_backward(sc, c)
    c = Case(rows, 5000, 24, dtype, key="low")
    c.h[:, 0] = 20
    c.w[:, 0] = -20
    _check_forward(sc, c)
    _check_backward(sc, c)


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
def test_equal_logits(sc, dtype):
    """All words alike: the loss is log(cols) exactly to the roundings, dw's columns are alike."""
    c = Case(20, 1000, 64, dtype, key="alike")
    c.w.copy_(c.w[:1].expand_as(c.w))
    _check_forward(sc, c)
    _check_backward(sc, c)


@pytest.mark.parametrize("rows", [9, 70, 140, 300])
@pytest.mark.parametrize("dtype", DTYPES, ids=str)
def test_rows_that_do_not_count_hold_anything(sc, rows, dtype):
    """NaN and infinities in rows without a label, with weight 0 or with an upstream gradient of 0."""
    c = Case(rows, 600, 64, dtype, key="junk")
    c.label[0], c.weight[0] = 3, 1.0  # at least one that counts
    c.dloss[0] = 1.0
    lse = c.exact()[1].float()
    clean = _backward(sc, c, lse, c.dloss)
    clean_loss = _forward(sc, c)[0]
    off = ~c.on()
    c.h[off] = NAN
    c.h[off, ::2] = INF
    loss, got_lse = _forward(sc, c)
    assert torch.equal(loss, clean_loss) and bool((loss[off] == 0).all()) and bool(got_lse[off].isnan().all())
    off |= c.dloss == 0
    c.h[off] = NAN
    lse[off] = NAN
    dh, dw = _backward(sc, c, lse, c.dloss)
    assert torch.equal(dh[~off], clean[0][~off]) and torch.equal(dw, clean[1])
    assert bool((dh[off] == 0).all())


def test_no_row_counts(sc):
    for dtype in DTYPES:
        c = Case(50, 300, 64, dtype)
        c.label.fill_(-100)
        loss, _ = _forward(sc, c)
        dh, dw = _backward(sc, c, torch.zeros(50, device="cuda"), c.dloss)
        assert not bool(loss.any()) and not bool(dh.any()) and not bool(dw.any())


def test_no_rows(sc):
    for dtype in DTYPES:
        c = Case(1, 300, 64, dtype)
        c.h, c.label, c.weight = c.h[:0], c.label[:0], c.weight[:0]
        empty = torch.empty(0, device="cuda")
        sc.scape_vocab_loss_forward(c.h, c.w, c.label, empty, empty)
        dw = torch.full_like(c.w.contiguous(), 7.0)
        sc.scape_vocab_loss_backward(c.h, c.w, c.label, empty, c.h, dw)
        torch.cuda.synchronize()
        assert not bool(dw.any())


@pytest.mark.parametrize("rows", [5, 200])
def test_a_bad_row_stays_in_its_row(sc, rows):
    """NaN in a row that counts shows in its loss, its dh and in dw, and in no other row."""
    c = Case(rows, 400, 64, torch.bfloat16)
    c.label[1], c.weight[1] = 5, 1.0
    c.dloss[1] = 1.0
    clean_loss, lse = _forward(sc, c)
    clean_h, _ = _backward(sc, c, lse, c.dloss)
    c.h[1, 3] = NAN
    loss, lse = _forward(sc, c)
    dh, dw = _backward(sc, c, lse, c.dloss)
    keep = torch.arange(rows, device="cuda") != 1
    assert bool(loss[1].isnan()) and torch.equal(loss[keep], clean_loss[keep])
    assert bool(dh[1].isnan().all()) and torch.equal(dh[keep], clean_h[keep])
    assert bool(dw.isnan().all())


def test_one_gradient_without_the_other(sc):
    for rows in (3, 100, 260):
        c = Case(rows, 900, 128, torch.float16)
        lse = c.exact()[1].float()
        dh, dw = _backward(sc, c, lse, c.dloss)
        assert torch.equal(_backward(sc, c, lse, c.dloss, want_w=False)[0], dh)
        assert torch.equal(_backward(sc, c, lse, c.dloss, want_h=False)[1], dw)


def test_factors_far_apart(sc):
    """float16 rows whose factors differ by 2^30, and all of them tiny or huge: dh keeps each row's own precision."""
    for base in (2.0 ** -60, 1.0, 2.0 ** 40):
        c = Case(48, 500, 64, torch.float16, key="far")
        c.weight = torch.full_like(c.weight, 1.0)
        c.label.clamp_(0, 499)
        c.dloss = base * 2.0 ** -(torch.arange(48, device="cuda") % 31).float()
        c.dloss[::3] *= -1
        lse = c.exact()[1].float()
        (dh, tol_h), (dw, tol_w), _ = _exact_grad(c, lse, c.dloss)
        got_h, got_w = _backward(sc, c, lse, c.dloss)
        # a value within the tolerance of the exact one is an infinity where the two together leave float16's range
        fits = dh.abs() + tol_h < 65504
        assert bool((((got_h.double() - dh).abs() <= tol_h) | ~fits).all())
        fits = dw.abs() + tol_w < 65504
        assert bool((((got_w.double() - dw).abs() <= tol_w) | ~fits).all())


def test_gradients_against_differences(sc):
    """Along random directions, against the loss' central difference in float64."""
    for dtype in DTYPES:
        c = Case(30, 200, 64, dtype, key="diff")
        lse = c.exact()[1].float()
        _, (_, tol_w), _ = _exact_grad(c, lse, None)
        (_, tol_h), _, _ = _exact_grad(c, lse, None)
        dh, dw = _backward(sc, c, lse, None)
        g = _gen("dir", dtype)
        vh = torch.randn(c.h.shape, generator=g, device="cuda", dtype=torch.float64)
        vw = torch.randn(c.w.shape, generator=g, device="cuda", dtype=torch.float64)

        def total(t):
            z = ((c.h.double() + t * vh) @ (c.w.double() + t * vw).t()) * c.scale
            at = torch.where(c.on(), c.label, 0).long()
            l = torch.logsumexp(z, 1) - z.gather(1, at[:, None])[:, 0]
            return float((torch.where(c.on(), c.weight.double(), 0.0) * l).sum())

        e = 1e-5
        slope = (total(e) - total(-e)) / (2 * e)
        got = float((dh.double() * vh).sum() + (dw.double() * vw).sum())
        # e^2/6 of the third derivative: moments of z' over the words, with z' of the size of sqrt(64) and less
        third = 6 * float(((vh @ c.w.double().t()).abs() + (c.h.double() @ vw.t()).abs()).amax()) ** 3
        assert abs(got - slope) <= float((tol_h * vh.abs()).sum() + (tol_w * vw.abs()).sum()) + e * e * third + 1e-9


def test_other_stream_and_repeats(sc):
    c = Case(150, 3000, 128, torch.bfloat16)
    want = _forward(sc, c)
    grads = _backward(sc, c, want[1], c.dloss)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for st in (s, None, s):
        got = _forward(sc, c, stream=st)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        again = _backward(sc, c, got[1], c.dloss, stream=st)
        assert torch.equal(again[0], grads[0]) and torch.equal(again[1], grads[1])


@pytest.mark.parametrize("rows", [5, 40, 200, 300])
def test_captured_and_replayed(sc, rows):
    """Forward and backward in one graph, replayed on new data with eager work between."""
    cap = Case(rows, 700, 64, torch.float16, key="cap")
    n, d = cap.h.shape
    loss, lse = torch.empty(n, device="cuda"), torch.empty(n, device="cuda")
    dh, dw = torch.empty(n, d, dtype=cap.dtype, device="cuda"), torch.empty(700, d, dtype=cap.dtype, device="cuda")
    ws = _bytes(max(sc.scape_vocab_loss_workspace_bytes(cap.h, cap.w), sc.scape_vocab_loss_workspace_bytes(cap.h, cap.w, grad=True)))

    def run():
        sc.scape_vocab_loss_forward(cap.h, cap.w, cap.label, loss, lse, weight=cap.weight, workspace=ws)
        sc.scape_vocab_loss_backward(cap.h, cap.w, cap.label, lse, dh, dw, weight=cap.weight, dloss=cap.dloss, workspace=ws)

    run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    for k in range(4):
        new = Case(rows, 700, 64, torch.float16, key=f"cap{k}")
        for name in ("h", "w", "label", "weight", "dloss"):
            getattr(cap, name).copy_(getattr(new, name))
        want = _forward(sc, new)
        grads = _backward(sc, new, want[1], new.dloss)
        for t in (loss, lse, dh, dw):
            t.fill_(3)
        ws.fill_(0x5A)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(loss, want[0]) and torch.equal(lse, want[1])
        assert torch.equal(dh, grads[0]) and torch.equal(dw, grads[1])


def test_two_streams_at_once(sc):
    cases = [Case(140, 2500, 192, torch.bfloat16, key=k) for k in "ab"]
    want = []
    for c in cases:
        loss, lse = _forward(sc, c)
        want.append((loss, lse, *_backward(sc, c, lse, c.dloss)))
    streams = [torch.cuda.Stream() for _ in cases]
    bufs = []
    for c in cases:
        n, d = c.h.shape
        bufs.append((torch.empty(n, device="cuda"), torch.empty(n, device="cuda"),
                     torch.empty(n, d, dtype=c.dtype, device="cuda"), torch.empty(2500, d, dtype=c.dtype, device="cuda"),
                     _bytes(sc.scape_vocab_loss_workspace_bytes(c.h, c.w)),
                     _bytes(sc.scape_vocab_loss_workspace_bytes(c.h, c.w, grad=True))))
    torch.cuda.synchronize()
    for _ in range(5):
        for c, s, (loss, lse, dh, dw, w1, w2) in zip(cases, streams, bufs):
            sc.scape_vocab_loss_forward(c.h, c.w, c.label, loss, lse, weight=c.weight, workspace=w1, stream=s)
            sc.scape_vocab_loss_backward(c.h, c.w, c.label, lse, dh, dw, weight=c.weight, dloss=c.dloss, workspace=w2,
                                         stream=s)
    torch.cuda.synchronize()
    for b, x in zip(bufs, want):
        for got, expect in zip(b, x):
            assert torch.equal(got, expect)


def test_rows_far_apart(sc):
    """Weights whose rows end behind 2^32 bytes."""
    cols, ld, dim, rows = 1100, 1 << 21, 64, 20
    buf = torch.zeros(cols * ld, dtype=torch.bfloat16, device="cuda")
    c = Case(rows, cols, dim, torch.bfloat16, key="far apart")
    w = buf.view(cols, ld)[:, :dim]
    w.copy_(c.w)
    near = _forward(sc, c)
    grads = _backward(sc, c, near[1], c.dloss)
    c.w = w
    far = _forward(sc, c)
    assert torch.equal(near[0], far[0]) and torch.equal(near[1], far[1])
    dh, dw = torch.empty_like(grads[0]).contiguous(), buf.view(cols, ld)[:, dim:2 * dim]
    ws = _bytes(sc.scape_vocab_loss_workspace_bytes(c.h, c.w, grad=True))
    sc.scape_vocab_loss_backward(c.h, c.w, c.label, far[1], dh, dw, scale=c.scale, weight=c.weight, dloss=c.dloss, workspace=ws)
    torch.cuda.synchronize()
    assert torch.equal(dh, grads[0]) and torch.equal(dw, grads[1])


def test_autograd_sees_what_was_written(sc):
    c = Case(4, 50, 64, torch.bfloat16)
    lse = c.exact()[1].float()
    for name in ("dh", "dw"):
        x = torch.randn(c.h.shape if name == "dh" else c.w.shape, device="cuda", dtype=torch.bfloat16, requires_grad=True)
        y = torch.tanh(x)
        ws = _bytes(sc.scape_vocab_loss_workspace_bytes(c.h, c.w, grad=True))
        sc.scape_vocab_loss_backward(c.h, c.w, c.label, lse, workspace=ws, **{name: y.detach()})
        with pytest.raises(RuntimeError, match="modified by an inplace"):
            y.sum().backward()
