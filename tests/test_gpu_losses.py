"""The loss operators on a GPU against plain implementations in float64: row
top-k, distillation from a teacher's top logits (loss, statistics, gradient),
router balance loss (counts, sums, loss, gradient).

Tolerances count roundings.  u = 2^-24 is half a step of float32 relative to
the value, HALF[dtype] half a step of an output type.  A float32 sum of
positive terms, n of them added one after another and the partial sums in a
tree of depth d, is off by at most (n + d) u relative; a term 2^x with x
rounded once and |x| <= X is off by X u ln 2 + 2 u (the exponential itself is
good to a step).
"""
import math
import zlib

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
TINY = {torch.float32: 2.0 ** -149, torch.bfloat16: 2.0 ** -126, torch.float16: 2.0 ** -25}  # an underflow's error
DTYPES = [torch.bfloat16, torch.float16, torch.float32]
INF, NAN = math.inf, math.nan


@pytest.fixture(scope="module", autouse=True)
def sc():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import sparse_communication_adam_amd as sc
    sc.lib()
    yield sc


def _rng(*key):
    """A generator seeded by what the arguments spell."""
    return torch.Generator().manual_seed(zlib.crc32("/".join(map(str, key)).encode()))


def _place(x, dtype, pad=0, shift=0):
    """x on the GPU, in rows `pad` elements apart from each other and
    starting `shift` elements into their buffer."""
    rows, cols = x.shape
    buf = torch.full((rows * (cols + pad) + shift + 8,), NAN, dtype=dtype, device="cuda")
    v = buf[shift:shift + rows * (cols + pad)].view(rows, cols + pad)[:, :cols]
    v.copy_(x.to(dtype))
    return v


def _bytes(n):
    return torch.full((max(n, 1),), 0xA5, dtype=torch.uint8, device="cuda")  # contents are arbitrary


# ---------------------------------------------------------------------------------------------------------------
# row top-k

def _topk_reference(z, k):
    """(val, idx) by value descending, then column ascending; -inf is none."""
    rows, cols = z.shape
    key = z.double()
    key = torch.where(z == INF, 1e300, key)
    key = torch.where(z.isnan(), 1e301, key)
    order = np.stack([np.lexsort((np.arange(cols), -key[r].numpy())) for r in range(rows)])[:, :k]
    idx = torch.from_numpy(order)
    val = z.gather(1, idx)
    return val, torch.where(val == -INF, -1, idx).to(torch.int32)


def _check_topk(sc, z, k, scale=1.0, lse=True, stream=None):
    rows, cols = z.shape
    val = torch.full((rows * k + 3,), 7.0, dtype=z.dtype, device="cuda")
    idx = torch.full((rows * k + 3,), -7, dtype=torch.int32, device="cuda")
    out = torch.full((rows + 3,), 7.0, device="cuda") if lse else None
    ws = _bytes(sc.scape_topk_rows_workspace_bytes(z, k))
    sc.scape_topk_rows(z, k, val, idx, out, scale=scale, workspace=ws, stream=stream)
    torch.cuda.synchronize()
    h = z.cpu()
    rv, ri = _topk_reference(h, k)
    assert torch.equal(idx[:rows * k].cpu().view(rows, k), ri)
    got = val[:rows * k].cpu().view(rows, k)
    assert torch.equal(got.nan_to_num(nan=12345.0), rv.nan_to_num(nan=12345.0))  # the values themselves; -0 == +0
    assert bool((idx[rows * k:] == -7).all()) and bool((val[rows * k:].float() == 7).all())
    if lse:
        x = h.double() * scale
        ref = torch.logsumexp(x, 1)
        ref = torch.where((h == INF).any(1) | h.isnan().any(1), torch.tensor(NAN, dtype=torch.float64), ref)
        o = out[:rows].cpu().double()
        fine = ref.isfinite()
        assert torch.equal(o.isnan(), ref.isnan()) and torch.equal(o[~fine & ~ref.isnan()], ref[~fine & ~ref.isnan()])
        # the sum: at most 128 terms a thread and a tree of 6 + 3 steps, terms with |x| up to the row's spread;
        # the scale's constant (u relative, times the exponents) and the last rounding
        big = x[fine].masked_fill(x[fine] == -INF, 0).abs().amax(1) if fine.any() else torch.zeros(0)
        tol = (128 + 9 + 2) * U + 4 * U * big + U * ref[fine].abs()
        assert bool(((o[fine] - ref[fine]).abs() <= tol).all())
        assert bool((out[rows:] == 7).all())


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
@pytest.mark.parametrize("rows,cols,k,pad,shift", [
    (1, 1, 1, 0, 0), (3, 2, 2, 0, 0), (5, 33, 7, 0, 1), (130, 60, 6, 0, 0), (1001, 64, 8, 0, 0), (7, 300, 32, 4, 3),
    (9, 1024, 32, 0, 0),                                   # short rows
    (2, 64, 40, 0, 0), (9, 1024, 33, 8, 0), (3, 1025, 5, 0, 0), (600, 2500, 17, 7, 5), (2, 4096, 1024, 0, 0),
    (520, 4097, 300, 0, 1),                                # a workgroup a row
    (1, 50304, 32, 0, 0), (2, 50257, 100, 47, 0), (1, 32000, 1024, 0, 1), (3, 16385, 1000, 0, 0), (2, 32769, 600, 0, 3),
    (2, 65535, 80, 0, 1), (5, 131072, 64, 0, 0), (1, 262144, 257, 0, 3),
])
def test_topk(sc, dtype, rows, cols, k, pad, shift):
    g = _rng("topk", dtype, rows, cols, k)
    z = _place(torch.randn(rows, cols, generator=g) * 3, dtype, pad, shift)
    _check_topk(sc, z, k, scale=0.5 if rows % 2 else 1.0)


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
@pytest.mark.parametrize("cols,k", [(64, 8), (1000, 32), (3000 + 1, 50), (20000, 1000), (60000, 64), (90000, 900)])
@pytest.mark.parametrize("kind", ["constant", "three values", "few left", "all masked", "specials", "zeros", "lowest"])
def test_topk_ties_and_specials(sc, dtype, cols, k, kind):
    rows = 3
    g = _rng("ties", dtype, cols, kind)
    if kind == "constant":
        x = torch.full((rows, cols), -1.5)
    elif kind == "three values":
        x = torch.randint(0, 3, (rows, cols), generator=g).float() - 1
    elif kind == "few left":  # fewer entries than slots
        x = torch.full((rows, cols), -INF)
        x[:, torch.randperm(cols, generator=g)[:k // 2]] = torch.randn(k // 2, generator=g)
    elif kind == "all masked":
        x = torch.full((rows, cols), -INF)
        x[1, cols // 2] = 0.25
    elif kind == "specials":
        x = torch.randn(rows, cols, generator=g)
        x[0, torch.randperm(cols, generator=g)[:5]] = NAN
        x[1, torch.randperm(cols, generator=g)[:3]] = INF
        x[1, torch.randperm(cols, generator=g)[:3]] = -INF
        x[2, 5], x[2, 7] = INF, NAN
    elif kind == "lowest":  # a mask of the type's lowest value
        x = torch.full((rows, cols), torch.finfo(dtype).min)
        x[1, ::3] = torch.randn(len(range(0, cols, 3)), generator=g)
        x[2] = 2.0 ** 15 if dtype == torch.float16 else 2.0 ** 127
    else:
        x = torch.where(torch.rand(rows, cols, generator=g) < 0.5, 0.0, -0.0)
    _check_topk(sc, _place(x, dtype, 0, 1), k)


def test_topk_without_lse_and_on_another_stream(sc):
    g = _rng("stream")
    z = _place(torch.randn(4, 5000, generator=g), torch.float32)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    _check_topk(sc, z, 9, lse=False, stream=s)


# ---------------------------------------------------------------------------------------------------------------
# distillation

class Case:
    """One distillation call's arguments on the GPU and its reference in float64."""

    def __init__(self, rows, cols, k, dtype, tail, scale=1.0, pad=0, shift=0, t_dtype=torch.float32, key=""):
        g = _rng("distill", rows, cols, k, dtype, tail, key)
        x = torch.randn(rows, cols, generator=g) * 2
        t = x + torch.randn(rows, cols, generator=g) * 0.7
        self.scale, self.tail = scale, tail
        top = torch.topk(t, min(k, cols), 1)
        self.val = torch.full((rows, k), 0.5)
        self.idx = torch.full((rows, k), -1, dtype=torch.int32)
        self.val[:, :top.values.shape[1]] = top.values
        self.idx[:, :top.indices.shape[1]] = top.indices.to(torch.int32)
        self.val = self.val.to(t_dtype)
        self.lse = torch.logsumexp(t.double() * scale, 1).float() if tail else None
        self.weight = torch.rand(rows, generator=g) + 0.5
        self.x, self.dtype, self.pad, self.shift = x, dtype, pad, shift

    def put(self):
        self.z = _place(self.x, self.dtype, self.pad, self.shift)
        self.h = self.z.cpu().double()
        return self

    def entries(self):
        """Per row, the entries that count: the first slot of each column inside the row."""
        rows, cols = self.h.shape
        for r in range(rows):
            seen, out = set(), []
            for j, i in enumerate(self.idx[r].tolist()):
                if 0 <= i < cols and i not in seen:
                    seen.add(i)
                    out.append((j, i))
            yield r, [j for j, _ in out], [i for _, i in out]

    def reference(self, factor):
        """loss, stats, dz with `factor` per row, each in float64."""
        rows, cols = self.h.shape
        loss, stats, dz = torch.zeros(rows).double(), torch.zeros(rows, 2).double(), torch.zeros(rows, cols).double()
        s = float(np.float32(self.scale))
        for r, slots, at in self.entries():
            if factor[r] == 0 or not at:
                continue
            x = self.h[r] * s
            lse = torch.logsumexp(x, 0)
            rest = torch.ones(cols, dtype=torch.bool)
            rest[at] = False
            tail = torch.logsumexp(x[rest], 0) if rest.any() else torch.tensor(-INF).double()
            stats[r, 0], stats[r, 1] = lse, tail - lse if lse > -INF else -INF
            if lse == -INF:
                continue
            t = self.val[r, slots].double() * s
            if self.tail:
                logq = t - self.lse[r].double()
                q = logq.exp()
                qt = max(0.0, 1 - float(q.sum())) if tail > -INF else 0.0
            elif bool((t > -INF).any()):
                logq = t - torch.logsumexp(t, 0)
                q, qt = logq.exp(), 0.0
            else:
                logq, q, qt = t, torch.zeros_like(t), 0.0
            kl = sum(float(a) * (float(b) - float(x[i]) + float(lse)) for a, b, i in zip(q, logq, at) if a > 0)
            if qt > 0:
                kl += qt * (math.log(qt) - float(tail - lse))
            loss[r] = factor[r] * kl
            d = torch.exp(x - lse) * (float(q.sum()) + qt)
            if qt > 0:
                d[rest] -= qt * torch.exp(x[rest] - tail)
            d[at] -= q
            dz[r] = d * s * factor[r]
        return loss, stats, dz

    def call(self, sc, grad=True, dz=None, stream=None):
        rows = self.z.shape[0]
        if grad and dz is None:
            dz = torch.full_like(self.z, 3.0)
        loss, stats = torch.full((rows,), 7.0, device="cuda"), torch.full((rows, 2), 7.0, device="cuda")
        self.dev = [t.cuda() if t is not None else None for t in (self.val, self.idx, self.lse, self.weight)]
        ws = _bytes(sc.scape_distill_workspace_bytes(self.z, self.idx.shape[1], grad))
        sc.scape_distill_forward(self.z, self.dev[0], self.dev[1], loss, stats, t_lse=self.dev[2], scale=self.scale,
                                 weight=self.dev[3], dz=dz, workspace=ws, stream=stream)
        torch.cuda.synchronize()
        return loss, stats, dz

    def bounds(self, factor):
        """What float32 arithmetic may be off by, per row: of p relative, and
        of the loss absolute.  Exponents go up to the row's spread X; a
        thread adds at most 32 terms and the row's 256th part (a row is cut
        only into more), then a tree of 9 steps."""
        x = (self.h * self.scale).masked_fill(~self.h.isfinite(), 0)
        X = 2 * x.abs().amax(1) + 1
        terms = max(128, 32 + self.h.shape[1] // 256)
        rel = (terms + 9 + 2 + 6) * U + 6 * U * X
        return rel, rel * 2 + U * (1 + X)


def _check_distill(c, factor, loss=None, stats=None, dz=None):
    rl, rs, rd = c.reference(factor)
    rel, absl = c.bounds(factor)
    if loss is not None:
        l, s = loss.cpu().double(), stats.cpu().double()
        inf = rl.isinf()
        assert torch.equal(l[inf], rl[inf])
        assert bool(((l - rl).abs()[~inf] <= (absl * factor.abs())[~inf] + U * rl[~inf].abs()).all()), (l - rl).abs().max()
        for col in (0, 1):
            fine = rs[:, col].isfinite()
            assert torch.equal(s[~fine, col], rs[~fine, col])
            assert bool(((s - rs)[fine, col].abs() <= rel[fine] + U * rs[fine, col].abs()).all())
    if dz is not None:
        d = dz.cpu().double()
        s = float(np.float32(c.scale))
        # p and the tail's factor, each relative, against p's part of the gradient and q's
        p = torch.softmax(c.h * s, 1).nan_to_num(0.0)
        part = (p + (rd / (s * torch.where(factor == 0, 1.0, factor.double()))[:, None]).abs()) * 2
        tol = (rel[:, None] * 2 * part + 4 * U * part) * s * factor.abs()[:, None].double()
        tol = tol + HALF[c.dtype] * rd.abs() * (1 + 1e-3) + TINY[c.dtype]
        worst = ((d - rd).abs() - tol).max()
        assert bool(((d - rd).abs() <= tol).all()), float(worst)


SHAPES = [(1, 1, 1, 0, 0), (3, 2, 1, 0, 1), (4, 40, 40, 0, 0), (5, 33, 7, 3, 0), (600, 130, 9, 0, 0), (3, 1000, 64, 0, 3),
          (530, 4099, 100, 5, 0), (2, 20000, 1024, 0, 1), (1, 50304, 50, 0, 0), (7, 50257, 100, 47, 0),
          (3, 131072, 300, 0, 0), (1, 262144, 20, 0, 1)]


@pytest.mark.parametrize("tail", [True, False], ids=["tail", "renormalised"])
@pytest.mark.parametrize("dtype", DTYPES, ids=str)
@pytest.mark.parametrize("rows,cols,k,pad,shift", SHAPES)
def test_distill(sc, rows, cols, k, pad, shift, dtype, tail):
    """Loss alone, loss with gradient, and the gradient from the statistics."""
    c = Case(rows, cols, k, dtype, tail, 0.5 if rows % 2 else 1.0, pad, shift, dtype if k % 2 else torch.float32).put()
    if rows > 2:
        c.weight[1] = 0
    w = c.weight.double()
    loss, stats, _ = c.call(sc, grad=False)
    _check_distill(c, w, loss, stats)
    loss2, stats2, dz = c.call(sc)
    assert torch.equal(loss, loss2) and torch.equal(stats, stats2)
    _check_distill(c, w, dz=dz)
    up = torch.rand(rows, generator=_rng("up", rows)) + 0.5
    out = torch.full((rows, cols + 3), 3.0, dtype=dtype, device="cuda")  # other alignment than z's
    sc.scape_distill_backward(c.z, c.dev[0], c.dev[1], stats, out[:, 1:cols + 1], t_lse=c.dev[2], scale=c.scale,
                              weight=c.dev[3], dloss=up.cuda())
    torch.cuda.synchronize()
    _check_distill(c, (c.weight * up).double(), dz=out[:, 1:cols + 1])
    assert bool((out[:, 0].float() == 3).all()) and bool((out[:, cols + 1:].float() == 3).all())


@pytest.mark.parametrize("rows,cols", [(600, 2000), (2, 50304), (2, 262144)],
                         ids=["whole rows", "few rows", "split rows"])
@pytest.mark.parametrize("tail", [True, False], ids=["tail", "renormalised"])
def test_distill_odd_rows(sc, rows, cols, tail):
    """Rows that hold little: no entry, entries outside the row, a column
    twice, masked logits, NaN under weight 0, no tail."""
    k = 12
    c = Case(rows, cols, k, torch.float32, tail, key="odd")
    r = rows - 1
    c.idx[0] = -1                                               # no entry
    c.idx[r, 3], c.idx[r, 5] = cols, -5                         # outside
    c.idx[r, 7], c.idx[r, 9] = c.idx[r, 2], c.idx[r, 2]         # again
    if rows > 8:
        c.idx[1, 0], c.idx[1, 1], c.idx[1, 2] = 2 ** 31 - 1, -2 ** 31, cols + 1
        c.x[2, 100:1900] = -INF
        c.x[2, c.idx[2].long()] = 0.5                           # masked columns, none of them an entry
        c.x[3] = -INF                                           # nothing at all
        c.x[4] = NAN
        c.weight[4] = 0                                         # padding: not read
        at = c.idx[5].long()
        keep = c.x[5, at].clone()
        c.x[5] = -INF
        c.x[5, at] = keep                                       # entries only: no tail
        c.x[6, c.idx[6, 0].long()] = -INF                       # an entry the student cannot give: inf
        c.val[7, 1] = -INF                                      # an entry without mass
        c.val[8] = -INF                                         # and a row of them
        if tail:
            c.lse[8] = 3.0
    c.put()
    w = c.weight.double()
    if rows > 8:
        c.h[4] = 0  # the reference skips it too
    loss, stats, dz = c.call(sc)
    _check_distill(c, w, loss, stats, dz)
    assert float(loss[0]) == 0 and not bool(dz[0].any()) and not bool(stats[0].any())
    back = torch.full_like(c.z, 5.0)
    sc.scape_distill_backward(c.z, c.dev[0], c.dev[1], stats, back, t_lse=c.dev[2], weight=c.dev[3])
    torch.cuda.synchronize()
    _check_distill(c, w, dz=back)
    if rows > 8:
        for t in (loss, dz, back):
            assert not bool(t[3].any()) and not bool(t[4].any())
        assert float(loss[6]) == INF


@pytest.mark.parametrize("rows,cols", [(600, 2000), (2, 50304), (2, 262144)],
                         ids=["whole rows", "few rows", "split rows"])
def test_distill_nan_stays_in_its_row(sc, rows, cols):
    c = Case(rows, cols, 5, torch.bfloat16, True, key="nan")
    c.x[0, 17] = NAN
    c.put()
    loss, stats, dz = c.call(sc)
    assert bool(loss[0].isnan()) and bool(dz[0].isnan().all())
    assert not bool(loss[1:].isnan().any()) and not bool(dz[1:].isnan().any())


@pytest.mark.parametrize("tail", [True, False], ids=["tail", "renormalised"])
@pytest.mark.parametrize("dtype", DTYPES, ids=str)
@pytest.mark.parametrize("rows,cols", [(600, 2000), (3, 50304), (3, 262144)],
                         ids=["whole rows", "few rows", "split rows"])
def test_distill_lowest_values(sc, rows, cols, dtype, tail):
    """Logits masked with the type's lowest value: a row of nothing else is a
    uniform one, and one with other logits left has no mass under the mask.
    The uniform row is the same as a row of zeros, bit for bit: only
    differences of its logits enter the loss and the forward gradient."""
    c = Case(rows, cols, 9, dtype, tail, key="lowest")
    low = torch.finfo(dtype).min
    c.x[0] = low
    c.x[1, 50:] = low
    c.x[1, c.idx[1, :4].long()] = low                          # entries under the mask, without teacher's mass
    c.val[1, :4] = -INF
    c.x[1, c.idx[1, 4:].long()] = 1.0
    c.x[2, :cols - 1] = low                                     # two logits left
    c.x[2, c.idx[2, 0].long()] = 0.0
    c.val[2, 1:] = -INF
    if tail:
        c.lse[2] = c.val[2, 0]
    c.put()
    loss, stats, dz = c.call(sc)
    assert bool(loss[:3].isfinite().all()) and bool(dz[:3].isfinite().all()) and bool(stats[:3, 0].isfinite().all())
    shown = [r for r in range(min(rows, 9)) if r != 0]
    w = c.weight.double()
    rl, _, rd = c.reference(w)
    rel = (max(128, 32 + cols // 256) + 9 + 2 + 6) * U + 6 * U * 40  # the masked terms are 0, the others within 20
    for r in shown[:2]:
        assert abs(float(loss[r]) - float(rl[r])) <= w[r] * (2 * rel + 41 * U) + U * abs(float(rl[r]))
        p = torch.softmax(c.h[r] * c.scale, 0)
        part = (p + (rd[r] / w[r]).abs()) * 2
        tol = (rel * 2 * part + 4 * U * part) * w[r] + HALF[dtype] * rd[r].abs() * 1.001 + TINY[dtype]
        assert bool(((dz[r].cpu().double() - rd[r]).abs() <= tol).all())
    c.x[0] = 0
    c.put()
    loss0, stats0, dz0 = c.call(sc)
    assert torch.equal(loss0, loss) and torch.equal(dz0, dz)
    assert float(stats[0, 1]) == float(stats0[0, 1]) and float(stats[0, 0]) < -6e4


@pytest.mark.parametrize("rows,cols", [(600, 2000), (3, 50304), (3, 262144)], ids=["whole rows", "few rows", "split rows"])
def test_distill_of_shifted_logits(sc, rows, cols):
    """2^18 more on every logit, with logits of so few bits that it is exact,
    changes no bit of the loss and of the forward gradient."""
    c = Case(rows, cols, 20, torch.float32, True, key="shifted")
    c.x = (c.x * 16).round() / 16
    c.put()
    loss, stats, dz = c.call(sc)
    c.x = c.x + 2.0 ** 18
    c.put()
    loss1, stats1, dz1 = c.call(sc)
    assert torch.equal(loss, loss1) and torch.equal(dz, dz1) and torch.equal(stats[:, 1], stats1[:, 1])
    assert bool(((stats1[:, 0] - stats[:, 0] - 2.0 ** 18).abs() <= 2.0 ** -6).all())  # half a step of 2^18 is 2^-6


@pytest.mark.parametrize("rows", [300, 520])
def test_distill_many_long_rows(sc, rows):
    """The longest rows, too many to be cut, against float64 on the device."""
    cols, k = 262144, 5
    z = torch.randn(rows, cols, generator=torch.Generator("cuda").manual_seed(rows), device="cuda")
    idx = torch.arange(k, device="cuda", dtype=torch.int32).repeat(rows, 1) * 50000 + 7
    val = z.gather(1, idx.long())
    loss, stats = torch.empty(rows, device="cuda"), torch.empty(rows, 2, device="cuda")
    sc.scape_distill_forward(z, val, idx, loss, stats, workspace=_bytes(sc.scape_distill_workspace_bytes(z, k)))
    torch.cuda.synchronize()
    assert sc.scape_distill_workspace_bytes(z, k) == rows * 8
    for r in range(rows):
        x = z[r].double()
        lse = torch.logsumexp(x, 0)
        q = torch.softmax(val[r].double(), 0)
        kl = (q * (q.log() - val[r].double() + lse)).sum()
        # a 256th of the row a thread and 9 steps, |x| < 6
        tol = (cols // 256 + 32 + 9 + 8 + 6 * 13) * U
        assert abs(float(lse) - float(stats[r, 0])) <= tol + U * float(lse)
        assert abs(float(kl) - float(loss[r])) <= 2 * tol + U * (14 + float(kl))


@pytest.mark.parametrize("rows,cols", [(600, 20000), (2, 20000), (2, 262144)],
                         ids=["whole rows", "few rows", "split rows"])
def test_distill_far_tail(sc, rows, cols):
    """A tail hundreds of e-folds below the entries keeps its terms: its sum
    is held against its own maximum."""
    k = 6
    c = Case(rows, cols, k, torch.float32, True, scale=4.0, key="far")
    c.x -= 30.0
    c.x[torch.arange(rows)[:, None], c.idx.long()] = torch.rand(rows, k, generator=_rng("far")) * 2 + 40
    c.val = c.x.gather(1, c.idx.long()) / 4 - 9.0
    c.lse = (torch.logsumexp(c.val.double() * 4.0, 1) + 0.7).float()  # half of the teacher's mass outside
    c.put()
    w = c.weight.double()
    loss, stats, dz = c.call(sc)
    _check_distill(c, w, loss, stats, dz)
    assert float(stats[:, 1].max()) < -100 and bool(dz.isfinite().all())
    back = torch.empty_like(c.z)
    sc.scape_distill_backward(c.z, c.dev[0], c.dev[1], stats, back, t_lse=c.dev[2], scale=4.0, weight=c.dev[3])
    # against log p_T of -200 and more, one step of the float32 statistics is 2^-24 of that
    ref = c.reference(w)[2]
    rel, _ = c.bounds(w)
    tol = (rel[:, None] * 2 + 2 * U * 400) * (ref.abs() + 4 * w[:, None] * torch.softmax(c.h * 4, 1)) * 2 + 2.0 ** -126
    assert bool(((back.cpu().double() - ref).abs() <= tol).all())


@pytest.mark.parametrize("rows,cols", [(600, 2000), (2, 50304), (3, 262144)], ids=str)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=str)
def test_distill_gradient_over_the_logits(sc, rows, cols, dtype):
    """dz may be z: the same bits as in a tensor of its own."""
    c = Case(rows, cols, 40, dtype, True, key="inplace", shift=1).put()
    loss, stats, dz = c.call(sc)
    keep = c.z.clone()
    loss2, stats2, _ = c.call(sc, dz=c.z)
    assert torch.equal(c.z, dz) and torch.equal(loss, loss2) and torch.equal(stats, stats2)
    back = torch.empty_like(keep)
    sc.scape_distill_backward(keep, c.dev[0], c.dev[1], stats, back, t_lse=c.dev[2], weight=c.dev[3])
    sc.scape_distill_backward(keep, c.dev[0], c.dev[1], stats, keep, t_lse=c.dev[2], weight=c.dev[3])
    torch.cuda.synchronize()
    assert torch.equal(keep, back)


@pytest.mark.parametrize("cols", [262144, 262143, 131075, 65537])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=str)
@pytest.mark.parametrize("shift", [0, 1, 3])
def test_distill_at_the_cuts(sc, cols, dtype, shift):
    """Entries at both ends of long rows and around every cut between parts,
    in a matrix that ends with its allocation (12 MiB and more of float32 are
    one of their own) or, shifted, begins inside a granule."""
    rows, n = 12, 16 // torch.empty(0, dtype=dtype).element_size()
    c = Case(rows, cols, 300, dtype, True, key="cuts", shift=shift)
    at = [0, 1, 2, cols - 1, cols - 2, cols - 3, cols - n, cols - n - 1]
    for cut in range(1024 * n, cols, 1024 * n):
        at += [cut - 1, cut, cut + 1, cut - n, cut + n]
    at = sorted({a for a in at if 0 <= a < cols})[-300:]
    c.idx[:, :len(at)] = torch.tensor(at, dtype=torch.int32)
    c.val[:, :len(at)] = c.x[:, at]
    if shift == 0:
        c.z = torch.empty(rows, cols, dtype=dtype, device="cuda").copy_(c.x)
        c.h = c.z.cpu().double()
    else:
        c.put()
    w = c.weight.double()
    loss, stats, dz = c.call(sc)
    _check_distill(c, w, loss, stats, dz)
    back = torch.full_like(c.z, 5.0)
    sc.scape_distill_backward(c.z, c.dev[0], c.dev[1], stats, back, t_lse=c.dev[2], weight=c.dev[3])
    torch.cuda.synchronize()
    _check_distill(c, w, dz=back)


@pytest.mark.parametrize("tail", [True, False], ids=["tail", "renormalised"])
def test_distill_gradient_against_differences(sc, tail):
    """Central differences of the kernel's own loss.  With step h = 2^-5 the
    loss's rounding (bounded as in Case.bounds) costs 2 e / (2 h), and the
    third derivative of a log-sum-exp, at most 1/2 for each of its two terms,
    h^2 / 6."""
    rows, cols, k, h = 6, 1500, 10, 2.0 ** -5
    c = Case(rows, cols, k, torch.float32, tail, key="fd")
    c.x = (c.x * 64).round() / 64  # so that x +- h is exact
    c.put()
    _, _, dz = c.call(sc)
    err = c.bounds(c.weight)[1]
    for col in [int(c.idx[0, 0]), int(c.idx[0, 5]), 3, 700, 1499]:
        z0 = c.z.clone()
        c.z[:, col] += h
        up = c.call(sc, grad=False)[0]
        c.z.copy_(z0)
        c.z[:, col] -= h
        down = c.call(sc, grad=False)[0]
        c.z.copy_(z0)
        fd = ((up.double() - down.double()) / (2 * h)).cpu()
        tol = c.weight.double() * (err / h + h * h / 6)
        assert bool(((fd - dz[:, col].cpu().double()).abs() <= tol).all()), col


def test_rows_beyond_32_bit_offsets(sc):
    """More than 2^32 elements in one matrix: the last rows are like the same
    rows alone."""
    rows, cols, k = 33000, 131072, 4
    z = torch.zeros(rows, cols, dtype=torch.bfloat16, device="cuda")
    last = torch.randn(600, cols, device="cuda").to(torch.bfloat16)
    z[-600:] = last
    outs = []
    for m in (z, last):
        n = m.shape[0]
        val = torch.empty(n, k, dtype=m.dtype, device="cuda")
        idx = torch.empty(n, k, dtype=torch.int32, device="cuda")
        lse = torch.empty(n, device="cuda")
        ws = _bytes(sc.scape_topk_rows_workspace_bytes(m, k))
        sc.scape_topk_rows(m, k, val, idx, lse, workspace=ws)
        loss, stats = torch.empty(n, device="cuda"), torch.empty(n, 2, device="cuda")
        ws = _bytes(sc.scape_distill_workspace_bytes(m, k))
        sc.scape_distill_forward(m, val, idx, loss, stats, t_lse=lse, scale=0.5, dz=m, workspace=ws)
        outs.append([val[-600:], idx[-600:], lse[-600:], loss[-600:], stats[-600:], m[-600:]])
    torch.cuda.synchronize()
    for a, b in zip(*outs):
        assert torch.equal(a, b)


# ---------------------------------------------------------------------------------------------------------------
# balance

def _router(tokens, experts, k, dtype, key=""):
    g = _rng("router", tokens, experts, k, dtype, key)
    x = torch.randn(tokens, experts, generator=g) * 1.5
    idx = torch.topk(x, k, 1).indices.to(torch.int32)
    idx[torch.rand(tokens, k, generator=g) < 0.05] = -1
    mask = (torch.rand(tokens, generator=g) < 0.9).to(torch.uint8) * 3
    return x, idx, mask


def _offsets(tokens, segments, g, lo=0, hi=None):
    cuts = torch.randint(lo, (tokens if hi is None else hi) + 1, (segments - 1,), generator=g).tolist()
    return sorted([lo, *cuts, tokens if hi is None else hi])


def _p(x, score):
    if score == "softmax":
        p = torch.softmax(x, 1)
        return p.nan_to_num(0.0), torch.ones_like(p)
    s = torch.sigmoid(x)
    t = s.sum(1, keepdim=True)
    return torch.where(t > 0, s / t, 0.0), 1 - s


def _balance_reference(x, idx, mask, edges, score, alpha, counts=None, n_tok=None, up=None):
    t, e = x.shape
    k = idx.shape[1]
    p, slope = _p(x, score)
    out = dict(counts=[], psum=[], n_tok=[], loss=[], dz=torch.full((t, e), NAN).double())
    for i, (a, b) in enumerate(zip(edges[:-1], edges[1:])):
        on = mask[a:b] != 0
        ch = idx[a:b][on].flatten()
        c = torch.bincount(ch[(ch >= 0) & (ch < e)].long(), minlength=e)
        n = int(on.sum())
        ps = p[a:b][on].sum(0)
        out["counts"].append(c)
        out["psum"].append(ps)
        out["n_tok"].append(n)
        out["loss"].append(alpha * e / (k * n * n) * float((c.double() * ps).sum()) if n else 0.0)
        c = c if counts is None else counts[i]
        n = n if n_tok is None else int(n_tok[i])
        G = (1.0 if up is None else float(up[i])) * alpha * e / (k * float(n) * n) if n else 0.0
        d = G * p[a:b] * slope[a:b] * (c.double() - (p[a:b] * c.double()).sum(1, keepdim=True))
        out["dz"][a:b] = torch.where(on[:, None], d, 0.0)
    return out


def _check_balance(sc, x, idx, mask, edges, dtype, score, pad=0, shift=0, alpha=0.01):
    tokens, experts = x.shape
    k, segs = idx.shape[1], len(edges) - 1
    z = _place(x, dtype, pad, shift)
    h = z.cpu().double()
    off = None if edges == [0, tokens] else torch.tensor(edges, dtype=torch.int32, device="cuda")
    m = None if mask is None else mask.cuda()
    href = torch.ones(tokens) if mask is None else mask
    counts = torch.full((segs, experts), -7, dtype=torch.int32, device="cuda")
    psum = torch.full((segs, experts), -7.0, device="cuda")
    n_tok = torch.full((segs,), -7, dtype=torch.int32, device="cuda")
    loss = torch.full((segs,), -7.0, device="cuda")
    ws = _bytes(sc.scape_balance_workspace_bytes(z, segs))
    sc.scape_balance_forward(z, idx.cuda(), counts, psum, n_tok, loss, alpha=alpha, offsets=off, mask=m, score=score,
                             workspace=ws)
    g = _rng("up", segs)
    up = torch.rand(segs, generator=g) + 0.5
    if dtype == torch.float16:
        up *= 1024.0 * max(tokens, 1)
    dz = torch.full((tokens, experts + pad), 5.0, dtype=dtype, device="cuda")[:, :experts]
    sc.scape_balance_backward(z, counts, n_tok, up.cuda(), dz, k=k, alpha=alpha, offsets=off, mask=m, score=score)
    again = torch.full((segs,), -7.0, device="cuda")
    sc.scape_balance_loss(counts, psum, n_tok, again, k, alpha=alpha)
    torch.cuda.synchronize()
    ref = _balance_reference(h, idx, href, edges, score, float(np.float32(alpha)), up=up)
    assert counts.cpu().tolist() == [c.tolist() for c in ref["counts"]]
    assert n_tok.cpu().tolist() == ref["n_tok"]
    # a score: the exponent's rounding (|x| <= X), a sum over at most 16 experts a lane and 6 steps, two divisions;
    # a sum of scores: a 256th of the tokens by 16 waves, or 65536 logits at once by 16 waves of up to 64 tokens, one
    # after another, then 6 steps over a wave and 1 + 8 over the waves
    X = float(h.masked_fill(~h.isfinite(), 0).abs().max()) * 2 + 1 if tokens else 1.0
    rel = U * (2 * X + 16 + 6 + 8)
    total = torch.stack(ref["psum"])
    seq = max(tokens / 4096 + 8, 64) + 15
    tol = total * (rel + U * seq) + 1e-37
    assert bool(((psum.cpu().double() - total).abs() <= tol).all())
    l = torch.tensor(ref["loss"], dtype=torch.float64)
    ltol = l.abs() * (rel + U * (seq + 1)) + 1e-37
    assert bool(((loss.cpu().double() - l).abs() <= ltol).all())
    assert bool(((again.cpu().double() - l).abs() <= ltol + 2 * U * l.abs()).all())
    d, rd = dz.cpu().double(), ref["dz"]
    inside = ~rd.isnan().any(1)
    assert bool((d[~inside] == 5).all())  # rows outside every segment
    p, _ = _p(h, score)
    seg = torch.zeros(tokens, dtype=torch.long)
    for i, (a, b) in enumerate(zip(edges[:-1], edges[1:])):
        seg[a:b] = i
    c = torch.stack(ref["counts"]).double()[seg] if tokens else torch.zeros(0, experts).double()
    n = torch.tensor(ref["n_tok"]).double()[seg].clamp(min=1)
    G = up.double()[seg] * alpha * experts / (k * n * n)
    tol = (G[:, None] * p * (c + (p * c).sum(1, keepdim=True))) * (3 * rel + U * 32)
    tol = tol + HALF[dtype] * rd.abs() * 1.001 + TINY[dtype]
    # past the type's largest value and half a step of it (a segment of one token, scaled for the others) inf is the
    # rounded value
    top = torch.finfo(dtype).max * (1 + torch.finfo(dtype).eps / 4)
    past = d.isinf() & (d.sign() == rd.sign()) & (rd.abs() + tol >= top)
    assert bool(((d - rd).abs()[inside] <= tol[inside]).logical_or(past[inside]).all())
    over = _place(x, dtype, pad, shift)
    sc.scape_balance_backward(over, counts, n_tok, up.cuda(), over, k=k, alpha=alpha, offsets=off, mask=m, score=score)
    torch.cuda.synchronize()
    assert torch.equal(over.cpu()[inside], dz.cpu()[inside])  # over the logits
    return counts, psum, n_tok, loss, dz


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", DTYPES, ids=str)
@pytest.mark.parametrize("tokens,experts,k,segments,pad,shift", [
    (1, 1, 1, 1, 0, 0), (1, 8, 2, 1, 0, 0), (7, 3, 2, 2, 0, 1), (129, 8, 2, 5, 0, 0), (1000, 60, 4, 3, 0, 0),
    (513, 64, 6, 1, 8, 0), (300, 100, 7, 40, 0, 3), (4097, 128, 8, 9, 0, 0), (700, 256, 16, 2, 0, 0),
    (257, 500, 3, 4, 0, 0), (90, 1024, 8, 2, 0, 0), (70000, 16, 2, 3, 0, 0),
    (1000, 61, 5, 3, 0, 1), (6000, 61, 5, 3, 3, 0), (30000, 2, 1, 6, 0, 0), (60000, 7, 2, 6, 1, 0), (9000, 9, 4, 7, 0, 0),
    (65536, 1, 1, 1, 0, 0), (300, 1001, 2, 1, 0, 1), (500, 4, 2, 3, 0, 0), (20000, 5, 2, 3, 0, 1), (20000, 32, 4, 300, 0, 0),
])
def test_balance(sc, tokens, experts, k, segments, pad, shift, dtype, score):
    x, idx, mask = _router(tokens, experts, k, dtype, score)
    edges = _offsets(tokens, segments, _rng("cuts", tokens, segments))
    _check_balance(sc, x, idx, mask if tokens > 1 else None, edges, dtype, score, pad, shift)


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
@pytest.mark.parametrize("tokens,experts", [(400, 24), (9000, 24)])
def test_balance_lowest_values(sc, tokens, experts, dtype):
    """Tokens of the type's lowest value have uniform scores; experts masked
    with it have none."""
    x, idx, mask = _router(tokens, experts, 2, dtype, "lowest")
    x[::7] = torch.finfo(dtype).min
    x[1::7, ::2] = torch.finfo(dtype).min
    z = _place(x, dtype)
    counts = torch.zeros(1, experts, dtype=torch.int32, device="cuda")
    psum, n_tok, loss = torch.zeros(1, experts, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda"), None
    outs = []
    for low in (z, _place(torch.where((x == x[0, 0]).all(1, keepdim=True), 0.0, x), dtype)):
        ws = _bytes(sc.scape_balance_workspace_bytes(low, 1))
        dz = torch.full_like(low, 5.0)
        sc.scape_balance_forward(low, idx.cuda(), counts, psum, n_tok, loss, mask=mask.cuda(), workspace=ws, alpha=0.01)
        sc.scape_balance_backward(low, counts, n_tok, None, dz, k=2, mask=mask.cuda(), alpha=0.01)
        torch.cuda.synchronize()
        outs.append((counts.clone(), psum.clone(), dz))
    assert bool(outs[0][1].isfinite().all()) and bool((outs[0][1] > 0).all())
    for a, b in zip(*outs):  # as if those tokens' logits were 0
        assert torch.equal(a, b)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_balance_odd_segments(sc, score):
    """Empty segments, tokens outside every segment, segments without a valid
    token, choices outside the experts, tokens without a finite logit, NaN in
    masked tokens."""
    x, idx, mask = _router(900, 24, 3, torch.float32, "odd")
    edges = [10, 10, 137, 400, 400, 401, 880, 880]
    mask[137:400] = 0
    mask[5] = mask[895] = 1
    idx[20, 0], idx[21, 1], idx[22] = 24, -9, 2 ** 31 - 1
    x[30] = -INF
    mask[30] = 1
    x[31, :20] = -INF
    x[200] = NAN
    mask[31] = mask[20] = mask[21] = mask[22] = 1
    x[mask == 0] = NAN
    z = x.clone()
    x[mask == 0] = 0  # the first round, with the reference, has 0 there; the second NaN
    counts, psum, n_tok, loss, dz = _check_balance(sc, x, idx, mask, edges, torch.float32, score)
    off = torch.tensor(edges, dtype=torch.int32, device="cuda")
    zn = z.cuda()
    again = [torch.empty_like(t) for t in (counts, psum, n_tok, loss)]
    ws = _bytes(sc.scape_balance_workspace_bytes(zn, len(edges) - 1))
    sc.scape_balance_forward(zn, idx.cuda(), *again, alpha=0.01, offsets=off, mask=mask.cuda(), score=score, workspace=ws)
    torch.cuda.synchronize()
    for a, b in zip((counts, psum, n_tok, loss), again):
        assert torch.equal(a, b)
    assert float(loss[0]) == 0 and int(n_tok[2]) == 0 and float(loss[2]) == 0
    dn = torch.full_like(zn, 5.0)
    up = (torch.rand(len(edges) - 1, generator=_rng("up", len(edges) - 1)) + 0.5).cuda()
    sc.scape_balance_backward(zn, counts, n_tok, up, dn, k=3, alpha=0.01, offsets=off, mask=mask.cuda(), score=score)
    assert torch.equal(dn, dz)
    sc.scape_balance_backward(zn, counts, n_tok, up, zn, k=3, alpha=0.01, offsets=off, mask=mask.cuda(), score=score)
    assert torch.equal(zn[10:880], dn[10:880])  # over the logits


def test_balance_without_tokens(sc):
    z = torch.zeros(0, 8, device="cuda")
    out = [torch.full((2, 8), -7, dtype=torch.int32, device="cuda"), torch.full((2, 8), -7.0, device="cuda"),
           torch.full((2,), -7, dtype=torch.int32, device="cuda"), torch.full((2,), -7.0, device="cuda")]
    ws = _bytes(sc.scape_balance_workspace_bytes(z, 2))
    sc.scape_balance_forward(z, torch.zeros(0, 2, dtype=torch.int32, device="cuda"), *out,
                             offsets=torch.zeros(3, dtype=torch.int32, device="cuda"), workspace=ws)
    assert not any(bool(t.any()) for t in out)


def test_balance_over_workers(sc):
    """Two workers' sums added: the loss and each worker's gradient are those
    of one batch that holds both."""
    x, idx, mask = _router(600, 16, 2, torch.float32, "workers")
    whole = _check_balance(sc, x, idx, mask, [0, 600], torch.float32, "softmax")
    parts = []
    for a, b in ((0, 250), (250, 600)):
        z = x[a:b].cuda()
        o = [torch.empty(1, 16, dtype=torch.int32, device="cuda"), torch.empty(1, 16, device="cuda"),
             torch.empty(1, dtype=torch.int32, device="cuda")]
        sc.scape_balance_forward(z, idx[a:b].cuda(), *o, alpha=0.01, mask=mask[a:b].cuda(),
                                 workspace=_bytes(sc.scape_balance_workspace_bytes(z)))
        parts.append((z, mask[a:b].cuda(), o))
    counts, psum, n_tok = (p + q for p, q in zip(parts[0][2], parts[1][2]))
    assert torch.equal(counts, whole[0]) and torch.equal(n_tok, whole[2])
    loss = torch.empty(1, device="cuda")
    sc.scape_balance_loss(counts, psum, n_tok, loss, 2, alpha=0.01)
    # sums of the same scores in another order: U for each of the additions that differ
    assert abs(float(loss) - float(whole[3])) <= 64 * U * float(whole[3])
    up = (torch.rand(1, generator=_rng("up", 1)) + 0.5).cuda()
    for (z, m, _), (a, b) in zip(parts, ((0, 250), (250, 600))):
        dz = torch.empty_like(z)
        sc.scape_balance_backward(z, counts, n_tok, up, dz, k=2, alpha=0.01, mask=m)
        assert torch.equal(dz, whole[4][a:b])


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_balance_gradient_against_differences(sc, score):
    """Central differences in float64 of the reference loss with the counts
    held: h = 1e-4 leaves h^2 / 6 times third derivatives of at most 6 times
    the loss's scale, and 1e-16 / h."""
    x, idx, mask = _router(40, 12, 2, torch.float32, "fd")
    *_, dz = _check_balance(sc, x, idx, mask, [0, 40], torch.float32, score)
    up = float(torch.rand(1, generator=_rng("up", 1)) + 0.5)
    ref = _balance_reference(x.double(), idx, mask, [0, 40], score, float(np.float32(0.01)))
    n, c = ref["n_tok"][0], ref["counts"][0].double()
    f = lambda y: up * 0.01 * 12 / (2 * n * n) * float((c * _p(y, score)[0][mask != 0].sum(0)).sum())  # noqa: E731
    size = up * 0.01 * 12 / (2 * n * n) * float(c.max())
    for t in range(0, 40, 7):
        for e in (0, 5, 11):
            d = torch.zeros(40, 12).double()
            d[t, e] = 1e-4
            fd = (f(x.double() + d) - f(x.double() - d)) / 2e-4
            assert abs(fd - float(dz[t, e])) <= size * (1e-8 + 64 * U) + 1e-11


# ---------------------------------------------------------------------------------------------------------------
# together

def _together(sc, bufs, stream=None):
    """One distillation micro-step as a program makes it: the teacher's
    records, the loss with its gradient, the loss and gradient apart, the
    router's choice, its balance loss and gradient."""
    b = bufs
    sc.scape_topk_rows(b["t"], 20, b["val"], b["idx"], b["lse"], workspace=b["ws1"], stream=stream)
    sc.scape_distill_forward(b["z"], b["val"], b["idx"], b["loss"], b["stats"], t_lse=b["lse"], weight=b["w"],
                             dz=b["dz"], workspace=b["ws2"], stream=stream)
    sc.scape_distill_backward(b["z"], b["val"], b["idx"], b["stats"], b["dz2"], t_lse=b["lse"], weight=b["w"],
                              stream=stream)
    sc.scape_topk_rows(b["r"], 2, b["rval"], b["ridx"], stream=stream)
    sc.scape_balance_forward(b["r"], b["ridx"], b["counts"], b["psum"], b["n_tok"], b["bloss"], alpha=0.01,
                             workspace=b["ws3"], stream=stream)
    sc.scape_balance_backward(b["r"], b["counts"], b["n_tok"], None, b["dr"], k=2, alpha=0.01, stream=stream)


def _together_buffers(sc, rows, cols, experts, key):
    g = _rng("together", key)
    f = lambda *s: torch.zeros(*s, device="cuda")  # noqa: E731
    i = lambda *s: torch.zeros(*s, dtype=torch.int32, device="cuda")  # noqa: E731
    z = torch.randn(rows, cols, generator=g).to(torch.bfloat16).cuda()
    b = dict(z=z, t=(z + torch.randn(rows, cols, generator=g).cuda()).to(torch.bfloat16),
             r=torch.randn(rows, experts, generator=g).cuda(), w=torch.rand(rows, generator=g).cuda() / rows,
             val=f(rows, 20).to(torch.bfloat16), idx=i(rows, 20), lse=f(rows), loss=f(rows), stats=f(rows, 2),
             dz=torch.zeros_like(z), dz2=torch.zeros_like(z), rval=f(rows, 2), ridx=i(rows, 2), counts=i(1, experts),
             psum=f(1, experts), n_tok=i(1), bloss=f(1), dr=f(rows, experts))
    b["ws1"] = _bytes(sc.scape_topk_rows_workspace_bytes(b["t"], 20))
    b["ws2"] = _bytes(sc.scape_distill_workspace_bytes(z, 20, grad=True))
    b["ws3"] = _bytes(sc.scape_balance_workspace_bytes(b["r"]))
    return b


OUTPUTS = ("val", "idx", "lse", "loss", "stats", "dz", "dz2", "rval", "ridx", "counts", "psum", "n_tok", "bloss", "dr")


@pytest.mark.parametrize("rows,cols", [(3, 50304), (640, 2000), (3, 262144)], ids=["few rows", "whole rows", "split rows"])
def test_captured_and_replayed(sc, rows, cols):
    """The micro-step captured into a graph, replayed with new inputs and with
    eager calls of the same program between the replays: every replay gives
    the eager call's bits."""
    cap = _together_buffers(sc, rows, cols, 16, "a")
    _together(sc, cap)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        _together(sc, cap)
    for n in range(4):
        eager = _together_buffers(sc, rows, cols, 16, n)
        for name in ("z", "t", "r", "w"):
            cap[name].copy_(eager[name])
        for name in OUTPUTS:
            cap[name].fill_(3)
        graph.replay()
        _together(sc, eager)
        torch.cuda.synchronize()
        for name in OUTPUTS:
            assert torch.equal(cap[name], eager[name]), (n, name)


@pytest.mark.parametrize("cols", [50304, 262144])
def test_two_streams_at_once(sc, cols):
    """Calls on two streams with workspaces of their own do not disturb each other."""
    a, b = (_together_buffers(sc, 5, cols, 16, k) for k in "xy")
    want = []
    for s in (a, b):
        _together(sc, s)
        torch.cuda.synchronize()
        want.append({n: s[n].clone() for n in OUTPUTS})
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(5):
        _together(sc, a, s1)
        _together(sc, b, s2)
    torch.cuda.synchronize()
    for s, w in zip((a, b), want):
        for n in OUTPUTS:
            assert torch.equal(s[n], w[n]), n


def test_a_training_step(sc):
    """The losses' gradients through a small model into the optimizer's step:
    two workers' batches, distilled from a teacher and balanced over experts,
    bf16 weight gradients in the optimizer's flat layout, one step."""
    g = _rng("train")
    h, vocab, experts, tokens, W = 64, 2048, 8, 96, 2
    cfg = sc.ScapeConfig(layer_numel=[vocab * h, experts * h], workers=W, keep_num=1, keep_den=10)
    from sparse_communication_adam_amd.state import ScapeState
    state = ScapeState(cfg)
    flat = torch.randn(state.layout.n_pad, generator=g).cuda() * 0.05
    state.set_params(flat)
    o0, o1 = state.layout.layer_offset
    teacher = torch.randn(vocab, h, generator=g).cuda() * 0.2
    for step in range(2):
        head = state.x[o0:o0 + vocab * h].view(vocab, h)
        router = state.x[o1:o1 + experts * h].view(experts, h)
        grads, stats = [], []
        for w in range(W):
            x = torch.randn(tokens, h, generator=g).cuda()
            b = dict(z=(x @ head.t()), t=(x @ teacher.t()), r=(x @ router.t()))
            zero = lambda *s, dtype=torch.float32: torch.zeros(*s, dtype=dtype, device="cuda")  # noqa: E731
            val, idx, lse = zero(tokens, 16), zero(tokens, 16, dtype=torch.int32), zero(tokens)
            sc.scape_topk_rows(b["t"], 16, val, idx, lse,
                               workspace=_bytes(sc.scape_topk_rows_workspace_bytes(b["t"], 16)))
            loss, st = zero(tokens), zero(tokens, 2)
            weight = torch.full((tokens,), 1.0 / tokens, device="cuda")
            dz = torch.empty_like(b["z"])
            sc.scape_distill_forward(b["z"], val, idx, loss, st, t_lse=lse, weight=weight, dz=dz,
                                     workspace=_bytes(sc.scape_distill_workspace_bytes(b["z"], 16, grad=True)))
            rval, ridx = zero(tokens, 2), zero(tokens, 2, dtype=torch.int32)
            sc.scape_topk_rows(b["r"], 2, rval, ridx)
            counts, psum = zero(1, experts, dtype=torch.int32), zero(1, experts)
            n_tok = zero(1, dtype=torch.int32)
            sc.scape_balance_forward(b["r"], ridx, counts, psum, n_tok,
                                     workspace=_bytes(sc.scape_balance_workspace_bytes(b["r"])))
            grads.append((x, dz, b, ridx, (val, idx, lse)))
            stats.append((counts, psum, n_tok))
        counts, psum, n_tok = (a + b for a, b in zip(*stats))
        bloss = torch.zeros(1, device="cuda")
        sc.scape_balance_loss(counts, psum, n_tok, bloss, 2, alpha=0.01)
        flat_grads = []
        for x, dz, b, ridx, (val, idx, lse) in grads:
            dr = torch.empty_like(b["r"])
            sc.scape_balance_backward(b["r"], counts, n_tok, None, dr, k=2, alpha=0.01)
            gr = torch.zeros(state.layout.n_pad, dtype=torch.bfloat16, device="cuda")
            gr[o0:o0 + vocab * h] = (dz.t() @ x).flatten().to(torch.bfloat16)
            gr[o1:o1 + experts * h] = (dr.t() @ x).flatten().to(torch.bfloat16)
            # the whole chain in float64 on the host: gradients of the same losses by autograd
            z = b["z"].cpu().double().requires_grad_()
            logq = val.cpu().double() - lse.cpu().double()[:, None]
            at = torch.log_softmax(z, 1).gather(1, idx.cpu().long())
            rest = 1 - logq.exp().sum(1)
            keep = torch.ones_like(z, dtype=torch.bool).scatter_(1, idx.cpu().long(), False)
            tail = torch.logsumexp(z.masked_fill(~keep, -INF), 1) - torch.logsumexp(z, 1)
            ((logq.exp() * (logq - at)).sum(1) + rest * (rest.log() - tail)).mean().backward()
            assert float((dz.cpu().double() - z.grad).norm() / z.grad.norm()) < 1e-5
            r = b["r"].cpu().double().requires_grad_()
            f = counts[0].cpu().double() * experts / (2 * float(n_tok))
            (0.01 * (f * torch.softmax(r, 1).sum(0) / float(n_tok)).sum()).backward()
            assert float((dr.cpu().double() - r.grad).norm() / r.grad.norm()) < 1e-5
            flat_grads.append(gr.view(torch.int16))
        before = state.x.clone()
        state.step(flat_grads)
        torch.cuda.synchronize()
        moved = (state.x != before).nonzero().numel()
        assert (moved == 0) == (step == 0)  # the first step's mask is empty
        if step:
            assert moved <= state.layout.k_total
    state.destroy()
