"""Tokens to their experts and back on a GPU, against plain implementations.

The sort and the gather are exact.  A combination is a float32 sum of k fused
products (each addition rounds once: k u of the sum of magnitudes, u = 2^-24)
rounded once to its type; the weight's gradient a float32 sum of dim exact or
once-rounded products in any order, (dim + 1) u of the sum of magnitudes; dy one
float32 product rounded once.
"""
import math
import zlib

import pytest
import torch

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
TINY = {torch.float32: 2.0 ** -149, torch.bfloat16: 2.0 ** -126, torch.float16: 2.0 ** -25}
DTYPES = [torch.bfloat16, torch.float16, torch.float32]
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
    return torch.Generator().manual_seed(zlib.crc32("/".join(map(str, key)).encode()))


def _place(x, dtype, pad=0, shift=0, fill=NAN):
    rows, cols = x.shape
    buf = torch.full((rows * (cols + pad) + shift + 8,), fill, dtype=dtype, device="cuda")
    v = buf[shift:shift + rows * (cols + pad)].view(rows, cols + pad)[:, :cols]
    v.copy_(x.to(dtype))
    return v


def _sort(sc, idx, experts, stream=None):
    tokens, k = idx.shape
    off = torch.full((experts + 3,), -7, dtype=torch.int32, device="cuda")
    row = torch.full((tokens * k + 3,), -7, dtype=torch.int32, device="cuda")
    ws = torch.full((max(1, sc.scape_expert_sort_workspace_bytes(idx, experts)),), 0xA5, dtype=torch.uint8, device="cuda")
    sc.scape_expert_sort(idx, experts, off, row, workspace=ws, stream=stream)
    torch.cuda.synchronize()
    assert bool((off[experts + 1:] == -7).all()) and bool((row[tokens * k:] == -7).all())
    return off[:experts + 1], row[:tokens * k].view(tokens, k)


def _plain_sort(idx, experts):
    e = idx.flatten().long()
    on = (e >= 0) & (e < experts)
    order = torch.argsort(torch.where(on, e, experts), stable=True)
    row = torch.full_like(e, -1)
    row[order] = torch.arange(e.numel())
    row[~on] = -1
    counts = torch.bincount(e[on], minlength=experts)
    return torch.cat([torch.zeros(1, dtype=torch.long), counts.cumsum(0)]).int(), row.int().view(idx.shape)


SORTS = [(0, 2, 5), (1, 1, 1), (1, 8, 64), (3, 2, 2), (63, 1, 7), (64, 4, 60), (65, 3, 1024), (257, 8, 256), (1000, 6, 64),
         (2049, 1, 9), (4096, 8, 128), (20000, 5, 1000), (131072, 8, 64), (300000, 4, 512)]


@pytest.mark.parametrize("tokens,k,experts", SORTS)
@pytest.mark.parametrize("kind", ["random", "one expert", "descending", "none", "odd values", "repeated"])
def test_sort(sc, tokens, k, experts, kind):
    g = _gen("sort", tokens, k, experts, kind)
    idx = torch.randint(0, experts, (tokens, k), generator=g, dtype=torch.int32)
    if kind == "one expert":
        idx.fill_(experts - 1)
    elif kind == "descending":
        idx = (experts - 1 - torch.arange(tokens * k) % experts).int().view(tokens, k)
    elif kind == "none":
        idx.fill_(-1)
    elif kind == "odd values":
        junk = torch.tensor([-1, -2 ** 31, experts, 2 ** 31 - 1], dtype=torch.int32)
        at = torch.rand(tokens, k, generator=g) < 0.3
        idx = torch.where(at, junk[torch.randint(0, 4, (tokens, k), generator=g)], idx)
    elif kind == "repeated":
        idx = idx[:, :1].expand(tokens, k).contiguous()
    off, row = _sort(sc, idx.cuda(), experts)
    want_off, want_row = _plain_sort(idx, experts)
    assert torch.equal(off.cpu(), want_off)
    assert torch.equal(row.cpu(), want_row)


def test_sort_of_many_choices(sc):
    """More choices than 512 blocks of 2048 hold."""
    g = torch.Generator(device="cuda").manual_seed(5)
    idx = torch.randint(-1, 37, (1 << 20, 3), generator=g, dtype=torch.int32, device="cuda")
    off, row = _sort(sc, idx, 37)
    want_off, want_row = _plain_sort(idx.cpu(), 37)
    assert torch.equal(off.cpu(), want_off) and torch.equal(row.cpu(), want_row)


class Case:
    def __init__(self, sc, tokens, k, experts, dim, dtype, pad=0, shift=0, key=""):
        g = _gen("move", tokens, k, experts, dim, dtype, key)
        idx = torch.randint(0, experts, (tokens, k), generator=g, dtype=torch.int32)
        idx[torch.rand(tokens, k, generator=g) < 0.1] = -1
        if tokens > 2:
            idx[1] = -1  # a token without any expert
        self.off, self.row = _sort(sc, idx.cuda(), experts)
        rows = tokens * k
        self.dtype, self.tokens, self.k, self.dim = dtype, tokens, k, dim
        self.x = _place(torch.randn(tokens, dim, generator=g), dtype, pad, shift)
        self.y = _place(torch.randn(rows, dim, generator=g), dtype, pad, shift)
        self.weight = torch.rand(tokens, k, generator=g).cuda() - 0.2
        self.weight[torch.rand(tokens, k, generator=g).cuda() < 0.1] = 0.0
        self.pad, self.shift = pad, shift

    def new(self, rows, fill=NAN):
        return _place(torch.full((rows, self.dim), fill), self.dtype, self.pad, self.shift)

    def picked(self):
        there = (self.row >= 0) & (self.row < self.y.shape[0])
        return self.y.double()[torch.where(there, self.row, 0).long()], there


def _untouched(t):
    """What lies between a placed matrix's rows and behind them is still NaN."""
    whole = t._base
    assert int(whole.isnan().sum()) == whole.numel() - t.numel() + int(t.isnan().sum())


def _check_moves(sc, c):
    rows = c.y.shape[0]
    y = c.new(rows, 5.0)
    sc.scape_expert_gather(c.x, c.row, y)
    want = torch.full((rows, c.dim), 5.0, dtype=c.dtype, device="cuda")
    t, j = torch.nonzero(c.row >= 0, as_tuple=True)
    want[c.row[t, j].long()] = c.x[t]
    torch.cuda.synchronize()
    assert torch.equal(y, want)
    _untouched(y)
    half, tiny = HALF[c.dtype], TINY[c.dtype]
    yy, there = c.picked()
    for weight in (c.weight, None):
        w = torch.where(there, 1.0 if weight is None else weight.double(), 0.0)
        parts = torch.where((w != 0)[:, :, None], w[:, :, None] * yy, 0.0)
        exact, size = parts.sum(1), parts.abs().sum(1)
        out = c.new(c.tokens)
        sc.scape_expert_combine(c.y, c.row, out, weight=weight)
        torch.cuda.synchronize()
        assert bool(((out.double() - exact).abs() <= c.k * U * size * (1 + half) + half * exact.abs() + tiny).all())
        _untouched(out)
        # gradients
        dout = c.x
        dy, dw = c.new(rows, 5.0), torch.full((c.tokens, c.k), 7.0, device="cuda")
        sc.scape_expert_combine_backward(c.y, c.row, dout, dy, weight=weight, dweight=dw)
        torch.cuda.synchronize()
        prod = yy * dout.double()[:, None]
        exact_w = torch.where(there, prod.sum(2), 0.0)
        tol = (c.dim + 1) * U * prod.abs().sum(2) + U * exact_w.abs()
        assert bool(((dw.double() - exact_w).abs() <= tol).all())
        full = torch.full((rows, c.dim), 5.0, dtype=torch.float64, device="cuda")
        full[c.row[t, j].long()] = w[t, j, None] * dout[t].double()
        assert bool(((dy.double() - full).abs() <= (half * (1 + U) + U) * full.abs() + tiny).all())
        _untouched(dy)
        # either alone, and over y itself
        dy2, dw2 = c.new(rows, 5.0), torch.full_like(dw, 7.0)
        sc.scape_expert_combine_backward(c.y, c.row, dout, dy2, weight=weight)
        sc.scape_expert_combine_backward(c.y, c.row, dout, weight=weight, dweight=dw2)
        own, dw3 = c.new(rows), torch.full_like(dw, 7.0)
        own.copy_(c.y)
        sc.scape_expert_combine_backward(own, c.row, dout, own, weight=weight, dweight=dw3)
        torch.cuda.synchronize()
        assert torch.equal(dy2, dy) and torch.equal(dw2, dw) and torch.equal(dw3, dw)
        assert torch.equal(own[c.row[t, j].long()], dy[c.row[t, j].long()])


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
@pytest.mark.parametrize("tokens,k,experts,dim,pad,shift", [
    (1, 1, 1, 1, 0, 0), (1, 6, 64, 2048, 0, 0), (3, 2, 4, 7, 0, 1), (5, 3, 8, 8, 3, 0), (33, 8, 16, 511, 0, 3),
    (130, 4, 8, 512, 8, 0), (64, 2, 5, 1001, 0, 0), (200, 1, 3, 1536, 1, 1), (17, 9, 40, 4100, 0, 0), (9, 70, 100, 130, 0, 0),
    (1000, 8, 64, 256, 0, 0), (6, 8, 8, 9000, 0, 5),
])
def test_moves(sc, tokens, k, experts, dim, pad, shift, dtype):
    _check_moves(sc, Case(sc, tokens, k, experts, dim, dtype, pad, shift))


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
@pytest.mark.parametrize("dim", [4, 9, 31, 33, 64, 65, 100, 129, 249, 257, 500, 513, 1025, 2047, 4101, 8195, 512, 1536])
def test_row_lengths(sc, dim, dtype):
    """Rows on either side of each way they are cut: lanes for a choice, granules a lane, a last granule that reaches back."""
    _check_moves(sc, Case(sc, 37, 5, 8, dim, dtype, dim % 3, dim % 2, key="rows"))


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
def test_what_does_not_count_holds_anything(sc, dtype):
    """NaN in rows that no place or only weights of 0 name; places outside y; a token without experts."""
    c = Case(sc, 40, 3, 8, 100, dtype, key="junk")
    clean = c.new(40)
    sc.scape_expert_combine(c.y, c.row, clean, weight=c.weight)
    used = torch.zeros(c.y.shape[0], dtype=torch.bool, device="cuda")
    t, j = torch.nonzero((c.row >= 0) & (c.weight != 0), as_tuple=True)
    used[c.row[t, j].long()] = True
    y = c.y.clone()
    y[~used] = NAN
    out = c.new(40)
    row = c.row.clone()
    row[c.row < 0] = torch.tensor([-1, -2 ** 31, y.shape[0], 2 ** 31 - 1], dtype=torch.int32, device="cuda")[
        torch.arange(int((c.row < 0).sum()), device="cuda") % 4]
    sc.scape_expert_combine(y, row, out, weight=c.weight)
    torch.cuda.synchronize()
    assert torch.equal(out, clean) and not bool(out[1].any())
    # the gradient of a weight of 0 is a row of +0 whatever dout holds, and its own gradient is not cut off
    c.weight[0], c.weight[2] = 0.0, 1.0
    dout = c.x.clone()
    dout[0] = INF
    dy, dw = torch.full_like(c.y, 5.0), torch.zeros(40, 3, device="cuda")
    sc.scape_expert_combine_backward(c.y, row, dout, dy, weight=c.weight, dweight=dw)
    g = torch.full_like(dy, 5.0)
    sc.scape_expert_gather(dout, row, g)
    torch.cuda.synchronize()
    for jj in range(3):
        r = int(c.row[0, jj])
        if r >= 0:
            assert not bool(dy[r].any())
            assert not bool(dw[0, jj].isfinite())
        r = int(c.row[2, jj])
        if r >= 0:
            assert torch.equal(dy[r], dout[2])
    assert not bool(dw[c.row < 0].any())
    named = torch.zeros(c.y.shape[0], dtype=torch.bool, device="cuda")
    named[c.row[c.row >= 0].long()] = True
    assert bool((dy[~named] == 5).all()) and bool((g[~named] == 5).all())


def test_fewer_rows_than_places(sc):
    """A y with room for the first rows only: places behind it are none."""
    c = Case(sc, 50, 2, 4, 64, torch.float32, key="room")
    full = torch.zeros(100, 64, device="cuda")
    sc.scape_expert_gather(c.x, c.row, full)
    part = torch.full((60, 64), 9.0, device="cuda")
    sc.scape_expert_gather(c.x, c.row, part[:40])
    torch.cuda.synchronize()
    assert torch.equal(part[:40], full[:40]) and bool((part[40:] == 9).all())
    out, want = torch.empty(50, 64, device="cuda"), torch.empty(50, 64, device="cuda")
    sc.scape_expert_combine(c.y[:40], c.row, out, weight=c.weight)
    sc.scape_expert_combine(c.y, torch.where(c.row < 40, c.row, -1), want, weight=c.weight)
    torch.cuda.synchronize()
    assert torch.equal(out, want)


def test_gather_and_combine_are_adjoint(sc):
    """<gather(x), y> = <x, combine(y)>, and differences of the weighted sum."""
    c = Case(sc, 60, 4, 8, 48, torch.float32, key="adjoint")
    g = torch.zeros_like(c.y)
    sc.scape_expert_gather(c.x, c.row, g)
    back = torch.empty_like(c.x)
    sc.scape_expert_combine(c.y, c.row, back)
    a, b = float((g.double() * c.y.double()).sum()), float((c.x.double() * back.double()).sum())
    size = float((g.double() * c.y.double()).abs().sum())
    assert abs(a - b) <= 6 * U * size
    # the weighted sum is bilinear: a central difference of step 1 is exact
    dout = torch.randn(60, 48, generator=_gen("up")).cuda()
    dy, dw = torch.zeros_like(c.y), torch.empty(60, 4, device="cuda")
    sc.scape_expert_combine_backward(c.y, c.row, dout, dy, weight=c.weight, dweight=dw)
    vy, vw = torch.randn(240, 48, generator=_gen("vy")).cuda().double(), torch.randn(60, 4, generator=_gen("vw")).cuda().double()
    yy, there = c.picked()
    vv = vy[torch.where(there, c.row, 0).long()]
    on = there & (c.weight != 0)

    def total(t):
        w = torch.where(there, c.weight.double() + t * vw, 0.0)
        return float(((w[:, :, None] * (yy + t * vv)).sum(1) * dout.double()).sum())

    slope = (total(1.0) - total(-1.0)) / 2
    got = float((dy.double() * vy).sum() + (dw.double() * vw).sum())
    size = float((dy.double() * vy).abs().sum() + ((yy * dout.double()[:, None]).abs().sum(2) * vw.abs()).sum())
    assert abs(got - slope) <= 60 * U * size and bool(on.any())


def test_streams_repeats_and_graphs(sc):
    c = Case(sc, 300, 4, 32, 264, torch.bfloat16, key="graph")
    g = _gen("graph idx")
    idx = torch.randint(-1, 32, (300, 4), generator=g, dtype=torch.int32).cuda()
    buf = dict(off=torch.empty(33, dtype=torch.int32, device="cuda"), row=torch.empty(300, 4, dtype=torch.int32, device="cuda"),
               y=torch.zeros(1200, 264, dtype=torch.bfloat16, device="cuda"), out=torch.empty_like(c.x.contiguous()),
               dy=torch.zeros(1200, 264, dtype=torch.bfloat16, device="cuda"), dw=torch.empty(300, 4, device="cuda"))
    ws = torch.empty(sc.scape_expert_sort_workspace_bytes(idx, 32), dtype=torch.uint8, device="cuda")

    def run(b, stream=None):
        sc.scape_expert_sort(idx, 32, b["off"], b["row"], workspace=ws, stream=stream)
        sc.scape_expert_gather(c.x, b["row"], b["y"], stream=stream)
        sc.scape_expert_combine(b["y"], b["row"], b["out"], weight=c.weight, stream=stream)
        sc.scape_expert_combine_backward(b["y"], b["row"], c.x, b["dy"], weight=c.weight, dweight=b["dw"], stream=stream)

    run(buf)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run(buf)
    s = torch.cuda.Stream()
    for k in range(4):
        idx.copy_(torch.randint(-1, 32, (300, 4), generator=g, dtype=torch.int32))
        c.x.copy_(torch.randn(300, 264, generator=g))
        eager = {n: torch.full_like(t, 3) for n, t in buf.items()}
        for t in buf.values():
            t.fill_(3)
        torch.cuda.synchronize()
        run(eager, s)
        torch.cuda.synchronize()
        ws.fill_(0x5A)
        graph.replay()
        torch.cuda.synchronize()
        for n in buf:
            assert torch.equal(buf[n], eager[n]), n


def test_rows_beyond_32_bit_offsets(sc):
    """y of over 2^32 bytes."""
    dim, rows, tokens = 8192, 300000, 64
    y = torch.zeros(rows, dim, dtype=torch.bfloat16, device="cuda")
    g = _gen("far")
    x = torch.randn(tokens, dim, generator=g).to(torch.bfloat16).cuda()
    row = (torch.arange(tokens, dtype=torch.int32) * 4600 + 9000).view(tokens, 1).cuda()
    row[-1] = rows - 1
    sc.scape_expert_gather(x, row, y)
    out = torch.empty_like(x)
    sc.scape_expert_combine(y, row, out)
    dy, dw = torch.zeros_like(y), torch.empty(tokens, 1, device="cuda")
    sc.scape_expert_combine_backward(y, row, x, dy, dweight=dw)
    torch.cuda.synchronize()
    assert torch.equal(out, x) and torch.equal(y[row[:, 0].long()], x) and torch.equal(dy, y)
    assert int((y != 0).any(1).sum()) == tokens


def test_the_most_tokens(sc):
    """As many tokens as a move takes, and one more is refused."""
    tokens = 2 ** 25
    x = (torch.arange(tokens, device="cuda", dtype=torch.int32) % 251).to(torch.bfloat16).view(tokens, 1)
    row = torch.arange(tokens - 1, -1, -1, device="cuda", dtype=torch.int32).view(tokens, 1)
    y, out, dy = torch.empty_like(x), torch.empty_like(x), torch.full_like(x, NAN)
    dw = torch.full((tokens, 1), NAN, device="cuda")
    sc.scape_expert_gather(x, row, y)
    assert torch.equal(y, x.flip(0))
    sc.scape_expert_combine(y, row, out)
    assert torch.equal(out, x)
    sc.scape_expert_combine_backward(y, row, x, dy, dweight=dw)
    assert torch.equal(dy, y) and torch.equal(dw, x.float() ** 2)
    more = torch.empty(tokens + 1, 1, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(sc.ScapeError):
        sc.scape_expert_gather(more, torch.zeros(tokens + 1, 1, dtype=torch.int32, device="cuda"), more)


def test_autograd_sees_what_was_written(sc):
    c = Case(sc, 10, 2, 4, 32, torch.float32, key="versions")
    x = torch.randn(20, 32, device="cuda", requires_grad=True)
    y = torch.tanh(x)
    sc.scape_expert_gather(c.x, c.row, y.detach())
    with pytest.raises(RuntimeError, match="modified by an inplace"):
        y.sum().backward()
