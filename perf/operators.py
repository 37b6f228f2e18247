"""The loss operators' measured cases: the top entries of each row, distillation from a teacher's top
logits, and the balance loss of a router, each in a plain form and through the framework's calls.

A case's "op" says which path it is:
  topk          the k largest entries of each row and the row's log-sum-exp (a teacher's records, a router's choice)
  distill       the distillation loss alone (evaluation, or a backward pass that comes later)
  distill_grad  the loss and the gradient of its sum in one call (a training step whose row weights are known)
  distill_back  the gradient from what the forward call kept and an upstream gradient for each row
  balance       per-expert counts, probability sums, token counts and the loss of each segment
  balance_back  the gradient with respect to the router's logits
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
SIZE = {"bf16": 2, "f16": 2, "f32": 4}


# --------------------------------------------------------------------------------------------------------------
# cases

def listed():
    return [
        # a teacher's records for one micro-batch of 4 sequences of 1024 tokens over a 32000-word vocabulary
        dict(name="topk teacher 4096x32000", op="topk", dtype="bf16", rows=4096, cols=32000, ld=32000, k=64, scale=1.0),
        # float32 logits of a 50257-word vocabulary in rows padded to 50304, softened by a temperature of 2
        dict(name="topk padded 1021x50257", op="topk", dtype="f32", rows=1021, cols=50257, ld=50304, k=100, scale=0.5),
        # one token at a time: a teacher that answers as it generates
        dict(name="topk one token 50304", op="topk", dtype="bf16", rows=1, cols=50304, ld=50304, k=32, scale=1.0),
        # a router's choice of 6 of 64 experts
        dict(name="topk router 65536x64", op="topk", dtype="f32", rows=65536, cols=64, ld=64, k=6, scale=1.0),
        # a handful of tokens: the smallest evaluation of the loss
        dict(name="distill 7x50304", op="distill", dtype="bf16", rows=7, cols=50304, ld=50304, k=50, scale=1.0,
             tail=True, teacher="f32"),
        # evaluation over two sequences, odd vocabulary without padding, teacher renormalised over its entries
        dict(name="distill 2048x50257", op="distill", dtype="f16", rows=2048, cols=50257, ld=50257, k=100, scale=0.5,
             tail=False, teacher="f16"),
        # the training step: loss and gradient of one micro-batch
        dict(name="distill_grad 4096x32000", op="distill_grad", dtype="bf16", rows=4096, cols=32000, ld=32000, k=64,
             scale=1.0, tail=True, teacher="bf16"),
        # the gradient alone, float32 logits
        dict(name="distill_back 1024x50304", op="distill_back", dtype="f32", rows=1024, cols=50304, ld=50304, k=128,
             scale=0.5, tail=True, teacher="f32"),
        # the balance loss over a whole batch
        dict(name="balance 131072x64", op="balance", dtype="f32", tokens=131072, experts=64, k=8, segments=1,
             score="softmax"),
        # one short batch of ragged sequences, few experts
        dict(name="balance 2000x8", op="balance", dtype="bf16", tokens=2000, experts=8, k=2, segments=7, score="softmax"),
        # gradients over many ragged sequences and many experts, sigmoid scores
        dict(name="balance_back 65536x256", op="balance_back", dtype="bf16", tokens=65536, experts=256, k=8, segments=33,
             score="sigmoid"),
        # gradients of one short batch
        dict(name="balance_back 4096x60", op="balance_back", dtype="f32", tokens=4096, experts=60, k=4, segments=1,
             score="softmax"),
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["topk", "topk", "distill", "distill_grad", "distill_back", "balance", "balance_back"])
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    if op.startswith("balance"):
        experts = _spread(rng, 4, 512)
        tokens = min(_spread(rng, 1, 131072), (1 << 24) // experts)
        return dict(op=op, dtype=dtype, tokens=tokens, experts=experts, k=rng.randint(1, min(16, experts)),
                    segments=_spread(rng, 1, min(64, tokens)), score=rng.choice(["softmax", "sigmoid"]))
    if op == "topk" and rng.random() < 0.4:
        cols = _spread(rng, 8, 512)
        rows = min(_spread(rng, 1, 131072), (1 << 24) // cols)
        k = rng.randint(1, min(16, cols))
        return dict(op=op, dtype=dtype, rows=rows, cols=cols, ld=cols, k=k, scale=1.0)
    cols = rng.choice([32000, 50257, 50304, _spread(rng, 1000, 131072)])
    rows = _spread(rng, 1, max(1, min(4096, (1 << 26) // cols)))
    case = dict(op=op, dtype=dtype, rows=rows, cols=cols, ld=cols + rng.choice([0, 0, 1, 40]), k=_spread(rng, 1, 256),
                scale=rng.choice([1.0, 1.0, 0.5, 0.25]))
    if op != "topk":
        case.update(tail=rng.random() < 0.5, teacher=rng.choice([dtype, "f32"]))
    return case


def work(case):
    op = case["op"]
    if op.startswith("balance"):
        t, e, k, s = case["tokens"], case["experts"], case["k"], case["segments"]
        b = SIZE[case["dtype"]]
        if op == "balance":  # logits, choices and mask read; counts, sums, tokens and loss written
            return dict(bytes=t * e * b + t * k * 4 + t + s * (8 * e + 8), flops=t * e * 8 + t * k)
        return dict(bytes=2 * t * e * b + t + s * (4 * e + 8), flops=t * e * 12)
    r, c, k, b = case["rows"], case["cols"], case["k"], SIZE[case["dtype"]]
    if op == "topk":  # logits read; values, indices and log-sum-exp written
        return dict(bytes=r * c * b + r * k * (b + 4) + r * 4, flops=r * c * 4)
    entries = r * k * (SIZE[case["teacher"]] + 4) + r * 16
    if op == "distill":
        return dict(bytes=r * c * b + entries + r * 12, flops=r * c * 4)
    return dict(bytes=2 * r * c * b + entries + r * 12, flops=r * c * 8)


# --------------------------------------------------------------------------------------------------------------
# inputs

def _logits(g, case, rows, cols, ld, teacher=False):
    """A student's logits in rows of `ld`, and a teacher's near them: a word's overall frequency, the context, and
    some words that stand out in it."""
    dev = dict(device="cuda", generator=g)
    z = torch.randn(rows, ld, **dev)
    z *= 1.5
    z += 2.0 * torch.randn(1, ld, **dev)
    hot = torch.randint(0, cols, (rows, min(8, cols)), **dev)
    z.scatter_add_(1, hot, 6.0 * torch.rand(rows, min(8, cols), **dev))
    other = None
    if teacher:
        other = (z + 0.7 * torch.randn(rows, ld, **dev)).to(DTYPES[case["dtype"]])[:, :cols]
    return z.to(DTYPES[case["dtype"]])[:, :cols], other


def _lse(z, scale):
    """log-sum-exp of each row in 64 bits, a block of rows at a time."""
    return torch.cat([torch.logsumexp(b.double() * scale, 1) for b in z.split(max(1, (1 << 25) // z.shape[1]))])


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    dev = dict(device="cuda", generator=g)
    new = lambda *shape, dtype=torch.float32: torch.empty(*shape, dtype=dtype, device="cuda")  # noqa: E731
    op, dt = case["op"], DTYPES[case["dtype"]]
    s = dict(case=case)
    if op.startswith("balance"):
        t, e, k, n = case["tokens"], case["experts"], case["k"], case["segments"]
        z = torch.randn(t, e, **dev) + 0.7 * torch.randn(1, e, **dev)
        idx = torch.topk(z, k, dim=1).indices.to(torch.int32)
        idx[torch.rand(t, k, **dev) < 0.02] = -1  # dropped for want of room
        s.update(z=z.to(dt), idx=idx, mask=(torch.rand(t, **dev) < 0.95).to(torch.uint8), alpha=0.01)
        cuts = torch.sort(torch.randint(0, t + 1, (n - 1,), **dev)).values
        ends = torch.tensor([0, t], device="cuda")
        s["offsets"] = torch.cat([ends[:1], cuts, ends[1:]]).to(torch.int32) if n > 1 else None
        if op == "balance":
            s.update(counts=new(n, e, dtype=torch.int32), psum=new(n, e), n_tok=new(n, dtype=torch.int32), loss=new(n))
        else:
            c, _, m, _ = _balance(s)
            up = 16.0 * t if case["dtype"] == "f16" else 1.0  # half floats are trained with a scaled loss
            s.update(counts=c, n_tok=m, dloss=up * (0.5 + torch.rand(n, **dev)), dz=torch.zeros(t, e, dtype=dt, device="cuda"))
        return s
    r, c, k = case["rows"], case["cols"], case["k"]
    z, t = _logits(g, case, r, c, case["ld"], teacher=op != "topk")
    s.update(z=z)
    if op == "topk":
        s.update(val=new(r, k, dtype=dt), idx=new(r, k, dtype=torch.int32), lse=new(r))
        return s
    top = torch.topk(t, k, dim=1)
    s.update(t_val=top.values.to(DTYPES[case["teacher"]]), t_idx=top.indices.to(torch.int32),
             t_lse=_lse(t, case["scale"]).float() if case["tail"] else None)
    short = torch.rand(r, 1, **dev) < 0.05  # rows with fewer entries than slots
    s["t_idx"] = torch.where(short & (torch.arange(k, device="cuda") >= (k + 1) // 2), -1, s["t_idx"]).to(torch.int32)
    up = 16384.0 if case["dtype"] == "f16" else 1.0  # half floats are trained with a scaled loss
    s["weight"] = torch.where(torch.rand(r, **dev) < 0.1, 0.0, up / r) * (0.5 + torch.rand(r, **dev))  # padding: 0
    if op == "distill_back":
        _, s["stats"] = _distill(s)
        s["dloss"] = 0.5 + torch.rand(r, **dev)
    else:
        s.update(loss=new(r), stats=new(r, 2))
    if op != "distill":
        s["dz"] = new(r, case["ld"], dtype=dt)[:, :c]
    return s


# --------------------------------------------------------------------------------------------------------------
# plain forms

def _topk(s):
    c = s["case"]
    z = s["z"].float()
    val, idx = torch.sort(z, dim=1, descending=True, stable=True)
    val, idx = val[:, :c["k"]], idx[:, :c["k"]].to(torch.int32)
    x = z * c["scale"]
    m = x.amax(1, keepdim=True)
    lse = m[:, 0] + torch.log(torch.exp(x - m).sum(1))
    return dict(val=val.to(s["z"].dtype), idx=torch.where(val == -math.inf, -1, idx), lse=lse)


def _teacher(s):
    """The entries' probabilities and their logarithms, the tail's, and which entries there are (64 bits: k a row)."""
    c = s["case"]
    there = s["t_idx"] >= 0
    t = torch.where(there, s["t_val"].double() * c["scale"], -math.inf)
    if s["t_lse"] is None:
        m = t.amax(1, keepdim=True)
        logq = t - (m + torch.log(torch.exp(t - m).sum(1, keepdim=True)))
    else:
        logq = t - s["t_lse"].double()[:, None]
    q = torch.exp(logq)
    rest = (1 - q.sum(1)).clamp(min=0) if s["t_lse"] is not None else torch.zeros_like(q[:, 0])
    return q, logq, rest, there


def _in_entries(s, there):
    r, c = s["z"].shape
    at = torch.where(there, s["t_idx"].long(), c)
    return torch.zeros(r, c + 1, dtype=torch.bool, device=at.device).scatter_(1, at, True)[:, :c]


def _sums(x):
    """log-sum-exp of each row: the sum in 32 bits, its logarithm and the maximum put together in 64."""
    m = x.amax(1, keepdim=True)
    return m[:, 0].double() + torch.log(torch.exp(x - m).sum(1).double())


def _distill(s):
    c = s["case"]
    x = s["z"].float() * c["scale"]
    q, logq, rest, there = _teacher(s)
    tail = _sums(x.masked_fill(_in_entries(s, there), -math.inf))
    at = torch.where(there, x.gather(1, s["t_idx"].long().clamp(min=0)).double(), -math.inf)
    lse = torch.logaddexp(tail, torch.logsumexp(at, 1))
    tail_p = -torch.log1p(torch.exp(at - tail[:, None]).sum(1))  # close to 0 where the entries hold little
    kl = torch.where(q > 0, q * (logq - at + lse[:, None]), 0.0).sum(1)
    kl = kl + torch.where(rest > 0, rest * (torch.log(rest.clamp(min=1e-300)) - tail_p), 0.0)
    on = s["weight"] != 0
    stats = torch.stack([lse, tail_p], 1)
    return torch.where(on, s["weight"] * kl, 0.0).float(), torch.where(on[:, None], stats, 0.0).float()


def _distill_back(s, stats, g):
    c = s["case"]
    x = s["z"].float() * c["scale"]
    q, _, rest, there = _teacher(s)
    whole = q.sum(1) + rest
    lse, tail_p = stats[:, 0].double(), stats[:, 1].double()
    d = torch.exp(x - stats[:, :1]) * (whole - torch.where(rest > 0, rest * torch.exp(-tail_p), 0.0)).float()[:, None]
    ii = torch.where(there, s["t_idx"].long(), 0)
    p_at = torch.exp(x.gather(1, ii).double() - lse[:, None])
    rows, slots = torch.nonzero(there, as_tuple=True)
    d[rows, ii[rows, slots]] = (p_at * whole[:, None] - q)[rows, slots].float()
    d *= (g * c["scale"])[:, None]
    return torch.where((g != 0)[:, None], d, 0.0).to(s["z"].dtype)


def _scores(z, score):
    if score == "softmax":
        e = torch.exp(z - z.amax(1, keepdim=True))
    else:
        e = 1 / (1 + torch.exp(-z))
    return e / e.sum(1, keepdim=True)


def _segment_of(s):
    t = s["z"].shape[0]
    if s["offsets"] is None:
        return torch.zeros(t, dtype=torch.long, device="cuda")
    return (torch.arange(t, device="cuda")[:, None] >= s["offsets"][None, 1:-1].long()).sum(1)


def _balance(s):
    c = s["case"]
    e, k, t = c["experts"], c["k"], c["tokens"]
    on = s["mask"] != 0
    ends = torch.tensor([0, t], device="cuda") if s["offsets"] is None else s["offsets"].long()

    def sums(x):  # of each segment's rows: long sums, in 64 bits
        run = torch.cumsum(x.double().t().contiguous(), 1)
        run = torch.cat([torch.zeros_like(run[:, :1]), run], 1)
        return (run[:, ends[1:]] - run[:, ends[:-1]]).t()

    psum = sums(torch.where(on[:, None], _scores(s["z"].float(), c["score"]), 0.0))
    n_tok = sums(on[:, None])[:, 0]
    took = torch.zeros(t, e + 1, device="cuda")
    took.scatter_add_(1, torch.where((s["idx"] >= 0) & on[:, None], s["idx"].long(), e),
                      torch.ones(1, 1, device="cuda").expand(t, k))
    counts = sums(took[:, :e])
    loss = s["alpha"] * e / k * (counts * psum).sum(1) / n_tok.clamp(min=1).square()
    return counts.to(torch.int32), psum.float(), n_tok.to(torch.int32), loss.float()


def _balance_back(s):
    c = s["case"]
    seg = _segment_of(s)
    z = s["z"].float()
    p = _scores(z, c["score"])
    f = s["counts"].float()[seg]
    d = p * (f - (p * f).sum(1, keepdim=True))
    if c["score"] == "sigmoid":
        d = d / (1 + torch.exp(z))
    n = s["n_tok"].double().clamp(min=1)
    g = (s["dloss"].double() * s["alpha"] * c["experts"] / c["k"] / n.square()).float()[seg]
    return torch.where((s["mask"] != 0)[:, None], d * g[:, None], 0.0).to(s["z"].dtype)


# --------------------------------------------------------------------------------------------------------------
# one pass

def _plain(s):
    op = s["case"]["op"]
    if op == "topk":
        return _topk(s)
    if op == "distill":
        loss, stats = _distill(s)
        return dict(loss=loss, stats=stats)
    if op == "distill_grad":
        loss, stats = _distill(s)
        return dict(loss=loss, stats=stats, dz=_distill_back(s, stats, s["weight"]))
    if op == "distill_back":
        return dict(dz=_distill_back(s, s["stats"], s["weight"] * s["dloss"]))
    if op == "balance":
        counts, psum, n_tok, loss = _balance(s)
        return dict(counts=counts, psum=psum, n_tok=n_tok, loss=loss)
    return dict(dz=_balance_back(s))


def _workspace(s, n_bytes):
    """The workspace that a program keeps for calls of one shape."""
    if "workspace" not in s:
        s["workspace"] = torch.empty(max(n_bytes, 1), dtype=torch.uint8, device="cuda")
    return s["workspace"]


def _own(s):
    import sparse_communication_adam_amd as sc
    c = s["case"]
    op = c["op"]
    if op == "topk":
        ws = _workspace(s, sc.scape_topk_rows_workspace_bytes(s["z"], c["k"]))
        sc.scape_topk_rows(s["z"], c["k"], s["val"], s["idx"], s["lse"], scale=c["scale"], workspace=ws)
        return dict(val=s["val"], idx=s["idx"], lse=s["lse"])
    if op in ("distill", "distill_grad"):
        dz = s.get("dz")
        ws = _workspace(s, sc.scape_distill_workspace_bytes(s["z"], c["k"], grad=dz is not None))
        sc.scape_distill_forward(s["z"], s["t_val"], s["t_idx"], s["loss"], s["stats"], t_lse=s["t_lse"],
                                 scale=c["scale"], weight=s["weight"], dz=dz, workspace=ws)
        out = dict(loss=s["loss"], stats=s["stats"])
        return out if dz is None else dict(out, dz=dz)
    if op == "distill_back":
        sc.scape_distill_backward(s["z"], s["t_val"], s["t_idx"], s["stats"], s["dz"], t_lse=s["t_lse"],
                                  scale=c["scale"], weight=s["weight"], dloss=s["dloss"])
        return dict(dz=s["dz"])
    if op == "balance":
        ws = _workspace(s, sc.scape_balance_workspace_bytes(s["z"], c["segments"]))
        sc.scape_balance_forward(s["z"], s["idx"], s["counts"], s["psum"], s["n_tok"], s["loss"], alpha=s["alpha"],
                                 offsets=s["offsets"], mask=s["mask"], score=c["score"], workspace=ws)
        return dict(counts=s["counts"], psum=s["psum"], n_tok=s["n_tok"], loss=s["loss"])
    if not s["counts"].is_contiguous():
        s["counts"] = s["counts"].contiguous()  # as the forward call writes them
    sc.scape_balance_backward(s["z"], s["counts"], s["n_tok"], s["dloss"], s["dz"], k=c["k"], alpha=s["alpha"],
                              offsets=s["offsets"], mask=s["mask"], score=c["score"])
    return dict(dz=s["dz"])


def run(state):
    return _own(state) if own else _plain(state)


# --------------------------------------------------------------------------------------------------------------
# the definitions in 64 bits

def _exact_rows(s, a, b):
    """Rows a..b of a distillation: the distributions, the log-sum-exp, the tail's log-probability and the loss."""
    c = s["case"]
    x = s["z"][a:b].double() * c["scale"]
    n, v = x.shape
    idx = s["t_idx"][a:b].long()
    there = idx >= 0
    # the teacher's distribution over v words and one more place for the tail
    t = s["t_val"][a:b].double() * c["scale"]
    if s["t_lse"] is None:
        q = torch.softmax(t.masked_fill(~there, -math.inf), 1)
    else:
        q = torch.exp(t - s["t_lse"][a:b, None].double()) * there
    full = torch.zeros(n, v + 1, dtype=torch.float64, device=x.device)
    full.scatter_add_(1, torch.where(there, idx, v), torch.where(there, q, 0.0))
    known = torch.zeros(n, v + 1, device=x.device, dtype=torch.bool).scatter_(1, torch.where(there, idx, v), True)[:, :v]
    full[:, v] = (1 - full[:, :v].sum(1)).clamp(min=0) if s["t_lse"] is not None else 0
    lse = torch.logsumexp(x, 1)
    tail = torch.logsumexp(x.masked_fill(known, -math.inf), 1)
    logp = torch.cat([torch.log_softmax(x, 1), (tail - lse)[:, None]], 1)
    kl = (torch.special.xlogy(full, full) - torch.where(full > 0, full * logp, 0.0)).sum(1)
    return x, full, known, lse, tail - lse, kl


def _exact_gradient(s, x, full, known, lse, tail_p, g):
    p = torch.exp(x - lse[:, None])
    share = torch.exp(x - (lse + tail_p)[:, None]).masked_fill(known, 0.0) * full[:, -1:]  # the tail's mass, spread as the student has it
    return (p * full.sum(1, keepdim=True) - full[:, :-1] - share) * (g * s["case"]["scale"])[:, None]


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "topk":
        z, k, c = s["z"], case["k"], case["cols"]
        vals, idxs = [], []
        step = max(1, (1 << 26) // c)
        down = torch.arange(c - 1, -1, -1, device="cuda")
        for a in range(0, case["rows"], step):
            bits = (z[a:a + step].float() + 0.0).view(torch.int32).long()
            key = torch.where(bits < 0, -(bits & 0x7FFFFFFF), bits) * (1 << 20) + down  # value, then the lower index
            at = torch.topk(key, k, dim=1).indices
            v = z[a:a + step].double().gather(1, at)
            vals.append(v)
            idxs.append(torch.where(v == -math.inf, -1, at))
        return dict(val=torch.cat(vals), idx=torch.cat(idxs).to(torch.int32), lse=_lse(z, case["scale"]))
    if op.startswith("distill"):
        w = s["weight"].double()
        loss, stats, dz = [], [], []
        step = max(1, (1 << 25) // case["cols"])
        for a in range(0, case["rows"], step):
            b = min(a + step, case["rows"])
            x, full, known, lse, tail_p, kl = _exact_rows(s, a, b)
            on = w[a:b] != 0
            if op != "distill_back":
                loss.append(torch.where(on, w[a:b] * kl, 0.0))
                stats.append(torch.where(on[:, None], torch.stack([lse, tail_p], 1), 0.0))
            if op != "distill":
                g = w[a:b]
                if op == "distill_back":  # from the statistics that it is given
                    g = g * s["dloss"][a:b].double()
                    lse, tail_p = s["stats"][a:b, 0].double(), s["stats"][a:b, 1].double()
                d = _exact_gradient(s, x, full, known, lse, tail_p, g)
                dz.append(torch.where((g != 0)[:, None], d, 0.0))
        out = {} if op == "distill_back" else dict(loss=torch.cat(loss), stats=torch.cat(stats))
        return out if op == "distill" else dict(out, dz=torch.cat(dz))
    z = s["z"].double()
    t, e = z.shape
    n, k = case["segments"], case["k"]
    if case["score"] == "softmax":
        p = torch.softmax(z, 1)
        slope = torch.ones_like(p)
    else:
        a = torch.sigmoid(z)
        p, slope = a / a.sum(1, keepdim=True), 1 - a
    edges = [0, t] if s["offsets"] is None else s["offsets"].tolist()
    on = s["mask"].bool()
    if op == "balance":
        counts, psum, n_tok, loss = [], [], [], []
        for a, b in zip(edges[:-1], edges[1:]):
            chosen = s["idx"][a:b][on[a:b]].flatten().long()
            counts.append(torch.bincount(chosen[chosen >= 0], minlength=e))
            psum.append(p[a:b][on[a:b]].sum(0))
            n_tok.append(on[a:b].sum())
            m = max(int(n_tok[-1]), 1)
            loss.append(s["alpha"] * ((counts[-1] * e / (k * m)) * (psum[-1] / m)).sum())
        return dict(counts=torch.stack(counts).to(torch.int32), psum=torch.stack(psum),
                    n_tok=torch.stack(n_tok).to(torch.int32), loss=torch.stack(loss))
    dz = torch.zeros_like(z)
    for i, (a, b) in enumerate(zip(edges[:-1], edges[1:])):
        f = s["counts"][i].double() * e / k
        m = max(int(s["n_tok"][i]), 1)
        up = s["dloss"][i].double() * s["alpha"] * f / m ** 2
        d = p[a:b] * slope[a:b] * (up - (p[a:b] * up).sum(1, keepdim=True))
        dz[a:b] = torch.where(on[a:b, None], d, 0.0)
    return dict(dz=dz)
