"""Measured cases of the operators between a model's last hidden states and the optimizer step, each in a plain form
and through the framework's calls.

A case's "op" says which path it is:
  loss          softmax cross entropy over a vocabulary, from hidden states and the head's weights (evaluation, or a
                forward pass whose backward pass comes later)
  grad          its gradients to the hidden states and to the head's weights
  clip          the gradient norms of a step's workers, of each of their layers, and the gradients clipped by them
  dispatch      a router's choices sorted by expert, and the tokens laid out in that order
  combine       the experts' outputs back in the tokens' order, weighted and summed
  combine_back  the gradients of that sum to the experts' outputs and to the weights
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
SIZE = {"bf16": 2, "f16": 2, "f32": 4}


# --------------------------------------------------------------------------------------------------------------
# cases

def _gpt_layers(n, h, f, v, pos):
    block = [h, h, 3 * h * h, 3 * h, h * h, h, h, h, f * h, f, h * f, h]
    return [v * h, pos * h] + block * n + [h, h]


def _llama_layers(n, h, ffn, v):
    return [v * h] + [h, 3 * h * h, h * h, h, 2 * ffn * h, h * ffn] * n + [h, v * h]


#: The parameter tensors of the repository's workloads, and two small sets.
MODELS = {
    "single": [1024 * 1024],
    "gpt-345m": _gpt_layers(24, 1024, 4096, 50304, 1024),
    "llama-0.55b": _llama_layers(16, 1536, 4096, 32000),
    "small": _llama_layers(2, 384, 1024, 1000),
    "ragged": [1000, 37, 1, 64, 4097, 33 * 65, 70000],
}


def listed():
    return [
        # a handful of tokens: the smallest evaluation of the loss
        dict(name="loss 7x50304x1024", op="loss", dtype="bf16", rows=7, cols=50304, dim=1024, scale=1.0),
        # evaluation over two sequences of 1024 tokens, odd vocabulary, softened logits
        dict(name="loss 2048x50257x1024", op="loss", dtype="f16", rows=2048, cols=50257, dim=1024, scale=0.5),
        # the backward pass of a short ragged batch
        dict(name="grad 333x50257x1536", op="grad", dtype="f16", rows=333, cols=50257, dim=1536, scale=1.0),
        # the backward pass of one micro-batch of 8 sequences of 1024 tokens under the 1.75B model's head
        dict(name="grad 8192x32000x2048", op="grad", dtype="bf16", rows=8192, cols=32000, dim=2048, scale=1.0),
        # two workers' gradients of the 345M model
        dict(name="clip gpt-345m", op="clip", model="gpt-345m", workers=2, interleaved=False, shared=False),
        # one layer, where launches count, in the interleaved layout
        dict(name="clip single", op="clip", model="single", workers=4, interleaved=True, shared=True),
        # a batch's tokens to 8 of 64 experts
        dict(name="dispatch 16384x2048", op="dispatch", dtype="bf16", tokens=16384, dim=2048, experts=64, k=8),
        # one token as it is generated
        dict(name="dispatch 1x2048", op="dispatch", dtype="bf16", tokens=1, dim=2048, experts=64, k=6),
        # the way back of such a batch
        dict(name="combine 16384x2048", op="combine", dtype="bf16", tokens=16384, dim=2048, experts=64, k=8),
        # a short batch whose rows are not a whole number of 16-byte pieces
        dict(name="combine 1000x1001", op="combine", dtype="f32", tokens=1000, dim=1001, experts=8, k=2),
        # gradients of the way back
        dict(name="combine_back 8192x4096", op="combine_back", dtype="bf16", tokens=8192, dim=4096, experts=256, k=8),
        # the same of a short batch
        dict(name="combine_back 2000x1536", op="combine_back", dtype="f16", tokens=2000, dim=1536, experts=60, k=4),
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["loss", "loss", "grad", "grad", "clip", "dispatch", "combine", "combine_back"])
    if op in ("loss", "grad"):
        cols = rng.choice([32000, 50257, 50304, _spread(rng, 1000, 131072)])
        dim = 8 * _spread(rng, 32, 512)
        most = 8192 * 32000 * 2048 // (cols * dim)
        return dict(op=op, dtype=rng.choice(["bf16", "bf16", "f16"]), rows=_spread(rng, 1, max(1, min(8192, most))),
                    cols=cols, dim=dim, scale=rng.choice([1.0, 1.0, 0.5]))
    if op == "clip":
        model = rng.choice(["single", "small", "ragged", "llama-0.55b"])
        most = 1 if model == "llama-0.55b" else 8
        return dict(op=op, model=model, workers=rng.randint(1, most), interleaved=rng.random() < 0.5,
                    shared=rng.random() < 0.5)
    k = rng.randint(1, 8)
    dim = rng.choice([8, 8, 1]) * _spread(rng, 16, 512)
    tokens = _spread(rng, 1, min(16384, (1 << 28) // (dim * k)))
    return dict(op=op, dtype=rng.choice(["bf16", "bf16", "f16", "f32"]), tokens=tokens, dim=dim,
                experts=max(k, _spread(rng, 4, 512)), k=k)


def work(case):
    op = case["op"]
    if op in ("loss", "grad"):
        n, v, d, b = case["rows"], case["cols"], case["dim"], SIZE[case["dtype"]]
        if op == "loss":  # hidden states and weights read; loss and log-sum-exp written
            return dict(bytes=(n + v) * d * b + n * 16, flops=2 * n * v * d)
        return dict(bytes=2 * (n + v) * d * b + n * 16, flops=6 * n * v * d)
    if op == "clip":
        n = sum(MODELS[case["model"]]) * case["workers"]
        return dict(bytes=4 * n, flops=4 * n)
    t, d, k, b = case["tokens"], case["dim"], case["k"], SIZE[case["dtype"]]
    if op == "dispatch":
        return dict(bytes=(1 + k) * t * d * b + 8 * t * k + 4 * case["experts"], flops=t * k)
    if op == "combine":
        return dict(bytes=(1 + k) * t * d * b + 8 * t * k, flops=2 * t * k * d)
    return dict(bytes=(1 + 2 * k) * t * d * b + 12 * t * k, flops=3 * t * k * d)


# --------------------------------------------------------------------------------------------------------------
# inputs

def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    dev = dict(device="cuda", generator=g)
    new = lambda *shape, dtype=torch.float32: torch.empty(*shape, dtype=dtype, device="cuda")  # noqa: E731
    op = case["op"]
    s = dict(case=case)
    if op in ("loss", "grad"):
        n, v, d, dt = case["rows"], case["cols"], case["dim"], DTYPES[case["dtype"]]
        w = torch.randn(v, d, **dev) * (0.9 / case["scale"] / math.sqrt(d))
        label = torch.randint(0, v, (n,), **dev)
        h = torch.randn(n, d, **dev)  # as a norm leaves them; the label's word stands out by 0 to 12
        h += w[label] * (12.0 / case["scale"] * torch.rand(n, 1, **dev) / w[label].square().sum(1, keepdim=True))
        label = torch.where(torch.rand(n, **dev) < 0.05, -100, label).to(torch.int32)  # prompts and padding
        up = 16384.0 if case["dtype"] == "f16" else 1.0  # half floats are trained with a scaled loss
        s.update(h=h.to(dt), w=w.to(dt), label=label, weight=(0.5 + torch.rand(n, **dev)) / n)
        if op == "loss":
            s.update(loss=new(n), lse=new(n))
        else:
            s["lse"] = _loss(s)[1]
            s.update(dloss=up * (0.5 + torch.rand(n, **dev)), dh=new(n, d, dtype=dt), dw=new(v, d, dtype=dt))
        return s
    if op == "clip":
        sizes, w = MODELS[case["model"]], case["workers"]
        padded = [(n + 63) // 64 * 64 for n in sizes]
        n_pad = sum(padded)
        flat = torch.zeros(w, n_pad, dtype=torch.bfloat16, device="cuda")  # 0 in the padding between layers
        sigma = torch.exp(torch.empty(len(sizes), **{"device": "cuda"}).uniform_(math.log(1e-5), math.log(1e-2), generator=g)).tolist()
        starts = [0]
        for p in padded:
            starts.append(starts[-1] + p)
        for a, n, x in zip(starts, sizes, sigma):
            flat[:, a:a + n] = x * torch.randn(w, n, **dev)
        s.update(starts=starts[:-1], sizes=sizes, n_pad=n_pad, norm=new(w + 1), layer_norm=new(w, len(sizes)))
        # clipped by a half or so; of a step's workers some are below the bound
        whole = torch.linalg.vector_norm(flat.float() if n_pad < 1 << 24 else flat, dim=1, dtype=torch.float32)
        s["max_norm"] = float(whole.mean()) * (0.4 + 0.3 * float(torch.rand(1, **dev)))
        if case["interleaved"]:
            s["g"] = flat.view(w, n_pad // 64, 64).transpose(0, 1).contiguous().view(-1)
            s["out"] = torch.zeros_like(s["g"])
        else:
            s["g"] = list(flat.unbind(0))
            s["out"] = list(torch.zeros_like(flat).unbind(0))
        return s
    t, d, k, e, dt = case["tokens"], case["dim"], case["k"], case["experts"], DTYPES[case["dtype"]]
    z = torch.randn(t, e, **dev) + 0.7 * torch.randn(1, e, **dev)  # some experts are chosen more often
    top = torch.topk(z, k, dim=1)
    idx = top.indices.to(torch.int32)
    idx[torch.rand(t, k, **dev) < 0.02] = -1  # dropped for want of room
    s.update(idx=idx, row=new(t, k, dtype=torch.int32), offsets=new(e + 1, dtype=torch.int32))
    if op == "dispatch":
        s.update(x=torch.randn(t, d, **dev).to(dt), y=torch.zeros(t * k, d, dtype=dt, device="cuda"))
        return s
    _, s["row"] = _sort(s)
    s.update(y=torch.randn(t * k, d, **dev).to(dt), weight=torch.softmax(top.values, 1), out=new(t, d, dtype=dt))
    if op == "combine_back":
        s.update(dout=torch.randn(t, d, **dev).to(dt), dy=torch.zeros(t * k, d, dtype=dt, device="cuda"),
                 dweight=new(t, k))
    return s


# --------------------------------------------------------------------------------------------------------------
# plain forms

def _logits(s):
    return (s["h"].float() @ s["w"].float().t()) * s["case"]["scale"]


def _counts_rows(s):
    """The rows whose label is a word, and a column to read in each row."""
    on = (s["label"] >= 0) & (s["label"] < s["case"]["cols"])
    return on, torch.where(on, s["label"], 0).long()


def _loss(s):
    z = _logits(s)
    on, at = _counts_rows(s)
    m = z.amax(1)
    lse = m + torch.log(torch.exp(z - m[:, None]).sum(1))
    loss = s["weight"] * (lse - z.gather(1, at[:, None])[:, 0])
    return torch.where(on, loss, 0.0), lse


def _grad(s):
    on, at = _counts_rows(s)
    p = torch.exp(_logits(s) - s["lse"][:, None])
    p.scatter_add_(1, at[:, None], torch.full_like(p[:, :1], -1.0))
    p *= torch.where(on, s["weight"] * s["dloss"] * s["case"]["scale"], 0.0)[:, None]
    return (p @ s["w"].float()).to(s["h"].dtype), (p.t() @ s["h"].float()).to(s["w"].dtype)


def _flat(s):
    """The workers' gradients as rows."""
    if s["case"]["interleaved"]:
        return s["g"].view(-1, s["case"]["workers"], 64).transpose(0, 1).reshape(s["case"]["workers"], -1)
    return torch.stack(s["g"])


def _clip(s):
    w = s["case"]["workers"]
    flat = _flat(s)
    squares = torch.stack([flat[:, a:a + n].double().square().sum(1) for a, n in zip(s["starts"], s["sizes"])], 1)
    whole = squares.sum(1)
    norm = torch.cat([whole, whole.mean()[None]]).sqrt()
    by = norm[w:].expand(w) if s["case"]["shared"] else norm[:w]
    f = torch.where(by > s["max_norm"], s["max_norm"] / by, 1.0).float()
    out = (flat.float() * f[:, None]).to(torch.bfloat16)
    if s["case"]["interleaved"]:
        out = out.view(w, -1, 64).transpose(0, 1).reshape(-1)
    else:
        out = list(out.unbind(0))
    return dict(norm=norm.float(), layer_norm=squares.sqrt().float(), out=out)


def _sort(s):
    c = s["case"]
    e = s["idx"].flatten().long()
    e = torch.where((e >= 0) & (e < c["experts"]), e, c["experts"])  # no choice: behind all
    at = torch.argsort(e, stable=True)
    row = torch.empty_like(at).scatter_(0, at, torch.arange(e.numel(), device="cuda"))
    row = torch.where(e < c["experts"], row, -1)
    counts = torch.zeros(c["experts"] + 1, dtype=torch.long, device="cuda").scatter_add_(0, e, torch.ones_like(e))
    offsets = torch.cat([torch.zeros_like(counts[:1]), torch.cumsum(counts[:-1], 0)])
    return offsets.to(torch.int32), row.view(c["tokens"], c["k"]).to(torch.int32)


def _dispatch(s):
    c = s["case"]
    offsets, row = _sort(s)
    y = torch.zeros(c["tokens"] * c["k"] + 1, c["dim"], dtype=s["x"].dtype, device="cuda")
    y[torch.where(row >= 0, row, c["tokens"] * c["k"]).long()] = s["x"][:, None].expand(-1, c["k"], -1)
    return dict(offsets=offsets, row=row, y=y[:-1])


def _picked(s):
    """Each token's k rows of y in 32 bits, and which there are."""
    there = s["row"] >= 0
    return s["y"][torch.where(there, s["row"], 0).long()].float(), there


def _combine(s):
    y, there = _picked(s)
    weight = torch.where(there, s["weight"], 0.0)
    return dict(out=torch.where((weight != 0)[:, :, None], weight[:, :, None] * y, 0.0).sum(1).to(s["y"].dtype))


def _combine_back(s):
    y, there = _picked(s)
    dout = s["dout"].float()[:, None]
    dweight = torch.where(there, (y * dout).sum(2), 0.0)
    dy = torch.zeros(s["y"].shape[0] + 1, s["y"].shape[1], dtype=s["y"].dtype, device="cuda")
    dy[torch.where(there, s["row"], s["y"].shape[0]).long()] = (s["weight"][:, :, None] * dout).to(dy.dtype)
    return dict(dy=dy[:-1], dweight=dweight)


# --------------------------------------------------------------------------------------------------------------
# one pass

def _plain(s):
    op = s["case"]["op"]
    if op == "loss":
        return dict(zip(("loss", "lse"), _loss(s)))
    if op == "grad":
        return dict(zip(("dh", "dw"), _grad(s)))
    return dict(clip=_clip, dispatch=_dispatch, combine=_combine, combine_back=_combine_back)[op](s)


def _workspace(s, query):
    """The workspace that a program keeps for calls of one shape."""
    if "workspace" not in s:
        s["workspace"] = torch.empty(max(query(), 1), dtype=torch.uint8, device="cuda")
    return s["workspace"]


def _context(s, sc):
    """The optimizer's context, which a program makes once for its parameters."""
    c = s["case"]
    key = (c["model"], c["workers"])
    if key not in _CONTEXTS:
        _CONTEXTS.clear()
        _CONTEXTS[key] = sc.Context(sc.ScapeConfig(layer_numel=s["sizes"], workers=c["workers"], keep_num=1, keep_den=100))
    return _CONTEXTS[key]


_CONTEXTS = {}


def _own(s):
    import sparse_communication_adam_amd as sc
    c = s["case"]
    op = c["op"]
    if op == "loss":
        ws = _workspace(s, lambda: sc.scape_vocab_loss_workspace_bytes(s["h"], s["w"], grad=False))
        sc.scape_vocab_loss_forward(s["h"], s["w"], s["label"], s["loss"], s["lse"], scale=c["scale"], weight=s["weight"],
                                    workspace=ws)
        return dict(loss=s["loss"], lse=s["lse"])
    if op == "grad":
        ws = _workspace(s, lambda: sc.scape_vocab_loss_workspace_bytes(s["h"], s["w"], grad=True))
        sc.scape_vocab_loss_backward(s["h"], s["w"], s["label"], s["lse"], s["dh"], s["dw"], scale=c["scale"],
                                     weight=s["weight"], dloss=s["dloss"], workspace=ws)
        return dict(dh=s["dh"], dw=s["dw"])
    if op == "clip":
        ctx = _context(s, sc)
        ws = _workspace(s, lambda: sc.scape_grad_norm_workspace_bytes(ctx))
        norm, clip = sc.scape_grad_norm, sc.scape_grad_clip
        if c["interleaved"]:
            norm, clip = sc.scape_grad_norm_interleaved, sc.scape_grad_clip_interleaved
        norm(ctx, s["g"], s["norm"], s["layer_norm"], workspace=ws)
        clip(ctx, s["g"], s["norm"], s["max_norm"], out=s["out"], shared=c["shared"])
        return dict(norm=s["norm"], layer_norm=s["layer_norm"], out=s["out"])
    if op == "dispatch":
        ws = _workspace(s, lambda: sc.scape_expert_sort_workspace_bytes(s["idx"], c["experts"]))
        sc.scape_expert_sort(s["idx"], c["experts"], s["offsets"], s["row"], workspace=ws)
        sc.scape_expert_gather(s["x"], s["row"], s["y"])
        return dict(offsets=s["offsets"], row=s["row"], y=s["y"])
    if op == "combine":
        sc.scape_expert_combine(s["y"], s["row"], s["out"], weight=s["weight"])
        return dict(out=s["out"])
    sc.scape_expert_combine_backward(s["y"], s["row"], s["dout"], s["dy"], weight=s["weight"], dweight=s["dweight"])
    return dict(dy=s["dy"], dweight=s["dweight"])


def run(state):
    return _own(state) if own else _plain(state)


# --------------------------------------------------------------------------------------------------------------
# the definitions in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op in ("loss", "grad"):
        h, w = s["h"].double(), s["w"].double()
        valid = s["label"] >= 0
        label = s["label"].long().clamp(min=0)
        weight = s["weight"].double() * valid
        loss, lse, dh, dw = [], [], [], torch.zeros_like(w)
        step = max(1, (1 << 27) // case["cols"])
        for a in range(0, case["rows"], step):
            hb, lb, wb = h[a:a + step], label[a:a + step], weight[a:a + step]
            z = torch.matmul(hb, w.t()).mul_(case["scale"])
            if op == "loss":
                lse.append(torch.logsumexp(z, 1))
                loss.append(wb * torch.nn.functional.cross_entropy(z, lb, reduction="none"))
                continue
            z.sub_(s["lse"][a:a + step, None].double()).exp_()  # from the log-sum-exp that it is given
            z[torch.arange(len(lb), device=z.device), lb] -= 1
            z.mul_((wb * s["dloss"][a:a + step].double() * case["scale"])[:, None])
            dh.append(torch.matmul(z, w))
            dw += torch.matmul(z.t(), hb)
        return dict(loss=torch.cat(loss), lse=torch.cat(lse)) if op == "loss" else dict(dh=torch.cat(dh), dw=dw)
    if op == "clip":
        w, il = case["workers"], case["interleaved"]
        g = s["g"].view(-1, w, 64).double() if il else [x.double() for x in s["g"]]
        worker = (lambda i: g[:, i].reshape(-1)) if il else (lambda i: g[i])
        layer = torch.stack([torch.stack([torch.linalg.vector_norm(worker(i)[a:a + n])
                                          for a, n in zip(s["starts"], s["sizes"])]) for i in range(w)])
        norm = torch.linalg.vector_norm(layer, dim=1)
        both = torch.cat([norm, (norm.square().sum() / w).sqrt()[None]])
        by = [float(both[w]) if case["shared"] else float(x) for x in norm]
        f = [min(1.0, s["max_norm"] / x) for x in by]
        if il:
            out = (g * torch.tensor(f, dtype=torch.float64, device="cuda")[None, :, None]).view(-1)
        else:
            out = [x * y for x, y in zip(g, f)]
        return dict(norm=both, layer_norm=layer, out=out)
    idx, k = s["idx"].flatten().tolist(), case["k"]
    if op == "dispatch":
        places = [[] for _ in range(case["experts"])]
        for i, e in enumerate(idx):
            if e >= 0:
                places[e].append(i)
        row, offsets, order = [-1] * len(idx), [0], []
        for p in places:
            for i in p:
                row[i] = len(order)
                order.append(i)
            offsets.append(len(order))
        y = torch.zeros_like(s["y"], dtype=torch.float64)
        y[:len(order)] = s["x"].double()[torch.tensor([i // k for i in order], dtype=torch.long, device="cuda")]
        return dict(offsets=torch.tensor(offsets, dtype=torch.int32, device="cuda"),
                    row=torch.tensor(row, dtype=torch.int32, device="cuda").view(-1, k), y=y)
    y, weight, row = s["y"].double(), s["weight"].double(), s["row"].long()
    if op == "combine":
        out = torch.zeros(case["tokens"], case["dim"], dtype=torch.float64, device="cuda")
        for j in range(k):
            t = torch.nonzero(row[:, j] >= 0)[:, 0]
            out[t] += weight[t, j, None] * y[row[t, j]]
        return dict(out=out)
    dout = s["dout"].double()
    dy, dweight = torch.zeros_like(y), torch.zeros_like(weight)
    for j in range(k):
        t = torch.nonzero(row[:, j] >= 0)[:, 0]
        dy[row[t, j]] = weight[t, j, None] * dout[t]
        dweight[t, j] = torch.linalg.vecdot(y[row[t, j]], dout[t])
    return dict(dy=dy, dweight=dweight)
