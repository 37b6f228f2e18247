"""Outputs of the vocabulary loss and the expert moves that lie over an input,
over one another or over the workspace are refused; rows of one between rows of
another, and what the header allows, are not."""
import ctypes
import os
import random

import pytest
import torch

P = ctypes.c_void_p
NAMES = ["head", "h", "w", "label", "weight", "loss", "lse", "dloss", "dh", "dw", "ws", "idx", "offsets", "row", "x", "y", "out",
         "dout", "dy", "dweight"]
AT = {n: (i + 1) << 40 for i, n in enumerate(NAMES)}  # far apart; nothing here is launched


@pytest.fixture(scope="module")
def sc():
    import sparse_communication_adam_amd as sc
    if not os.path.exists(sc.LIB_PATH):
        sc.build()
    return sc


def _call(sc, fn, at):
    """The call with its pointers where `at` says; every case below overlaps, so none is launched."""
    from sparse_communication_adam_amd._scape import _Head
    a = dict(AT)
    a.update(at)
    p = {n: P(v) for n, v in a.items()}
    lib = sc.lib()
    head = ctypes.byref(_Head(a["h"], 96, a["w"], 64, 1, 10, 100, 64, a["label"], a["weight"], 1.0))
    if fn == "forward":
        rc = lib.scape_vocab_loss_forward(head, p["loss"], p["lse"], p["ws"], 1 << 30, None)
    elif fn == "backward":
        rc = lib.scape_vocab_loss_backward(head, p["lse"], p["dloss"], p["dh"], 96, p["dw"], 64, p["ws"], 1 << 30, None)
    elif fn == "sort":
        rc = lib.scape_expert_sort(p["idx"], 5000, 2, 8, p["offsets"], p["row"], p["ws"], 1 << 20, None)
    elif fn == "gather":
        rc = lib.scape_expert_gather(p["x"], 1, 10, 64, 64, p["row"], 2, p["y"], 20, 96, None)
    elif fn == "combine":
        rc = lib.scape_expert_combine(p["y"], 1, 20, 64, 96, p["row"], p["weight"], 10, 2, p["out"], 64, None)
    else:
        rc = lib.scape_expert_combine_backward(p["y"], 1, 20, 64, 96, p["row"], p["weight"], p["dout"], 64, 10, 2, p["dy"], 96,
                                               p["dweight"], None)
    return rc, sc.scape_last_error()


H_END, W_END = AT["h"] + (9 * 96 + 64) * 2, AT["w"] + 100 * 128   # first bytes behind h and w
CASES = (
    [("forward", c) for c in [
        dict(lse=AT["loss"]), dict(lse=AT["loss"] + 36), dict(lse=AT["loss"] - 36), dict(loss=AT["label"]), dict(lse=AT["label"]),
        dict(loss=AT["weight"] + 4), dict(lse=AT["weight"]), dict(loss=H_END - 4), dict(lse=W_END - 4), dict(loss=AT["ws"]),
        dict(ws=AT["h"]), dict(ws=AT["weight"] + 32), dict(ws=W_END - 16), dict(lse=AT["ws"] + 16)]]
    + [("backward", c) for c in [
        dict(dh=AT["h"]), dict(dh=AT["h"] + 192), dict(dh=AT["h"] - 192 * 9), dict(dh=AT["h"] + 16), dict(dh=AT["h"] + 80),
        dict(dh=AT["w"]), dict(dw=AT["w"]), dict(dw=AT["w"] + 99 * 128), dict(dw=AT["w"] - 99 * 128), dict(dw=AT["h"]),
        dict(dw=AT["dh"]), dict(dh=W_END - 16), dict(dh=AT["dw"] - 192 * 9 - 112), dict(dh=AT["label"]), dict(dw=AT["weight"]),
        dict(dh=AT["lse"]), dict(dw=AT["dloss"] - 99 * 128), dict(ws=AT["h"]), dict(ws=AT["dh"]), dict(ws=AT["dw"] + 128),
        dict(ws=AT["lse"]), dict(ws=H_END - 16)]]
    + [("sort", c) for c in [
        dict(row=AT["idx"] + 4), dict(row=AT["idx"] - 4), dict(offsets=AT["idx"]), dict(offsets=AT["row"] + 39996), dict(ws=AT["idx"]),
        dict(ws=AT["row"]), dict(offsets=AT["ws"])]]
    + [("gather", c) for c in [dict(y=AT["x"]), dict(y=AT["x"] + 1278), dict(y=AT["x"] - 19 * 192 - 126), dict(y=AT["row"])]]
    + [("combine", c) for c in [dict(out=AT["y"]), dict(out=AT["y"] + 19 * 192 + 126), dict(out=AT["row"]), dict(out=AT["weight"] + 76)]]
    + [("backward of combine", c) for c in [
        dict(dy=AT["y"] + 2), dict(dy=AT["y"] + 192), dict(dy=AT["y"] + 66), dict(dy=AT["dout"]), dict(dy=AT["row"]),
        dict(dy=AT["weight"]), dict(dweight=AT["weight"]), dict(dweight=AT["row"]), dict(dweight=AT["y"]), dict(dweight=AT["dout"]),
        dict(dweight=AT["dy"] + 19 * 192 + 124)]])


@pytest.mark.parametrize("fn,at", CASES, ids=[f"{f}-{'-'.join(c)}-{i}" for i, (f, c) in enumerate(CASES)])
def test_overlaps_are_refused(sc, fn, at):
    code, text = _call(sc, fn, at)
    assert code == -1 and " overlaps " in text


@pytest.fixture
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return torch.device("cuda")


@pytest.mark.gpu
def test_any_two_places_in_one_buffer(sc, gpu):
    """The gather of x into y somewhere in one buffer: right where no element is shared, refused where one is."""
    rng = random.Random(7)
    size, seen = 6000, [0, 0]
    for trial in range(400):
        n, k, dim = rng.randint(1, 12), rng.randint(1, 3), rng.randint(1, 40)
        m = n * k + rng.randint(0, 2)
        ld_x = dim + rng.choice([0, 0, 3, 41, 90])
        ld_y = ld_x if rng.random() < 0.6 and ld_x >= dim else dim + rng.randint(0, 90)
        x0, y0 = rng.randint(0, 400), rng.randint(0, 400)
        buf = torch.randn(size, device=gpu).to(torch.bfloat16)
        x = buf.as_strided((n, dim), (ld_x, 1), x0)
        y = buf.as_strided((m, dim), (ld_y, 1), y0)
        taken = torch.zeros(size, dtype=torch.int32)
        taken.as_strided((n, dim), (ld_x, 1), x0).fill_(1)
        over = bool(taken.as_strided((m, dim), (ld_y, 1), y0).any())
        row = torch.randperm(m, device=gpu)[:n * k].to(torch.int32).view(n, k)
        seen[over] += 1
        if over:
            with pytest.raises(sc.ScapeError, match="y overlaps x"):
                sc.scape_expert_gather(x, row, y)
            continue
        want = buf.clone()
        w = want.as_strided((m, dim), (ld_y, 1), y0)
        w[row.long().reshape(-1)] = x.repeat_interleave(k, 0)
        sc.scape_expert_gather(x, row, y)
        assert torch.equal(buf, want), trial
    assert min(seen) > 40


@pytest.mark.gpu
def test_hidden_states_and_gradients_beside_each_other(sc, gpu):
    """dh in the other half of h's rows, dw in the other half of w's."""
    for rows in (5, 140, 300):
        g = torch.Generator(device=gpu).manual_seed(rows)
        both_h = torch.randn(rows, 128, device=gpu, generator=g).to(torch.bfloat16)
        both_w = (torch.randn(500, 128, device=gpu, generator=g) / 8).to(torch.bfloat16)
        h, dh, w, dw = both_h[:, :64], both_h[:, 64:], both_w[:, 64:], both_w[:, :64]
        label = torch.randint(0, 500, (rows,), device=gpu, generator=g).to(torch.int32)
        weight = torch.rand(rows, device=gpu, generator=g)
        n = max(sc.scape_vocab_loss_workspace_bytes(h, w), sc.scape_vocab_loss_workspace_bytes(h, w, grad=True))
        ws = torch.zeros(n, dtype=torch.uint8, device=gpu)
        loss, lse = torch.zeros(rows, device=gpu), torch.zeros(rows, device=gpu)
        want_h, want_w = torch.zeros(rows, 64, device=gpu, dtype=torch.bfloat16), torch.zeros(500, 64, device=gpu, dtype=torch.bfloat16)
        sc.scape_vocab_loss_forward(h, w, label, loss, lse, weight=weight, workspace=ws)
        sc.scape_vocab_loss_backward(h, w, label, lse, want_h, want_w, weight=weight, workspace=ws)
        sc.scape_vocab_loss_backward(h, w, label, lse, dh, dw, weight=weight, workspace=ws)
        assert torch.equal(dh, want_h) and torch.equal(dw, want_w)
        with pytest.raises(sc.ScapeError, match="dh overlaps h"):
            sc.scape_vocab_loss_backward(h, w, label, lse, both_h[:, 56:120], dw, weight=weight, workspace=ws)
        over = weight.clone()  # the loss in its weights' place
        sc.scape_vocab_loss_forward(h, w, label, over, lse, weight=over, workspace=ws)
        assert torch.equal(over, loss)


@pytest.mark.gpu
def test_places_over_choices(sc, gpu):
    """row may be idx."""
    for tokens, k, experts in ((1, 2, 4), (100, 3, 7), (3000, 8, 64), (70000, 2, 1024)):
        idx = torch.randint(-1, experts, (tokens, k), device=gpu).to(torch.int32)
        off, row = torch.zeros(experts + 1, dtype=torch.int32, device=gpu), torch.zeros_like(idx)
        ws = torch.zeros(max(1, sc.scape_expert_sort_workspace_bytes(idx, experts)), dtype=torch.uint8, device=gpu)
        sc.scape_expert_sort(idx, experts, off, row, workspace=ws)
        off2 = torch.zeros_like(off)
        sc.scape_expert_sort(idx, experts, off2, idx, workspace=ws)
        assert torch.equal(idx, row) and torch.equal(off, off2)
