"""Refusals of the vocabulary loss, the expert moves and the gradient norms, on
the host: every bad argument is turned down with its code and a text before
anything is launched, by the C ABI and by the Python binding.  No GPU."""
import ctypes
import os

import pytest
import torch

P = ctypes.c_void_p
INF, NAN = float("inf"), float("nan")


@pytest.fixture(scope="module")
def sc():
    import sparse_communication_adam_amd as sc
    if not os.path.exists(sc.LIB_PATH):
        sc.build()
    return sc


@pytest.fixture(scope="module")
def lib(sc):
    return sc.lib()


HEAD = dict(h=64, ld_h=64, w=128, ld_w=64, dtype=1, rows=4, cols=100, dim=64, label=64, weight=64, scale=1.0)


def _head(**kw):
    from sparse_communication_adam_amd._scape import _Head
    d = dict(HEAD)
    d.update(kw)
    return ctypes.byref(_Head(*[d[n] for n in HEAD]))


FORWARD = dict(head={}, loss=64, lse=64, ws=64, ws_bytes=1 << 40, stream=0)
BACKWARD = dict(head={}, lse=64, dloss=64, dh=256, ld_dh=64, dw=512, ld_dw=64, ws=64, ws_bytes=1 << 40, stream=0)
SORT = dict(idx=64, tokens=10, k=2, experts=8, offsets=64, row=64, ws=64, ws_bytes=1 << 30, stream=0)
GATHER = dict(x=64, dtype=1, tokens=10, dim=16, ld_x=16, row=64, k=2, y=128, rows=20, ld_y=16, stream=0)
COMBINE = dict(y=128, dtype=1, rows=20, dim=16, ld_y=16, row=64, weight=64, tokens=10, k=2, out=64, ld_out=16, stream=0)
COMBINE_BACK = dict(y=128, dtype=1, rows=20, dim=16, ld_y=16, row=64, weight=64, dout=64, ld_dout=16, tokens=10, k=2,
                    dy=256, ld_dy=16, dweight=64, stream=0)
POINTERS = {"loss", "lse", "ws", "stream", "dloss", "dh", "dw", "idx", "offsets", "row", "x", "y", "weight", "out",
            "dout", "dy", "dweight"}


def _call(lib, fn, base, **change):
    args = dict(base)
    args.update(change)
    out = []
    for name, v in args.items():
        if name == "head":
            out.append(None if v is None else _head(**v))
        else:
            out.append(P(v) if name in POINTERS else v)
    return getattr(lib, fn)(*out)


HEADS = [(None, -1)] + [
    (c, e) for c, e in [
        (dict(dtype=0), -1), (dict(dtype=3), -1), (dict(rows=-1), -2), (dict(rows=(1 << 20) + 1), -2), (dict(cols=0), -2),
        (dict(cols=262145), -2), (dict(dim=0), -2), (dict(dim=-8), -2), (dict(dim=63), -2), (dict(dim=65544, ld_h=65544), -2),
        (dict(ld_h=56), -2), (dict(ld_w=56), -2), (dict(ld_h=68), -3), (dict(ld_w=65), -3), (dict(h=0), -1), (dict(w=0), -1),
        (dict(h=72), -3), (dict(w=136), -3), (dict(ld_h=1 << 22), -2), (dict(ld_w=1 << 60), -2), (dict(label=0), -1),
        (dict(label=66), -3), (dict(weight=66), -3), (dict(scale=0.0), -1), (dict(scale=-1.0), -1), (dict(scale=INF), -1),
        (dict(scale=NAN), -1)]]
MOVES = [(dict(dtype=3), -1), (dict(tokens=-1), -2), (dict(tokens=(1 << 25) + 1), -2), (dict(dim=0), -2), (dict(rows=-1), -2),
         (dict(dim=1 << 25), -2), (dict(k=0), -2), (dict(k=-1), -2), (dict(tokens=1 << 25, k=64), -2), (dict(row=0), -1), (dict(row=66), -3),
         (dict(ld_y=15), -2), (dict(y=0), -1), (dict(y=129), -3), (dict(ld_y=1 << 60), -2)]
CASES = (
    [("scape_vocab_loss_forward", FORWARD, dict(head=c), e) for c, e in HEADS]
    + [("scape_vocab_loss_forward", FORWARD, c, e) for c, e in [
        (dict(loss=0), -1), (dict(loss=66), -3), (dict(lse=0), -1), (dict(lse=66), -3), (dict(ws=0), -1),
        (dict(ws_bytes=8), -2), (dict(ws=72), -3)]]
    + [("scape_vocab_loss_backward", BACKWARD, dict(head=c), e) for c, e in HEADS]
    + [("scape_vocab_loss_backward", BACKWARD, c, e) for c, e in [
        (dict(lse=0), -1), (dict(lse=66), -3), (dict(dloss=66), -3), (dict(dh=264), -3), (dict(dw=520), -3),
        (dict(ld_dh=56), -2), (dict(ld_dw=56), -2), (dict(ld_dh=68), -3), (dict(ld_dw=1 << 22), -2), (dict(ws=0), -1),
        (dict(ws_bytes=8), -2), (dict(ws=72), -3)]]
    + [("scape_expert_sort", SORT, c, e) for c, e in [
        (dict(tokens=-1), -2), (dict(tokens=(1 << 30) + 1), -2), (dict(k=0), -2), (dict(experts=0), -2),
        (dict(experts=1025), -2), (dict(tokens=1 << 30), -2), (dict(idx=0), -1), (dict(idx=66), -3), (dict(offsets=0), -1),
        (dict(offsets=66), -3), (dict(row=0), -1), (dict(row=66), -3), (dict(tokens=5000, ws_bytes=8), -2),
        (dict(tokens=5000, ws=0), -1), (dict(tokens=5000, ws=72), -3)]]
    + [("scape_expert_gather", GATHER, c, e) for c, e in MOVES + [
        (dict(x=0), -1), (dict(x=65), -3), (dict(ld_x=15), -2)]]
    + [("scape_expert_combine", COMBINE, c, e) for c, e in MOVES + [
        (dict(out=0), -1), (dict(out=65), -3), (dict(ld_out=15), -2), (dict(weight=66), -3)]]
    + [("scape_expert_combine_backward", COMBINE_BACK, c, e) for c, e in MOVES + [
        (dict(dout=0), -1), (dict(dout=65), -3), (dict(ld_dout=15), -2), (dict(weight=66), -3), (dict(dweight=66), -3),
        (dict(dy=257), -3), (dict(ld_dy=15), -2), (dict(dy=128, ld_dy=17), -2)]])


@pytest.mark.parametrize("fn,base,change,code", CASES,
                         ids=[f"{f[6:]}-{'-'.join(f'{k}={v}' for k, v in c.items())}" for f, _, c, _ in CASES])
def test_bad_arguments_are_refused(sc, lib, fn, base, change, code):
    assert _call(lib, fn, base, **change) == code
    assert sc.scape_last_error()


def test_nothing_to_do_enqueues_nothing(lib):
    none = dict(rows=0, h=0, label=0, weight=0)
    assert _call(lib, "scape_vocab_loss_forward", FORWARD, head=none, loss=0, lse=0, ws=0, ws_bytes=0) == 0
    assert _call(lib, "scape_vocab_loss_backward", BACKWARD, head=none, lse=0, dh=0, dw=0, ws=0, ws_bytes=0) == 0
    assert _call(lib, "scape_vocab_loss_backward", BACKWARD, head=none, lse=0, dw=0, ws=0, ws_bytes=0) == 0
    assert _call(lib, "scape_vocab_loss_backward", BACKWARD, dh=0, dw=0, ws=0, ws_bytes=0) == 0
    assert _call(lib, "scape_expert_gather", GATHER, tokens=0, x=0, row=0) == 0
    assert _call(lib, "scape_expert_gather", GATHER, rows=0, y=0) == 0
    assert _call(lib, "scape_expert_combine", COMBINE, tokens=0, out=0, row=0) == 0
    assert _call(lib, "scape_expert_combine_backward", COMBINE_BACK, tokens=0, dout=0, row=0) == 0
    assert _call(lib, "scape_expert_combine_backward", COMBINE_BACK, dy=0, dweight=0) == 0


def test_workspace_queries(sc, lib):
    b = ctypes.c_int64(-1)
    for q in (lib.scape_vocab_loss_workspace, lib.scape_vocab_grad_workspace):
        assert q(1, 7, 50304, 1024, ctypes.byref(b)) == 0 and b.value > 0
        assert q(2, 0, 50304, 1024, ctypes.byref(b)) == 0 and b.value == 0
        assert q(0, 7, 50304, 1024, ctypes.byref(b)) == -1
        assert q(1, 7, 50304, 1023, ctypes.byref(b)) == -2
        assert q(1, 7, 50304, 1024, None) == -1
    # the logits are not kept: a batch's workspace is far below them
    assert lib.scape_vocab_loss_workspace(1, 65536, 131072, 4096, ctypes.byref(b)) == 0
    assert b.value < 65536 * 131072 * 4 // 64
    assert lib.scape_vocab_grad_workspace(1, 65536, 131072, 4096, ctypes.byref(b)) == 0
    assert b.value < 65536 * 131072 * 2 // 4
    assert lib.scape_expert_sort_workspace(1, 8, 64, ctypes.byref(b)) == 0
    assert lib.scape_expert_sort_workspace(1 << 27, 8, 1024, ctypes.byref(b)) == 0 and 0 < b.value <= 1024 * 512 * 4
    assert lib.scape_expert_sort_workspace(1, 8, 0, ctypes.byref(b)) == -2
    assert lib.scape_expert_sort_workspace(1, 8, 64, None) == -1
    h, w = torch.zeros(7, 64, dtype=torch.bfloat16), torch.zeros(100, 64, dtype=torch.bfloat16)
    assert sc.scape_vocab_loss_workspace_bytes(h, w) > 0 and sc.scape_vocab_loss_workspace_bytes(h, w, grad=True) > 0
    assert lib.scape_grad_norm_workspace(None, ctypes.byref(b)) == -1


def test_gradient_norms_refuse_without_a_context(lib):
    g = (ctypes.c_void_p * 1)(64)
    assert lib.scape_grad_norm(None, g, P(64), None, P(64), 1 << 20, None) == -1
    assert lib.scape_grad_norm_interleaved(None, P(64), P(64), None, P(64), 1 << 20, None) == -1
    assert lib.scape_grad_clip(None, g, P(64), 1.0, 0, g, None) == -1
    assert lib.scape_grad_clip_interleaved(None, P(64), P(64), 1.0, 0, P(64), None) == -1


def test_binding_refuses_before_the_library(sc):
    """Wrong types, shapes, strides and devices are Python errors."""
    bf, f32, i32 = torch.bfloat16, torch.float32, torch.int32
    h, w, lab = torch.zeros(4, 64, dtype=bf), torch.zeros(100, 64, dtype=bf), torch.zeros(4, dtype=i32)
    loss, lse, ws = torch.zeros(4), torch.zeros(4), torch.zeros(1 << 24, dtype=torch.uint8)
    idx, off, row = torch.zeros(4, 2, dtype=i32), torch.zeros(9, dtype=i32), torch.zeros(4, 2, dtype=i32)
    y = torch.zeros(8, 64, dtype=bf)
    fwd, bwd = sc.scape_vocab_loss_forward, sc.scape_vocab_loss_backward
    cases = [
        (TypeError, lambda: fwd([1.0], w, lab, loss, lse, workspace=ws)),
        (TypeError, lambda: fwd(h.double(), w, lab, loss, lse, workspace=ws)),
        (ValueError, lambda: fwd(h, w.half(), lab, loss, lse, workspace=ws)),
        (ValueError, lambda: fwd(h, w[:, :56], lab, loss, lse, workspace=ws)),
        (ValueError, lambda: fwd(h, w.t(), lab, loss, lse, workspace=ws)),
        (TypeError, lambda: fwd(h, w, lab.long(), loss, lse, workspace=ws)),
        (ValueError, lambda: fwd(h, w, lab[:3], loss, lse, workspace=ws)),
        (ValueError, lambda: fwd(h, w, lab, loss[:3], lse, workspace=ws)),
        (TypeError, lambda: fwd(h, w, lab, loss, None, workspace=ws)),
        (TypeError, lambda: fwd(h, w, lab, loss, lse.half(), workspace=ws)),
        (ValueError, lambda: fwd(h, w, lab, loss, lse, weight=loss[:3], workspace=ws)),
        (ValueError, lambda: fwd(h, w, lab, loss, lse)),                            # no workspace
        (ValueError, lambda: fwd(h, w, lab, loss, lse, workspace=ws)),              # right, but on the host
        (ValueError, lambda: bwd(h, w, lab, lse, dh=h[:3], workspace=ws)),
        (ValueError, lambda: bwd(h, w, lab, lse, dw=w.half(), workspace=ws)),
        (ValueError, lambda: bwd(h, w, lab, lse, dh=h, dloss=loss[:3], workspace=ws)),
        (ValueError, lambda: bwd(h, w, lab, lse, dh=h, dw=w)),
        (ValueError, lambda: bwd(h, w, lab, lse, dh=h, dw=w, workspace=ws)),
        (ValueError, lambda: sc.scape_expert_sort(idx[0], 8, off, row, workspace=ws)),
        (TypeError, lambda: sc.scape_expert_sort(idx.long(), 8, off, row, workspace=ws)),
        (ValueError, lambda: sc.scape_expert_sort(idx, 9, off, row, workspace=ws)),
        (ValueError, lambda: sc.scape_expert_sort(idx, 8, off, row[:3], workspace=ws)),
        (ValueError, lambda: sc.scape_expert_sort(idx, 8, off, row)),
        (ValueError, lambda: sc.scape_expert_sort(idx, 8, off, row, workspace=ws)),
        (ValueError, lambda: sc.scape_expert_gather(h[:3], row, y)),
        (ValueError, lambda: sc.scape_expert_gather(h, row, y[:, :32])),
        (ValueError, lambda: sc.scape_expert_gather(h, row, y.half())),
        (TypeError, lambda: sc.scape_expert_gather(h, row.long(), y)),
        (ValueError, lambda: sc.scape_expert_gather(h, row, y)),
        (ValueError, lambda: sc.scape_expert_combine(y, row, h[:3])),
        (ValueError, lambda: sc.scape_expert_combine(y, row, h, weight=torch.zeros(4, 1))),
        (TypeError, lambda: sc.scape_expert_combine(y, row, h, weight=torch.zeros(4, 2, dtype=bf))),
        (ValueError, lambda: sc.scape_expert_combine(y, row, h)),
        (ValueError, lambda: sc.scape_expert_combine_backward(y, row, h, dy=y[:7])),
        (ValueError, lambda: sc.scape_expert_combine_backward(y, row, h[:2], dy=y)),
        (ValueError, lambda: sc.scape_expert_combine_backward(y, row, h, dy=y, dweight=torch.zeros(3))),
        (ValueError, lambda: sc.scape_expert_combine_backward(y, row, h, dy=y)),
    ]
    for kind, call in cases:
        with pytest.raises(kind):
            call()
    with pytest.raises(sc.ScapeError) as e:
        sc.scape_vocab_loss_workspace_bytes(h.float(), w.float())
    assert e.value.code == -1
    with pytest.raises(sc.ScapeError) as e:
        sc.scape_vocab_loss_workspace_bytes(torch.zeros(4, 63, dtype=bf), torch.zeros(9, 63, dtype=bf))
    assert e.value.code == -2
