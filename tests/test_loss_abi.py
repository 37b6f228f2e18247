"""The loss operators' refusals, on the host: every bad argument is turned
down with its code and a text before anything is launched, by the C ABI and by
the Python binding.  No GPU."""
import ctypes
import os

import pytest
import torch

P = ctypes.c_void_p


@pytest.fixture(scope="module")
def sc():
    import sparse_communication_adam_amd as sc
    if not os.path.exists(sc.LIB_PATH):
        sc.build()
    return sc


@pytest.fixture(scope="module")
def lib(sc):
    return sc.lib()


def _teacher(lib, **kw):
    from sparse_communication_adam_amd._scape import _Teacher
    d = dict(val=64, dtype=1, idx=64, lse=64, k=4)
    d.update(kw)
    return ctypes.byref(_Teacher(*[d[n] for n in ("val", "dtype", "idx", "lse", "k")]))


# each call with valid arguments of a shape that needs no workspace, as a dict
# in the order of the C signature; a test changes one of them
TOPK = dict(z=64, dtype=1, rows=4, cols=100, ld=100, k=5, scale=1.0, val=64, idx=64, lse=64, ws=0, ws_bytes=0, stream=0)
FORWARD = dict(z=64, dtype=1, rows=2000, cols=100, ld=100, teacher={}, scale=1.0, weight=64, loss=64, stats=64, dz=128,
               ld_dz=100, ws=0, ws_bytes=0, stream=0)
BACKWARD = dict(z=64, dtype=1, rows=2000, cols=100, ld=100, teacher={}, scale=1.0, weight=64, stats=64, dloss=64, dz=128,
                ld_dz=100, stream=0)
BALANCE = dict(logits=64, dtype=0, tokens=10, experts=8, ld=8, idx=64, k=2, offsets=64, segments=3, mask=64, score=0,
               alpha=1.0, counts=64, psum=64, n_tok=64, loss=64, ws=64, ws_bytes=1 << 20, stream=0)
BALANCE_LOSS = dict(counts=64, psum=64, n_tok=64, segments=3, experts=8, k=2, alpha=1.0, loss=64, stream=0)
BALANCE_BACK = dict(logits=64, dtype=0, tokens=10, experts=8, ld=8, k=2, offsets=64, segments=3, mask=64, score=0,
                    alpha=1.0, counts=64, n_tok=64, dloss=64, dlogits=128, ld_d=8, stream=0)
POINTERS = {"z", "val", "idx", "lse", "ws", "stream", "weight", "loss", "stats", "dz", "dloss", "logits", "offsets",
            "mask", "counts", "psum", "n_tok", "dlogits"}


def _call(lib, fn, base, **change):
    args = dict(base)
    args.update(change)
    out = []
    for name, v in args.items():
        if name == "teacher":
            out.append(None if v is None else _teacher(lib, **v))
        else:
            out.append(P(v) if name in POINTERS else v)
    return getattr(lib, fn)(*out)


INF, NAN = float("inf"), float("nan")
ROWS = [  # of every call on rows
    (dict(dtype=3), -1), (dict(dtype=-1), -1), (dict(rows=-1), -2), (dict(cols=0), -2), (dict(cols=262145, ld=262145), -2),
    (dict(ld=99), -2), (dict(z=0), -1), (dict(z=65), -3), (dict(scale=0.0), -1), (dict(scale=-1.0), -1),
    (dict(scale=INF), -1), (dict(scale=NAN), -1), (dict(rows=1 << 40), -2), (dict(ld=1 << 60), -2),
]
CASES = (
    [("scape_topk_rows", TOPK, c, e) for c, e in ROWS + [
        (dict(k=0), -2), (dict(k=101), -2), (dict(k=1025, cols=5000, ld=5000), -2), (dict(val=0), -1), (dict(val=65), -3),
        (dict(idx=0), -1), (dict(idx=66), -3), (dict(lse=66), -3),
        (dict(rows=1, cols=131072, ld=131072), -1),                                    # a split row: no workspace
        (dict(rows=1, cols=131072, ld=131072, ws=64, ws_bytes=8), -2),                 # too small
        (dict(rows=1, cols=131072, ld=131072, ws=72, ws_bytes=1 << 20), -3)]]          # misaligned
    + [("scape_distill_forward", FORWARD, c, e) for c, e in ROWS + [
        (dict(teacher=None), -1), (dict(teacher=dict(val=0)), -1), (dict(teacher=dict(val=65)), -3),
        (dict(teacher=dict(dtype=7)), -1), (dict(teacher=dict(idx=0)), -1), (dict(teacher=dict(idx=66)), -3),
        (dict(teacher=dict(lse=66)), -3), (dict(teacher=dict(k=0)), -2), (dict(teacher=dict(k=1025)), -2),
        (dict(weight=66), -3), (dict(loss=0), -1), (dict(loss=66), -3), (dict(stats=0), -1), (dict(stats=66), -3),
        (dict(dz=129), -3), (dict(ld_dz=99), -2), (dict(dz=64, ld_dz=101), -2),
        (dict(rows=1, cols=262144, ld=262144, ld_dz=262144), -1)]]  # a split row: no workspace
    + [("scape_distill_backward", BACKWARD, c, e) for c, e in ROWS + [
        (dict(teacher=None), -1), (dict(teacher=dict(k=1025)), -2), (dict(dz=0), -1), (dict(dz=129), -3),
        (dict(ld_dz=99), -2), (dict(dz=64, ld_dz=101), -2), (dict(stats=0), -1), (dict(dloss=66), -3),
        (dict(weight=66), -3)]]
    + [("scape_balance_forward", BALANCE, c, e) for c, e in [
        (dict(dtype=9), -1), (dict(tokens=-1), -2), (dict(tokens=(1 << 30) + 1), -2), (dict(experts=0), -2),
        (dict(experts=1025, ld=1025), -2), (dict(ld=7), -2), (dict(k=0), -2), (dict(k=9), -2), (dict(logits=0), -1),
        (dict(logits=66), -3), (dict(idx=0), -1), (dict(idx=66), -3), (dict(offsets=0), -1), (dict(offsets=66), -3),
        (dict(segments=0), -2), (dict(score=2), -1), (dict(alpha=NAN), -1), (dict(counts=0), -1), (dict(psum=66), -3),
        (dict(n_tok=0), -1), (dict(loss=66), -3), (dict(ws=0), -1), (dict(ws_bytes=16), -2), (dict(ws=72), -3),
        (dict(tokens=1 << 30, k=8, ws_bytes=1 << 40), -2)]]
    + [("scape_balance_loss", BALANCE_LOSS, c, e) for c, e in [
        (dict(counts=0), -1), (dict(psum=0), -1), (dict(n_tok=66), -3), (dict(loss=0), -1), (dict(k=9), -2),
        (dict(segments=0), -2), (dict(experts=0), -2), (dict(alpha=INF), -1)]]
    + [("scape_balance_backward", BALANCE_BACK, c, e) for c, e in [
        (dict(dtype=9), -1), (dict(tokens=-1), -2), (dict(experts=0), -2), (dict(ld=7), -2), (dict(ld_d=7), -2),
        (dict(k=9), -2), (dict(logits=0), -1), (dict(dlogits=0), -1), (dict(dlogits=130), -3),
        (dict(dlogits=64, ld_d=9), -2), (dict(offsets=0), -1), (dict(score=-1), -1), (dict(counts=0), -1),
        (dict(n_tok=0), -1), (dict(dloss=66), -3), (dict(alpha=NAN), -1)]])


@pytest.mark.parametrize("fn,base,change,code", CASES,
                         ids=[f"{f[6:]}-{'-'.join(f'{k}={v}' for k, v in c.items())}" for f, _, c, _ in CASES])
def test_bad_arguments_are_refused(sc, lib, fn, base, change, code):
    assert _call(lib, fn, base, **change) == code
    assert sc.scape_last_error()


def test_no_rows_enqueue_nothing(lib):
    assert _call(lib, "scape_topk_rows", TOPK, rows=0, z=0, val=0, idx=0, lse=0) == 0
    empty = dict(val=0, idx=0, lse=0)
    assert _call(lib, "scape_distill_forward", FORWARD, rows=0, z=0, teacher=empty, loss=0, stats=0, dz=0) == 0
    assert _call(lib, "scape_distill_backward", BACKWARD, rows=0, z=0, teacher=empty, stats=0, dz=0) == 0
    assert _call(lib, "scape_balance_backward", BALANCE_BACK, tokens=0, logits=0, dlogits=0, counts=0, n_tok=0) == 0


def test_workspace_queries(sc, lib):
    b = ctypes.c_int64(-1)
    assert lib.scape_topk_rows_workspace(1, 4096, 32000, 64, ctypes.byref(b)) == 0 and b.value == 0
    assert lib.scape_topk_rows_workspace(1, 1 << 20, 64, 8, ctypes.byref(b)) == 0 and b.value == 0
    assert lib.scape_topk_rows_workspace(1, 1, 50304, 32, ctypes.byref(b)) == 0 and b.value == 0
    assert lib.scape_topk_rows_workspace(1, 1, 131072, 32, ctypes.byref(b)) == 0 and b.value > 0
    assert lib.scape_topk_rows_workspace(0, 4096, 262144, 64, ctypes.byref(b)) == 0 and b.value > 0  # too long for one
    assert lib.scape_distill_workspace(1, 4096, 32000, 64, ctypes.byref(b)) == 0 and b.value == 0
    assert lib.scape_distill_workspace(1, 1, 50304, 64, ctypes.byref(b)) == 0 and b.value == 0
    assert lib.scape_distill_workspace(1, 1, 262144, 64, ctypes.byref(b)) == 0 and b.value > 0
    assert lib.scape_balance_workspace(131072, 64, 1, ctypes.byref(b)) == 0 and b.value > 0
    assert lib.scape_topk_rows_workspace(1, 1, 50304, 32, None) == -1
    assert lib.scape_distill_workspace(1, 1, 50304, 0, ctypes.byref(b)) == -2
    assert lib.scape_balance_workspace(1, 0, 1, ctypes.byref(b)) == -2
    z = torch.zeros(1, 262144, dtype=torch.bfloat16)
    assert sc.scape_topk_rows_workspace_bytes(z, 32) > 0 and sc.scape_distill_workspace_bytes(z, 32, grad=True) > 0
    assert sc.scape_balance_workspace_bytes(torch.zeros(7, 8), 2) > 0


def test_row_limits_of_a_launch(lib):
    """A launch counts its threads in 32 bits: more rows than that are refused
    (nothing is read, so no such matrix is needed)."""
    b = ctypes.c_int64()
    assert lib.scape_topk_rows_workspace(1, 1 << 22, 2048, 8, ctypes.byref(b)) == 0
    assert lib.scape_topk_rows_workspace(1, 1 << 23, 2048, 8, ctypes.byref(b)) == -2
    assert lib.scape_topk_rows_workspace(1, 1 << 25, 64, 8, ctypes.byref(b)) == 0
    assert lib.scape_topk_rows_workspace(1, (1 << 25) + 1, 64, 8, ctypes.byref(b)) == -2
    assert lib.scape_distill_workspace(1, 1 << 23, 2048, 8, ctypes.byref(b)) == -2


def test_binding_refuses_before_the_library(sc):
    """Wrong types, shapes, strides and devices are Python errors."""
    z = torch.zeros(4, 100)
    val, idx = torch.zeros(4, 5), torch.zeros(4, 5, dtype=torch.int32)
    loss, stats = torch.zeros(4), torch.zeros(4, 2)
    cases = [
        (TypeError, lambda: sc.scape_topk_rows(z.double(), 5, val, idx)),
        (TypeError, lambda: sc.scape_topk_rows([1.0], 5, val, idx)),
        (ValueError, lambda: sc.scape_topk_rows(z[0], 5, val, idx)),
        (ValueError, lambda: sc.scape_topk_rows(z.t(), 4, val, idx)),
        (ValueError, lambda: sc.scape_topk_rows(z[:1].expand(4, 100), 5, val, idx)),  # rows on top of each other
        (ValueError, lambda: sc.scape_topk_rows(z, 5, val[:3], idx)),
        (TypeError, lambda: sc.scape_topk_rows(z, 5, val.half(), idx)),
        (TypeError, lambda: sc.scape_topk_rows(z, 5, val, idx.long())),
        (ValueError, lambda: sc.scape_topk_rows(z, 5, val, idx)),  # right, but on the host
        (ValueError, lambda: sc.scape_distill_forward(z, val, idx[:, :4], loss, stats)),
        (ValueError, lambda: sc.scape_distill_forward(z, val[:3], idx[:3], loss, stats)),
        (TypeError, lambda: sc.scape_distill_forward(z, val.double(), idx, loss, stats)),
        (ValueError, lambda: sc.scape_distill_forward(z, val, idx, loss, stats, dz=z.half())),
        (ValueError, lambda: sc.scape_distill_forward(z, val, idx, loss, stats, dz=z[:, :50])),
        (ValueError, lambda: sc.scape_distill_forward(z, val, idx, loss[:3], stats)),
        (ValueError, lambda: sc.scape_distill_forward(z, val, idx, loss, stats[:3])),
        (TypeError, lambda: sc.scape_distill_backward(z, val, idx, stats, None)),
        (ValueError, lambda: sc.scape_balance_forward(z, idx[:2], idx, val, idx)),
        (ValueError, lambda: sc.scape_balance_backward(z, idx, idx, None, val, k=2)),
        (ValueError, lambda: sc.scape_balance_loss(idx[0], val, idx, loss, 2)),
    ]
    for i, (kind, call) in enumerate(cases):
        with pytest.raises(kind):
            call()
    with pytest.raises(sc.ScapeError) as e:
        sc.scape_topk_rows(z, 101, torch.zeros(4, 101), torch.zeros(4, 101, dtype=torch.int32))
    assert e.value.code == -2
    with pytest.raises(ValueError, match="workspace"):
        big = torch.zeros(1, 50304)
        sc.scape_topk_rows(big, 2, torch.zeros(1, 2), torch.zeros(1, 2, dtype=torch.int32))
    counts, n_tok = torch.zeros(1, 100, dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError, match="GPU"):
        sc.scape_balance_backward(z, counts, n_tok, None, torch.zeros_like(z), k=2)
    with pytest.raises(ValueError, match="GPU"):
        sc.scape_balance_loss(counts, torch.zeros(1, 100), n_tok, torch.zeros(1), 2)
