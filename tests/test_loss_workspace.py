"""The workspace of a distillation: a loss alone needs none for its gradient.
No GPU."""
import ctypes
import os

import pytest
import torch


@pytest.fixture(scope="module")
def sc():
    import sparse_communication_adam_amd as sc
    if not os.path.exists(sc.LIB_PATH):
        sc.build()
    return sc


LONG = [(300, 262144, torch.float32), (7, 50304, torch.float32), (2000, 131072, torch.bfloat16)]


@pytest.mark.parametrize("rows,cols,dtype", LONG, ids=str)
def test_loss_of_long_rows_needs_no_workspace(sc, rows, cols, dtype):
    z = torch.empty(rows, cols, dtype=dtype, device="meta")
    assert sc.scape_distill_workspace_bytes(z, 5, grad=False) == 0
    assert sc.scape_distill_workspace_bytes(z, 5, grad=True) == rows * 8
    assert sc.scape_distill_workspace_bytes(z, 5) == rows * 8  # enough for either


def test_split_rows_need_less_without_the_gradient(sc):
    z = torch.empty(2, 262144, device="meta")
    loss, grad = (sc.scape_distill_workspace_bytes(z, 5, grad=g) for g in (False, True))
    assert 0 < loss < grad == sc.scape_distill_workspace_bytes(z, 5)


def test_the_call_asks_for_what_it_needs(sc):
    """Without a workspace: a loss alone comes as far as the check of the
    devices, with a gradient it is told how many bytes it needs."""
    z = torch.empty(7, 50304)
    val, idx = torch.zeros(7, 3), torch.zeros(7, 3, dtype=torch.int32)
    loss, stats = torch.zeros(7), torch.zeros(7, 2)
    with pytest.raises(ValueError, match="GPU"):
        sc.scape_distill_forward(z, val, idx, loss, stats)
    with pytest.raises(ValueError, match="workspace of 56 bytes"):
        sc.scape_distill_forward(z, val, idx, loss, stats, dz=torch.empty_like(z))


def test_library_query(sc):
    lib, b = sc.lib(), ctypes.c_int64(-1)
    assert lib.scape_distill_loss_workspace(0, 300, 262144, 5, ctypes.byref(b)) == 0 and b.value == 0
    assert lib.scape_distill_loss_workspace(0, 2, 262144, 5, ctypes.byref(b)) == 0 and b.value > 0
    assert lib.scape_distill_loss_workspace(0, 2, 262144, 0, ctypes.byref(b)) == -2
    assert lib.scape_distill_loss_workspace(7, 2, 262144, 5, ctypes.byref(b)) == -1
    assert lib.scape_distill_loss_workspace(0, 2, 262144, 5, None) == -1
