"""What the vocabulary gradient's workspace holds, and the gradient where it holds
most: P of a piece is 2^27 elements, or 4096 words of every row where that is
more; copies of h; and sums of dh only where more than one launch adds to them."""
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


def _bytes(sc, dtype, rows, cols, dim):
    b = ctypes.c_int64()
    assert sc.lib().scape_vocab_grad_workspace(dtype, rows, cols, dim, ctypes.byref(b)) == 0
    return b.value


def _up(n, to):
    return -(-n // to) * to


@pytest.mark.parametrize("dtype", [1, 2])
def test_no_sums_where_one_launch_writes_dh(sc, dtype):
    """8192 rows of 2048 are 256 tiles of dh, a round of the CUs: no splits, and up to 2^27 / 8192 words one piece."""
    rows, dim, cols = 8192, 2048, 16000
    most = rows * 16 + 16 + 4096 + rows * dim * 2 + rows * _up(cols, 256) * 2
    assert most - 4096 <= _bytes(sc, dtype, rows, cols, dim) <= most
    two = _bytes(sc, dtype, rows, 32000, dim)  # in two pieces: dh is summed in between
    assert two >= rows * 16 + rows * dim * 2 + rows * 16000 * 2 + rows * dim * 4


@pytest.mark.parametrize("rows", [1, 300, 8192, 32768, 32769, 100000, 1 << 20])
def test_bound(sc, rows):
    dim, cols = 2048, 262144  # from 8192 rows on a round of tiles of dh, which is not split
    pad = _up(rows, 256)
    elements = max(1 << 27, 4096 * pad)
    sums = 128 * rows * dim * 4 if rows < 8192 else rows * dim * 4
    got = _bytes(sc, 1, rows, cols, dim)
    assert got <= elements * 2 + pad * 16 + 16 + rows * dim * 2 + sums
    if rows > 32768:
        assert got >= 4096 * rows * 2 * 0.9


@pytest.fixture
def on_gpu(sc):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    yield sc
    torch.cuda.empty_cache()


SHAPES = [
    (33000, 8190, 24),     # P of 4096 words: more than 2^27 elements, in two pieces
    (1100, 131072, 32),    # tiles of 192 tokens, in two pieces
    (8192, 16000, 64),     # one piece and no sums of dh
    (40, 3001, 4096), (200, 2500, 5120), (300, 1500, 2048), (600, 2000, 1536),  # dims of models
]


@pytest.mark.gpu
@pytest.mark.parametrize("rows,cols,dim", SHAPES)
def test_gradients(on_gpu, rows, cols, dim):
    import test_gpu_vocab_loss as v
    for dtype in v.DTYPES:
        c = v.Case(rows, cols, dim, dtype, key="memory")
        v._check_forward(on_gpu, c)
        v._check_backward(on_gpu, c)
