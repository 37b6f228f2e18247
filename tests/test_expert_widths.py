"""Gates, their gradients, places and layer norms of another width than the
call's are turned down by the binding; on the host, before any device check."""
import os

import pytest
import torch


@pytest.fixture(scope="module")
def sc():
    import sparse_communication_adam_amd as sc
    if not os.path.exists(sc.LIB_PATH):
        sc.build()
    return sc


TOKENS, K, EXPERTS = 4, 2, 8
WRONG = [(TOKENS, EXPERTS), (TOKENS, K + 1), (K + 1, TOKENS), (1, EXPERTS + 1), (TOKENS, EXPERTS, 1), (2, TOKENS, K + 2), (TOKENS * K, 2 * K)]
RIGHT = [(TOKENS, K), (TOKENS + 3, K), (TOKENS * K,), (TOKENS * K + 5,), (TOKENS, K, 1), (2, 2, K), (1, TOKENS, K), (TOKENS * K, 1),
         (1, TOKENS * K)]


def _calls(sc, dtype_of_weight=torch.float32):
    bf, i32 = torch.bfloat16, torch.int32
    h, y, row = torch.zeros(TOKENS, 64, dtype=bf), torch.zeros(8, 64, dtype=bf), torch.zeros(TOKENS, K, dtype=i32)
    off, ws = torch.zeros(EXPERTS + 1, dtype=i32), torch.zeros(1 << 16, dtype=torch.uint8)
    new = lambda shape, dt=dtype_of_weight: torch.zeros(*shape, dtype=dt)  # noqa: E731
    return {
        "combine": lambda s: sc.scape_expert_combine(y, row, h, weight=new(s)),
        "weight": lambda s: sc.scape_expert_combine_backward(y, row, h, dy=y, weight=new(s)),
        "dweight": lambda s: sc.scape_expert_combine_backward(y, row, h, dy=y, dweight=new(s)),
        "row": lambda s: sc.scape_expert_sort(row, EXPERTS, off, new(s, i32), workspace=ws),
    }


@pytest.mark.parametrize("name", ["combine", "weight", "dweight", "row"])
def test_other_widths_are_refused(sc, name):
    for shape in WRONG:
        with pytest.raises(ValueError, match=r"must be \[4, 2\]"):
            _calls(sc)[name](shape)


@pytest.mark.parametrize("name", ["combine", "weight", "dweight", "row"])
def test_flat_and_longer_ones_are_taken(sc, name):
    """These go on to the next check: the tensors are not on a GPU."""
    for shape in RIGHT:
        with pytest.raises(ValueError, match="must be on the GPU"):
            _calls(sc)[name](shape)


def test_one_choice_and_one_token(sc):
    bf, i32 = torch.bfloat16, torch.int32
    y = torch.zeros(8, 64, dtype=bf)
    for tokens, k in ((5, 1), (1, 3), (1, 1)):
        row, out = torch.zeros(tokens, k, dtype=i32), torch.zeros(tokens, 64, dtype=bf)
        for shape, text in [((tokens, k), "on the GPU"), ((tokens * k,), "on the GPU"), ((tokens, EXPERTS), "must be"),
                            ((tokens, k + 1), "must be")]:
            with pytest.raises(ValueError, match=text):
                sc.scape_expert_combine(y, row, out, weight=torch.zeros(*shape))


@pytest.mark.gpu
def test_layer_norms_of_another_width(sc):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    ctx = sc.Context(sc.ScapeConfig(layer_numel=[100, 200, 5], workers=2, keep_num=1, keep_den=10))
    g = [torch.ones(ctx.layout.n_pad, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    norm = torch.zeros(3, device="cuda")
    ws = torch.zeros(sc.scape_grad_norm_workspace_bytes(ctx), dtype=torch.uint8, device="cuda")
    with pytest.raises(ValueError, match=r"must be \[2, 3\]"):
        sc.scape_grad_norm(ctx, g, norm, torch.zeros(3, 3 + 1, device="cuda"), workspace=ws)
    layer = torch.zeros(2, 3, device="cuda")
    sc.scape_grad_norm(ctx, g, norm, layer, workspace=ws)
    assert torch.equal(layer, torch.tensor([[100.0, 200.0, 5.0]] * 2, device="cuda").sqrt())
