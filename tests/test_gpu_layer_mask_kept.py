"""The mask of a checkpointed step is that of its forward pass."""
import pytest
import torch

from tests.test_gpu_encoder import make
from tests.test_gpu_encoder_joins import joined

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.mark.parametrize("kind", ["plain", "joined"])
def test_a_mask_that_takes_the_next_batch_meanwhile(kind):
    layer, x, dy, _ = make(200, 1500, 2, 128, 8, 256, "bf16", seed=3)
    if kind == "joined":
        layer = joined(layer, 7, True, 2)
    mask = torch.zeros(2, 200, dtype=torch.bool, device=DEV)
    mask[1, 100:] = True
    _, kept = layer.forward_checkpointed(x, key_padding_mask=mask)
    want = layer.backward_checkpointed(kept, dy)
    static = x.clone()
    _, kept = layer.forward_checkpointed(static, key_padding_mask=mask)
    mask.logical_not_()  # as a captured graph's inputs are written again
    static.zero_()
    got = layer.backward_checkpointed(kept, dy)
    assert all(torch.equal(got[k], v) for k, v in want.items() if v is not None)
