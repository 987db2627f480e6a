"""Clipping of tensors so large that a block takes runs of many chunks, in one
tensor and across several, and the error of their sums."""
import pytest
import torch

import graph_sparse_head_gb300 as pmha
from tests import test_gpu_clip as small
from tests.test_gpu_clip import DEV

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


def make(sizes, dtypes, offset=0):
    """Tensors of these sizes, each `offset` values behind a 16-byte boundary, of different scales."""
    out = []
    for i, (n, t) in enumerate(zip(sizes, dtypes)):
        g = torch.Generator(device=DEV).manual_seed(i)
        flat = torch.randn(n + offset, generator=g, device=DEV).mul_(0.02 * 3 ** (i % 7)).to(t)
        out.append(flat[offset:])
    return out


# a block takes some 3, 14 and 1 chunks of these; the second set's tensors end inside a chunk, the third's runs go
# across tensors of several chunks each
SETS = [((8_000_000, 40_000_000, 3_000_000), (F32, BF16, F32)),
        ((8_000_001, 39_999_993, 3_000_017), (BF16, F32, BF16)),
        ((200_003,) * 300, (F32, BF16) * 150)]


@pytest.mark.parametrize("sizes,dtypes", SETS, ids=["whole", "ragged", "many"])
@pytest.mark.parametrize("offset", [0, 1])
@pytest.mark.parametrize("separate", [False, True])
@pytest.mark.parametrize("max_norm", [1.0, 1e9])
def test_long_runs(sizes, dtypes, offset, separate, max_norm):
    grads = make(sizes, dtypes, offset)
    out = [torch.full_like(g, 7.0) for g in grads] if separate else None
    small.check(grads, max_norm, out)


def test_a_value_anywhere_counts():
    # all zeros but one: every chunk of every run is read, and scaled
    sizes, dtypes = SETS[1]
    grads = [torch.zeros(n, dtype=t, device=DEV) for n, t in zip(sizes, dtypes)]
    for i, n in enumerate(sizes):
        for at in (0, 65535, 65536, n // 2, n - 40000, n - 1):
            grads[i][at] = 3.0
            assert float(pmha.pmha_clip_grad_norm(grads, 1.5)) == 3.0
            assert abs(float(grads[i][at]) - 1.5) <= 2.0 ** -9 * 1.5
            grads[i][at] = 0.0
    assert not any(bool(g.any()) for g in grads)


@pytest.mark.parametrize("dtype,n", [(BF16, 1_000_000_000), (F32, 500_000_000)], ids=["bf16", "f32"])
@pytest.mark.parametrize("offset", [0, 1])
def test_equal_values(dtype, n, offset):
    # Additions of equal values are all off to the same side: chains of k squares by up to k / 2 roundings of their
    # sum, the norm by half as much. 128 squares at most are added in float32: 2^-19; a chain of all of a thread's
    # squares here would have some 4,000 (float32: 2,100).
    g = torch.full((n + offset,), 0.0123, dtype=dtype, device=DEV)[offset:]
    value = float(g[0])
    norm = pmha.pmha_clip_grad_norm([g], 1e9)
    want = value * float(n) ** 0.5
    assert abs(float(norm) - want) <= (2.0 ** -19 + 2.0 ** -24) * want
