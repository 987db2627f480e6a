"""What the C ABI of the encoder operators offers beyond the Python calls: both of
the norm's outputs at once, sums that are not kept, single gradients, gradients
aligned to their elements only, clipping without a table of outputs."""
import ctypes
import itertools

import pytest
import torch

import graph_sparse_head_gb300 as pmha
from graph_sparse_head_gb300 import _lib
from tests import _encoder_ref as ref
from tests.test_gpu_ffn import BF16, DEV, F32, make

pytestmark = pytest.mark.gpu
CODE = {F32: 0, BF16: 1}


def stream():
    return torch.cuda.current_stream().cuda_stream


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("width", [7, 48, 128, 257, 1000, 2048])
@pytest.mark.parametrize("keep", [True, False])
def test_both_outputs_of_the_norm(width, dtype, keep):
    g = torch.Generator().manual_seed(width)
    sizes = torch.tensor([1.0, 2.0 ** 40, 2.0 ** 52, 2.0 ** 62, 1e30, 1e38, 1e-10])[:, None]
    x, r = ((sizes * torch.randn(7, width, generator=g)).to(dtype).to(DEV) for _ in range(2))
    w = (1 + 0.2 * torch.randn(width, generator=g)).to(dtype).to(DEV)
    out, s = torch.empty_like(x), torch.empty_like(x)
    q = torch.empty(7, width, dtype=torch.float8_e4m3fn, device=DEV)
    scale = torch.empty(7, device=DEV)
    st = _lib.load().pmha_rms_norm(CODE[dtype], 7, width, x.data_ptr(), r.data_ptr(), w.data_ptr(), ref.EPS,
                                   s.data_ptr() if keep else None, out.data_ptr(), q.data_ptr(), scale.data_ptr(), stream())
    _lib.check(st, "pmha_rms_norm")
    wq, wscale, ws = pmha.pmha_rms_norm_quantized(x, w, ref.EPS, residual=r)
    # as bits: the sum of a row of 1e38 may be infinite, its scale NaN
    assert torch.equal(q.view(torch.uint8), wq.view(torch.uint8))
    assert torch.equal(scale.view(torch.int32), wscale.view(torch.int32))
    assert not keep or torch.equal(s, ws)
    finite = ws.isfinite().all(-1)
    assert int(finite.sum()) >= 6 and bool(wscale[finite].isfinite().all()) and bool(wscale[~finite].isnan().all())
    out, y = out[finite], ref.norm(ws[finite], w)[0]
    ref.assert_within("out", out, y, 1.01 * (ref.stat_tol(width) + ref.half_ulp(dtype)) * y.abs()
                      + torch.finfo(dtype).smallest_normal)


# on the tensor cores with and without the tokens kept on the chip, padded, few values in float32, float32
@pytest.mark.parametrize("rows,E,F,dtype", [(3000, 128, 200, BF16), (3000, 256, 264, BF16), (2000, 320, 264, BF16),
                                            (5000, 100, 171, BF16), (20, 24, 40, BF16), (300, 33, 65, F32)])
@pytest.mark.parametrize("offset", [0, 1])
def test_single_gradients(rows, E, F, dtype, offset):
    p, x, dy = make(rows, E, F, dtype)
    full = pmha.pmha_ffn_backward(p, x, dy)
    names = ("wg", "wu", "wd", "bg", "bu", "bd")
    lib = _lib.load()
    s = p.as_struct()
    need = lib.pmha_ffn_backward_workspace_size(ctypes.byref(s), rows)
    ws = torch.empty(need, dtype=torch.uint8, device=DEV)
    sets = [(n,) for n in names] + [("wd", "bd"), ("wg", "bu"), ("wu", "wd"), ("bg", "bu", "bd")]
    for some, with_dx in itertools.product(sets, (False, True)):
        ws.fill_(255)  # NaN wherever a value is read before it is written
        g = _lib.PmhaFfnGrads()
        flat = {n: torch.full((full["d" + n].numel() + 8,), 7.0, dtype=dtype, device=DEV) for n in some}
        for n in some:
            setattr(g, n, flat[n].data_ptr() + offset * flat[n].element_size())
        dx = torch.empty_like(x) if with_dx else None
        st = lib.pmha_ffn_backward(ctypes.byref(s), x.data_ptr(), dy.data_ptr(), rows, dx.data_ptr() if with_dx else None,
                                   ctypes.byref(g), ws.data_ptr(), need, stream())
        _lib.check(st, "pmha_ffn_backward")
        pmha.pmha_device_status()
        for n in some:
            want = full["d" + n].flatten()
            assert torch.equal(flat[n][offset:offset + want.numel()], want), (some, n)
            assert bool((flat[n][:offset] == 7).all()) and bool((flat[n][offset + want.numel():] == 7).all())
        assert not with_dx or torch.equal(dx, full["dx"])


def test_clip_without_a_table_of_outputs():
    grads = [torch.randn(n, device=DEV).to(t) for n, t in ((100, F32), (70_001, BF16), (200_000, F32))]
    want = [torch.empty_like(g) for g in grads]
    norm = pmha.pmha_clip_grad_norm(grads, 0.5, out=want)
    lib, n = _lib.load(), len(grads)
    got = torch.empty((), device=DEV)
    need = lib.pmha_clip_grad_norm_workspace_size(n)
    ws = torch.empty(need, dtype=torch.uint8, device=DEV)
    st = lib.pmha_clip_grad_norm(n, (ctypes.c_void_p * n)(*(g.data_ptr() for g in grads)), None,
                                 (ctypes.c_int64 * n)(*(g.numel() for g in grads)),
                                 (ctypes.c_int * n)(*(CODE[g.dtype] for g in grads)), 0.5, got.data_ptr(), ws.data_ptr(),
                                 need, stream())
    _lib.check(st, "pmha_clip_grad_norm")
    assert torch.equal(got, norm) and all(torch.equal(a, b) for a, b in zip(grads, want))
