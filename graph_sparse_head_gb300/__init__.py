"""Edge-packed multi-head attention on GB300 (sm_103a).

Thin Python binding over the C ABI of include/pmha.h. Every step of the layer
runs in the library's CUDA kernels; this module only checks tensor shapes,
passes device pointers and the current torch CUDA stream, and allocates
output / workspace tensors with torch. There is no CPU path: without a built
libpmha.so or without a GPU every call raises.

The layer (kpnn2 0.3.0 API reference, "PackedMultiheadAttention"): each
query token attends only to the key tokens along the live edges
(source_index[e], target_index[e]); scores q_t . k_s / sqrt(d) are
softmaxed over the edges into each target, weight the values, and the heads'
mixes go through out_proj.

Around it stands the rest of an encoder and of its training step: the norm of
the residual sum (pmha_rms_norm), the gated feed-forward block (pmha_ffn_*),
their gradients, clipping by the global norm (pmha_clip_grad_norm), and
PackedEncoderLayer, which runs them together with the layer.
"""
from __future__ import annotations

import contextlib
import ctypes
import dataclasses
import itertools
import operator
import struct

import torch

from . import _lib
from ._lib import (PMHA_ACT_GELU, PMHA_ACT_SILU, PMHA_BF16, PMHA_F32, PMHA_WEIGHTS_AVG, PMHA_WEIGHTS_NONE, PMHA_WEIGHTS_PER_HEAD,
                   PmhaError)

__all__ = [
    "Graph", "Params", "PackedMultiheadAttention", "PmhaError", "pmha_build_csr", "pmha_graph_info",
    "pmha_graph_split_info",
    "pmha_graph_export", "pmha_forward", "pmha_forward_host", "pmha_edge_weights",
    "pmha_forward_workspace_size", "pmha_edge_weights_workspace_size", "pmha_forward_host_workspace_size",
    "pmha_device_status", "pmha_profile_enable", "pmha_profile_read", "pmha_launch_count",
    "pmha_backward", "pmha_backward_workspace_size", "pmha_graph_export_by_source",
    "WMODES",
    "FfnParams", "FfnQuantizedParams", "PackedEncoderLayer", "quantize_rows",
    "pmha_rms_norm", "pmha_rms_norm_quantized", "pmha_rms_norm_backward",
    "pmha_ffn_forward", "pmha_ffn_forward_quantized", "pmha_ffn_backward",
    "pmha_ffn_forward_workspace_size", "pmha_ffn_forward_quantized_workspace_size",
    "pmha_ffn_backward_workspace_size", "pmha_clip_grad_norm",
]

WMODES = {"none": PMHA_WEIGHTS_NONE, "avg": PMHA_WEIGHTS_AVG, "per_head": PMHA_WEIGHTS_PER_HEAD}
_DTYPES = {torch.float32: PMHA_F32, torch.bfloat16: PMHA_BF16}
ACTS = {"silu": PMHA_ACT_SILU, "gelu": PMHA_ACT_GELU}


def _stream_ptr(stream) -> int:
    s = torch.cuda.current_stream() if stream is None else stream
    return int(s.cuda_stream)


def _ptr(t) -> int | None:
    return None if t is None else int(t.data_ptr())


class Graph:
    """A built per-target edge view (owns the library's pmha_graph)."""

    def __init__(self, handle: int, device: torch.device):
        self._h = ctypes.c_void_p(handle)
        self.device = device
        nnz, L, S, md = (ctypes.c_int64() for _ in range(4))
        _lib.check(_lib.load().pmha_graph_info(self._h, ctypes.byref(nnz), ctypes.byref(L), ctypes.byref(S),
                                               ctypes.byref(md)), "pmha_graph_info")
        self.nnz, self.query_features, self.key_features, self.max_in_degree = nnz.value, L.value, S.value, md.value

    @property
    def handle(self) -> ctypes.c_void_p:
        if self._h is None:
            raise RuntimeError("graph was destroyed")
        return self._h

    def destroy(self) -> None:
        if self._h is not None and _lib._lib is not None:
            torch.cuda.synchronize(self.device)
            _lib.load().pmha_graph_destroy(self._h)
        self._h = None

    def __del__(self):
        try:
            self.destroy()
        except Exception:
            pass


@dataclasses.dataclass
class Params:
    """The four projections (q_proj, k_proj, v_proj, out_proj): (E, E) weights
    stored (out, in) and (E,) biases (None for bias=False), on one CUDA device,
    all float32 or all bfloat16."""
    wq: torch.Tensor
    wk: torch.Tensor
    wv: torch.Tensor
    wo: torch.Tensor
    bq: torch.Tensor | None
    bk: torch.Tensor | None
    bv: torch.Tensor | None
    bo: torch.Tensor | None
    num_heads: int

    @property
    def embed_dim(self) -> int:
        return int(self.wq.shape[0])

    @property
    def dtype(self) -> torch.dtype:
        return self.wq.dtype

    def as_struct(self) -> _lib.PmhaParams:
        E = self.embed_dim
        if self.dtype not in _DTYPES:
            raise TypeError(f"parameters must be float32 or bfloat16, not {self.dtype}")
        for n in ("wq", "wk", "wv", "wo"):
            w = getattr(self, n)
            if tuple(w.shape) != (E, E) or w.dtype != self.dtype or not w.is_cuda or not w.is_contiguous():
                raise ValueError(f"{n} must be a contiguous ({E}, {E}) CUDA tensor of dtype {self.dtype}")
        for n in ("bq", "bk", "bv", "bo"):
            b = getattr(self, n)
            if b is not None and (tuple(b.shape) != (E,) or b.dtype != self.dtype or not b.is_cuda
                                  or not b.is_contiguous()):
                raise ValueError(f"{n} must be None or a contiguous ({E},) CUDA tensor of dtype {self.dtype}")
        return _lib.PmhaParams(E, int(self.num_heads), _DTYPES[self.dtype],
                               _ptr(self.wq), _ptr(self.wk), _ptr(self.wv), _ptr(self.wo),
                               _ptr(self.bq), _ptr(self.bk), _ptr(self.bv), _ptr(self.bo))

    @staticmethod
    def from_arrays(arrays: dict, num_heads: int, dtype: torch.dtype, device="cuda") -> "Params":
        def t(x):
            return None if x is None else torch.as_tensor(x).to(device=device, dtype=dtype).contiguous()
        return Params(t(arrays["wq"]), t(arrays["wk"]), t(arrays["wv"]), t(arrays["wo"]),
                      t(arrays.get("bq")), t(arrays.get("bk")), t(arrays.get("bv")), t(arrays.get("bo")),
                      num_heads)


def pmha_build_csr(source_index: torch.Tensor, target_index: torch.Tensor, query_features: int,
                   key_features: int, add_self_loops: bool = False, stream=None) -> Graph:
    """Validate the packed edge index (device int64) and build the per-target view."""
    for n, t in (("source_index", source_index), ("target_index", target_index)):
        if not (isinstance(t, torch.Tensor) and t.is_cuda and t.dtype == torch.int64 and t.dim() == 1):
            raise TypeError(f"{n} must be a 1-D int64 CUDA tensor")
    src, tgt = source_index.contiguous(), target_index.contiguous()
    if src.numel() != tgt.numel():
        raise ValueError("source_index and target_index differ in length")
    out = ctypes.c_void_p()
    with torch.cuda.device(src.device):
        st = _lib.load().pmha_build_csr(_ptr(src), _ptr(tgt), src.numel(), int(query_features), int(key_features),
                                        int(bool(add_self_loops)), _stream_ptr(stream), ctypes.byref(out))
    _lib.check(st, "pmha_build_csr")
    return Graph(out.value, src.device)


def pmha_graph_info(graph: Graph) -> dict:
    return {"nnz": graph.nnz, "query_features": graph.query_features, "key_features": graph.key_features,
            "max_in_degree": graph.max_in_degree}


def pmha_graph_split_info(graph: Graph) -> dict:
    """How the build split the targets: heavy targets (tensor-core path) and the light edges."""
    n, th, ln = (ctypes.c_int64() for _ in range(3))
    _lib.check(_lib.load().pmha_graph_split_info(graph.handle, ctypes.byref(n), ctypes.byref(th), ctypes.byref(ln)),
               "pmha_graph_split_info")
    return {"n_heavy": n.value, "heavy_min_degree": th.value, "light_nnz": ln.value}


def pmha_graph_export(graph: Graph, stream=None):
    """(row_ptr, col, perm) as int32 CUDA tensors."""
    dev = graph.device
    row_ptr = torch.empty(graph.query_features + 1, dtype=torch.int32, device=dev)
    col = torch.empty(graph.nnz, dtype=torch.int32, device=dev)
    perm = torch.empty(graph.nnz, dtype=torch.int32, device=dev)
    _lib.check(_lib.load().pmha_graph_export(graph.handle, _ptr(row_ptr), _ptr(col), _ptr(perm),
                                             _stream_ptr(stream)), "pmha_graph_export")
    return row_ptr, col, perm


def pmha_graph_export_by_source(graph: Graph, stream=None):
    """(src_row_ptr, target) of the per-source view as int32 CUDA tensors."""
    dev = graph.device
    src_row_ptr = torch.empty(graph.key_features + 1, dtype=torch.int32, device=dev)
    target = torch.empty(graph.nnz, dtype=torch.int32, device=dev)
    _lib.check(_lib.load().pmha_graph_export_by_source(graph.handle, _ptr(src_row_ptr), _ptr(target),
                                                       _stream_ptr(stream)), "pmha_graph_export_by_source")
    return src_row_ptr, target


def pmha_forward_workspace_size(graph: Graph, params: Params, batch: int, wmode: str = "none") -> int:
    p = params.as_struct()
    return int(_lib.load().pmha_forward_workspace_size(graph.handle, ctypes.byref(p), int(batch), WMODES[wmode]))


def pmha_edge_weights_workspace_size(graph: Graph, params: Params, batch: int, wmode: str = "avg") -> int:
    p = params.as_struct()
    return int(_lib.load().pmha_edge_weights_workspace_size(graph.handle, ctypes.byref(p), int(batch),
                                                            WMODES[wmode]))


def pmha_forward_host_workspace_size(graph: Graph, params: Params, batch: int, wmode: str = "none") -> int:
    p = params.as_struct()
    return int(_lib.load().pmha_forward_host_workspace_size(graph.handle, ctypes.byref(p), int(batch),
                                                            WMODES[wmode]))


def _workspace(nbytes: int, device, workspace):
    if workspace is not None:
        if not isinstance(workspace, torch.Tensor) or workspace.device != device or not workspace.is_contiguous():
            raise ValueError(f"workspace must be a contiguous tensor on {device}")
        if workspace.numel() * workspace.element_size() < nbytes:
            raise ValueError(f"workspace holds fewer than the {nbytes} bytes needed")
        return workspace
    return torch.empty(max(nbytes, 1), dtype=torch.uint8, device=device)


def _check_dest(name, t, shape, dtype, device):
    """A result tensor the caller supplies: exactly `shape` and `dtype`,
    contiguous, on `device` (None: a host tensor). The kernels write it whole,
    so anything smaller or strided is refused before a launch."""
    if not isinstance(t, torch.Tensor) or tuple(t.shape) != tuple(shape) or t.dtype != dtype \
            or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {tuple(shape)} tensor of {dtype}")
    if device is None:
        if t.is_cuda:
            raise ValueError(f"{name} must be a host tensor here")
    elif t.device != device:
        raise ValueError(f"{name} must live on {device}")


def _check_placement(graph, params, device):
    """The graph and every parameter tensor on the device of the call."""
    if graph.device != device:
        raise ValueError(f"the graph was built on {graph.device}, the call runs on {device}")
    for n in ("wq", "wk", "wv", "wo", "bq", "bk", "bv", "bo"):
        t = getattr(params, n)
        if t is not None and t.device != device:
            raise ValueError(f"parameter {n} lives on {t.device}, the call runs on {device}")


def _check_tokens(name, x, batch, seq, E, dtype, device):
    if not isinstance(x, torch.Tensor) or x.dim() != 3 or tuple(x.shape) != (batch, seq, E):
        raise ValueError(f"{name} must have shape ({batch}, {seq}, {E})")
    if x.dtype != dtype or x.device != device or not x.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor on {device}")


def _check_mask(mask, batch, S, on_device, device=None):
    """key_padding_mask: None, or a contiguous (B, S) bool / uint8 tensor (nonzero = key dropped)."""
    if mask is None:
        return None
    if not isinstance(mask, torch.Tensor) or tuple(mask.shape) != (batch, S) or \
            mask.dtype not in (torch.bool, torch.uint8) or not mask.is_contiguous():
        raise ValueError(f"key_padding_mask must be a contiguous ({batch}, {S}) bool or uint8 tensor")
    if on_device and mask.device != device:
        raise ValueError(f"key_padding_mask must live on {device}")
    if not on_device and mask.is_cuda:
        raise ValueError("key_padding_mask must be a host tensor here")
    return _ptr(mask)


def _weights_shape(graph, batch, H, wmode):
    return (batch, graph.nnz) if wmode == "avg" else (batch, graph.nnz, H)


def pmha_forward(graph: Graph, params: Params, query: torch.Tensor, key: torch.Tensor, value: torch.Tensor,
                 wmode: str = "none", out: torch.Tensor | None = None, weights: torch.Tensor | None = None,
                 workspace: torch.Tensor | None = None, stream=None, key_padding_mask: torch.Tensor | None = None,
                 check: bool = False):
    """One forward pass on device tensors: query (B, L, E), key / value (B, S, E),
    key_padding_mask (B, S) bool (True = key dropped) or None.
    Returns (output (B, L, E), weights or None). The call returns once the work
    is queued; check=True waits for it and raises what the kernels flagged (for
    bfloat16 layers: an fp16 intermediate out of range, i.e. invalid outputs)."""
    B = int(query.shape[0])
    E, H = params.embed_dim, int(params.num_heads)
    dev = query.device
    _check_tokens("query", query, B, graph.query_features, E, params.dtype, dev)
    _check_tokens("key", key, B, graph.key_features, E, params.dtype, dev)
    _check_tokens("value", value, B, graph.key_features, E, params.dtype, dev)
    mp = _check_mask(key_padding_mask, B, graph.key_features, True, dev)
    _check_placement(graph, params, dev)
    p = params.as_struct()
    lib = _lib.load()
    wm = WMODES[wmode]
    if out is None:
        out = torch.empty_like(query)
    else:
        _check_dest("out", out, (B, graph.query_features, E), params.dtype, dev)
    if wm != PMHA_WEIGHTS_NONE:
        if weights is None:
            weights = torch.empty(_weights_shape(graph, B, H, wmode), dtype=torch.float32, device=dev)
        else:
            _check_dest("weights", weights, _weights_shape(graph, B, H, wmode), torch.float32, dev)
    need = lib.pmha_forward_workspace_size(graph.handle, ctypes.byref(p), B, wm)
    if need == 0:
        _lib.check(_lib.PMHA_OK + 1, "pmha_forward_workspace_size")
    ws = _workspace(need, dev, workspace)
    with torch.cuda.device(dev):
        st = lib.pmha_forward(graph.handle, ctypes.byref(p), _ptr(query), _ptr(key), _ptr(value), mp, B, _ptr(out), wm,
                              _ptr(weights) if wm != PMHA_WEIGHTS_NONE else None, _ptr(ws),
                              ws.numel() * ws.element_size(), _stream_ptr(stream))
    _lib.check(st, "pmha_forward")
    if check:
        with torch.cuda.device(dev):
            pmha_device_status(stream)
    return out, (weights if wm != PMHA_WEIGHTS_NONE else None)


def pmha_forward_host(graph: Graph, params: Params, query: torch.Tensor, key: torch.Tensor, value: torch.Tensor,
                      out: torch.Tensor, wmode: str = "none", weights: torch.Tensor | None = None,
                      workspace: torch.Tensor | None = None, stream=None, device=None,
                      key_padding_mask: torch.Tensor | None = None):
    """Forward pass on HOST tensors (pinned for asynchronous copies): the library
    copies the inputs in, runs the layer and copies out (and weights) back, all
    on the stream. Synchronize the stream before reading `out`."""
    B = int(query.shape[0])
    dev = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
    if dev.type == "cuda" and dev.index is None:
        dev = torch.device("cuda", torch.cuda.current_device())
    E, H = params.embed_dim, int(params.num_heads)
    for n, x, seq in (("query", query, graph.query_features), ("key", key, graph.key_features),
                      ("value", value, graph.key_features), ("out", out, graph.query_features)):
        if x.is_cuda or tuple(x.shape) != (B, seq, E) or x.dtype != params.dtype or not x.is_contiguous():
            raise ValueError(f"{n} must be a contiguous host tensor ({B}, {seq}, {E}) of {params.dtype}")
    mp = _check_mask(key_padding_mask, B, graph.key_features, False)
    _check_placement(graph, params, dev)
    wm = WMODES[wmode]
    if wm != PMHA_WEIGHTS_NONE and weights is not None:
        _check_dest("weights", weights, _weights_shape(graph, B, H, wmode), torch.float32, None)
    p = params.as_struct()
    lib = _lib.load()
    need = lib.pmha_forward_host_workspace_size(graph.handle, ctypes.byref(p), B, wm)
    ws = _workspace(need, dev, workspace)
    with torch.cuda.device(dev):
        st = lib.pmha_forward_host(graph.handle, ctypes.byref(p), _ptr(query), _ptr(key), _ptr(value), mp, B,
                                   _ptr(out),
                                   wm, _ptr(weights) if wm != PMHA_WEIGHTS_NONE else None, _ptr(ws),
                                   ws.numel() * ws.element_size(), _stream_ptr(stream))
    _lib.check(st, "pmha_forward_host")
    return out, weights


def pmha_edge_weights(graph: Graph, params: Params, query: torch.Tensor, key: torch.Tensor, wmode: str = "avg",
                      weights: torch.Tensor | None = None, workspace: torch.Tensor | None = None, stream=None,
                      key_padding_mask: torch.Tensor | None = None):
    """Per-edge softmax weights only (no value projection, mix or out_proj)."""
    B = int(query.shape[0])
    E, H = params.embed_dim, int(params.num_heads)
    dev = query.device
    _check_tokens("query", query, B, graph.query_features, E, params.dtype, dev)
    _check_tokens("key", key, B, graph.key_features, E, params.dtype, dev)
    if wmode not in ("avg", "per_head"):
        raise ValueError("wmode must be 'avg' or 'per_head'")
    mp = _check_mask(key_padding_mask, B, graph.key_features, True, dev)
    _check_placement(graph, params, dev)
    p = params.as_struct()
    lib = _lib.load()
    wm = WMODES[wmode]
    if weights is None:
        weights = torch.empty(_weights_shape(graph, B, H, wmode), dtype=torch.float32, device=dev)
    else:
        _check_dest("weights", weights, _weights_shape(graph, B, H, wmode), torch.float32, dev)
    need = lib.pmha_edge_weights_workspace_size(graph.handle, ctypes.byref(p), B, wm)
    ws = _workspace(need, dev, workspace)
    with torch.cuda.device(dev):
        st = lib.pmha_edge_weights(graph.handle, ctypes.byref(p), _ptr(query), _ptr(key), mp, B, wm, _ptr(weights),
                                   _ptr(ws), ws.numel() * ws.element_size(), _stream_ptr(stream))
    _lib.check(st, "pmha_edge_weights")
    return weights


def pmha_backward_workspace_size(graph: Graph, params: Params, batch: int) -> int:
    p = params.as_struct()
    return int(_lib.load().pmha_backward_workspace_size(graph.handle, ctypes.byref(p), int(batch)))


def pmha_backward(graph: Graph, params: Params, query: torch.Tensor, key: torch.Tensor, value: torch.Tensor,
                  dout: torch.Tensor, key_padding_mask: torch.Tensor | None = None, input_grads: bool = True,
                  param_grads: bool = True, workspace: torch.Tensor | None = None, stream=None) -> dict:
    """Gradients of the layer for dout = dLoss/d(output): recomputes the forward
    from (query, key, value) and returns {"dquery", "dkey", "dvalue"} in the layer
    dtype (one shared tensor when inputs are one tensor, holding the sum) and
    {"dwq", "dwk", "dwv", "dwo", "dbq", "dbk", "dbv", "dbo"} in float32 (None
    for biases the layer does not have)."""
    B = int(query.shape[0])
    E = params.embed_dim
    dev = query.device
    _check_tokens("query", query, B, graph.query_features, E, params.dtype, dev)
    _check_tokens("key", key, B, graph.key_features, E, params.dtype, dev)
    _check_tokens("value", value, B, graph.key_features, E, params.dtype, dev)
    _check_tokens("dout", dout, B, graph.query_features, E, params.dtype, dev)
    mp = _check_mask(key_padding_mask, B, graph.key_features, True, dev)
    _check_placement(graph, params, dev)
    p = params.as_struct()
    lib = _lib.load()
    out = {}
    gx = [None, None, None]
    if input_grads:
        made = {}
        for i, (name, x) in enumerate((("dquery", query), ("dkey", key), ("dvalue", value))):
            if x.data_ptr() not in made:
                made[x.data_ptr()] = torch.empty_like(x)
            out[name] = made[x.data_ptr()]
            gx[i] = _ptr(out[name])
    g = _lib.PmhaGrads()
    if param_grads:
        for n in ("wq", "wk", "wv", "wo"):
            out["d" + n] = torch.empty((E, E), dtype=torch.float32, device=dev)
            setattr(g, n, _ptr(out["d" + n]))
        for n in ("bq", "bk", "bv", "bo"):
            if getattr(params, n) is None:
                out["d" + n] = None
            else:
                out["d" + n] = torch.empty(E, dtype=torch.float32, device=dev)
                setattr(g, n, _ptr(out["d" + n]))
    need = lib.pmha_backward_workspace_size(graph.handle, ctypes.byref(p), B)
    if need == 0:
        _lib.check(_lib.PMHA_OK + 5, "pmha_backward_workspace_size (unsupported shape)")
    ws = _workspace(need, dev, workspace)
    with torch.cuda.device(dev):
        st = lib.pmha_backward(graph.handle, ctypes.byref(p), _ptr(query), _ptr(key), _ptr(value), mp, B, _ptr(dout),
                               gx[0], gx[1], gx[2], ctypes.byref(g), _ptr(ws), ws.numel() * ws.element_size(),
                               _stream_ptr(stream))
    _lib.check(st, "pmha_backward")
    return out


def pmha_device_status(stream=None) -> None:
    """Synchronize the stream; raise if a kernel flagged a condition since the last
    check: a bounded device-side wait gave up, or an fp16 intermediate overflowed."""
    _lib.check(_lib.load().pmha_device_status(_stream_ptr(stream)), "pmha_device_status")


def pmha_profile_enable(on: bool = True) -> None:
    _lib.check(_lib.load().pmha_profile_enable(int(bool(on))), "pmha_profile_enable")


def pmha_profile_read() -> dict:
    """{stage: (launches, total_ms)} since the last read."""
    n_max = 256  # the library has some 50 stages
    names = ctypes.create_string_buffer(32 * n_max)
    launches = (ctypes.c_int64 * n_max)()
    totals = (ctypes.c_double * n_max)()
    n = ctypes.c_int()
    _lib.check(_lib.load().pmha_profile_read(n_max, names, launches, totals, ctypes.byref(n)), "pmha_profile_read")
    out = {}
    for i in range(min(n.value, n_max)):
        name = names.raw[32 * i:32 * i + 32].split(b"\0", 1)[0].decode()
        out[name] = (int(launches[i]), float(totals[i]))
    return out


def pmha_launch_count() -> int:
    return int(_lib.load().pmha_launch_count())


class PackedMultiheadAttention:
    """The layer as one object: a built graph plus parameters, called like
    kpnn2's PackedMultiheadAttention.forward on batch-first device tensors:
    ``out, w = layer(query, key, value, key_padding_mask=None, need_weights=False,
    average_attn_weights=True)``.
    Reuses one workspace tensor across calls on the current stream."""

    def __init__(self, source_index, target_index, query_features: int, key_features: int, params: Params,
                 add_self_loops: bool = False, device="cuda"):
        dev = torch.device(device)
        src = torch.as_tensor(source_index, dtype=torch.int64).to(dev)
        tgt = torch.as_tensor(target_index, dtype=torch.int64).to(dev)
        self.graph = pmha_build_csr(src, tgt, query_features, key_features, add_self_loops)
        self.params = params
        self.num_heads = params.num_heads
        self.embed_dim = params.embed_dim
        self.nnz = self.graph.nnz
        self._ws = None

    def __call__(self, query, key, value, key_padding_mask=None, need_weights: bool = False,
                 average_attn_weights: bool = True):
        wmode = "none" if not need_weights else ("avg" if average_attn_weights else "per_head")
        B = int(query.shape[0])
        need = pmha_forward_workspace_size(self.graph, self.params, B, wmode)
        if self._ws is None or self._ws.numel() < need:
            self._ws = torch.empty(need, dtype=torch.uint8, device=query.device)
        return pmha_forward(self.graph, self.params, query, key, value, wmode, workspace=self._ws,
                            key_padding_mask=key_padding_mask)


# ---------------------------------------------------------------- the encoder around the layer
# These calls are short on the GPU (a norm of a small batch takes 4 us), so the
# checks in front of them are written for few Python operations.
_HERE = contextlib.nullcontext()
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)  # the pointer alone, without a Stream object
_T = torch.Tensor


def _on(index, stream):
    """Runs a call on `stream` of device `index`: what is allocated inside
    belongs to that stream, so that its memory is not handed out again before
    the stream has passed the call."""
    if stream is not None:
        if stream.device.index != index:
            raise ValueError(f"the stream belongs to {stream.device}, the call runs on cuda:{index}")
        return torch.cuda.stream(stream)
    return _HERE if torch.cuda.current_device() == index else torch.cuda.device(index)


def _stream_of(index, stream) -> int:
    if stream is not None:
        return stream.cuda_stream
    return _raw_stream(index) if _raw_stream is not None else torch.cuda.current_stream(index).cuda_stream


def _library():
    return _lib._lib if _lib._lib is not None else _lib.load()


def _rows_of(name, x, dtype=None):
    """(shape, rows, width, device index) of a contiguous CUDA tensor (..., width)."""
    if not isinstance(x, _T) or not x.is_cuda or not x.is_contiguous() or not x.dim() \
            or (x.dtype not in _DTYPES if dtype is None else x.dtype is not dtype):
        raise ValueError(f"{name} must be a contiguous CUDA tensor (..., width) of "
                         f"{'float32 or bfloat16' if dtype is None else dtype}")
    shape = x.shape
    width = shape[-1]
    return shape, x.numel() // width if width else 0, width, x.get_device()


def _like(name, t, shape, dtype, index):
    """Pointer of a contiguous tensor of this shape, type and device (None: none)."""
    if t is None:
        return None
    if not isinstance(t, _T) or t.shape != shape or t.dtype is not dtype or t.get_device() != index \
            or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {tuple(shape)} tensor of {dtype} on cuda:{index}")
    return t.data_ptr()


def pmha_rms_norm(x: torch.Tensor, weight: torch.Tensor | None, eps: float, residual: torch.Tensor | None = None,
                  out: torch.Tensor | None = None, stream=None):
    """Root-mean-square norm over the last axis of s = x + residual:
    s / sqrt(mean(s^2) + eps) * weight. Returns (out, s), s rounded to x's type
    as the norm takes it, or (out, None) without a residual."""
    shape, rows, width, dev = _rows_of("x", x)
    dtype = x.dtype
    w = _like("weight", weight, (width,), dtype, dev)
    r = _like("residual", residual, shape, dtype, dev)
    o = _like("out", out, shape, dtype, dev)
    with _on(dev, stream):
        if out is None:
            out = torch.empty_like(x)
            o = out.data_ptr()
        s = None if residual is None else torch.empty_like(x)
        st = _library().pmha_rms_norm(_DTYPES[dtype], rows, width, x.data_ptr(), r, w, eps,
                                      None if s is None else s.data_ptr(), o, None, None, _stream_of(dev, stream))
    if st:
        _lib.check(st, "pmha_rms_norm")
    return out, s


def pmha_rms_norm_quantized(x: torch.Tensor, weight: torch.Tensor | None, eps: float,
                            residual: torch.Tensor | None = None, stream=None):
    """pmha_rms_norm with its output in 8 bits: (q, scale, s) with q in
    float8_e4m3fn, scale (...,) float32, norm ~ q * scale[..., None]; every q is
    the formula's value, computed to some 46 bits and rounded once. What pmha_ffn_forward_quantized takes."""
    shape, rows, width, dev = _rows_of("x", x)
    dtype = x.dtype
    w = _like("weight", weight, (width,), dtype, dev)
    r = _like("residual", residual, shape, dtype, dev)
    with _on(dev, stream):
        q = torch.empty_like(x, dtype=torch.float8_e4m3fn)
        scale = torch.empty(shape[:-1], dtype=torch.float32, device=x.device)
        s = None if residual is None else torch.empty_like(x)
        st = _library().pmha_rms_norm(_DTYPES[dtype], rows, width, x.data_ptr(), r, w, eps,
                                      None if s is None else s.data_ptr(), None, q.data_ptr(), scale.data_ptr(),
                                      _stream_of(dev, stream))
    if st:
        _lib.check(st, "pmha_rms_norm")
    return q, scale, s


def pmha_rms_norm_backward(x: torch.Tensor, weight: torch.Tensor | None, eps: float, dout: torch.Tensor,
                           dsum: torch.Tensor | None = None, input_grad: bool = True, param_grad: bool = True,
                           stream=None) -> dict:
    """Gradients of the norm of x (with a residual: of the sum that pmha_rms_norm
    returned): {"dx", "dweight"}; dx, in x's type, is the gradient of both
    summands and includes dsum, the sum's gradient from its other uses; dweight
    is float32 (None without a weight)."""
    shape, rows, width, dev = _rows_of("x", x)
    dtype = x.dtype
    w = _like("weight", weight, (width,), dtype, dev)
    dy = _like("dout", dout, shape, dtype, dev)
    if dout is None:
        raise ValueError("dout is missing")
    ds = _like("dsum", dsum, shape, dtype, dev)
    lib = _library()
    with _on(dev, stream):
        dx = torch.empty_like(x) if input_grad else None
        dw = ws = None
        need = 0
        if param_grad and weight is not None:
            dw = torch.empty(width, dtype=torch.float32, device=x.device)
            need = lib.pmha_rms_norm_backward_workspace_size(_DTYPES[dtype], rows, width)
            ws = torch.empty(need, dtype=torch.uint8, device=x.device)
        st = lib.pmha_rms_norm_backward(_DTYPES[dtype], rows, width, x.data_ptr(), w, eps, dy, ds, _ptr(dx), _ptr(dw),
                                        _ptr(ws), need, _stream_of(dev, stream))
    if st:
        _lib.check(st, "pmha_rms_norm_backward")
    return {"dx": dx, "dweight": dw}


def _table(code, values):
    """A host array for the library (the format's C type, one of each value)."""
    return struct.pack(f"{len(values)}{code}", *values)


_dtype_of = operator.attrgetter("dtype")


def pmha_clip_grad_norm(grads, max_norm: float, out=None, stream=None) -> torch.Tensor:
    """Scales the gradients (an iterable of contiguous float32 / bfloat16 CUDA
    tensors of one device; None entries are skipped) by
    min(1, max_norm / (norm + 1e-6)), norm the 2-norm of all their values, and
    returns the norm before scaling as a float32 scalar on the device. In place,
    or into the tensors of `out` (one for each gradient, same type and number of
    values)."""
    grads = list(grads)
    outs = grads if out is None else list(out)
    if len(outs) != len(grads):
        raise ValueError("out must have one tensor for each gradient")
    if any(map(operator.is_, grads, itertools.repeat(None))):
        keep = [i for i, g in enumerate(grads) if g is not None]
        grads, outs = [grads[i] for i in keep], outs if out is None else [outs[i] for i in keep]
        if out is None:
            outs = grads
    if not grads:
        raise ValueError("no gradients: the call needs a tensor to know its device")
    n = len(grads)
    # each step is one pass of a C-level map over the tensors: a stack of layers has hundreds
    gp = op = list(map(_T.data_ptr, grads))  # TypeError for what is no tensor
    sizes = list(map(_T.numel, grads))
    types = list(map(_dtype_of, grads))
    devices = set(map(_T.get_device, grads))
    dense = all(map(_T.is_contiguous, grads))
    if out is not None:
        op = list(map(_T.data_ptr, outs))
        devices.update(map(_T.get_device, outs))
        dense = dense and all(map(_T.is_contiguous, outs))
        if list(map(_T.numel, outs)) != sizes or list(map(_dtype_of, outs)) != types:
            raise ValueError("each output must have its gradient's type and number of values")
    if not dense or len(devices) > 1 or -1 in devices:
        raise ValueError("gradients and outputs must be contiguous CUDA tensors on one device")
    bf16 = torch.bfloat16
    if types.count(torch.float32) + types.count(bf16) != n:
        raise TypeError("gradients must be float32 or bfloat16")
    kinds = _table("i", [PMHA_BF16 if t is bf16 else PMHA_F32 for t in types])
    gt = _table("q", gp)
    dev = devices.pop()
    lib = _library()
    need = lib.pmha_clip_grad_norm_workspace_size(n)
    with _on(dev, stream):
        device = grads[0].device
        norm = torch.empty((), dtype=torch.float32, device=device)
        ws = torch.empty(need, dtype=torch.uint8, device=device)
        st = lib.pmha_clip_grad_norm(n, gt, gt if op is gp else _table("q", op), _table("q", sizes), kinds, max_norm,
                                     norm.data_ptr(), ws.data_ptr(), need, _stream_of(dev, stream))
    if st:
        _lib.check(st, "pmha_clip_grad_norm")
    return norm


def _ffn_struct(p, dtype):
    """Checks a block's tensors and lists them for the library; dtype: of its gate and up weights (None: wd's)."""
    wd = p.wd
    if not isinstance(wd, _T) or wd.dim() != 2 or wd.dtype not in _DTYPES or not wd.is_cuda or not wd.is_contiguous():
        raise ValueError("wd must be a contiguous (E, F) CUDA tensor of float32 or bfloat16")
    E, F = wd.shape
    t, dev = wd.dtype, wd.get_device()
    act = ACTS.get(p.act)
    if act is None:
        raise ValueError(f"act must be one of {sorted(ACTS)}")
    g = _like("wg", p.wg, (F, E), dtype or t, dev)
    u = _like("wu", p.wu, (F, E), dtype or t, dev)
    if g is None or u is None:
        raise ValueError("wg and wu are missing")
    return _lib.PmhaFfnParams(E, F, _DTYPES[t], act, None if dtype else g, None if dtype else u, wd.data_ptr(),
                              _like("bg", p.bg, (F,), t, dev), _like("bu", p.bu, (F,), t, dev),
                              _like("bd", p.bd, (E,), t, dev))


@dataclasses.dataclass
class FfnParams:
    """A gated feed-forward block, (act(x wg^T + bg) * (x wu^T + bu)) wd^T + bd:
    wg, wu (F, E) and wd (E, F) stored (out, in), biases (F,), (F,), (E,) or None,
    all float32 or all bfloat16 on one CUDA device; act "silu" or "gelu" (erf)."""
    wg: torch.Tensor
    wu: torch.Tensor
    wd: torch.Tensor
    bg: torch.Tensor | None = None
    bu: torch.Tensor | None = None
    bd: torch.Tensor | None = None
    act: str = "silu"

    def as_struct(self) -> _lib.PmhaFfnParams:
        return _ffn_struct(self, None)


@dataclasses.dataclass
class FfnQuantizedParams:
    """A bfloat16 block whose gate and up weights are float8_e4m3fn with one
    float32 scale for each of their F rows (quantize_rows makes them)."""
    wg: torch.Tensor
    wg_scale: torch.Tensor
    wu: torch.Tensor
    wu_scale: torch.Tensor
    wd: torch.Tensor
    bg: torch.Tensor | None = None
    bu: torch.Tensor | None = None
    bd: torch.Tensor | None = None
    act: str = "silu"

    def as_struct(self) -> _lib.PmhaFfnParams:
        return _ffn_struct(self, torch.float8_e4m3fn)

    def quantized_struct(self) -> _lib.PmhaFfnQuantized:
        F, dev = self.wg.shape[0], self.wd.get_device()
        gs = _like("wg_scale", self.wg_scale, (F,), torch.float32, dev)
        us = _like("wu_scale", self.wu_scale, (F,), torch.float32, dev)
        if gs is None or us is None:
            raise ValueError("wg_scale and wu_scale are missing")
        return _lib.PmhaFfnQuantized(self.wg.data_ptr(), self.wu.data_ptr(), gs, us)

    @staticmethod
    def from_params(params: FfnParams) -> "FfnQuantizedParams":
        """The block with its gate and up weights quantized, once, when a model is loaded."""
        return FfnQuantizedParams(*quantize_rows(params.wg), *quantize_rows(params.wu), params.wd, params.bg,
                                  params.bu, params.bd, params.act)


def quantize_rows(w: torch.Tensor):
    """(q, scale) of a weight matrix: q float8_e4m3fn, scale float32 a row,
    max|row| / 448 (at least 2^-64), w ~ q * scale[:, None]. A step of loading a
    model, in torch operations; tokens are quantized by pmha_rms_norm_quantized."""
    f = w.float()
    scale = (f.abs().amax(-1) / 448.0).clamp_min(2.0 ** -64)
    return (f / scale[..., None]).clamp(-448.0, 448.0).to(torch.float8_e4m3fn), scale


_NO_SIZE = ctypes.c_size_t(-1).value


def _ffn_size(fn, p, rows, where) -> int:
    need = fn(ctypes.byref(p), rows)
    if need == _NO_SIZE:  # the size functions make the checks of their calls
        message = (_lib.load().pmha_last_error() or b"").decode()
        raise PmhaError(5 if "must be a multiple" in message else 1, where, message)
    return need


def pmha_ffn_forward_workspace_size(params: FfnParams, rows: int) -> int:
    return _ffn_size(_library().pmha_ffn_forward_workspace_size, params.as_struct(), int(rows), "pmha_ffn_forward")


def pmha_ffn_forward_quantized_workspace_size(params: FfnQuantizedParams, rows: int) -> int:
    return _ffn_size(_library().pmha_ffn_forward_quantized_workspace_size, params.as_struct(), int(rows),
                     "pmha_ffn_forward_quantized")


def pmha_ffn_backward_workspace_size(params: FfnParams, rows: int) -> int:
    return _ffn_size(_library().pmha_ffn_backward_workspace_size, params.as_struct(), int(rows), "pmha_ffn_backward")


def _ffn_tokens(name, x, p, wd, dtype):
    shape, rows, width, dev = _rows_of(name, x, dtype)
    if width != p.embed_dim or dev != wd.get_device():
        raise ValueError(f"{name} must be (..., {p.embed_dim}) on {wd.device}")
    return shape, rows, dev


def _scratch(x, need, workspace):
    """(pointer, bytes, the tensor to keep) of the workspace, the caller's or a new one."""
    if workspace is not None:
        ws = _workspace(need, x.device, workspace)
        return ws.data_ptr(), ws.numel() * ws.element_size(), ws
    if not need:
        return None, 0, None
    ws = torch.empty(need, dtype=torch.uint8, device=x.device)  # half of new_empty's host time
    return ws.data_ptr(), need, ws


def pmha_ffn_forward(params: FfnParams, x: torch.Tensor, residual: torch.Tensor | None = None,
                     out: torch.Tensor | None = None, workspace: torch.Tensor | None = None, stream=None):
    """The gated feed-forward block on tokens x (..., E), plus the residual."""
    p = params.as_struct()
    dtype = params.wd.dtype
    shape, rows, dev = _ffn_tokens("x", x, p, params.wd, dtype)
    r = _like("residual", residual, shape, dtype, dev)
    o = _like("out", out, shape, dtype, dev)
    lib = _library()
    need = _ffn_size(lib.pmha_ffn_forward_workspace_size, p, rows, "pmha_ffn_forward")
    with _on(dev, stream):
        if out is None:
            out = torch.empty_like(x)
            o = out.data_ptr()
        wp, wn, keep = _scratch(x, need, workspace)
        st = lib.pmha_ffn_forward(ctypes.byref(p), x.data_ptr(), r, rows, o, wp, wn, _stream_of(dev, stream))
    if st:
        _lib.check(st, "pmha_ffn_forward")
    return out


def pmha_ffn_forward_quantized(params: FfnQuantizedParams, x: torch.Tensor, x_scale: torch.Tensor,
                               residual: torch.Tensor | None = None, out: torch.Tensor | None = None,
                               workspace: torch.Tensor | None = None, stream=None):
    """pmha_ffn_forward for tokens in float8_e4m3fn with a float32 scale each (what
    pmha_rms_norm_quantized returns) and a quantized block; residual and result
    are bfloat16."""
    p, q = params.as_struct(), params.quantized_struct()
    dtype = params.wd.dtype
    shape, rows, dev = _ffn_tokens("x", x, p, params.wd, torch.float8_e4m3fn)
    xs = _like("x_scale", x_scale, shape[:-1], torch.float32, dev)
    if xs is None:
        raise ValueError("x_scale is missing")
    r = _like("residual", residual, shape, dtype, dev)
    o = _like("out", out, shape, dtype, dev)
    lib = _library()
    need = _ffn_size(lib.pmha_ffn_forward_quantized_workspace_size, p, rows, "pmha_ffn_forward_quantized")
    with _on(dev, stream):
        if out is None:
            out = torch.empty_like(x, dtype=dtype)
            o = out.data_ptr()
        wp, wn, keep = _scratch(x, need, workspace)
        st = lib.pmha_ffn_forward_quantized(ctypes.byref(p), ctypes.byref(q), x.data_ptr(), xs, r, rows, o, wp, wn,
                                            _stream_of(dev, stream))
    if st:
        _lib.check(st, "pmha_ffn_forward_quantized")
    return out


def pmha_ffn_backward(params: FfnParams, x: torch.Tensor, dout: torch.Tensor, input_grads: bool = True,
                      param_grads: bool = True, workspace: torch.Tensor | None = None, stream=None) -> dict:
    """Gradients of the block for dout = dLoss/d(block(x)), the hidden rows
    recomputed from x: {"dx", "dwg", "dwu", "dwd", "dbg", "dbu", "dbd"} in the
    block's type (None for biases it does not have). A residual's gradient is
    dout itself."""
    p = params.as_struct()
    dtype = params.wd.dtype
    shape, rows, dev = _ffn_tokens("x", x, p, params.wd, dtype)
    dy = _like("dout", dout, shape, dtype, dev)
    if dout is None:
        raise ValueError("dout is missing")
    lib = _library()
    need = _ffn_size(lib.pmha_ffn_backward_workspace_size, p, rows, "pmha_ffn_backward")
    out = {}
    g = _lib.PmhaFfnGrads()
    with _on(dev, stream):
        dx = None
        if input_grads:
            out["dx"] = dx = torch.empty_like(x)
        if param_grads:
            for n in ("wg", "wu", "wd", "bg", "bu", "bd"):
                t = getattr(params, n)
                out["d" + n] = d = None if t is None else torch.empty_like(t)
                if d is not None:
                    setattr(g, n, d.data_ptr())
        wp, wn, keep = _scratch(x, need, workspace)
        st = lib.pmha_ffn_backward(ctypes.byref(p), x.data_ptr(), dy, rows, _ptr(dx), ctypes.byref(g), wp, wn,
                                   _stream_of(dev, stream))
    if st:
        _lib.check(st, "pmha_ffn_backward")
    return out


class PackedEncoderLayer:
    """One pre-norm encoder layer around the packed attention, on tokens
    x (B, n, E) of one graph with query_features == key_features:

        a = attention(norm1(x));  s = x + a;  y = s + block(norm2(s))

    ``layer(x)`` runs it (residual and norm2 in one pass over the tokens);
    ``layer.backward(x, dy)`` returns the gradients of x and of every parameter
    for dy = dLoss/dy, recomputing the forward pass; ``layer.clip_grads`` scales
    them by their global norm."""

    def __init__(self, graph: Graph, attention: Params, norm1: torch.Tensor, norm2: torch.Tensor, block: FfnParams,
                 eps: float = 1e-6):
        if graph.query_features != graph.key_features:
            raise ValueError("an encoder layer needs a graph with query_features == key_features")
        if not isinstance(block, FfnParams):
            raise TypeError("block must be FfnParams (the layer has a backward pass; a block in 8 bits is called beside it)")
        E = attention.embed_dim
        for n, t in (("norm1", norm1), ("norm2", norm2)):
            _like(n, t, (E,), attention.dtype, attention.wq.get_device())
        if block.wd.dtype != attention.dtype or block.wd.shape[0] != E:
            raise ValueError(f"the block must have width {E} and type {attention.dtype}")
        block.as_struct()  # checks its tensors
        self.graph, self.attention, self.block = graph, attention, block
        self.norm1, self.norm2, self.eps = norm1, norm2, float(eps)

    def _attend(self, x, key_padding_mask):
        n1, _ = pmha_rms_norm(x, self.norm1, self.eps)
        a, _ = pmha_forward(self.graph, self.attention, n1, n1, n1, key_padding_mask=key_padding_mask)
        n2, s = pmha_rms_norm(a, self.norm2, self.eps, residual=x)
        return n1, s, n2

    def __call__(self, x: torch.Tensor, key_padding_mask: torch.Tensor | None = None) -> torch.Tensor:
        _, s, n2 = self._attend(x, key_padding_mask)
        return pmha_ffn_forward(self.block, n2, residual=s)

    def backward(self, x: torch.Tensor, dy: torch.Tensor, key_padding_mask: torch.Tensor | None = None) -> dict:
        """{"dx", "dnorm1", "dnorm2", and the keys of pmha_backward's and
        pmha_ffn_backward's parameter gradients}."""
        n1, s, n2 = self._attend(x, key_padding_mask)
        gb = pmha_ffn_backward(self.block, n2, dy)
        g2 = pmha_rms_norm_backward(s, self.norm2, self.eps, gb.pop("dx"), dsum=dy)
        ds = g2["dx"]  # of x and of the attention's output
        ga = pmha_backward(self.graph, self.attention, n1, n1, n1, ds, key_padding_mask=key_padding_mask)
        dn1 = ga.pop("dquery")  # one tensor: the sum over the three roles
        del ga["dkey"], ga["dvalue"]
        g1 = pmha_rms_norm_backward(x, self.norm1, self.eps, dn1, dsum=ds)
        return {"dx": g1["dx"], "dnorm1": g1["dweight"], "dnorm2": g2["dweight"], **ga, **gb}

    @staticmethod
    def clip_grads(grads: dict, max_norm: float) -> torch.Tensor:
        """Scales the parameter gradients of backward() in place; returns their norm."""
        return pmha_clip_grad_norm([t for n, t in grads.items() if n != "dx"], max_norm)
