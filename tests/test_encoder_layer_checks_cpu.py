"""CPU: what PackedEncoderLayer refuses when it is made, not when it first runs."""
import types

import pytest
import torch

import graph_sparse_head_gb300 as pmha


def attention(E=32):
    w = [torch.zeros(E, E) for _ in range(4)]
    return pmha.Params(*w, None, None, None, None, 4)


def test_a_block_in_8_bits_is_refused():
    graph = types.SimpleNamespace(query_features=8, key_features=8)
    w = torch.zeros(64, 32)
    block = pmha.FfnQuantizedParams(*pmha.quantize_rows(w), *pmha.quantize_rows(w), torch.zeros(32, 64))
    with pytest.raises(TypeError, match="FfnParams"):
        pmha.PackedEncoderLayer(graph, attention(), None, None, block)


def test_a_graph_between_two_token_sets_is_refused():
    graph = types.SimpleNamespace(query_features=8, key_features=9)
    with pytest.raises(ValueError, match="query_features"):
        pmha.PackedEncoderLayer(graph, attention(), None, None, None)
