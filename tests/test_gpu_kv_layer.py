"""The example layer: the cache's calls together with the linears, prompts in one
step and a replayed graph of single tokens, against the parts in 64 bits."""
import importlib.util
import os

import pytest
import torch

from conftest import ROOT
from kv_helpers import attention

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def example():
    from nvfp4_w4a4_decode_gb300 import build as nvbuild
    nvbuild.build()
    path = os.path.join(ROOT, "examples", "paged_attention_layer.py")
    spec = importlib.util.spec_from_file_location("paged_attention_layer", path)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


@pytest.mark.parametrize("kw", [dict(), dict(prompts=(1, 130, 16, 64), steps=9, head_dim=128, q_heads=14, kv_heads=2,
                                             hidden=1024, page_size=32)])
def test_layer(example, kw):
    nv = example.nv
    nv.device_status(clear=True)
    layer, table, lens, inputs, outputs = example.run(**kw)
    assert nv.device_status() == 0
    assert lens == [len(x) for x in inputs]
    used = table[table >= 0]
    assert len(used.unique()) == len(used)  # no page twice
    assert (table >= 0).sum(1).tolist() == [-(-n // layer.cache.page_size) for n in lens]
    for r, (x, y) in enumerate(zip(inputs, outputs)):
        # every row again in one call over the finished cache: causality makes them the same rows
        q, _, _ = layer.split(layer.project(x, layer.qkv, layer.x_g))
        out, _, _, _, _ = attention(layer.cache, q, table[r:r + 1], [lens[r]], [lens[r]])
        # the attention's bfloat16 rounding may move single 4-bit codes of the o linear's input:
        # a step of at most 2/6 of a block's maximum each, rare; rows agree to a few percent
        want = layer.project(out.to(torch.bfloat16).flatten(1), layer.o, layer.cache.v_g)
        off = (y.float() - want.float()).norm() / want.float().norm()
        assert off < 0.03, off
        cos = torch.nn.functional.cosine_similarity(y.float().flatten(), example.dense(layer, x).flatten(), dim=0)
        assert cos > 0.95, cos
