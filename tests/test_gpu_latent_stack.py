"""Several layers over latent caches as one step whose inputs come in one copy."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import ops_ref as R
from devutil import bf16_dev, i32_dev
from test_gpu_latent import INV, pkv, same  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("N", [16, 128])
def test_a_stacks_inputs_in_one_copy(pkv, N):  # noqa: F811
    from paged_kv_decode_slot_gb300.step import LatentDecodeStep, LayerStack, PackedInputs, StepGraph
    r = np.random.default_rng(N)
    ctx, new = [100, 1, 700], lambda *shape: bf16_dev(R.to_bf16(r.standard_normal(shape)))
    tab, pool = R.tables(r, ctx)
    inv, base = torch.from_numpy(INV).cuda(), [new(pool, 16, 576) for _ in range(2)]
    make = lambda: LayerStack([LatentDecodeStep(torch.zeros(3, 1, 576, device="cuda").bfloat16(), torch.zeros(3, 1, N, 192, device="cuda").bfloat16()[..., 128:],
                                                torch.zeros(3, 1, N, 576, device="cuda").bfloat16(), c.clone(), i32_dev(np.zeros((3, tab.shape[1]))),
                                                i32_dev([0, 0, 0]), 0.07, inv) for c in base])
    stack = make()
    assert stack.input_names() == ("block_tables", "context_lens", "kv_new.0", "q_rope.0", "q.0", "kv_new.1", "q_rope.1", "q.1")
    assert len(stack.inputs()) == 8
    packed = PackedInputs(stack, stack.input_names())
    graph = StepGraph(stack)
    inputs = dict(zip(stack.input_names(), [i32_dev(tab), i32_dev(ctx)] + [new(*t.shape) for t in stack.inputs()[2:]]))
    for n, t in inputs.items():
        packed.host[n].copy_(t)
    packed.upload(graph.stream)
    with torch.cuda.stream(graph.stream):
        graph.replay()
    torch.cuda.synchronize()
    for i, layer in enumerate(stack.layers):
        s = LatentDecodeStep(inputs[f"kv_new.{i}"], inputs[f"q_rope.{i}"], inputs[f"q.{i}"].clone(), base[i].clone(), inputs["block_tables"],
                             inputs["context_lens"], 0.07, inv)
        s.run()
        assert same(s.out, layer.out) and same(s.lse, layer.lse) and same(s.latent_cache, layer.latent_cache) and same(s.q, layer.q)
