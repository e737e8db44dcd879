"""The MoE layer and the output head inside a serving step, against the oracle on the attention rows and layer outputs
that the step itself made: eagerly and in a captured decode step whose buffers are poisoned before each replay (every
kernel of the step is launched to overlap its predecessor's end). test_gpu_serving_step.py checks the append, the
attention and the sampling of the same step.

Bounds: the layer contract's (gpu_layer.check_output); the head's in fp32 against its fp64 form, as in
test_gpu_lm_head.py."""
import numpy as np
import pytest
import torch

import nvfp4_weight_only_flint_b200 as fm
import oracle
import synth
from gpu_layer import check_output, cuda_to_bits
from test_gpu_serving_step import D, HKV, HQ, DH, V, Step

pytestmark = pytest.mark.gpu


def _check_layers(s, b, last):
    torch.cuda.synchronize()
    x = cuda_to_bits(b["att"].view(-1, D).index_select(0, last))
    router = s.router.cpu().numpy().view(np.uint16)
    ids, _, gap = oracle.topk(oracle.router_logits(x, router), s.layer.w.k)
    assert (gap > 1e-6).all()  # no routing near a tie
    ref = s.layer.oracle_forward(x, router, ids, residual_bits=x)
    check_output(cuda_to_bits(b["moe"]), ref["out"], "layer of the step")
    ref = oracle.dense_gemv(s.head_oracle, cuda_to_bits(b["moe"]))
    got = b["logits"].cpu().numpy().astype(np.float64)
    for t in range(s.B):
        d = got[t] - ref[t]
        assert np.linalg.norm(d) <= 5e-3 * np.linalg.norm(ref[t])
        assert np.abs(d).max() <= 2e-2 * np.sqrt(np.mean(ref[t] ** 2))
    for ws in (s.layer.ws, s.ws_head):
        assert fm.flint_moe_get_status(ws) == (0, 0)
    assert int(s.status.item()) == 0


@pytest.mark.parametrize("e4m3", [False, True])
def test_layer_and_head_of_a_serving_step(e4m3):
    B, prompts = 4, [37, 5, 64, 1]
    s = Step(B, 120, sum(prompts), e4m3)
    g = torch.Generator().manual_seed(3)  # the head as Step draws it
    torch.randperm(s.n_pages, generator=g)
    for _ in range(2):
        torch.rand(DH, generator=g)
    s.head_oracle = oracle.quantize((torch.randn((V, D), generator=g) * 0.2).numpy())
    assert np.array_equal(s.head[0].cpu().numpy(), s.head_oracle.codes)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    g = torch.Generator().manual_seed(17)
    qkv_of = lambda T: torch.randn((T, HQ + 2 * HKV, DH), generator=g).to(torch.bfloat16).cuda()  # noqa: E731
    params = [torch.full((B,), 0.8, device="cuda"), i32([50, 0, 3, 0]), torch.full((B,), 0.9, device="cuda"),
              torch.rand(B, generator=g).cuda()]
    starts = [sum(prompts[:i]) for i in range(B + 1)]
    last = i32([x - 1 for x in starts[1:]]).long()
    b = s.run(qkv_of(sum(prompts)), i32(starts), i32(prompts), sum(prompts), max(prompts), last, *params)
    _check_layers(s, b, last)
    q_start, kv_len, qkv = i32(list(range(B + 1))), i32([x + 1 for x in prompts]), qkv_of(B)
    last = torch.arange(B, device="cuda")
    call = lambda: s.run(qkv, q_start, kv_len, B, 1, last, *params)  # noqa: E731
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        b = call()
    for step in range(1, 4):
        kv_len.copy_(i32([x + step for x in prompts]))
        qkv.copy_(qkv_of(B))
        for name in ("q", "att", "moe", "logits"):
            b[name].fill_(float("nan"))
        graph.replay()
        _check_layers(s, b, last)
