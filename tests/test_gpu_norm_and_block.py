"""The RMS norm right before the block of affine 4-bit experts, whose router begins while the norm still runs."""
from __future__ import annotations

import pytest

import expert_ffn_gb300 as mx
import synth

pytestmark = pytest.mark.gpu


# the multi-launch path (fp32, more tokens than the single launch takes), the single launch and the grouped products
@pytest.mark.parametrize("T,act", [(8, "f32"), (40, "f32"), (1, "bf16"), (40, "bf16")])
@pytest.mark.parametrize("captured", [False, True])
def test_norm_then_block(T, act, captured):
    """The block has the norm's rows of this call, not of the one before."""
    import torch
    from tests import gpu_util as gu
    cfg = synth.small_config(T=T, D=512, E=32, K=4, I=128, S=128, act=act, seed=T)
    dev = mx.DeviceLayer(synth.make_layer(cfg), gu.act_code(cfg))
    dtype = torch.float32 if act == "f32" else torch.bfloat16
    g = torch.Generator(device="cuda")
    g.manual_seed(T)
    x, h, out = (torch.zeros(T, 512, dtype=dtype, device="cuda") for _ in range(3))
    idx, w = torch.empty(T, 4, dtype=torch.int32, device="cuda"), torch.empty(T, 4, device="cuda")
    ws = gu.Workspace(mx.workspace_bytes(dev.layout, T))

    def block(rows, to):
        mx.layer_forward_ex(rows, T, dev, to, idx, w, ws.t, ws.nbytes, stream=torch.cuda.current_stream())

    def run():
        mx.fp8_rmsnorm(x, out=h)
        block(h, out)

    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        run()
        if captured:
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=side):
                run()
        for _ in range(20):
            x.copy_(torch.randn(T, 512, device="cuda", generator=g).to(dtype))
            graph.replay() if captured else run()
            side.synchronize()
            want = torch.empty_like(out)
            block(h.clone(), want)
            side.synchronize()
            assert torch.equal(out, want)
            assert torch.allclose(h.float().pow(2).mean(1), torch.ones(T, device="cuda"), atol=0.02)
        mx.workspace_check(ws.t, side)
