"""The layer's tensor-core path with other work between its calls: weights
that come from memory rather than from the L2, copies that share the memory
with them and grouped products in the same stream change when each of a
layer's copies lands, and in which order.  The output is the same bits every
time, as every sum has a fixed order.

The expert GEMM's two conversion sets share an odd ring of weight slots; a
set that waits for a slot too early reads the slot's weights of three steps
before, a whole tile wrong, and only when two copies land out of order."""
import numpy as np
import pytest
import torch

import quantized_moe_expert_fwd_gb300 as q
from tests import gpu_util as G
from workloads import gen

pytestmark = pytest.mark.gpu

DIMS = gen.LayerDims(hidden=1024, n_experts=32, top_k=4, inter=256, shared_inter=256)


@pytest.mark.parametrize("between", ["flush", "copies", "grouped"])
def test_layer_keeps_its_bits(between):
    dev, T, calls = G.dev(), 40, 8
    dl = q.DeviceLayer(gen.draw_layer(DIMS, 5), dev)
    x = torch.from_numpy(np.random.default_rng(6).standard_normal((T, 1024))).to(dev, torch.bfloat16)
    out = torch.zeros(calls, T, 1024, dtype=torch.bfloat16, device=dev)
    ws = q.make_workspace(DIMS, T, dev)
    q.moe_layer_forward(DIMS, dl, x, out[0], ws)
    torch.cuda.synchronize()
    want = out[0].clone()

    big = torch.zeros(1 << 26, device=dev)                  # 256 MB, above the L2
    E, N = 8, 512
    gws = q.make_grouped_workspace(dev)
    offs = torch.tensor([0, 9, 9, 40, 41, 100, 160, 160, 200], dtype=torch.int32, device=dev)
    gx = torch.zeros(200, 1024, dtype=torch.bfloat16, device=dev)
    gw = torch.zeros(E, N, 1024, dtype=torch.bfloat16, device=dev)
    gy = torch.zeros(200, N, dtype=torch.bfloat16, device=dev)

    side, other = torch.cuda.Stream(), torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other.wait_stream(torch.cuda.current_stream())
    wrong = torch.zeros((), dtype=torch.int64, device=dev)
    with torch.cuda.stream(side):
        for i in range(400):
            if between == "copies":
                with torch.cuda.stream(other):
                    big[:1 << 25].copy_(big[1 << 25:])
            for k in range(calls):
                if between == "flush":
                    big.fill_(float(i))
                elif between == "grouped":
                    q.moe_grouped_mm(gx, gw, offs, gy, gws)
                q.moe_layer_forward(DIMS, dl, x, out[k], ws)
            wrong += (out != want).flatten(1).any(1).sum()
            out.zero_()
            if i % 20 == 19:
                side.synchronize()
                other.synchronize()
    torch.cuda.synchronize()
    assert q.moe_get_device_status(ws) == q.STRATA_OK
    assert int(wrong) == 0
