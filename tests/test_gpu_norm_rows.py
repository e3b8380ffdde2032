"""The layer norm's backward where every workgroup takes several rows, the
last time not all of them, for each number of threads that a row may have.
Tolerances as in test_gpu_norm."""
import pytest
import torch

import oracle.train_ops as ops
import synth
from helpers import dev, to_np
from test_gpu_norm import DT, EPS, _check_backward, _f64, _inputs

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import routing_grouped_gemm_router_amd as moe

# T, d, type, threads of a row
ROWS = [(33001, 32, "bf16", 4), (16500, 96, "bf16", 8), (8300, 160, "bf16", 16), (4200, 256, "bf16", 32),
        (4200, 320, "bf16", 32), (4200, 544, "bf16", 64), (700, 2048, "bf16", 256), (600, 16384, "bf16", 1024),
        (16500, 32, "f32", 8), (8300, 96, "f32", 16), (700, 1056, "f32", 256), (600, 6176, "f32", 1024),
        (600, 8224, "f32", 1024), (600, 16384, "f32", 1024)]


@pytest.mark.parametrize("T,d,dt,threads", ROWS)
@pytest.mark.parametrize("act8", [False, True])
def test_backward_over_several_rows(T, d, dt, threads, act8):
    x, ds, ga, _ = _inputs(T, d, dt, T + d)
    dy = dev(synth.normal((T, d), 8, 2, 1.0), DT[dt])
    c = moe.MOE_BF16 if dt == "bf16" else moe.MOE_F32
    groups = moe.moe_layer_norm_backward_workspace_size(c, T, d) // (8 * d)
    slots = groups * max(256 // threads, 1)
    assert T > slots and T % slots                          # a second pass, uneven
    f = moe.moe_layer_norm(x, ga, None, EPS, act8=act8)
    s = ops.act8_decode(to_np(f["x8"]).view("int8"), to_np(f["x8_scale"])) if act8 else _f64(x)
    src = f if act8 else dict(f, x=x)
    b = moe.moe_layer_norm_backward(src, dy, ga, ds)
    _check_backward(b, s, f, dy, ga, ds, dt, T, "rows")
    assert torch.equal(moe.moe_layer_norm_backward(src, dy, ga, ds)["dweight"], b["dweight"])
