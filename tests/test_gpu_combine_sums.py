"""The combine backward's dots where a token has a wave or more, within the
roundings of that order: nv vectors of N elements dealt to 64 threads are N
ceil(nv / 64) products a thread at most, each one rounding (a fused
multiply-add), and 6 additions in the wave; with 256 threads fewer products, 6
additions and 4 over the waves. So N ceil(nv / 64) + 10 roundings at most."""
import numpy as np
import pytest
import torch

import oracle.train_ops as ops
import synth
from helpers import dev, to_np
from test_gpu_act8 import DT, U, _near, _routing

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import routing_grouped_gemm_router_amd as moe


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("T,d,E,k", [(33, 288, 8, 2), (64, 2080, 16, 4), (3000, 1056, 8, 4), (5, 8224, 8, 8),
                                     (2100, 2048, 8, 4), (3, 16384, 4, 4)])
def test_dots_of_wide_rows(dt, T, d, E, k):
    idx, g, pos, R = _routing(T, E, k, T + d)
    y, go = dev(synth.normal((R, d), 4, 0, 2.0), DT[dt]), dev(synth.normal((T, d), 4, 1, 1.0), DT[dt])
    q, s = moe.moe_act8_store(y)
    b = moe.moe_combine_backward_act8(go, q, s, torch.from_numpy(g).cuda(), torch.from_numpy(idx).cuda(),
                                      torch.from_numpy(pos).cuda(), E)
    v = ops.act8_decode(to_np(q).view(np.int8), to_np(s))[pos]
    o = to_np(go).astype(np.float64)[:, None]
    n = 8 if dt == "bf16" else 4
    roundings = n * -(-(d // n) // 64) + 10
    _near(to_np(b["dgate"]), (o * v).sum(2), roundings * U * np.abs(o * v).sum(2) + 2.0 ** -126, "dgate")
