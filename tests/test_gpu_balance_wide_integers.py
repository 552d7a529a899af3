"""Expert ids and sequence offsets held in 64 bits: those past 32 bits are
clamped like any other out of range, not taken for their low 32 bits."""

import numpy as np
import pytest
import torch

from oracle import training as R

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,E,k", [(50, 9, 3), (700, 300, 2)])
def test_values_past_32_bits(gpu_lib, T, E, k):
    from moe_layer_router_amd import layer as L
    rng = np.random.default_rng(T)
    l = rng.normal(size=(T, E)).astype(np.float32)
    ids = rng.integers(0, E, size=(T, k))
    ids[3, 0], ids[4, 1], ids[5, 0] = 2 ** 32 + 1, -2 ** 32 + 1, 2 ** 31 + 2
    off = np.array([-2 ** 33 + 7, 20, 2 ** 32 + 30])
    out = L.balance_loss(torch.from_numpy(l).cuda(), torch.from_numpy(ids).cuda(), alpha=1.0,
                         seq_offsets=torch.from_numpy(off).cuda())
    torch.cuda.synchronize()
    ref = R.balance_loss(l, ids, 1.0, off)
    assert np.array_equal(out["counts"].cpu().numpy(), ref["counts"])
    # fp32 sums over at most T tokens, as the operator's own test derives them
    assert abs(float(out["loss"].cpu()[0]) - ref["loss"]) <= (68 + T) * 2.0 ** -24 * ref["loss"]
