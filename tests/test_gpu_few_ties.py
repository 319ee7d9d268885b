"""Near ties of the router among keys far above 1, where fp32 has steps that are coarse
beside the scores: the choice is still that of 64 bits."""
import math

import pytest
import torch

from tests.test_gpu_few import BF16, DEV, TOL, layer64, layer_weights, moe

pytestmark = pytest.mark.gpu


def rivals(g, X, z):
    """An fp32 row w of terms near 1 whose products with every row of X (64 bits) are z but
    for its rounding: a fixed part plus one that X does not see."""
    vh = torch.linalg.svd(X, full_matrices=True)[2]
    fixed = torch.linalg.pinv(X) @ torch.full((X.shape[0],), z, dtype=torch.float64)
    free = vh[X.shape[0]:]
    n = free.T @ (free @ torch.randn(X.shape[1], generator=g, dtype=torch.float64))
    return (fixed + n).float()


@pytest.mark.parametrize("bias", [4096.0, -4100.0, 0.75 * 2**17])
@pytest.mark.parametrize("seed", range(3))
def test_keys_on_both_sides_of_a_rounding_border(moe, bias, seed):
    """Two experts whose keys lie a few 2^-24 apart and on the border between two fp32
    values: the nearest of them may be in the wrong order, one step apart."""
    g = torch.Generator().manual_seed(seed)
    T, H = 32, 512
    w = layer_weights(g, H, 4, 64)
    x = torch.randn(T, H, generator=g).to(BF16)
    step = 2.0**(math.floor(math.log2(abs(bias))) - 23)
    s = 0.5 + step / 2  # bias + s lies midway between two fp32 values
    assert torch.tensor(bias + s, dtype=torch.float64).float().item() != bias + s
    z = math.log(s / (1 - s))
    w["router_w"][0], w["router_w"][1] = (rivals(g, x.double(), z).to(DEV) for _ in range(2))
    w["router_bias"][:] = torch.tensor([bias, bias, bias - 100, bias - 100])
    want = layer64(w, x.to(DEV), 1)
    off = (moe.layer_few(x.to(DEV), w, 1).double() - want).norm(dim=1) / want.norm(dim=1)
    assert bool((off <= TOL).all()), off.tolist()
