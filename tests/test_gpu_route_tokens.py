"""GPU: a token's experts and weights go by its own logits, whatever the tokens
beside it hold, and by rules that hold where scores are NaN."""
import math

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu


def at_a_cut(g, pairs):
    """Logits and biases (float32) of 2 * pairs experts, sigmoid scores in [0.5, 1).
    The second of a pair has the sum p + bias on a multiple of 2^-43, where the 42
    mantissa bits that sums are compared by change, with p rounded to float64: one
    unit less in p's last place and it equals the first one's, of the lower index."""
    z = np.repeat(np.sort(g.uniform(0.3, 1.8, pairs).astype(np.float32)), 2)
    b = np.zeros(2 * pairs, dtype=np.float32)
    for i in range(0, 2 * pairs, 2):
        p = 1 / (1 + math.exp(-float(z[i])))
        cut = math.ceil(p * 2.0 ** 43) * 2.0 ** -43
        b[i + 1] = cut - p                       # at most ten bits: exact
        assert p + float(b[i + 1]) == cut
        b[i] = cut - 2.0 ** -44 - p
    return z, b


@pytest.mark.parametrize("E", [16, 32, 64])
@pytest.mark.parametrize("far", [700.0, -700.0, float("inf"), float("nan")])
def test_route_neighbours(gpu_lib, E, far):
    """One token of four has a logit that the short form of the sigmoid does not
    take. Sums on the border between two choices show a difference of one unit in a
    score's last place: the other three tokens' results keep their bits."""
    print("neighbours", E, far, flush=True)
    g = np.random.default_rng([94, E])
    M, top = 40 * E + 4, 16
    for trial in range(25):
        zs, bs = at_a_cut(g, 8)
        z = torch.full((M, E), -float("inf"))
        z[:, :16] = torch.from_numpy(zs)
        b = torch.zeros(E)
        b[:16] = torch.from_numpy(bs)
        clean = gpu_lib.moe_route(z.cuda(), top, bias=b.cuda(), scoring="sigmoid")
        z[::4, 3] = far
        got = gpu_lib.moe_route(z.cuda(), top, bias=b.cuda(), scoring="sigmoid")
        rest = torch.arange(M) % 4 != 0
        for was, now in zip(clean, got):
            assert torch.equal(was.cpu()[rest], now.cpu()[rest]), trial
