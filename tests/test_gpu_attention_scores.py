"""GPU: attention over the FP8 cache with scores of any size."""
import pytest
import torch

import layer_ref as R
from test_gpu_attention_weights import one_exponent, set_token
from test_gpu_attention_windows import WIDTHS
from test_gpu_layer_ops import gen, ints, to_gpu

pytestmark = pytest.mark.gpu


# tokens that outweigh all before them, and the sizes of their keys
STEPS = {0: 4.0, 3: 9.0, 20: 18.0, 70: 44.0, 150: 88.0}


def codes_of(value):
    return int((R.E4M3[:127] == value).nonzero()[0, 0])


@pytest.mark.parametrize("size", [2.0 ** 4, 2.0 ** 13, 2.0 ** 18, 2.0 ** 22, 2.0 ** 26, 2.0 ** 50])
@pytest.mark.parametrize("width", WIDTHS)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("lens,new", [([200], [1]), ([200, 90], [2, 3]), ([200, 160], [190, 60]), ([200] * 5, [70] * 5)])
def test_large_scores(gpu_lib, lens, new, d, width, size):
    """Scores so large that their float32 steps are many powers of two: each row
    is the value of the one token that outweighs the others, exactly."""
    print("attend large scores", lens, new, d, width, size, flush=True)
    one_token_each(gpu_lib, lens, new, d, width, size, STEPS, 1.0)


def one_token_each(lib, lens, new, d, width, size, steps, other):
    h, hq, block = 1, 2, 32
    g = gen(42, d)
    table, cu, ref = one_exponent(g, lens, new, h, block, d, width)
    for s, n in enumerate(lens):
        for t in range(n):
            set_token(ref, table, s, t, codes_of(steps.get(t, other)), int(g.integers(0x20, 0x50)))
        for b in range(-(-n // block)):
            ref["vs"][int(table[s, b])] = 127 + b % 3
    q = torch.zeros(cu[-1], hq, d, dtype=torch.bfloat16)
    want = torch.zeros(cu[-1], hq, d, dtype=torch.float64)
    for s, n in enumerate(lens):
        _, v, _ = R.held_values(ref, table, s, n)
        for i in range(new[s]):
            p = n - new[s] + i
            q[cu[s] + i] = size * (1 + (i % 128) / 128)
            want[cu[s] + i] = v[max(t for t in steps if t <= p)]
    got = lib.attention_fp8_kv(q.cuda(), to_gpu(lib, ref), table.cuda(), ints(lens), ints(cu)).cpu().double()
    # four significant bits a value, off by a few 2^-24 before it is rounded to bf16
    bad = (got != want).any(-1)
    assert not bool(bad.any()), (int(bad.sum()), got[bad][0, :4].tolist(), want[bad][0, :4].tolist())


@pytest.mark.parametrize("width", WIDTHS)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("lens,new", [([200], [1]), ([200, 90], [2, 3]), ([200, 160], [190, 60]), ([200] * 5, [200] * 5)])
def test_scores_far_below_zero(gpu_lib, lens, new, d, width):
    """Rows all of whose scores lie below -10^30: still the token that outweighs the others."""
    print("attend scores below zero", lens, new, d, width, flush=True)
    one_token_each(gpu_lib, lens, new, d, width, -2.0 ** 100, {0: 352.0, 3: 176.0, 20: 88.0, 70: 44.0, 150: 9.0}, 448.0)
