"""GPU: attention over the FP8 cache where many weights far below a row's
largest make up its output."""
import pytest
import torch

import layer_ref as R
from test_gpu_attention_windows import WIDTHS
from test_gpu_layer_ops import gen, ints, make_batch, random_cache, to_gpu

pytestmark = pytest.mark.gpu


def one_exponent(g, lens, new, h, block, d, width):
    """A batch and a cache of zeros at scale 1."""
    table, cu, n = make_batch(g, lens, new, block, width_extra=-(-width // block))
    ref = random_cache(g, n, h, block, d)
    for x in ("k", "v"):
        ref[x].zero_()
        ref[x + "s"].fill_(127)
    return table, cu, ref


def set_token(ref, table, s, t, k, v):
    """Every value of token t of sequence s: codes k and v."""
    b = ref["k"].shape[2]
    ref["k"][int(table[s, t // b]), :, t % b] = k
    ref["v"][int(table[s, t // b]), :, :, t % b] = v


@pytest.mark.parametrize("width", WIDTHS)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("lens,new", [([512], [1]), ([700, 330], [2, 3]), ([400], [60]), ([300, 500], [130, 1]), ([500] * 5, [70] * 5)])
def test_weights_far_below_the_largest(gpu_lib, lens, new, d, width):
    """One token of every 64 outweighs each of the others by 2^26, and has no
    value where theirs is 1: the output is what they weigh together.

    Tolerance: the rounding to bf16, 2^-8; the weights in fp16, 2^-11 relatively
    or 2^-32 of the largest where they are subnormal; the scores as in
    layer_ref.attention."""
    print("attend small weights", lens, new, d, width, flush=True)
    h, hq, block = 2, 4, 32
    table, cu, ref = one_exponent(gen(41), lens, new, h, block, d, width)
    for s, n in enumerate(lens):
        for t in range(n):
            heavy = t % 64 == 5
            set_token(ref, table, s, t, 0x3C if heavy else 0x00, 0x00 if heavy else 0x38)     # 1.5, 0 and 0, 1
    q = torch.full((cu[-1], hq, d), 1.5 if d == 64 else 1.0625, dtype=torch.bfloat16)
    want, _ = R.attention(q, ref, table, lens, cu, d ** -0.5, 0)
    got = gpu_lib.attention_fp8_kv(q.cuda(), to_gpu(gpu_lib, ref), table.cuda(), ints(lens), ints(cu)).cpu().double()
    score = 1.5 * d * float(q[0, 0, 0]) * d ** -0.5
    rel = 2.0 ** -8 + 2.0 ** -11 + 2 * ((d + 3) * 2.0 ** -23 * score * 1.4427 + 2.0 ** -20)
    for s, n in enumerate(lens):
        for i in range(new[s]):
            p = n - new[s] + i
            heavy = (p + 59) // 64                                       # of the p + 1 tokens seen
            assert heavy > 0
            r = cu[s] + i
            off = (got[r] - want[r]).abs()
            assert bool((off <= rel * want[r] + (p + 1) * 2.0 ** -32 / heavy).all()), (s, i, float(got[r, 0, 0]), float(want[r, 0, 0]))
