"""GPU: qk_norm_rope where a head holds an infinity, and over large batches."""
import pytest
import torch

import layer_ref as R
from test_gpu_layer_ops import bf16, gen

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("layout", ["half_split", "interleaved"])
@pytest.mark.parametrize("d,rope", [(64, 32), (128, 64), (256, 32)])
def test_an_infinity_beside_the_rotated_dims(gpu_lib, d, rope, layout):
    """An infinite value makes its head's root infinite: its own quotient is NaN,
    every other one 0, as there are no pairs behind the rotated dims."""
    print("norm infinity", d, rope, layout, flush=True)
    g = gen(50, d)
    M, hq, hk = 3, 3, 1
    q, k = bf16(g, M, hq, d), bf16(g, M, hk, d)
    q[1, 2, rope + 4] = float("inf")
    q[2, 0, d - 1] = float("-inf")
    qw, kw = bf16(g, d) + 1, bf16(g, d) + 1
    pos = torch.tensor([3, 0, 7])
    cs = gpu_lib.rope_cos_sin_table(10000.0, 10, rope)
    got = gpu_lib.qk_norm_rope(q.cuda(), k.cuda(), qw.cuda(), kw.cuda(), pos.cuda(), cs, head_dim=d, rope_layout=layout)
    for x, src, w in ((got[0], q, qw), (got[1], k, kw)):
        ref, tol = R.norm_rope(src, w, pos, cs.cpu(), 1e-6, layout == "interleaved")
        x = x.cpu().double()
        plain = ref.isfinite()
        assert torch.equal(x.isnan(), ref.isnan()) and torch.equal(x[~plain & ~ref.isnan()], ref[~plain & ~ref.isnan()])
        assert bool(((x - ref).abs() <= tol)[plain].all())


@pytest.mark.parametrize("layout", ["half_split", "interleaved"])
@pytest.mark.parametrize("M,hq,hk,d,rope", [(2101, 64, 8, 128, 64), (4203, 56, 9, 64, 64), (1003, 64, 8, 256, 96)])
def test_batches_past_the_caches(gpu_lib, M, hq, hk, d, rope, layout):
    """Batches of more than 32 MiB, which are loaded and stored past the caches:
    as column ranges of one projection's rows, into new tensors and in place."""
    print("norm", M, hq, hk, d, rope, layout, flush=True)
    assert M * (hq + hk) * d * 2 > 32 << 20
    g = gen(51, d)
    x = bf16(g, M, (hq + hk) * d + 16)
    q, k = x[:, : hq * d], x[:, hq * d + 8 : (hq + hk) * d + 8]
    qw, kw = bf16(g, d) + 1, bf16(g, d) + 1
    pos = torch.from_numpy(g.integers(0, 500, M))
    cs = gpu_lib.rope_cos_sin_table(10000.0, 500, rope)
    xd = x.cuda()
    qd, kd = xd[:, : hq * d], xd[:, hq * d + 8 : (hq + hk) * d + 8]
    args = (qw.cuda(), kw.cuda(), pos.cuda(), cs)
    got = gpu_lib.qk_norm_rope(qd, kd, *args, head_dim=d, rope_layout=layout)
    for y, src, w, h in ((got[0], q, qw, hq), (got[1], k, kw, hk)):
        ref, tol = R.norm_rope(src.reshape(M, h, d), w, pos, cs.cpu(), 1e-6, layout == "interleaved")
        off = (y.cpu().double().view(M, h, d) - ref).abs()
        assert bool((off <= tol).all()), float((off / tol.clamp_min(1e-300)).max())
    keep = xd.clone()
    gpu_lib.qk_norm_rope(qd, kd, *args, head_dim=d, rope_layout=layout, q_out=qd, k_out=kd)
    keep[:, : hq * d], keep[:, hq * d + 8 : (hq + hk) * d + 8] = got
    assert torch.equal(xd, keep)
