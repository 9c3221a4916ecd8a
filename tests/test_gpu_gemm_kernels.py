"""GPU: every kernel of the FP8 product, at sizes off its tiles that the rule
sends to it, with padded operands and outputs, nothing written beside them."""
import pytest
import torch

import layer_ref as R
from test_gemm_sizes_cpu import KERNEL_SIZES
from test_gpu_layer_ops import exact_operands, gen

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kernel,M,N,K", KERNEL_SIZES)
def test_each_kernel(gpu_lib, kernel, M, N, K):
    """Sums that are exact in every order (test_gpu_layer_ops.exact_operands):
    equal to the float64 product rounded to bf16."""
    print("gemm", kernel, M, N, K, flush=True)
    assert gpu_lib.debug_fp8_gemm_kernel(M, N, K) == kernel
    a, words, w, ws = exact_operands(gen(60, M, N, K), M, N, K)
    ref = (R.dequant_rows(a, words) @ R.dequant_tiles(w, ws).T).to(torch.bfloat16).cuda()
    out = gpu_lib.fp8_gemm_1x128_128x128(a.cuda(), words.cuda(), w.cuda(), ws.cuda())
    assert torch.equal(out, ref)
    ap = torch.full((M, K + 32), 0x7F, dtype=torch.uint8)
    ap[:, :K] = a
    wp = torch.full((N, K + 16), 0x7F, dtype=torch.uint8)
    wp[:, :K] = w
    wsp = torch.full((ws.shape[0], ws.shape[1] + 1), 255, dtype=torch.uint8)
    wsp[:, : ws.shape[1]] = ws
    mn = torch.full((words.shape[1], M + 5), -1, dtype=torch.int32)          # every scale byte NaN
    mn[:, :M] = words.T
    ap, wp, wsp, mn = ap.cuda()[:, :K], wp.cuda()[:, :K], wsp.cuda()[:, : ws.shape[1]], mn.cuda().T[:M]
    for pad, first in ((0, 0), (-N % 8, 0), (8 - N % 8, 8), (3, 1)):        # 16-byte stores in the second and third
        buf = torch.full((M + 2, N + first + pad), 7.0, dtype=torch.bfloat16, device="cuda")
        gpu_lib.fp8_gemm_1x128_128x128(ap, mn, wp, wsp, out=buf[1:M + 1, first:first + N])
        want = torch.full_like(buf, 7.0)
        want[1:M + 1, first:first + N] = ref
        assert torch.equal(buf, want), (pad, first)
