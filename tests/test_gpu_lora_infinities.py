"""GPU: infinities through low-rank adapters."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rank", [8, 32, 40, 128])
@pytest.mark.parametrize("N,tokens", [(300, 5), (8, 70), (5, 3)])
@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_an_infinite_input_gives_infinities(gpu_lib, rank, N, tokens, sign):
    """A > 0 and a sign for each row of B: A x is +-inf in every entry, and B (A x),
    a sum of infinities of one sign, is that and not NaN. The other rows keep their bits."""
    print("lora inf", rank, N, tokens, sign, flush=True)
    g = torch.Generator().manual_seed(rank)
    K = 136
    index = (torch.arange(tokens) % 3 - 1).to(torch.int32).cuda()
    groups = gpu_lib.group_rows(index, 2)
    a = (torch.rand(2, rank, K, generator=g) + 0.5).to(torch.bfloat16)
    side = torch.where(torch.rand(2, N, 1, generator=g) < 0.5, -1.0, 1.0)
    b = ((torch.rand(2, N, rank, generator=g) + 0.5) * side).to(torch.bfloat16)
    x, out = torch.randn(tokens, K, generator=g).to(torch.bfloat16), torch.randn(tokens, N, generator=g).to(torch.bfloat16)
    plain = gpu_lib.lora_add(out.cuda(), x.cuda(), a.cuda(), b.cuda(), groups).cpu()
    bad = x.clone()
    bad[0, 7] = bad[1, K - 1] = bad[2, 0] = sign * float("inf")      # tokens of no adapter, of 0 and of 1
    got = gpu_lib.lora_add(out.cuda(), bad.cuda(), a.cuda(), b.cuda(), groups).cpu()
    for m, adapter in ((1, 0), (2, 1)):
        assert torch.equal(got[m].float(), sign * side[adapter, :, 0] * float("inf"))
    rest = torch.ones(tokens, dtype=torch.bool)
    rest[1:3] = False
    assert torch.equal(got[rest], plain[rest])
