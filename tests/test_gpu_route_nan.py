"""GPU: the order of the experts where a token's scores are NaN."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("M,E", [(6, 96), (9, 300), (41 * 16, 16), (41 * 64, 64)])
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid", "sqrt_softplus"])
@pytest.mark.parametrize("renormalize", [False, True])
@pytest.mark.parametrize("bias", [False, True])
def test_route_nan_logits_come_first(gpu_lib, M, E, scoring, renormalize, bias):
    """Experts whose logits are NaN come before all others, the lower index first,
    and those of -inf after all others; so under softmax too, where one NaN makes every
    score of its token NaN and the logits decide between the others."""
    print("nan order", M, E, scoring, renormalize, bias, flush=True)
    g = torch.Generator().manual_seed(E)
    z = torch.randn(M, E, generator=g)
    b = (0.01 * torch.randn(E, generator=g)).cuda() if bias else None
    good = gpu_lib.moe_route(z.cuda(), 4, bias=b, scoring=scoring, renormalize=renormalize)
    nan, inf = float("nan"), float("inf")
    z[1, 11] = nan
    z[2, [13, 5]] = nan
    z[3] = -inf
    z[3, 14], z[3, 9] = nan, 1.0
    z[4, 12] = inf
    w, e = (t.cpu() for t in gpu_lib.moe_route(z.cuda(), 4, bias=b, scoring=scoring, renormalize=renormalize))
    assert e[1, 0] == 11 and math_nan(w[1, 0])
    assert e[2, :2].tolist() == [5, 13] and math_nan(w[2, :2])
    assert e[3].tolist() == [14, 9, 0, 1] and math_nan(w[3, 0])
    if scoring == "softmax" or not bias:
        assert e[4, 0] == 12
    if scoring == "softmax" and bias:
        # sums of NaN: the logits' order
        order = torch.sort(z[1], descending=True, stable=True).indices.tolist()
        order.remove(11)
        assert e[1, 1:].tolist() == order[:3]
    for row in range(5):
        assert len(set(e[row].tolist())) == 4 and 0 <= int(e[row].min()) and int(e[row].max()) < E
    assert torch.equal(w[5:], good[0].cpu()[5:]) and torch.equal(e[5:], good[1].cpu()[5:])
    assert torch.equal(w[0], good[0].cpu()[0]) and torch.equal(e[0], good[1].cpu()[0])


def math_nan(t):
    return bool(torch.isnan(t).all())
