"""GPU: attention over the FP8 cache with windows that no sequence reaches."""
import pytest
import torch

from test_gpu_layer_ops import attend, gen

pytestmark = pytest.mark.gpu


# Tables that keep a batch of few rows in the prompt kernel, and that do not.
WIDTHS = [1, 2100, 9000]


@pytest.mark.parametrize("window", [2 ** 31 - 1, 2 ** 31 - 20, 2 ** 30])
@pytest.mark.parametrize("width", WIDTHS)
@pytest.mark.parametrize("hq,h,d", [(1, 1, 64), (4, 2, 128), (16, 2, 64)])
@pytest.mark.parametrize("lens,new", [([25], [20]), ([25, 40, 130], [20, 3, 1]), ([300, 20], [200, 16])])
def test_windows_past_every_length(gpu_lib, lens, new, hq, h, d, width, window):
    """A window that no sequence reaches is no window, to the bit."""
    print("attend window", lens, new, hq, h, d, width, window, flush=True)
    args, out = attend(gpu_lib, gen(40, hq, d, len(lens)), lens, new, hq, h, d, 16, window=window, extra=-(-width // 16))
    assert torch.equal(out, gpu_lib.attention_fp8_kv(*args))
