"""Arguments of the layer's entry points on the GPU: stream handles, sizes past 32 bits."""
import pytest
import torch

import gated_delta_rule_95_b200 as g

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def test_the_default_stream_by_its_handle():
    # handle 0 is the default stream: a call on it waits for what is queued there, whatever stream is current
    assert torch.cuda.default_stream().cuda_stream == 0
    x, w, side = torch.zeros(64, 256, device="cuda"), torch.ones(256, device="cuda"), torch.cuda.Stream()
    new = torch.randn(64, 256, device="cuda")
    want = g.gdn2_layer_norm_fwd(new, w)[0]
    torch.cuda.synchronize()
    torch.cuda._sleep(200_000_000)  # about 0.1 s, on the default stream
    x.copy_(new)
    with torch.cuda.stream(side):
        y = g.gdn2_layer_norm_fwd(x, w, stream=0)[0]
    torch.cuda.synchronize()
    assert torch.equal(y, want)


def test_more_rows_than_the_library_counts():
    # 2^32 + 5 rows are not 5
    if torch.cuda.mem_get_info()[0] < 30e9:
        pytest.skip("needs 26 GB of device memory")
    x, w = torch.empty(2 ** 32 + 5, 1, dtype=BF, device="cuda"), torch.ones(1, device="cuda")
    for call in (lambda: g.gdn2_layer_norm_fwd(x, w, want_stats=False), lambda: g.gdn2_short_conv(x.view(1, -1, 1), torch.ones(1, 4, device="cuda")),
                 lambda: g.gdn2_short_conv_bwd(x.view(1, -1, 1), x.view(1, -1, 1), torch.ones(1, 4, device="cuda"))):
        with pytest.raises(ValueError, match="gdn2_"):
            call()
    torch.cuda.empty_cache()
