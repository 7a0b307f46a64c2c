"""Arguments of the layer's entry points on the GPU: sizes past 32 bits."""
import pytest
import torch

import gated_delta_rule_95_b200 as g

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


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
