"""Layer norm and its backward on the GPU with many rows to a block: every kernel's walk over the rows goes round
several times (the sums' two buffers, the ring's stages and their phases, the columns' sums carried
over turns), with rows left over in the last turn.  Definitions and tolerances as in test_gpu_norm."""
import pytest
import torch

import gated_delta_rule_95_b200 as g
from tests.test_gpu_norm import _check_bwd, _check_fwd, _draw

pytestmark = pytest.mark.gpu

# 592 blocks: single elements held by a block (1001), by part of a warp with one row (33) and two rows at once (1), 16-byte
# vectors held by a warp (512, 256 in fp32), by part of one (64) and by one thread (8, 4 in fp32), by a block of 64 or 128
CASES = [(5003, 1001), (3001, 3001), (20003, 33), (9001, 250), (400001, 1), (40003, 512), (30001, 256), (100001, 64), (700001, 8),
         (600001, 4), (12001, 1000), (6007, 2048)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,cols", CASES)
def test_many_rows(rows, cols, dtype):
    s, dy, w, b = _draw((rows, cols), 1, dtype), _draw((rows, cols), 2, dtype), _draw((cols,), 3), _draw((cols,), 4)
    ds = _draw((rows, cols), 5, dtype) if cols % 3 else None
    sd, wd = s.cuda(), w.cuda()
    out = g.gdn2_layer_norm_fwd(sd, wd, b.cuda())
    r = g.gdn2_layer_norm_bwd(dy.cuda(), sd, wd, out[2], out[3], None if ds is None else ds.cuda())
    torch.cuda.synchronize()
    _check_fwd(s, None, w, b, out, 1e-5, dtype)
    _check_bwd(dy, s, w, out[2], out[3], ds, r, dtype)
    assert g.gdn2_device_status() == 0


# the last width of each way to hold a row and the first of the next (threads of a row, vectors of a thread, blocks of 128,
# 256, 512 and 1024 threads, rows that no block holds), for vectors and for single elements
EDGES = [128, 132, 255, 257, 260, 264, 511, 513, 520, 1023, 1025, 2052, 4095, 4096, 4097, 4100, 4104, 8191, 8193, 32768, 32772, 32776]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("cols", EDGES)
def test_widths_at_the_edges(cols, dtype):
    rows = 7
    s, dy, w, b = _draw((rows, cols), 6, dtype), _draw((rows, cols), 7, dtype), _draw((cols,), 8), _draw((cols,), 9)
    r, ds = _draw((rows, cols), 10, dtype), _draw((rows, cols), 11, dtype)
    out = g.gdn2_layer_norm_fwd(s.cuda(), w.cuda(), b.cuda(), r.cuda())
    d = g.gdn2_layer_norm_bwd(dy.cuda(), out[1], w.cuda(), out[2], out[3], ds.cuda())
    torch.cuda.synchronize()
    _check_fwd(s, r, w, b, out, 1e-5, dtype)
    _check_bwd(dy, out[1].cpu(), w, out[2], out[3], ds, d, dtype)
    assert g.gdn2_device_status() == 0
