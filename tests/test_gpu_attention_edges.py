"""Attention over a context at its edges, on either of its kernels: rows, sequences and parts without keys."""

import numpy as np
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
import rank_decomposed_gb300 as lr  # noqa: E402
from test_gpu_attention import Batch, close  # noqa: E402


@pytest.fixture(autouse=True, params=[1, 2], ids=["rows", "tiles"])
def kernel(request):
    lr.lib.lr_test_attention_kernel(request.param)
    yield request.param
    lr.lib.lr_test_attention_kernel(0)


def _sees(b):
    """Whether each row sees a token."""
    own = [n - k + j + 1 for n, k in zip(b.lens, b.qs) for j in range(k)]
    return np.asarray([b.prefix > 0 or s > 0 for s in own])


@pytest.mark.parametrize("nh,nkv,hd,lens,qs,bps", [
    (2, 2, 128, [40], [200], 3),                       # of two row tiles the first sees nothing; one key range
    (2, 2, 64, [40, 0], [200, 130], 3),
    (8, 1, 128, [5, 3], [30, 9], 2),                   # the same with eight heads a key head
    (2, 2, 128, [40], [200], 80),                      # room for several key ranges
    (80, 80, 64, [5] * 128 + [0] * 60, None, 1),       # packed rows, the second tile's sequences empty
    (80, 80, 64, [0] * 128 + [5] * 60, None, 1),       # the first tile's
    (4, 4, 128, [0] * 128 + [33] * 70, None, 3),
])
def test_a_row_tile_without_keys_beside_one_with_keys(nh, nkv, hd, lens, qs, bps):
    b = Batch(41, nh, nkv, hd, 0, lens, qs=qs, bps=bps)
    want, mag = b.want()
    sees = _sees(b)
    assert sees.any() and not sees.all()
    flush = torch.empty(1 << 28, dtype=torch.uint8, device="cuda")
    for i in range(4):
        flush.fill_(i)                                 # inputs come from memory, not from L2
        out = b.run()
        assert int(b.status.item()) == 0
        close(out, want, mag)
        assert not out[torch.from_numpy(~sees).cuda()].any()
