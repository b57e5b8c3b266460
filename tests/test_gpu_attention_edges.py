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


@pytest.mark.parametrize("nh,nkv,hd,prefix,lens,qs,bps", [
    (2, 2, 64, 0, [40], [200], 3),                     # one key range, two row tiles, one of them without keys
    (8, 8, 128, 40, [40], [100], 3),                   # one key range, one row tile on both rings
    (8, 1, 128, 3000, [90] * 40, None, 8),             # packed rows, several key ranges
])
def test_every_warp_gives_up_together(kernel, nh, nkv, hd, prefix, lens, qs, bps):
    """Loads that never come: the launch reports it and ends whichever of its warps notices first."""
    if kernel == 1:
        pytest.skip("the kernel by rows waits for its own copies alone")
    b = Batch(47, nh, nkv, hd, prefix, lens, qs=qs, bps=bps)
    lr.lib.lr_test_stall_producer(1)
    try:
        b.run()
    finally:
        lr.lib.lr_test_stall_producer(0)
    assert int(b.status.item()) == lr.LR_ERR_TIMEOUT
    b.status.zero_()
    close(b.run(), *b.want())
    assert int(b.status.item()) == 0
