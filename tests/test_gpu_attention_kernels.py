"""Every test of the shared-prefix attention on either of its kernels, whichever its sizes would choose."""

import pytest

torch = pytest.importorskip("torch")
import rank_decomposed_gb300 as lr  # noqa: E402
from test_gpu_attention import *  # noqa: E402,F401,F403
from test_gpu_attention import Batch, close  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True, params=[1, 2], ids=["rows", "tiles"])
def kernel(request):
    lr.lib.lr_test_attention_kernel(request.param)
    yield request.param
    lr.lib.lr_test_attention_kernel(0)


@pytest.mark.parametrize("nh,nkv,hd,prefix,lens,qs", [
    (1, 1, 128, 1, [1], None),                                 # one row, one head, two keys
    (64, 1, 128, 40, [3, 0, 17], None),                        # the most heads a key head, two query rows a tile
    (33, 1, 64, 500, [9, 100, 33, 20], [9, 1, 33, 2]),         # three query rows a tile, 99 of 128 rows used
    (12, 4, 64, 3000, [1 + i % 7 for i in range(79)], None),
    (40, 8, 128, 100, [20] * 57, None),
    (16, 2, 64, 128, [256, 128, 16], [2, 3, 1]),               # contexts that end with a tile and a group of keys
])
def test_more_shapes(nh, nkv, hd, prefix, lens, qs):
    b = Batch(31, nh, nkv, hd, prefix, lens, qs=qs)
    out = b.run()
    assert int(b.status.item()) == 0
    close(out, *b.want())


@pytest.mark.parametrize("qs", [[0, 30, 200], [0, 1, 2]])
def test_a_prefix_length_is_reported_when_the_first_sequence_has_no_rows(qs):
    b = Batch(33, 8, 2, 64, 64, [5, 40, 208], qs=qs, pcap=4)
    b.d["prefix_len"].fill_(65)
    close(b.run(), *b.want())
    assert int(b.status.item()) == lr.LR_ERR_INDEX_RANGE


@pytest.mark.parametrize("nh,nkv,hd,n", [(8, 1, 128, 700), (4, 4, 64, 513)])
def test_a_prompt_alone(nh, nkv, hd, n):
    """Many row tiles of one sequence, the last of them first: every row sees itself and what is before it."""
    b = Batch(34, nh, nkv, hd, 0, [n], qs=[n])
    out = b.run()
    assert int(b.status.item()) == 0
    close(out, *b.want())


def test_a_stalled_load_is_reported_and_the_next_call_is_right(kernel):
    """The producers of the tiles issue nothing: every wait of the launch runs out, and it returns."""
    for qs in (None, [30, 1, 200]):
        b = Batch(32, 8, 1, 128, 700, [90, 21, 210], qs=qs)
        lr.lib.lr_test_stall_producer(1)
        try:
            out = b.run()
        finally:
            lr.lib.lr_test_stall_producer(0)
        if kernel == 1:  # the kernel by rows waits for its own copies alone
            assert int(b.status.item()) == 0
            close(out, *b.want())
            continue
        assert int(b.status.item()) == lr.LR_ERR_TIMEOUT
        b.status.zero_()
        close(b.run(), *b.want())
        assert int(b.status.item()) == 0
