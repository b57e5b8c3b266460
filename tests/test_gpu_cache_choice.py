"""Which kernel a call over a cache in 8 bits or with a window takes: its results are those of that kernel, bit by bit."""

import pytest

from test_gpu_cache_attention import Cached, close

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
import rank_decomposed_gb300 as lr  # noqa: E402


def _taken(b):
    """Results of the chosen kernel, and whether they are those by rows and those on tiles."""
    outs = []
    try:
        for which in (0, 1, 2):
            lr.lib.lr_test_attention_kernel(which)
            outs.append(b.run(out=torch.empty(b.m, b.nh * b.hd, device="cuda")))
            assert int(b.status.item()) == 0
    finally:
        lr.lib.lr_test_attention_kernel(0)
    return outs[0], torch.equal(outs[0], outs[1]), torch.equal(outs[0], outs[2])


# by rows, on tiles: measured times in us of batches whose sequences are all of the first one's length
@pytest.mark.parametrize("nh,nkv,hd,n,own,q,prefix,eight,window", [
    (64, 8, 128, 256, 700, 1, 0, True, 0),          # 71, 168
    (64, 8, 128, 256, 200, 1, 0, True, 0),          # 33, 61
    (8, 2, 64, 128, 4000, 1, 100, True, 0),         # 62, 108
    (56, 56, 128, 64, 50, 2, 0, True, 0),           # 28, 43
    (32, 32, 128, 256, 200, 1, 300, False, 100),    # 139, 471
    (32, 32, 128, 256, 200, 4, 0, False, 100),      # 141, 479
    (56, 56, 128, 128, 200, 1, 0, False, 500),      # 123, 413
])
def test_many_short_sequences_go_by_rows(nh, nkv, hd, n, own, q, prefix, eight, window):
    """The capacities are those of the longest sequence; the others are short."""
    qs = None if q == 1 else [min(q, 1 + i % 40) for i in range(n)]
    b = Cached(61, nh, nkv, hd, prefix, [own] + [1 + i % 40 for i in range(n - 1)], qs=qs, eight=eight, window=window)
    out, rows, tiles = _taken(b)
    assert rows and not tiles
    few = [0, 1, 2, 3, n - 1]                       # (the oracle takes some of them)
    keep = [r for i in few for r in range(b.starts[i], b.starts[i + 1])]
    b.starts = [0] + [sum(b.qs[i] for i in few[:k + 1]) for k in range(len(few))]
    b.lens, b.table = [b.lens[i] for i in few], b.table[few]
    close(out[keep], *b.want(q=b.q[keep]), f32=True, eight=eight)


@pytest.mark.parametrize("nh,nkv,hd,n,own,q,prefix,eight,window", [
    (64, 8, 128, 64, 100, 1, 4096, True, 0),
    (64, 8, 128, 4, 500, 100, 1000, True, 0),
    (64, 8, 128, 1, 1500, 1500, 0, False, 512),
])
def test_long_prefixes_and_prompts_go_on_tiles(nh, nkv, hd, n, own, q, prefix, eight, window):
    _, rows, tiles = _taken(Cached(62, nh, nkv, hd, prefix, [own] * n, qs=None if q == 1 else [q] * n, eight=eight, window=window))
    assert tiles and not rows
