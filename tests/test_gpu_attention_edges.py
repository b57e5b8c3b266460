"""Attention over a context at its edges, on either of its kernels: rows, sequences and parts without keys."""

import numpy as np
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
import oracle  # noqa: E402
import rank_decomposed_gb300 as lr  # noqa: E402
from test_gpu_attention import Batch, _f64, _i32, close  # noqa: E402


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


@pytest.mark.parametrize("prefix,qs", [(64, None), (0, None), (64, [40, 1, 20]), (0, [40, 1, 20]), (64, [2, 1, 3]), (700, None)])
def test_lengths_and_row_offsets_are_reported_where_there_are_no_pages(prefix, qs):
    b = Batch(42, 8, 2, 64, prefix, [0, 0, 0], qs=qs)
    b.d["block_table"] = torch.empty(3, 0, dtype=torch.int32, device="cuda")
    want = b.want()
    close(b.run(), *want)
    assert int(b.status.item()) == 0
    for bad in (1, -1, 1 << 30):
        b.status.zero_()
        b.d["lengths"][1] = bad
        close(b.run(), *want)
        assert int(b.status.item()) == lr.LR_ERR_INDEX_RANGE, bad
    b.d["lengths"][1] = 0
    if qs is not None:
        for i, bad in ((1, b.starts[2] + 1), (2, b.m + 1), (0, -1)):
            b.status.zero_()
            b.d["q_start"][i] = bad
            b.run()
            assert int(b.status.item()) == lr.LR_ERR_INDEX_RANGE, (i, bad)
            b.d["q_start"][i] = b.starts[i]
        b.status.zero_()
        b.d["max_q"] -= 1
        b.run()
        assert int(b.status.item()) == lr.LR_ERR_INDEX_RANGE


@pytest.mark.parametrize("lens", [[30, 7, 1], [0, 0, 0]])
def test_a_prefix_length_is_reported_where_there_are_no_prefix_pages(lens):
    b = Batch(43, 8, 2, 64, 0, lens)
    b.d.update(prefix_blocks=torch.empty(0, dtype=torch.int32, device="cuda"), prefix_len=_i32([0]))
    want = b.want()
    close(b.run(), *want)
    assert int(b.status.item()) == 0
    for bad in (1, -1):
        b.status.zero_()
        b.d["prefix_len"].fill_(bad)
        close(b.run(), *want)
        assert int(b.status.item()) == lr.LR_ERR_INDEX_RANGE, bad


@pytest.mark.parametrize("qs", [[3, 0, 5], [70, 0, 5]])
@pytest.mark.parametrize("stale", [-7, 1 << 30])
def test_the_length_of_a_sequence_without_rows_is_not_reported(qs, stale):
    """A place of the batch that is empty may hold any length, whichever kernel runs."""
    b = Batch(44, 8, 2, 64, 100, [80, 0, 33], qs=qs)
    b.d["lengths"][1] = stale
    close(b.run(), *b.want())
    assert int(b.status.item()) == 0


@pytest.mark.parametrize("qs,max_q", [([10, 30, 5], 29), ([10, 30, 5], 12), ([2, 7, 3], 5), ([70, 300, 20], 260)])
def test_rows_up_to_max_q_of_a_sequence_with_more_are_right(qs, max_q):
    b = Batch(45, 8, 2, 64, 100, [40, 310, 33], qs=qs)
    b.d["max_q"] = max_q
    out = b.run()
    assert int(b.status.item()) == lr.LR_ERR_INDEX_RANGE
    want, mag = b.want()
    keep = [r for i, (s, n) in enumerate(zip(b.starts, qs)) for r in range(s, s + min(n, max_q))]
    close(out[keep], want[keep], mag[keep])


@pytest.mark.parametrize("nh,nkv,hd,n,bps", [(8, 1, 128, 3, 4), (4, 4, 64, 5, 4), (8, 1, 128, 60, 4), (4, 4, 128, 200, 4),
                                             (80, 80, 64, 3, 1), (8, 2, 64, 9, 300)])
@pytest.mark.parametrize("ragged", [False, True])
def test_scores_of_minus_infinity(nh, nkv, hd, n, bps, ragged):
    """Such a key has no weight beside others; a row whose tokens all have that score is NaN, as its softmax is."""
    qs = [1 + i % 2 for i in range(n)] if ragged else None
    for prefix in (0, 70):
        lens = [i % 3 * 7 for i in range(n)]            # sequences 0, 3, .. see the prefix alone
        b = Batch(46, nh, nkv, hd, prefix, lens, qs=qs, bps=bps)
        b.q.view(b.m, nh, hd)[:, :, 0] = 1.0
        low = b.rows_of(b.prefix_blocks, prefix)        # all of the prefix, all of some sequences, a part of others
        for i in range(n):
            rows = b.rows_of(b.table[i], lens[i])
            low += rows if i % 2 else rows[: len(rows) // 2]
        b.kp.view(-1, nkv, hd)[low, :, 0] = float("-inf")
        with np.errstate(invalid="ignore"):
            kp, vp = (np.where(np.isnan(x), 0.0, x) for x in (_f64(b.kp), _f64(b.vp)))
            want, mag = oracle.prefix_attention(_f64(b.q), kp, vp, nh, nkv, hd, b.br, b.prefix_blocks.numpy(), prefix,
                                                b.table.numpy(), b.lens, b.starts, hd ** -0.5)
        out = b.run()
        assert int(b.status.item()) == 0
        nan = np.isnan(want)
        assert nan.any() and not nan.all()
        assert np.array_equal(np.isnan(_f64(out)), nan)
        ok = ~nan.any(1)
        close(out[torch.from_numpy(ok).cuda()], want[ok], mag[ok])


def test_a_workspace_for_the_largest_batch_serves_smaller_ones(kernel):
    """Sized once, by the rule, for 300 sequences; the calls need more of it, less of it or nothing as sizes change."""
    lr.lib.lr_test_attention_kernel(0)                 # the kernel that the sizes choose
    full = Batch(48, 16, 2, 128, 700, [1 + i % 40 for i in range(300)])
    ws = full.workspace()
    for n in (1, 2, 9, 40, 130, 300):
        b = Batch(49, 16, 2, 128, 700, [1 + i % 40 for i in range(n)])
        assert lr.prefix_attention_workspace_bytes(n, 16, b.cache(), **b.d) <= ws.numel()
        ws.fill_(0xFF)
        out = b.run(ws=ws)
        assert int(b.status.item()) == 0
        close(out, *b.want())
