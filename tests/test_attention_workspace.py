"""The workspace rule of the shared-prefix attention without a GPU: what it promises to programs that allocate once."""

import ctypes
import random

import pytest

torch = pytest.importorskip("torch")
import rank_decomposed_gb300 as lr  # noqa: E402

HEADS = [(64, 8, 128), (32, 32, 128), (8, 2, 64), (4, 4, 64), (40, 8, 128), (64, 1, 128), (7, 1, 64), (1, 1, 128),
         (4096, 4096, 64)]


def _desc(heads, br, prefix_pages, n_seq, pages, max_q, ragged):
    nh, nkv, hd = heads
    cache = lr.KvCache(0x100000, 0x200000, nkv * hd, 1 << 16, br, nkv, hd)
    return lr.AttnDesc(cache, nh, 0.1, 0x100 if prefix_pages else None, prefix_pages, 0x200 if prefix_pages else None, n_seq,
                       0x300 if ragged else None, max_q if ragged else 1, 0x400, pages, 0x500)


def _rule(M, *a):
    return lr.lib.lr_prefix_attention_workspace_bytes(M, ctypes.byref(_desc(*a)))


def _sizes(rng):
    spread = lambda hi: int(round(2 ** rng.uniform(0, hi)))  # noqa: E731
    return spread(14), spread(13) - 1, spread(10) - 1, spread(9) - 1, spread(12)  # M, prefix pages, n_seq, pages, max_q


def test_the_rule_does_not_fall_as_sizes_grow():
    rng = random.Random(1)
    for _ in range(4000):
        heads, br, ragged = rng.choice(HEADS), rng.choice((16, 48, 64)), rng.random() < 0.5
        a, b = _sizes(rng), _sizes(rng)
        low, high = [tuple(f(x, y) for x, y in zip(a, b)) for f in (min, max)]
        small, large = (_rule(s[0], heads, br, *s[1:], ragged) for s in (low, high))
        assert small <= large, (heads, br, low, high)
        assert large == _rule(high[0], heads, br, *high[1:4], 1, False)   # neither max_q nor q_start enter it


@pytest.mark.parametrize("forced", [0, 1, 2])
def test_no_smaller_call_needs_more(forced):
    """A call names what it needs when it refuses a workspace of no bytes."""
    if torch.cuda.is_available():
        pytest.skip("a call that needs nothing would be launched")
    rng = random.Random(2)
    lr.lib.lr_test_attention_kernel(forced)
    try:
        seen = 0
        for _ in range(6000):
            heads, br, ragged = rng.choice(HEADS), rng.choice((16, 48, 64)), rng.random() < 0.5
            large = _sizes(rng)
            M, pre, n, pages, mq = (rng.choice((x, rng.randint(min(x, 1), x))) for x in large)
            if not ragged:
                n = min(n, M)
            d = _desc(heads, br, pre, n, pages, mq, ragged)
            w = heads[0] * heads[2]
            st = lr.lib.lr_prefix_attention(0x10000, w, 0x20000, w, 0, M, ctypes.byref(d), 0x30000, 0, None, None)
            assert st in (lr.LR_ERR_INVALID_ARG, lr.LR_ERR_CUDA, lr.LR_ERR_UNSUPPORTED)
            if st == lr.LR_ERR_INVALID_ARG:
                assert "workspace 0 <" in lr.last_error(), lr.last_error()
                need = int(lr.last_error().split("<")[1].split()[0])
                assert need <= _rule(large[0], heads, br, *large[1:], ragged), (heads, br, large, (M, pre, n, pages, mq, ragged))
                seen += 1
        assert seen > 2000
    finally:
        lr.lib.lr_test_attention_kernel(0)


def test_one_workspace_for_a_decode_batch_of_any_size():
    """512 prefix pages and 32 own pages of 16 rows, 64 heads over 8: the call needs 18 MB at 64 rows, none at 512."""
    sizes = [_rule(M, (64, 8, 128), 16, 512, M, 32, 1, False) for M in (1, 64, 256, 512, 4096)]
    assert sizes == sorted(sizes) and sizes[1] >= 18 << 20 and sizes[-1] < 48 << 20


@pytest.mark.parametrize("kernel", [0, 1, 2])
@pytest.mark.parametrize("nh,nkv,n_seq,mq", [(32, 8, 1 << 29, 5), (8, 8, 1 << 30, 1)])
def test_too_many_sequences_for_a_launch_are_refused_before_anything_is_enqueued(kernel, nh, nkv, n_seq, mq):
    d, w = _desc((nh, nkv, 128), 16, 3, n_seq, 4, mq, True), nh * 128
    lr.lib.lr_test_attention_kernel(kernel)
    try:
        st = lr.lib.lr_prefix_attention(0x10000, w, 0x20000, w, 0, 9, ctypes.byref(d), 0x30000, 1 << 40, None, None)
    finally:
        lr.lib.lr_test_attention_kernel(0)
    assert st == lr.LR_ERR_UNSUPPORTED and "one launch" in lr.last_error()
