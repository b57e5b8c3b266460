"""The block over its context at prefill sizes and on the attention's tensor-core tiles, with either MLP."""

import numpy as np
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
import rank_decomposed_gb300 as lr  # noqa: E402
import test_gpu_block_cached as base  # noqa: E402
from test_gpu_block_cached import rows_of  # noqa: E402

MHA = dict(n_heads=4, n_kv=4, hd=128, ranks=(128, 128, 128, 128, 192, 192, 192))
RELU = dict(mlp="relu")
CONFIGS = [dict(), dict(d=1024, n_heads=8, n_kv=1, hd=128), MHA, RELU, dict(MHA, **RELU)]
NAMES = ["gqa", "mqa", "mha", "relu", "relu mha"]


@pytest.fixture(params=[0, 2], ids=["chosen", "tiles"])
def kernel(request):
    lr.lib.lr_test_attention_kernel(request.param)
    yield request.param
    lr.lib.lr_test_attention_kernel(0)


def _model(monkeypatch, n_seq, seed, prefix, pages, over):
    """A model whose shared prefix has `prefix` tokens and whose sequences have `pages` pages each."""
    monkeypatch.setattr(base, "P", prefix)
    monkeypatch.setattr(base, "CAP", pages)
    m = base.Model(n_seq, seed, **over)
    table = torch.from_numpy(lr.rope_table(prefix + 16 * pages, m.cfg["hd"])).cuda()
    m.map.cos_sin, m.table = table, table.double().cpu().numpy()
    return m


def _turns(m, seed, prefix, lens):
    starts = [0] + list(np.cumsum(lens))
    m.step(seed, [prefix + t for k in lens for t in range(k)], [r for b, k in enumerate(lens) for r in rows_of(m.pages[b], 0, k)],
           True, m.pages.numpy(), lens, starts, max(lens))


def _decode(m, seed, prefix, lens):
    rows, count, _ = lr.remap_build(lens, m.pages.numpy(), base.BR, 1, len(lens))
    assert count == len(lens)
    m.step(seed, [prefix + k - 1 for k in lens], rows, True, m.pages.numpy(), lens)


@pytest.mark.parametrize("over", CONFIGS, ids=NAMES)
def test_a_long_prompt_long_turns_and_decode(monkeypatch, kernel, over):
    """More than 256 rows: the projections are fused launches, and the attention is on tiles."""
    prefix, lens = 300, [7, 130, 1, 97, 64]
    m = _model(monkeypatch, len(lens), 41, prefix, 9, over)
    m.step(1, range(prefix), rows_of(m.prefix_pages, 0, prefix), False, m.prefix_pages.numpy()[None], [prefix], [0, prefix], prefix)
    _turns(m, 2, prefix, lens)
    for s in range(2):
        lens = [k + 1 for k in lens]
        _decode(m, 3 + s, prefix, lens)


@pytest.mark.parametrize("over", [dict(), MHA], ids=["gqa", "mha"])
def test_a_wide_decode_batch(monkeypatch, kernel, over):
    """Packed tiles behind the append: decode sizes, and more rows than the decode projections take."""
    for n in (70, 270):
        prefix, lens = 120, [1 + i % 5 for i in range(n)]
        m = _model(monkeypatch, n, 42, prefix, 1, over)
        m.step(1, range(prefix), rows_of(m.prefix_pages, 0, prefix), False, m.prefix_pages.numpy()[None], [prefix],
               [0, prefix], prefix)
        _turns(m, 2, prefix, lens)
        _decode(m, 3, prefix, [k + 1 for k in lens])
