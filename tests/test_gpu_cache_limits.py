"""What attention over caches in 8 bits and with windows reports and how precise it is at the ends of its ranges."""

import numpy as np
import pytest

from test_gpu_attention import _f64, _i32
from test_gpu_cache_attention import F8, Cached, close

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
import rank_decomposed_gb300 as lr  # noqa: E402


@pytest.fixture(params=[0, 1, 2], ids=["chosen", "rows", "tiles"])
def kernel(request):
    lr.lib.lr_test_attention_kernel(request.param)
    yield request.param
    lr.lib.lr_test_attention_kernel(0)


@pytest.mark.parametrize("eight,window,sinks", [(True, 0, 0), (True, 40, 4), (False, 40, 4)])
@pytest.mark.parametrize("lens,qs", [([30, 7, 1], None), ([0, 0, 0], None), ([9, 3000], None), ([60, 30, 5], [50, 30, 5])])
def test_a_prefix_length_is_reported_where_there_are_no_prefix_pages(kernel, lens, qs, eight, window, sinks):
    """Whether the results of a call go straight to out or are joined."""
    b = Cached(43, 8, 2, 64, 0, lens, qs=qs, eight=eight, window=window, sinks=sinks)
    b.d.update(prefix_blocks=torch.empty(0, dtype=torch.int32, device="cuda"), prefix_len=_i32([0]))
    want = b.want()
    close(b.run(), *want, eight=eight)
    assert int(b.status.item()) == 0
    for bad in (1, -1):
        b.status.zero_()
        b.d["prefix_len"].fill_(bad)
        close(b.run(), *want, eight=eight)
        assert int(b.status.item()) == lr.LR_ERR_INDEX_RANGE, bad


