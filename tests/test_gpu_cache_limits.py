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


@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("qs", [None, [40, 33, 70]])
@pytest.mark.parametrize("prefix", [0, 160])
def test_small_weights_beside_a_large_one(kernel, prefix, qs, hd):
    """In every 16 keys one of weight 1 and value 0 and 15 of weight e^-18 and value 1.  Such a weight is 2^-25.97, and an
    f16 of it times 2^7 is a multiple of 2^-24, off by 2^-25 at most: the sum of 15 by 15 / 16 of 2^-32 of the weights of 1.
    (A reference that lags behind the maximum only leaves more bits.)"""
    b = Cached(51, 8, 2, hd, prefix, [64, 160, 320], qs=qs)
    b.q.fill_(0)
    b.q.view(b.m, 8, hd)[:, :, 0] = 1.0
    for codes, scale in ((b.k8, b.ks), (b.v8, b.vs)):
        scale.fill_(1.0)
        codes.view(torch.uint8).zero_()
    k, v = (x.view(torch.uint8).view(b.pages, 16, 2, hd) for x in (b.k8, b.v8))
    code = lambda x: int(torch.tensor(x).to(F8).view(torch.uint8))  # noqa: E731
    k[:, 3, :, 0] = code(18.0)
    v[:] = code(1.0)
    v[:, 3] = 0
    out = torch.empty(b.m, 8 * hd, device="cuda")
    b.run(out=out, scale=1.0)
    assert int(b.status.item()) == 0
    want, mag = b.want(scale=1.0)
    if qs is None:   # (rows of turns end inside a group)
        w = np.exp(-18.0)
        assert np.allclose(want, 15 * w / (1 + 15 * w), rtol=1e-12)
    large = np.exp(-18.0) * np.ones_like(want)
    sees = want > 0.5                                 # a row that sees no key of weight 1 is exactly 1
    off = np.abs(_f64(out) - want)
    assert np.all(off[~sees] <= (18 * 2.0 ** -32 + 2.0 ** -10 * (mag + large))[~sees]), float(off[~sees].max())
    assert np.all(off[sees] <= 2.0 ** -10)


@pytest.mark.parametrize("kexp,vexp", [(124, 0), (124, -112), (-112, 100)])
@pytest.mark.parametrize("qs", [None, [60, 33, 3]])
def test_queries_and_scales_at_the_ends_of_the_range(kernel, qs, kexp, vexp):
    """Scales of K of some 2^118 under queries of 2^-124, bf16's subnormal numbers among them, and the reverse."""
    b = Cached(52, 8, 2, 128, 64, [90, 80, 200], qs=qs, sizes=0)
    b.ks *= 2.0 ** kexp
    b.vs *= 2.0 ** vexp
    q = b.q.float() * torch.exp2(-12.0 * (torch.arange(b.q.shape[1], device="cuda") % 2))   # every second one 2^-12 of it
    b.q = (q * 2.0 ** -kexp).bfloat16()
    out = torch.empty(b.m, 1024, device="cuda")
    b.run(out=out)
    assert int(b.status.item()) == 0
    close(out, *b.want(), f32=True)


@pytest.mark.parametrize("eight,window", [(True, 0), (False, 0), (True, 300)])
@pytest.mark.parametrize("prefix", [129, 272, 700])
@pytest.mark.parametrize("hd,nh,nkv,lens,qs", [(128, 3, 3, [20], None), (64, 40, 5, [0, 7], None), (128, 8, 1, [80, 1], [0, 1]),
                                               (64, 8, 2, [60, 30, 5], [50, 30, 5])])
def test_padding_rows_behind_a_prefix_of_several_tiles(kernel, hd, nh, nkv, lens, qs, prefix, eight, window):
    """Queries of NaN in rows of no sequence, whose results are joined from several parts of the prefix: zeros."""
    b = Cached(53, nh, nkv, hd, prefix, lens, qs=qs, eight=eight, window=window)
    pad = torch.full((3, nh * hd), float("nan"), dtype=torch.bfloat16, device="cuda")
    out = torch.full((b.m + 3, nh * hd), 7.0, device="cuda")
    b.run(out=out, q=torch.cat([b.q, pad]))
    assert int(b.status.item()) == 0
    assert not out[b.m:].any()
    close(out[:b.m], *b.want(), f32=True, eight=eight)


LARGE = [16, 19, 21]      # scores under 2^22 on every kernel; by rows of all sizes


@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("qs", [None, [40, 1, 70]])
@pytest.mark.parametrize("size", LARGE + [24, 28, 40])
def test_one_key_takes_all_among_large_scores(kernel, size, qs, hd):
    """Scores of some 2^size, in natural units, and a key whose score is far above the others': its values, whatever the
    scales of its page and of others are.  (A power of two times a code, and once f16's half step.)"""
    if size not in LARGE and kernel != 1:
        pytest.skip("by rows only")
    b = Cached(55, 8, 2, hd, 90, [64, 160, 320], qs=qs)
    g = torch.Generator().manual_seed(size)
    codes = lambda lo, hi, *shape: torch.randint(lo, hi, shape, generator=g).float().to(F8).view(torch.uint8).cuda()  # noqa: E731
    b.q.fill_(0)
    q, k, v = b.q.view(b.m, 8, hd), *(x.view(torch.uint8).view(b.pages, 16, 2, hd) for x in (b.k8, b.v8))
    q[:, :, 0] = 2.0 ** (size - 8)
    k.zero_()
    k[..., 0] = codes(1, 200, b.pages, 16, 2)
    v.copy_(codes(-400, 400, *v.shape))
    first = int(b.prefix_blocks[2])                       # a token of the prefix, which every row sees
    k[first, 7, :, 0] = int(torch.tensor(256.0).to(F8).view(torch.uint8))
    b.ks.fill_(1.0)
    b.vs.copy_(torch.exp2(torch.randint(-6, 6, (b.pages, 2), generator=g).float()).cuda())
    b.vs[first] = torch.tensor([2.0 ** -6, 2.0 ** 5], device="cuda")
    out = torch.empty(b.m, 8 * hd, device="cuda")
    b.run(out=out, scale=0.9)
    assert int(b.status.item()) == 0
    want = (b.v8.view(b.pages, 16, 2, hd)[first, 7].float() * b.vs[first][:, None]).double().repeat_interleave(4, 0).view(1, -1)
    assert torch.all((out.double() - want).abs() <= 2.0 ** -10 * want.abs())


@pytest.mark.parametrize("qs", [None, [40, 1, 70]])
@pytest.mark.parametrize("size", LARGE + [24, 28, 40])
def test_scores_that_differ_by_little_beside_their_size(kernel, size, qs):
    """Maxima lag behind by what the reference allows.  Results are averages of the values all the same."""
    if size not in LARGE and kernel != 1:
        pytest.skip("by rows only")
    b = Cached(54, 8, 2, 128, 90, [64, 160, 320], qs=qs)
    g = torch.Generator().manual_seed(size)
    rand = lambda n, *shape: torch.randint(0, n, shape, generator=g).cuda()  # noqa: E731
    code = lambda x: int(torch.tensor(x).to(F8).view(torch.uint8))  # noqa: E731
    b.q.fill_(0)
    q, k, v = b.q.view(b.m, 8, 128), *(x.view(torch.uint8).view(b.pages, 16, 2, 128) for x in (b.k8, b.v8))
    q[:, :, 0], q[:, :, 1] = 2.0 ** (size - 8), 1.0
    k.zero_()
    k[..., 0] = code(256.0)
    k[..., 1] = torch.arange(0.0, 24.0).to(F8).view(torch.uint8).cuda()[rand(24, b.pages, 16, 2)]
    v[:] = code(448.0)
    b.ks.fill_(1.0)
    b.vs.copy_(torch.exp2(rand(3, b.pages, 2).float()))
    out = torch.empty(b.m, 1024, device="cuda")
    b.run(out=out, scale=0.9)
    assert int(b.status.item()) == 0
    got = _f64(out)
    assert np.all(got >= 448 * (1 - 2.0 ** -10)) and np.all(got <= 448 * 4 * (1 + 2.0 ** -10))
