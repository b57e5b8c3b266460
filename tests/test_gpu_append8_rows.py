"""The append to a cache in 8 bits where rows and heads have no number to scale by: heads of zeros under a norm, rows of
NaN, and rows that are skipped, in calls whose warps hold one run of rows, several, or a part of one."""

import numpy as np
import pytest

from test_gpu_append8 import _cache, _check, _copy, _err, _f64
from test_gpu_heads import _map, _rand, _status, _want

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
import rank_decomposed_gb300 as lr  # noqa: E402

# hd, rows a page, key heads, tokens at least: a warp holds 16 rows (32 with heads of 64, 8 with 256), a CTA four times as
# many, and beyond that pages are walked; long calls give a warp several runs, without a norm two heads, too
SIZES = [(128, 16, 2, 20), (128, 16, 8, 900), (64, 16, 40, 1200), (128, 64, 2, 100), (128, 64, 8, 900), (64, 64, 8, 900),
         (128, 256, 2, 300), (64, 256, 8, 1200), (192, 5, 3, 40), (256, 48, 8, 700)]


def _runs(br, least):
    """(page, first row in the page, tokens) of runs of all lengths, whose first rows open a page or follow others."""
    lengths = [1, br, 2, 1, 1, 3, br - 1, 1, 2 * br + 3, 1, br // 2 + 1, 1, 1, 5, 1]
    runs, page, m, i = [], 0, 0, 0
    while m < least or i < len(lengths):
        n, first = max(1, lengths[i % len(lengths)]), 0 if i % 3 == 0 else (5 * i) % br
        runs.append((page, first, n))
        page += (first + n - 1) // br + 1 + i % 2
        m, i = m + n, i + 1
    return runs


class Call:
    """An append of keys and values to the rows of `runs`; run[i] is the run of token i, place[i] its place there."""

    def __init__(self, hd, br, nkv, least, norm, style, dtype, eps=1e-6, seed=1):
        self.hd, self.br, self.nkv, self.style = hd, br, nkv, style
        self.runs = _runs(br, least)
        at = [(page * br + first + j, i, j) for i, (page, first, n) in enumerate(self.runs) for j in range(n)]
        self.rows, self.run, self.place = (np.array(x) for x in zip(*at))
        self.m = len(at)
        self.cache = _cache(int(self.rows.max()) // br + 2, br, nkv, hd, seed)
        self.hm = _map(hd, norm, hd if style == "half" else 32, style, seed + 10)
        self.hm.eps = eps
        self.k, self.v = (_rand((self.m, nkv * hd), seed + s, dtype) for s in (20, 30))
        self.pos = torch.randint(0, 5000, (self.m,), generator=torch.Generator().manual_seed(seed)).int()

    def heads(self, x):
        return x.view(self.m, self.nkv, self.hd)

    def check(self, status=0):
        """Against the oracle, whose call has only the rows at positions within the table."""
        before, st = _copy(self.cache), _status()
        i32 = lambda a: torch.as_tensor(a, dtype=torch.int32).cuda()  # noqa: E731
        lr.kv_append(self.k, self.v, i32(self.pos), i32(self.rows), self.hm, self.cache, st)
        torch.cuda.synchronize()
        assert int(st.item()) == status
        ok = np.flatnonzero((self.pos.numpy() >= 0) & (self.pos.numpy() < 5000))
        with np.errstate(invalid="ignore"):
            kx = _want(self.k[ok], self.hm, self.hm.k_gain, self.pos.numpy()[ok], self.style)
            vx = _f64(self.v[ok])
        kx, vx = kx.reshape(-1, self.nkv, self.hd), vx.reshape(-1, self.nkv, self.hd)
        rows = self.rows[ok].tolist()
        with np.errstate(invalid="ignore"):
            _check(self.cache.k_pool, self.cache.k_scale, before.k_pool, before.k_scale, kx, rows, self.br, _err(kx))
            _check(self.cache.v_pool, self.cache.v_scale, before.v_pool, before.v_scale, vx, rows, self.br, 0 * np.nan_to_num(vx))


@pytest.mark.parametrize("hd,br,nkv,least", SIZES)
@pytest.mark.parametrize("style,dtype,eps", [("half", torch.bfloat16, 1e-6), ("pair", torch.float32, 1e-5), ("half", torch.float32, 1e-12)])
def test_heads_of_zeros_with_a_norm(hd, br, nkv, least, style, dtype, eps):
    """Zeros stay zeros: in pages of nothing else, beside rows that are not, and behind a page's earlier rows of zeros."""
    c = Call(hd, br, nkv, least, True, style, dtype, eps)
    run, first = torch.from_numpy(c.run).cuda(), torch.from_numpy(c.place).cuda() == 0
    for x in (c.heads(c.k), c.heads(c.v)):
        x[:, -1] = 0
        x[run % 4 == 0] = 0
        x[(run % 4 == 1), 0] = 0
        x[(run % 4 == 2) & first] = 0
    for i, (page, at, n) in enumerate(c.runs):
        if at > 0 and i % 2:                        # what the page holds is zeros, too
            for pool, scale in ((c.cache.k_pool, c.cache.k_scale), (c.cache.v_pool, c.cache.v_scale)):
                pool.view(torch.uint8)[page * br:page * br + at] = 0
                scale[page] = 2.0 ** -120
    c.check()


@pytest.mark.parametrize("hd,br,nkv,least", SIZES)
@pytest.mark.parametrize("norm,style,dtype", [(True, "half", torch.bfloat16), (False, "pair", torch.float32), (False, "half", torch.bfloat16)])
def test_rows_of_nan(hd, br, nkv, least, norm, style, dtype):
    """A row without a finite element counts for nothing in its page's scale: alone, as all of a run, and among others.
    With a norm one NaN makes a head's row of them."""
    c = Call(hd, br, nkv, least, norm, style, dtype)
    run, place = torch.from_numpy(c.run).cuda(), torch.from_numpy(c.place).cuda()
    k, v = c.heads(c.k), c.heads(c.v)
    for rows in (run % 3 == 1, place % 7 == 3):     # whole runs; some rows of the others
        k[rows, 0, 3 if norm else slice(None)] = float("nan")
        v[rows, 0] = float("nan")
        k[rows, -1] = float("nan")
    v[run % 5 == 2] = float("nan")
    c.check()


@pytest.mark.parametrize("hd,br,nkv,least", SIZES)
@pytest.mark.parametrize("norm,style,dtype", [(True, "half", torch.bfloat16), (False, "pair", torch.float32), (False, "half", torch.bfloat16)])
def test_skipped_rows_are_none_of_a_page_s_new_rows(hd, br, nkv, least, norm, style, dtype):
    """Positions out of range: the first row of a run, its first ones, all of them.  A page without a new row keeps its
    scales, and in one whose first rows are skipped those before the first new one keep what they stand for."""
    c = Call(hd, br, nkv, least, norm, style, dtype)
    for i, (page, at, n) in enumerate(c.runs):
        rows = np.flatnonzero(c.run == i)
        bad = {0: rows, 1: rows[:1], 2: rows[:3], 3: rows[:0], 4: rows[:-1], 5: rows[1::2], 6: rows[:40]}[i * 5 % 7]
        c.pos[bad] = 5000 if i % 2 else -1
    c.check(lr.LR_ERR_INDEX_RANGE)
