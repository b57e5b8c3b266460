"""GPU parity of attention over a shared prefix and own paged tokens."""

import numpy as np
import pytest

import oracle

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
import rank_decomposed_gb300 as lr  # noqa: E402


def _f64(t):
    return t.double().cpu().numpy()


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


class Batch:
    """A batch whose pool holds NaN wherever no token of it lies."""

    def __init__(self, seed, nh, nkv, hd, prefix, lens, qs=None, br=16, extra=3, loud=2.0, bps=None, pcap=None):
        g = torch.Generator().manual_seed(seed)
        self.nh, self.nkv, self.hd, self.br, self.prefix, self.lens = nh, nkv, hd, br, prefix, lens
        self.qs = [1] * len(lens) if qs is None else qs
        self.starts = [0] + list(np.cumsum(self.qs))
        self.m = int(self.starts[-1])
        pb = pcap or -(-prefix // br)
        bps = bps or max([1] + [-(-n // br) for n in lens])
        perm = torch.randperm(pb + len(lens) * bps + extra, generator=g).int()
        self.pages = perm.numel()
        self.prefix_blocks, self.table = perm[:pb].contiguous(), perm[pb:pb + len(lens) * bps].view(len(lens), bps).contiguous()
        w = nkv * hd
        kp, vp = (torch.full((self.pages * br, w), float("nan")) for _ in range(2))
        at = self.rows_of(self.prefix_blocks, prefix)
        for b, n in enumerate(lens):
            at = at + self.rows_of(self.table[b], n)
        if at:
            kp[at] = torch.randn(len(at), w, generator=g) * loud
            vp[at] = torch.randn(len(at), w, generator=g) + 0.25
        self.kp, self.vp = kp.bfloat16().cuda(), vp.bfloat16().cuda()
        self.q = torch.randn(self.m, nh * hd, generator=g).bfloat16().cuda()
        self.ragged = qs is not None
        self.d = dict(prefix_blocks=self.prefix_blocks.cuda() if pb else None, prefix_len=_i32([prefix]) if pb else None,
                      block_table=self.table.cuda(), lengths=_i32(lens), q_start=_i32(self.starts) if self.ragged else None,
                      max_q=max([1] + self.qs))
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")

    def rows_of(self, pages, n):
        return [int(pages[t // self.br]) * self.br + t % self.br for t in range(n)]

    def cache(self):
        return lr.PagedKV(self.kp, self.vp, self.nkv, self.hd, self.br)

    def workspace(self, m=None):
        n = lr.prefix_attention_workspace_bytes(m or max(1, self.m), self.nh, self.cache(), **self.d)
        return torch.full((max(n, 256),), 0xFF, dtype=torch.uint8, device="cuda")   # NaNs, if read unwritten

    def run(self, out=None, q=None, ws=None, **kw):
        q = self.q if q is None else q
        out = torch.full((q.shape[0], self.nh * self.hd), 7.0, dtype=torch.bfloat16, device="cuda") if out is None else out
        lr.prefix_attention(q, self.nh, self.cache(), out=out, workspace=ws if ws is not None else self.workspace(q.shape[0]),
                            status=self.status, **dict(self.d, **kw))
        torch.cuda.synchronize()
        return out

    def want(self, scale=None, q=None, rows=None):
        scale = self.hd ** -0.5 if scale is None else scale
        return oracle.prefix_attention(_f64(self.q if q is None else q), np.nan_to_num(_f64(self.kp)), np.nan_to_num(_f64(self.vp)),
                                       self.nh, self.nkv, self.hd, self.br, self.prefix_blocks.numpy(), self.prefix,
                                       self.table.numpy(), self.lens, self.starts, scale)


def close(y, want, mag, f32=False):
    """Each probability is off by 2^-8 of itself (its rounding to bf16), so a result by 2^-8 sum p |v|; a bf16 result
    rounds once more, by 2^-8 of itself; fp32 scores and sums add a sixteenth of the first."""
    bound = 2.0 ** -8 * (17 / 16 * mag + (0 if f32 else np.abs(want))) + 1e-30
    got = _f64(y)
    assert np.all(np.isfinite(got))
    worst = float((np.abs(got - want) / bound).max()) if want.size else 0.0
    assert worst <= 1.0, worst


DECODE = [  # nh, nkv, hd, prefix, own lengths, rows a page
    (8, 2, 64, 200, [1, 17, 40], 16),
    (64, 8, 128, 1000, [5, 1, 16, 33, 250, 128], 16),
    (4, 4, 128, 77, [1], 16),
    (32, 32, 128, 130, [3, 64, 200], 16),
    (14, 2, 128, 300, [9, 10, 11], 48),            # seven heads a key head, pages that are no power of two
    (6, 2, 64, 1, [1, 2], 64),                     # a prefix of one token
    (8, 1, 128, 129, [31, 1, 100, 7, 64, 65, 3, 2, 90, 12, 13, 14, 15, 16, 17, 18, 19], 32),   # 136 rows a key head
    (40, 8, 64, 511, [100] * 20, 16),              # 100 rows a key head
    (8, 8, 64, 640, [20 + i for i in range(140)], 16),   # 140 rows a key head, one head each
    (64, 8, 128, 4100, [20] * 40, 64),             # 320 rows a key head, several key ranges
    (64, 1, 64, 900, [40, 41, 42, 43, 44], 16),    # all heads share one key head: 320 rows
]


@pytest.mark.parametrize("nh,nkv,hd,prefix,lens,br", DECODE)
def test_one_row_a_sequence_matches_oracle(nh, nkv, hd, prefix, lens, br):
    b = Batch(1, nh, nkv, hd, prefix, lens, br=br)
    out = b.run()
    assert int(b.status.item()) == 0
    close(out, *b.want())


RAGGED = [  # nh, nkv, hd, prefix, own lengths, query rows, rows a page
    (8, 2, 64, 100, [30, 7, 64], [30, 3, 1], 16),
    (8, 1, 128, 260, [150, 40, 129], [150, 17, 100], 16),
    (8, 8, 128, 131, [300, 3], [130, 3], 16),
    (6, 2, 128, 64, [200, 128, 90], [200, 128, 70], 32),
    (7, 1, 64, 500, [257], [257], 16),             # seven heads: 126 rows of a tile of 128 hold queries
    (16, 2, 128, 700, [400, 1, 300, 0, 260], [400, 0, 290, 0, 5], 64),
    (4, 4, 64, 33, [600, 500], [600, 33], 16),
]


@pytest.mark.parametrize("nh,nkv,hd,prefix,lens,qs,br", RAGGED)
def test_ragged_rows_match_oracle(nh, nkv, hd, prefix, lens, qs, br):
    b = Batch(2, nh, nkv, hd, prefix, lens, qs=qs, br=br)
    out = b.run()
    assert int(b.status.item()) == 0
    close(out, *b.want())


FEW_ROWS = [  # some query rows a sequence, packed into tiles that cut through sequences
    (8, 2, 64, 100, [30, 7, 64, 9, 150], [3, 1, 7, 9, 2], 16),
    (8, 1, 128, 300, [5, 140, 2, 0, 33, 260], [5, 8, 8, 0, 0, 7], 16),       # rows before their tokens, no rows
    (4, 4, 128, 131, [40 + i for i in range(20)], [1 + i % 9 for i in range(20)], 32),
    (2, 2, 64, 0, [130 * (i % 3) + 1 for i in range(150)], [1 + i % 3 for i in range(150)], 16),   # two tiles, no prefix
    (28, 4, 128, 700, [20, 300, 129], [9, 9, 9], 48),                        # seven heads a key head
    (6, 3, 128, 0, [0] * 12, [3] * 12, 16),                                  # nothing to see at all
]


@pytest.mark.parametrize("nh,nkv,hd,prefix,lens,qs,br", FEW_ROWS)
def test_few_rows_a_sequence_match_oracle(nh, nkv, hd, prefix, lens, qs, br):
    b = Batch(22, nh, nkv, hd, prefix, lens, qs=qs, br=br)
    out = b.run()
    assert int(b.status.item()) == 0
    close(out, *b.want())


@pytest.mark.parametrize("nh,nkv,hd,n,bad", [(8, 1, 128, 40, 7), (8, 1, 128, 3, 1), (4, 4, 64, 200, 130), (64, 8, 128, 20, 0),
                                             (16, 2, 64, 1, 0)])
@pytest.mark.parametrize("what", [float("nan"), float("inf")])
def test_one_sequence_s_values_do_not_reach_another(nh, nkv, hd, n, bad, what):
    """NaN or infinities among a sequence's own values show in its rows alone, though rows share their tiles."""
    b = Batch(23, nh, nkv, hd, 260, [5 + 37 * i % 200 for i in range(n)])
    want, mag = b.want()
    clean = b.run()
    b.vp[b.rows_of(b.table[bad], b.lens[bad])] = what
    out = b.run()
    rest = [i for i in range(n) if i != bad]
    assert not torch.isfinite(out[bad]).any()
    assert torch.equal(out[rest], clean[rest])
    close(out[rest], want[rest], mag[rest])


@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("nh,nkv", [(8, 2), (2, 2), (16, 1)])
def test_rows_that_see_nothing_are_zero(hd, nh, nkv):
    """No prefix, no own tokens, more rows than tokens, sequences without rows, rows of no sequence."""
    b = Batch(3, nh, nkv, hd, 0, [0, 2, 30, 5], qs=[3, 5, 0, 5])
    out = b.run()
    want, mag = b.want()
    assert int(b.status.item()) == 0
    close(out, want, mag)
    assert not out[:6].any()                       # three of the empty sequence, three that precede its two tokens
    b = Batch(4, nh, nkv, hd, 50, [0, 1])          # an own length of zero leaves the prefix
    close(b.run(), *b.want())
    b = Batch(5, nh, nkv, hd, 40, [4, 9], qs=[2, 3])
    q = torch.cat([b.q, b.q[:4]])
    out = b.run(q=q)
    close(out[:5], *b.want())
    assert not out[5:].any()


def test_no_shared_part_and_no_own_part():
    b = Batch(6, 8, 2, 128, 0, [100, 37, 1])
    assert b.d["prefix_blocks"] is None
    close(b.run(), *b.want())
    b = Batch(7, 8, 2, 128, 300, [0, 0])           # nothing of their own
    close(b.run(), *b.want())
    b.d["block_table"] = torch.empty(2, 0, dtype=torch.int32, device="cuda")
    close(b.run(), *b.want())


@pytest.mark.parametrize("rows", ["decode", "ragged"])
def test_capacities_beyond_the_lengths_do_not_matter(rows):
    """Tables with room for far more tokens, whose unused entries are no pages at all."""
    qs = None if rows == "decode" else [40, 1, 20]
    b = Batch(8, 8, 1, 128, 140, [90, 3, 21], qs=qs, bps=300, pcap=400)
    want = b.want()
    b.d["prefix_blocks"][9:] = -1
    for i, n in enumerate(b.lens):
        b.d["block_table"][i, -(-n // 16):] = 1 << 30
    out = b.run()
    assert int(b.status.item()) == 0
    close(out, *want)


def test_fp32_output_strided_rows_scale_and_joint_pool():
    b = Batch(9, 16, 2, 64, 333, [50, 60, 70])
    pool = torch.cat([b.kp, b.vp, b.kp], 1)        # [K | V | other] rows
    b.kp, b.vp = pool[:, :128], pool[:, 128:256]
    wide = torch.zeros(3, 16 * 64 + 24, dtype=torch.bfloat16, device="cuda")
    wide[:, 8:8 + 1024] = b.q
    out = torch.full((3, 1024 + 8), 7.0, dtype=torch.float32, device="cuda")
    b.run(out=out[:, :1024], q=wide[:, 8:8 + 1024], scale=0.31)
    close(out[:, :1024], *b.want(scale=0.31), f32=True)
    assert torch.all(out[:, 1024:] == 7.0)


@pytest.mark.parametrize("hd,nh,nkv,n", [(128, 8, 1, 3), (128, 8, 1, 40), (64, 4, 4, 5), (64, 8, 2, 70)])
def test_large_scores_and_one_key_that_takes_all(hd, nh, nkv, n):
    """Scores of some hundreds in natural units, rising along the keys: maxima move in every tile."""
    b = Batch(10, nh, nkv, hd, 600, [30 + i % 40 for i in range(n)], loud=30.0)
    at = b.rows_of(b.prefix_blocks, 600)
    b.kp[at] *= torch.linspace(0.1, 2.0, 600, device="cuda")[:, None].bfloat16()
    out = b.run()
    want, mag = b.want()
    # a score of 1000 natural units has an fp32 error of about 1000 * 2^-22, which the power turns into a relative one
    bound = 2.0 ** -8 * (17 / 16 * mag + np.abs(want)) + 2.0 ** -11 * (mag + 1)
    assert np.all(np.abs(_f64(out) - want) <= bound)


def test_results_do_not_depend_on_the_run():
    for qs in (None, [60, 200, 3]):
        b = Batch(11, 8, 1, 128, 2000, [90, 210, 33], qs=qs)
        first = b.run()
        for _ in range(3):
            assert torch.equal(b.run(), first)


@pytest.mark.parametrize("qs", [None, [30, 1, 200]])
def test_lengths_outside_their_capacity_are_clamped_and_reported(qs):
    b = Batch(12, 8, 2, 64, 64, [48, 16, 208], qs=qs, bps=13, pcap=4)
    b.kp.nan_to_num_(0.5), b.vp.nan_to_num_(0.25)
    b.d["prefix_len"].fill_(65)
    close(b.run(), *b.want())
    assert int(b.status.item()) == lr.LR_ERR_INDEX_RANGE
    for bad, clamped in ((-5, 0), (1 << 30, 208)):
        b.status.zero_(), b.d["prefix_len"].fill_(64)
        b.d["lengths"][1] = bad
        b.lens[1] = clamped
        close(b.run(), *b.want())
        assert int(b.status.item()) == lr.LR_ERR_INDEX_RANGE


def test_row_offsets_that_are_wrong_are_reported():
    """Only the report and the untouched rows around the output are promised."""
    for starts, max_q in (([0, 40, 20, 50], 50), ([-3, 10, 20, 50], 50), ([0, 10, 20, 1 << 30], 50), ([0, 30, 31, 50], 29)):
        b = Batch(13, 8, 2, 64, 64, [48, 16, 200], qs=[10, 10, 30])
        b.d.update(q_start=_i32(starts), max_q=max_q)
        out = torch.full((52, 512), 7.0, dtype=torch.bfloat16, device="cuda")
        b.run(out=out[1:51])
        assert int(b.status.item()) == lr.LR_ERR_INDEX_RANGE, starts
        assert torch.all(out[0] == 7.0) and torch.all(out[51] == 7.0)
    for starts, max_q in (([0, 8, 4, 10], 8), ([-3, 2, 6, 10], 8), ([0, 2, 6, 1 << 30], 8), ([0, 3, 4, 10], 5)):
        b = Batch(13, 8, 2, 64, 64, [48, 16, 200], qs=[2, 2, 6])
        b.d.update(q_start=_i32(starts), max_q=max_q)
        out = torch.full((12, 512), 7.0, dtype=torch.bfloat16, device="cuda")
        b.run(out=out[1:11])
        assert int(b.status.item()) == lr.LR_ERR_INDEX_RANGE, starts
        assert torch.all(out[0] == 7.0) and torch.all(out[11] == 7.0)


@pytest.mark.parametrize("n", [3, 40])
def test_pages_outside_the_pool_read_as_zeros_and_are_reported(n):
    b = Batch(14, 8, 1, 128, 200, [40] * n)
    b.prefix_blocks[5], b.table[1, 0], b.table[2, 1] = -1, b.pages, 1 << 30
    b.d.update(prefix_blocks=b.prefix_blocks.cuda(), block_table=b.table.cuda())
    out = b.run()
    assert int(b.status.item()) == lr.LR_ERR_REMAP_RANGE
    close(out, *b.want())


def test_offsets_beyond_32_bits():
    """Pools of more than 2^31 elements each, with the batch's pages at their ends."""
    nkv, hd, br = 8, 128, 16
    pages = (1 << 31) // (nkv * hd * br) + 64
    b = Batch(15, 64, nkv, hd, 150, [33, 70, 1])
    kp = torch.zeros(pages * br, nkv * hd, dtype=torch.bfloat16, device="cuda")
    vp = torch.zeros_like(kp)
    shift = pages - b.pages
    kp[shift * br:], vp[shift * br:] = b.kp, b.vp
    want = b.want()
    b.kp, b.vp = kp, vp
    b.d.update(prefix_blocks=b.d["prefix_blocks"] + shift, block_table=b.d["block_table"] + shift)
    close(b.run(), *want)
    b2 = Batch(16, 64, nkv, hd, 150, [133, 70], qs=[100, 70])
    kp[shift * br:], vp[shift * br:] = 0, 0
    shift = pages - b2.pages
    kp[shift * br:], vp[shift * br:] = b2.kp, b2.vp
    want = b2.want()
    b2.kp, b2.vp = kp, vp
    b2.d.update(prefix_blocks=b2.d["prefix_blocks"] + shift, block_table=b2.d["block_table"] + shift)
    close(b2.run(), *want)


@pytest.mark.parametrize("ragged", [False, True])
def test_captured_once_it_serves_other_batches(ragged):
    """On a stream of its own, in a graph: new lengths, offsets, pages and queries between replays."""
    first = Batch(17, 16, 2, 128, 500, [100, 30, 5, 64], qs=[40, 30, 1, 10] if ragged else None, bps=30, pcap=60)
    later = Batch(18, 16, 2, 128, 900, [10, 400, 77, 1], qs=[10, 2, 77, 1] if ragged else None, bps=30, pcap=60)
    m = 100 if ragged else 4
    first.d["max_q"] = 80 if ragged else 1
    q = torch.zeros(m, 16 * 128, dtype=torch.bfloat16, device="cuda")
    out = torch.zeros_like(q)
    q[:first.m] = first.q
    ws, s = first.workspace(m), torch.cuda.Stream()
    call = lambda: lr.prefix_attention(q, 16, first.cache(), out=out, workspace=ws, status=first.status, stream=s, **first.d)
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        call()
    s.synchronize()
    close(out[:first.m], *first.want())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        call()
    assert later.kp.shape == first.kp.shape
    q.zero_()
    q[:later.m] = later.q
    first.kp.copy_(later.kp), first.vp.copy_(later.vp)
    for k in ("prefix_blocks", "prefix_len", "block_table", "lengths") + (("q_start",) if ragged else ()):
        first.d[k].copy_(later.d[k])
    out.fill_(7.0), ws.fill_(0xFF)
    g.replay()
    torch.cuda.synchronize()
    assert int(first.status.item()) == 0
    close(out[:later.m], *later.want())
    assert not out[later.m:].any()


def test_two_streams_with_workspaces_of_their_own():
    a, b = Batch(19, 8, 1, 128, 3000, [50] * 30), Batch(20, 32, 32, 64, 700, [300] * 8)
    s, t = torch.cuda.Stream(), torch.cuda.Stream()
    oa, ob = torch.zeros_like(a.q), torch.zeros_like(b.q)
    wa, wb = a.workspace(), b.workspace()
    torch.cuda.synchronize()
    for _ in range(5):
        lr.prefix_attention(a.q, a.nh, a.cache(), out=oa, workspace=wa, status=a.status, stream=s, **a.d)
        lr.prefix_attention(b.q, b.nh, b.cache(), out=ob, workspace=wb, status=b.status, stream=t, **b.d)
    torch.cuda.synchronize()
    close(oa, *a.want())
    close(ob, *b.want())
