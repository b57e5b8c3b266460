"""The decomposed block over a real context: prompt, shared prefix, ragged turns and decode steps against the oracle."""

import numpy as np
import pytest

import oracle
import synth
from lr_testutil import assert_parity
from test_gpu_block import SMALL, make_layer

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
import rank_decomposed_gb300 as lr  # noqa: E402

P, BR, CAP = 50, 16, 6          # prefix tokens, rows a page, pages a sequence


def _i32(v):
    return torch.tensor(np.asarray(v), dtype=torch.int32, device="cuda")


class Model:
    """Two layers with their caches, on the device and in the oracle."""

    def __init__(self, n_seq, seed, **over):
        self.cfg = cfg = dict(SMALL, **over)
        self.layers = [make_layer(seed, i, cfg) for i in range(2)]
        nh, nkv, hd = cfg["n_heads"], cfg["n_kv"], cfg["hd"]
        g = torch.Generator().manual_seed(seed)
        self.gains = [(1 + 0.2 * torch.randn(hd, generator=g)).bfloat16() for _ in range(2)]
        table = torch.from_numpy(lr.rope_table(256, hd)).cuda()
        self.map = lr.HeadMap(hd, norm=True, q_gain=self.gains[0].cuda(), k_gain=self.gains[1].cuda(), rot_dim=hd,
                              cos_sin=table)
        self.table = table.double().cpu().numpy()
        pages = -(-P // BR) + n_seq * CAP
        perm = torch.randperm(pages, generator=g).int()
        self.prefix_pages, self.pages = perm[:-(-P // BR)].contiguous(), perm[-(-P // BR):].view(n_seq, CAP).contiguous()
        # stale rows hold NaN
        self.dev = [[torch.full((pages * BR, nkv * hd), float("nan"), dtype=torch.bfloat16, device="cuda") for _ in "kv"]
                    for _ in self.layers]
        self.ref = [[np.zeros((pages * BR, nkv * hd)) for _ in "kv"] for _ in self.layers]
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")

    def context(self, layer, pos, rows, prefix, table, lengths, q_start, max_q, n_active=None):
        cfg = self.cfg
        return lr.Context(lr.PagedKV(*self.dev[layer], cfg["n_kv"], cfg["hd"], BR), self.map, pos, rows,
                          self.prefix_pages.cuda() if prefix else None, _i32([P]) if prefix else None, table, lengths,
                          q_start=q_start, max_q=max_q, n_active=n_active)

    def oracle_step(self, h, pos, rows, prefix, table, lengths, q_start):
        cfg, half = self.cfg, self.cfg["hd"] // 2
        nh, nkv, hd = cfg["n_heads"], cfg["n_kv"], cfg["hd"]
        cos, sin = self.table[pos, :half], self.table[pos, half:]
        for (_, host), (kp, vp) in zip(self.layers, self.ref):
            batch = lambda q: oracle.prefix_attention(  # noqa: E731
                q, kp, vp, nh, nkv, hd, BR, self.prefix_pages.numpy(), P if prefix else 0, table, lengths, q_start,
                hd ** -0.5)[0]
            h = oracle.block_forward_cached(h, host, nh, nkv, hd, kp, vp, rows, cos, sin,
                                            [g.double().numpy() for g in self.gains], "half", batch)
        return h

    def step(self, seed, pos, rows, prefix, table, lengths, q_start=None, max_q=1):
        """One pass of new tokens through both layers, compared with the oracle."""
        m = len(pos)
        h0 = oracle.widen_bf16(synth.bf16_normal(seed, synth.make_tag(0, 0, synth.KIND_X), (m, self.cfg["d"])))
        h = torch.from_numpy(h0.astype(np.float32)).cuda()
        for i, (blk, _) in enumerate(self.layers):
            ctx = self.context(i, _i32(pos), _i32(rows), prefix, _i32(table), _i32(lengths),
                               None if q_start is None else _i32(q_start), max_q)
            scratch = torch.full((lr.block_cached_scratch_bytes(m, blk, ctx),), 0xFF, dtype=torch.uint8, device="cuda")
            lr.block_forward_cached(h, blk, ctx, scratch, self.status)
        torch.cuda.synchronize()
        assert int(self.status.item()) == 0
        starts = np.arange(m + 1) if q_start is None else q_start
        ref = self.oracle_step(h0, np.asarray(pos), np.asarray(rows), prefix, table, lengths, starts)
        got = h.cpu().numpy().astype(np.float64)
        assert_parity(got - h0, ref - h0, "delta of %d rows" % m)


def rows_of(pages, lo, hi):
    return [int(pages[t // BR]) * BR + t % BR for t in range(lo, hi)]


@pytest.mark.parametrize("over", [dict(), dict(d=1024, n_heads=8, n_kv=1, hd=128)])
def test_prompt_shared_prefix_turns_and_decode(over):
    n = 5
    m = Model(n, 31, **over)
    # the shared prefix, as a sequence of its own
    m.step(1, range(P), rows_of(m.prefix_pages, 0, P), False, m.prefix_pages.numpy()[None], [P], [0, P], P)
    # turns of unequal lengths behind it
    lens = [7, 33, 1, 20, 12]
    starts = [0] + list(np.cumsum(lens))
    pos = [P + t for k in lens for t in range(k)]
    rows = [r for b, k in enumerate(lens) for r in rows_of(m.pages[b], 0, k)]
    m.step(2, pos, rows, True, m.pages.numpy(), lens, starts, max(lens))
    # decode steps, with rows from the preparation scan
    for s in range(3):
        lens = [k + 1 for k in lens]
        rows, count, _ = lr.remap_build(lens, m.pages.numpy(), BR, 1, n)
        assert count == n
        m.step(3 + s, [P + k - 1 for k in lens], rows, True, m.pages.numpy(), lens)


def test_decode_step_is_captured_once_and_replayed():
    """Fixed buffers for up to 8 rows: the graph serves growing lengths and fewer active rows."""
    cap = 8
    m = Model(cap, 32)
    m.step(1, range(P), rows_of(m.prefix_pages, 0, P), False, m.prefix_pages.numpy()[None], [P], [0, P], P)
    lens = [3 + 5 * b for b in range(cap)]
    starts = [0] + list(np.cumsum(lens))
    m.step(2, [P + t for k in lens for t in range(k)], [r for b, k in enumerate(lens) for r in rows_of(m.pages[b], 0, k)],
           True, m.pages.numpy(), lens, starts, max(lens))
    d = m.cfg["d"]
    h = torch.zeros(cap, d, dtype=torch.float32, device="cuda")
    pos, rows, lengths, act = _i32([0] * cap), _i32([0] * cap), _i32([0] * cap), _i32([0])
    ctxs = [m.context(i, pos, rows, True, m.pages.cuda(), lengths, None, 1, n_active=act) for i in range(2)]
    need = max(lr.block_cached_scratch_bytes(cap, blk, c) for (blk, _), c in zip(m.layers, ctxs))
    scratch = torch.full((need,), 0xFF, dtype=torch.uint8, device="cuda")

    def fill(seed, n):
        for b in range(n):
            lens[b] += 1
        r, count, _ = lr.remap_build(lens[:n], m.pages.numpy()[:n], BR, 1, n)
        assert count == n
        h0 = oracle.widen_bf16(synth.bf16_normal(seed, synth.make_tag(0, 0, synth.KIND_X), (n, d)))
        h.zero_(), pos.zero_(), rows.fill_(-1), lengths.zero_()
        h[:n] = torch.from_numpy(h0.astype(np.float32)).cuda()
        pos[:n], rows[:n], lengths[:n] = _i32([P + k - 1 for k in lens[:n]]), _i32(r[:n]), _i32(lens[:n])
        act.fill_(n)
        return h0, np.asarray([P + k - 1 for k in lens[:n]]), r[:n]

    def run(stream):
        for (blk, _), c in zip(m.layers, ctxs):
            lr.block_forward_cached(h, blk, c, scratch, m.status, stream=stream)

    s = torch.cuda.Stream()
    act.zero_()
    torch.cuda.synchronize()
    run(s)
    s.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        run(s)
    for seed, n in ((10, 8), (11, 3), (12, 8)):
        h0, p, r = fill(seed, n)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert int(m.status.item()) == 0
        ref = m.oracle_step(h0, p, r, True, m.pages.numpy(), lens[:n], np.arange(n + 1))
        assert_parity(h[:n].cpu().numpy().astype(np.float64) - h0, ref - h0, "replay of %d rows" % n)
