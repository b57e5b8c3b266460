"""Cached-attention entry points without a GPU: the host table, argument checks, workspace rule, oracle pins."""

import ctypes

import numpy as np
import pytest

import oracle
import rank_decomposed_gb300 as lr

BIG = 1 << 40


def test_rope_table_matches_oracle_angles_at_far_positions():
    n, rot = 70000, 32
    t = lr.rope_table(n, rot, 10000.0)
    a = oracle.rope_angles(np.arange(n), rot)
    want = np.concatenate([np.cos(a), np.sin(a)], axis=1)
    # one rounding to fp32 of values at most 1, and the 64-bit angle's own (70000 * 2^-53)
    assert np.abs(t - want).max() <= 2.0 ** -25 + 1e-10


def test_rope_table_refusals():
    out = np.zeros(64, np.float32)
    f = lambda n, rot, theta, p=out.ctypes.data: lr.lib.lr_rope_table(n, rot, theta, p)
    assert f(0, 16, 1e4, None) == lr.LR_OK
    assert f(4, 16, 1e4) == lr.LR_OK
    for a in ((-1, 16, 1e4), (4, 0, 1e4), (4, 7, 1e4), (4, 16, 0.0), (4, 16, float("nan")), (4, 16, float("inf"))):
        assert f(*a) == lr.LR_ERR_INVALID_ARG
    assert f(4, 16, 1e4, None) == lr.LR_ERR_INVALID_ARG


def _map(hd=128, rot=128, **kw):
    d = lr.HeadMapDesc(hd, 1, 1e-6, 0x1000, 0x2000, rot, lr.ROT_HALF, 0x3000, 100)
    for k, v in kw.items():
        setattr(d, k, v)
    return d


def _rope(hm=None, M=4, q=0x10000, ldq=1024, nh=8, k=0x20000, ldk=256, nkv=2, dt=lr.LR_BF16, pos=0x100, qo=0x30000,
          ldqo=1024, ko=0x40000, ldko=256):
    hm = hm or _map()
    return lr.lib.lr_qk_norm_rope(q, ldq, nh, k, ldk, nkv, dt, M, pos, None, ctypes.byref(hm), qo, ldqo, ko, ldko, None,
                                  None)


def test_qk_norm_rope_refusals_launch_nothing():
    assert _rope(M=0, q=None, pos=None) == lr.LR_OK
    assert _rope(nh=0, nkv=0) == lr.LR_OK
    bad = lr.LR_ERR_INVALID_ARG
    for kw in (dict(q=None), dict(q=0x10008), dict(ldq=1000), dict(ldq=1028), dict(k=None), dict(qo=None), dict(ko=None),
               dict(ldko=128), dict(dt=7), dict(M=-1), dict(nh=-1), dict(pos=None), dict(M=1 << 31),
               dict(dt=lr.LR_F32, qo=0x10000),                      # in place with another type
               dict(qo=0x10000, ldq=1032)):                         # in place with another stride
        assert _rope(**kw) == bad, kw
    for kw in (dict(eps=-1.0), dict(eps=float("nan")), dict(q_gain=0x1008), dict(rot_style=5), dict(cos_sin=None),
               dict(cos_sin=0x3004), dict(max_pos=0), dict(head_dim=0), dict(rot_dim=-16)):
        assert _rope(hm=_map(**kw)) == bad, kw
    for kw in (dict(head_dim=96), dict(head_dim=320), dict(rot_dim=24), dict(rot_dim=144)):
        assert _rope(hm=_map(**kw)) == lr.LR_ERR_UNSUPPORTED, kw
    assert "rot_dim" in lr.last_error()
    assert lr.lib.lr_qk_norm_rope(0x10000, 1024, 8, 0x20000, 256, 2, 0, 4, 0x100, None, None, 0x30000, 1024, 0x40000,
                                  256, None, None) == bad


def _cache(**kw):
    c = lr.KvCache(0x100000, 0x200000, 256, 64, 16, 2, 128)
    for k, v in kw.items():
        setattr(c, k, v)
    return c


def _append(cache=None, hm=None, M=4, k=0x1000, v=0x2000, q=0x3000, nh=8, rows=0x200, pos=0x100, qo=0x4000):
    hm, cache = hm or _map(), cache or _cache()
    return lr.lib.lr_kv_append(k, 256, v, 256, q, 1024, nh, lr.LR_BF16, M, pos, rows, None, ctypes.byref(hm),
                               ctypes.byref(cache), qo, 1024, None, None)


def test_kv_append_refusals_launch_nothing():
    assert _append(M=0) == lr.LR_OK
    for kw in (dict(k=None), dict(v=None), dict(v=0x2002), dict(q=None), dict(qo=None), dict(rows=None), dict(pos=None),
               dict(hm=_map(hd=64, rot=64))):
        assert _append(**kw) == lr.LR_ERR_INVALID_ARG, kw
    for kw in (dict(k=None), dict(v=0x200008), dict(ld=250), dict(ld=128), dict(n_kv_heads=0), dict(block_rows=0),
               dict(pool_blocks=-1), dict(pool_blocks=1 << 28)):
        assert _append(cache=_cache(**kw)) == lr.LR_ERR_INVALID_ARG, kw


def _desc(**kw):
    d = lr.AttnDesc(_cache(), 8, 0.1, 0x100, 10, 0x200, 3, 0x300, 5, 0x400, 4, 0x500)
    for k, v in kw.items():
        setattr(d, k, v)
    return d


def _attn(d=None, M=9, q=0x10000, ldq=1024, out=0x20000, ldo=1024, dt=lr.LR_BF16, ws=0x30000, ws_bytes=BIG):
    d = d or _desc()
    return lr.lib.lr_prefix_attention(q, ldq, out, ldo, dt, M, ctypes.byref(d), ws, ws_bytes, None, None)


def test_prefix_attention_refusals_launch_nothing():
    assert _attn(M=0) == lr.LR_OK
    bad, no = lr.LR_ERR_INVALID_ARG, lr.LR_ERR_UNSUPPORTED
    need = lr.lib.lr_prefix_attention_workspace_bytes(9, ctypes.byref(_desc()))
    assert need > 0
    for kw in (dict(q=None), dict(out=None), dict(q=0x10002), dict(ldq=1000), dict(ldo=1028), dict(dt=3), dict(M=-1),
               dict(ws=None), dict(ws=0x30010), dict(ws_bytes=need - 1)):
        assert _attn(**kw) == bad, kw
    for kw in (dict(n_heads=7), dict(n_heads=0), dict(scale=0.0), dict(scale=float("nan")), dict(scale=float("inf")),
               dict(prefix_blocks=None), dict(prefix_len=None), dict(cap_prefix_blocks=-1), dict(n_seq=-1),
               dict(lengths=None), dict(block_table=None), dict(max_q=0), dict(q_start=None),  # max_q 5 without q_start
               dict(cap_prefix_blocks=1 << 28), dict(blocks_per_seq=1 << 28),
               dict(q_start=None, max_q=1, n_seq=10),                                          # more sequences than rows
               dict(cache=_cache(ld=100)), dict(cache=_cache(k=None))):
        assert _attn(d=_desc(**kw)) == bad, kw
    for kw in (dict(cache=_cache(head_dim=192, ld=512)), dict(cache=_cache(block_rows=8)), dict(n_heads=2 * 65)):
        assert _attn(d=_desc(**kw), ldq=1 << 15, ldo=1 << 15) == no, kw
    assert lr.lib.lr_prefix_attention(0x10000, 1024, 0x20000, 1024, 0, 9, None, 0x30000, BIG, None, None) == bad


def test_workspace_covers_capacities_and_is_zero_for_nothing():
    f = lambda M, **kw: lr.lib.lr_prefix_attention_workspace_bytes(M, ctypes.byref(_desc(**kw)))
    assert f(0) == 0 and f(-3) == 0
    assert lr.lib.lr_prefix_attention_workspace_bytes(9, None) == 0
    assert f(9, cap_prefix_blocks=100) >= f(9) > 0


def test_workspace_of_refused_head_groups_is_zero():
    """More query heads a key head than a tile has rows: refused by the call, and no division by zero before it."""
    for nh in (130, 256, 260, 1 << 20):
        d = _desc(n_heads=nh)
        assert lr.lib.lr_prefix_attention_workspace_bytes(9, ctypes.byref(d)) == 0
        assert _attn(d=d, ldq=1 << 28, ldo=1 << 28) == lr.LR_ERR_UNSUPPORTED
    f = lambda M, **kw: lr.lib.lr_prefix_attention_workspace_bytes(M, ctypes.byref(_desc(**kw)))
    assert f(1 << 39) == 0 and f(1 << 62) == 0
    f((1 << 31) - 1, n_seq=1 << 30, cache=_cache(n_kv_heads=1 << 14), n_heads=1 << 14, max_q=1 << 25)  # counts that wrap
    many = _desc(n_heads=512, cache=_cache(n_kv_heads=1))
    b = _block(n_heads=512, n_kv_heads=1)
    b.f[0], b.f[3] = lr.Factor(0x10000, 0x20000, 512, 65536, 64), lr.Factor(0x30000, 0x40000, 65536, 512, 64)
    for i in (1, 2):
        b.f[i] = lr.Factor(0x50000, 0x60000, 512, 128, 64)
    assert lr.lib.lr_block_forward_cached(0x1000, 9, ctypes.byref(b), ctypes.byref(_context(attn=many)), 0x100000, BIG,
                                          None, None) == lr.LR_ERR_UNSUPPORTED


def _block(**kw):
    b = lr.BlockDesc()
    b.d_model, b.d_ff, b.n_heads, b.n_kv_heads, b.head_dim, b.eps = 512, 1024, 8, 2, 128, 1e-6
    io = [(512, 1024), (512, 256), (512, 256), (1024, 512), (512, 1024), (512, 1024), (1024, 512)]
    for i, (a, o) in enumerate(io):
        b.f[i] = lr.Factor(0x10000 * (i + 1), 0x10000 * (i + 20), a, o, 64)
    for k, v in kw.items():
        setattr(b, k, v)
    return b


def _context(attn=None, heads=None, pos=0x100, rows=0x200):
    return lr.ContextDesc(attn or _desc(), heads or _map(), pos, rows, None)


def test_block_forward_cached_refusals_launch_nothing():
    def call(b=None, c=None, M=9, h=0x1000, ws=0x100000, ws_bytes=BIG):
        b = b or _block()
        c = _context() if c is None else c
        return lr.lib.lr_block_forward_cached(h, M, ctypes.byref(b), ctypes.byref(c), ws, ws_bytes, None, None)

    bad = lr.LR_ERR_INVALID_ARG
    assert call(M=0) == lr.LR_OK
    need = lr.lib.lr_block_cached_scratch_bytes(9, ctypes.byref(_block()), ctypes.byref(_context()))
    assert need > lr.lib.lr_block_scratch_bytes(9, ctypes.byref(_block()))
    for kw in (dict(h=None), dict(h=0x1004), dict(ws=None), dict(ws=0x100010), dict(ws_bytes=need - 1), dict(M=-1),
               dict(c=_context(pos=None)), dict(c=_context(rows=None)), dict(c=_context(heads=_map(hd=64, rot=64))),
               dict(c=_context(attn=_desc(n_heads=4))), dict(c=_context(attn=_desc(lengths=None))),
               dict(c=_context(attn=_desc(scale=-1.0))), dict(c=_context(attn=_desc(cache=_cache(n_kv_heads=1)))),
               dict(b=_block(n_kv_heads=3))):
        assert call(**kw) == bad, kw
    assert call(c=_context(attn=_desc(cache=_cache(block_rows=24)))) == lr.LR_ERR_UNSUPPORTED
    assert lr.lib.lr_block_forward_cached(0x1000, 4, ctypes.byref(_block()), None, 0x100000, BIG, None, None) == bad


def test_status_string_of_index_range():
    assert "range" in lr.status_string(lr.LR_ERR_INDEX_RANGE)


# ---------------------------------------------------------------- binding
def test_binding_refuses_wrong_tensors():
    """Types, shapes and strides that the calls cannot take; no call reaches a GPU (streams are numbers here)."""
    torch = pytest.importorskip("torch")
    b16 = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)  # noqa: E731
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
    hm = lambda **kw: lr.HeadMap(**dict(dict(head_dim=64, norm=True, q_gain=b16(64), rot_dim=64,  # noqa: E731
                                             cos_sin=torch.zeros(8, 64)), **kw))
    m, st = 0, i32(1)

    def rope(q=b16(m, 128), k=b16(m, 64), pos=i32(m), heads=None, qo=b16(m, 128), ko=b16(m, 64), n=None):
        lr.qk_norm_rope(q, k, pos, heads or hm(), qo, ko, st, n_active=n, stream=1)

    rope()                                              # no rows: nothing to do
    rope(q=None, qo=None)
    for kw in (dict(q=torch.zeros(m, 128).half(), k=None), dict(qo=torch.zeros(m, 128)), dict(k=torch.zeros(m, 64)),
               dict(pos=torch.zeros(m, dtype=torch.int64)), dict(heads=hm(q_gain=torch.zeros(64))),
               dict(heads=hm(k_gain=b16(128)[::2])), dict(heads=hm(cos_sin=b16(8, 64))), dict(n=i32(1, 1)),
               dict(pos=i32(m, 1))):
        with pytest.raises(TypeError):
            rope(**kw)
    for kw in (dict(q=None, k=None), dict(q=b16(m, 100), qo=b16(m, 100)), dict(qo=b16(m, 64)), dict(qo=b16(2, 128)),
               dict(q=b16(128)), dict(q=b16(128, 3).t()), dict(pos=i32(3)), dict(heads=hm(cos_sin=torch.zeros(8, 32))),
               dict(heads=hm(q_gain=b16(32))), dict(heads=hm(head_dim=0, q_gain=None))):
        with pytest.raises(ValueError):
            rope(**kw)
    with pytest.raises(OverflowError):
        rope(heads=hm(rot_style=1 << 40))
    with pytest.raises(AttributeError):
        rope(heads=7)
    with pytest.raises(lr.LrError):
        rope(heads=hm(eps=-1.0))

    pools = b16(64, 192)
    cache = lambda **kw: lr.PagedKV(**dict(dict(k_pool=pools[:, :128], v_pool=pools[:, 64:], n_kv_heads=2,  # noqa: E731
                                                head_dim=64), **kw))

    def append(k=b16(m, 128), v=b16(m, 128), pos=i32(m), rows=i32(m), c=None, q=None, qo=None):
        lr.kv_append(k, v, pos, rows, hm(), c or cache(), st, q=q, q_out=qo, stream=1)

    append()
    append(q=b16(m, 256), qo=b16(m, 256))
    assert cache().c().ld == 192 and cache().c().pool_blocks == 4
    for kw in (dict(k=b16(m, 64)), dict(v=b16(m, 64)), dict(rows=i32(2)), dict(q=b16(m, 100), qo=b16(m, 100)),
               dict(c=cache(v_pool=b16(64, 128))), dict(c=cache(block_rows=48)), dict(c=cache(block_rows=0)),
               dict(c=cache(n_kv_heads=3)), dict(c=cache(k_pool=pools[:32, :128]))):
        with pytest.raises(ValueError):
            append(**kw)
    with pytest.raises(TypeError):
        append(v=torch.zeros(m, 128))

    def attend(q=b16(m, 256), out=b16(m, 256), pages=i32(3), n=i32(1), table=i32(2, 4), lens=i32(2), start=i32(3)):
        lr.prefix_attention(q, 4, cache(), pages, n, table, lens, out=out, workspace=None, status=st, q_start=start,
                            max_q=5, stream=1)

    attend()
    attend(out=torch.zeros(m, 256), pages=None, n=None)
    for kw in (dict(q=b16(m, 128)), dict(out=b16(m, 128)), dict(table=i32(3, 4)), dict(start=i32(4))):
        with pytest.raises(ValueError):
            attend(**kw)
    for kw in (dict(q=torch.zeros(m, 256)), dict(lens=None), dict(table=i32(4)), dict(table=i32(4, 2).t()),
               dict(pages=torch.zeros(3)), dict(out=torch.zeros(m, 256).double())):
        with pytest.raises(TypeError):
            attend(**kw)


# ------------------------------------------------------------ oracle pins
def test_oracle_rotation_keeps_pair_norms_and_adds_angles():
    rng = np.random.default_rng(0)
    x = rng.standard_normal((3, 2 * 64))
    for style in ("half", "pair"):
        a1, a2 = oracle.rope_angles([3, 5, 9], 32), oracle.rope_angles([4, 1, 30], 32)
        turn = lambda t, a: oracle.map_heads(t, 64, None, 0.0, np.cos(a), np.sin(a), style)
        assert np.allclose(turn(turn(x, a1), a2), turn(x, a1 + a2), atol=1e-12)
        assert np.allclose(np.linalg.norm(turn(x, a1)), np.linalg.norm(x))
        assert np.array_equal(turn(x, a1).reshape(3, 2, 64)[..., 32:], x.reshape(3, 2, 64)[..., 32:])


def test_oracle_scores_depend_on_distance_alone():
    rng = np.random.default_rng(1)
    q, k = rng.standard_normal((1, 64)), rng.standard_normal((1, 64))
    def score(p, t):
        turn = lambda x, n: oracle.map_heads(x, 64, None, 0.0, np.cos(oracle.rope_angles([n], 64)),
                                             np.sin(oracle.rope_angles([n], 64)), "half")
        return float((turn(q, p) @ turn(k, t).T)[0, 0])
    assert abs(score(100, 60) - score(1040, 1000)) < 1e-9


def test_oracle_prefix_attention_is_attention_over_the_joined_context():
    """Pages shuffled and split into prefix and own tokens give plain attention over the same tokens in order."""
    rng = np.random.default_rng(2)
    d, nkv, nh, br = 8, 2, 4, 4
    K, V = rng.standard_normal((11, nkv * d)), rng.standard_normal((11, nkv * d))
    kp, vp = np.full((24, nkv * d), np.nan), np.full((24, nkv * d), np.nan)
    pre, own = [4, 1], [5, 0]
    for t in range(11):
        at = pre[t // br] * br + t % br if t < 6 else own[(t - 6) // br] * br + (t - 6) % br
        kp[at], vp[at] = K[t], V[t]
    q = rng.standard_normal((3, nh * d))
    out, _ = oracle.prefix_attention(q, kp, vp, nh, nkv, d, br, pre, 6, [own], [5], [0, 3], 0.3)
    for j in range(3):
        for h in range(nh):
            n, c = 9 + j, slice(h // 2 * d, h // 2 * d + d)
            w = np.exp(0.3 * K[:n, c] @ q[j, h * d:(h + 1) * d])
            assert np.allclose(out[j, h * d:(h + 1) * d], w @ V[:n, c] / w.sum())
    empty, _ = oracle.prefix_attention(q, kp, vp, nh, nkv, d, br, pre, 0, [own], [1], [0, 3], 0.3)
    assert not empty[:2].any() and empty[2].any()      # one own token: the first two rows see nothing
