"""GPU parity of the head norms, the position rotation and the append to a paged cache."""

import numpy as np
import pytest

import oracle

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
import rank_decomposed_gb300 as lr  # noqa: E402

STYLE = {"half": lr.ROT_HALF, "pair": lr.ROT_PAIR}


def _rand(shape, seed, dtype):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * 1.5).to(dtype).cuda()


def _f64(t):
    return t.double().cpu().numpy()


def _status():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


def _map(hd, norm, rot, style, seed, max_pos=5000):
    gains = [(1 + 0.3 * _rand((hd,), seed + i, torch.float32)).bfloat16() for i in range(2)] if norm else [None, None]
    table = torch.from_numpy(lr.rope_table(max_pos, rot)).cuda() if rot else None
    return lr.HeadMap(hd, norm=norm, eps=1e-5, q_gain=gains[0], k_gain=gains[1], rot_dim=rot, rot_style=STYLE[style],
                      cos_sin=table)


def _want(x, hm, gain, pos, style):
    t = np.zeros((x.shape[0], 0)) if hm.rot_dim == 0 else _f64(hm.cos_sin)[pos]
    half = hm.rot_dim // 2
    g = None if not hm.norm else (np.ones(hm.head_dim) if gain is None else _f64(gain))
    return oracle.map_heads(_f64(x), hm.head_dim, g, hm.eps, t[:, :half], t[:, half:], style)


def _close(y, want, hd):
    """One rounding to bf16 (2^-8 of the value), and fp32 arithmetic: some hundred roundings of 2^-24 of the largest
    element of the head that enters a sum or a pair."""
    want = want.reshape(want.shape[0], -1, hd)
    bound = 2.0 ** -8 * np.abs(want) + 256 * 2.0 ** -24 * np.abs(want).max(-1, keepdims=True)
    err = np.abs(_f64(y).reshape(want.shape) - want)
    assert np.all(err <= bound), float((err / bound).max())


@pytest.mark.parametrize("hd,rot,style,norm,dtype,m,nh,nkv", [
    (64, 64, "half", True, torch.bfloat16, 1, 8, 2),
    (128, 128, "half", True, torch.bfloat16, 37, 64, 8),
    (128, 32, "pair", True, torch.float32, 5, 32, 32),
    (128, 96, "half", False, torch.float32, 700, 7, 1),
    (192, 192, "half", True, torch.bfloat16, 9, 3, 1),
    (192, 64, "pair", False, torch.bfloat16, 3, 5, 5),
    (256, 256, "half", True, torch.float32, 11, 4, 2),
    (256, 16, "half", True, torch.bfloat16, 1000, 6, 3),
    (64, 0, "half", True, torch.bfloat16, 33, 8, 8),
    (64, 16, "pair", False, torch.bfloat16, 2500, 56, 56),
])
def test_qk_norm_rope_matches_oracle(hd, rot, style, norm, dtype, m, nh, nkv):
    """q and k are slices of one joint projection output; the outputs have padded rows."""
    hm = _map(hd, norm, rot, style, 7)
    x = _rand((m, (nh + nkv) * hd + 8), 1, dtype)
    q, k = x[:, :nh * hd], x[:, nh * hd:(nh + nkv) * hd]
    pos = torch.randint(0, 5000, (m,), generator=torch.Generator().manual_seed(2), dtype=torch.int32)
    pos[-1] = 4999
    qb = torch.full((m, nh * hd + 16), 3.0, dtype=torch.bfloat16, device="cuda")
    kb = torch.full((m, nkv * hd + 8), 3.0, dtype=torch.bfloat16, device="cuda")
    st = _status()
    lr.qk_norm_rope(q, k, pos.cuda(), hm, qb[:, :nh * hd], kb[:, :nkv * hd], st)
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    _close(qb[:, :nh * hd], _want(q, hm, hm.q_gain, pos.numpy(), style), hd)
    _close(kb[:, :nkv * hd], _want(k, hm, hm.k_gain, pos.numpy(), style), hd)
    assert torch.all(qb[:, nh * hd:] == 3.0) and torch.all(kb[:, nkv * hd:] == 3.0)   # padding untouched


def test_qk_norm_rope_in_place_one_side_and_active_rows():
    hm = _map(128, True, 128, "half", 3)
    k = _rand((40, 4 * 128), 5, torch.bfloat16)
    before = k.clone()
    pos = torch.arange(40, dtype=torch.int32, device="cuda") * 100
    n = torch.tensor([29], dtype=torch.int32, device="cuda")
    st = _status()
    lr.qk_norm_rope(None, k, pos, hm, None, k, st, n_active=n)
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    _close(k[:29], _want(before[:29], hm, hm.k_gain, pos[:29].cpu().numpy(), "half"), 128)
    assert torch.equal(k[29:], before[29:])


def test_unit_gain_zero_rows_and_values_outside_the_rotation():
    """A zero head stays zero under its norm; infinities past rot_dim stay where they are."""
    hm = lr.HeadMap(64, norm=True, eps=1e-6, rot_dim=0)
    q = torch.zeros(3, 128, dtype=torch.bfloat16, device="cuda")
    q[1] = 2.0
    out = torch.full_like(q, 5.0)
    st = _status()
    lr.qk_norm_rope(q, None, None, hm, out, None, st)
    assert torch.equal(out[0], torch.zeros_like(out[0])) and torch.equal(out[1], torch.ones_like(out[1]))
    for style in ("half", "pair"):
        hm = _map(64, False, 32, style, 1)
        x = _rand((4, 64), 8, torch.bfloat16)
        x[:, 32:] = float("inf")
        x[2, 40] = float("nan")
        y = torch.zeros_like(x)
        lr.qk_norm_rope(x, None, torch.tensor([0, 9, 100, 4999], dtype=torch.int32, device="cuda"), hm, y, None, st)
        torch.cuda.synchronize()
        assert torch.isfinite(y[:, :32].float()).all()
        # a NaN stays one (its payload does not: it passes through fp32), all else keeps its bits
        assert torch.equal(torch.isnan(y), torch.isnan(x)) and torch.equal(y[:, 32:].nan_to_num(), x[:, 32:].nan_to_num())
    assert int(st.item()) == 0


def test_positions_outside_the_table_give_zero_rows_and_are_reported():
    hm = _map(64, True, 64, "half", 1, max_pos=50)
    q = _rand((4, 128), 3, torch.bfloat16)
    out = torch.full_like(q, 5.0)
    st = _status()
    lr.qk_norm_rope(q, None, torch.tensor([49, 50, -1, 0], dtype=torch.int32, device="cuda"), hm, out, None, st)
    torch.cuda.synchronize()
    assert int(st.item()) == lr.LR_ERR_INDEX_RANGE
    assert not out[1:3].any()
    _close(out[[0, 3]], _want(q[[0, 3]], hm, hm.q_gain, [49, 0], "half"), 64)


@pytest.mark.parametrize("hd,nkv,nh,dtype,m,joint", [
    (128, 8, 64, torch.bfloat16, 64, False),
    (128, 32, 0, torch.float32, 301, False),
    (64, 2, 8, torch.bfloat16, 1, True),
    (192, 3, 6, torch.float32, 77, True),
])
def test_kv_append_writes_its_rows_alone(hd, nkv, nh, dtype, m, joint):
    """Scattered rows of separate pools, or of one pool of [K | V] rows; every other row keeps its bits."""
    hm = _map(hd, True, hd, "half", 4)
    w = nkv * hd
    pool = _rand((48 * 16, 2 * w), 5, torch.bfloat16)
    kp, vp = (pool[:, :w], pool[:, w:]) if joint else (pool[:, :w].contiguous(), pool[:, w:].contiguous())
    kb, vb = kp.clone(), vp.clone()
    x = _rand((m, (nh + 2 * nkv) * hd), 6, dtype)
    q, k, v = x[:, :nh * hd], x[:, nh * hd:nh * hd + w], x[:, nh * hd + w:]
    g = torch.Generator().manual_seed(9)
    rows = torch.randperm(48 * 16, generator=g)[:m].int()
    pos = torch.randint(0, 5000, (m,), generator=g, dtype=torch.int32)
    qo = torch.zeros(m, nh * hd, dtype=torch.bfloat16, device="cuda") if nh else None
    st = _status()
    lr.kv_append(k, v, pos.cuda(), rows.cuda(), hm, lr.PagedKV(kp, vp, nkv, hd, 16), st, q=q if nh else None, q_out=qo)
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    at = rows.long().cuda()
    _close(kp[at], _want(k, hm, hm.k_gain, pos.numpy(), "half"), hd)
    assert torch.equal(vp[at], v.bfloat16())
    if nh:
        _close(qo, _want(q, hm, hm.q_gain, pos.numpy(), "half"), hd)
    rest = torch.ones(48 * 16, dtype=torch.bool, device="cuda")
    rest[at] = False
    assert torch.equal(kp[rest], kb[rest]) and torch.equal(vp[rest], vb[rest])


def test_kv_append_skips_and_reports_bad_rows_and_positions():
    hm = _map(64, False, 64, "half", 4, max_pos=100)
    k, v, q = (_rand((5, 128), i, torch.bfloat16) for i in (1, 2, 3))
    for rows, pos, code, kept in (([3, 64, 5, -1, 7], [1, 2, 3, 4, 5], lr.LR_ERR_REMAP_RANGE, [0, 2, 4]),
                                  ([3, 4, 5, 6, 7], [1, 100, 3, 4, -7], lr.LR_ERR_INDEX_RANGE, [0, 2, 3])):
        kp = torch.full((64, 128), 3.0, dtype=torch.bfloat16, device="cuda")
        vp, qo, st = kp.clone(), torch.full_like(q, 5.0), _status()
        lr.kv_append(k, v, torch.tensor(pos, dtype=torch.int32, device="cuda"),
                     torch.tensor(rows, dtype=torch.int32, device="cuda"), hm, lr.PagedKV(kp, vp, 2, 64), st, q=q, q_out=qo)
        torch.cuda.synchronize()
        assert int(st.item()) == code
        at = [rows[i] for i in kept]
        _close(kp[at], _want(k[kept], hm, None, [pos[i] for i in kept], "half"), 64)
        assert torch.equal(vp[at], v[kept])
        rest = [r for r in range(64) if r not in at]
        assert torch.all(kp[rest] == 3.0) and torch.all(vp[rest] == 3.0)
        if code == lr.LR_ERR_INDEX_RANGE:
            assert not qo[[1, 4]].any()


def test_append_then_rotation_of_reconstructed_keys_agree():
    """Keys rotated on the way into the cache equal keys stored unrotated and rotated in place afterwards."""
    m, w = 96, 4 * 64
    hm = _map(64, True, 64, "half", 2)
    k, v = _rand((m, w), 1, torch.bfloat16), _rand((m, w), 2, torch.bfloat16)
    pos = torch.arange(m, dtype=torch.int32, device="cuda")
    kp, vp = torch.zeros(m, w, dtype=torch.bfloat16, device="cuda"), torch.zeros(m, w, dtype=torch.bfloat16, device="cuda")
    st = _status()
    lr.kv_append(k, v, pos, pos, hm, lr.PagedKV(kp, vp, 4, 64), st)
    lr.qk_norm_rope(None, k, pos, hm, None, k, st)
    torch.cuda.synchronize()
    assert int(st.item()) == 0 and torch.equal(kp, k)


def test_append_on_a_side_stream_in_a_graph():
    """Captured once on its own stream, replayed for another batch of fewer rows."""
    hm = _map(128, True, 128, "half", 6)
    k, v, q = _rand((16, 256), 1, torch.bfloat16), _rand((16, 256), 2, torch.bfloat16), _rand((16, 512), 3, torch.bfloat16)
    kp = torch.zeros(64, 256, dtype=torch.bfloat16, device="cuda")
    vp, qo, st = kp.clone(), torch.zeros_like(q), _status()
    pos = torch.arange(16, dtype=torch.int32, device="cuda")
    rows = pos + 30
    n = torch.tensor([16], dtype=torch.int32, device="cuda")
    call = lambda s: lr.kv_append(k, v, pos, rows, hm, lr.PagedKV(kp, vp, 2, 128), st, q=q, q_out=qo, n_active=n, stream=s)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        call(s)
    s.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        call(s)
    kp.zero_(), vp.zero_()
    k.copy_(_rand((16, 256), 11, torch.bfloat16)), pos.add_(1000), n.fill_(7)
    g.replay()
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    _close(kp[30:37], _want(k[:7], hm, hm.k_gain, np.arange(1000, 1007), "half"), 128)
    assert torch.equal(vp[30:37], v[:7]) and not kp[37:].any() and not vp[37:].any()
