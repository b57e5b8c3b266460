"""Tensors that the kernels could not follow are refused by the binding: on the host, empty, or of another type.

No call here reaches a GPU: each has a tensor that is refused, or no rows.
"""

import pytest

torch = pytest.importorskip("torch")
import rank_decomposed_gb300 as lr  # noqa: E402


class OnGpu:
    """A tensor that says it is on the GPU."""

    is_cuda = True

    def __init__(self, t):
        self.t = t

    def __getattr__(self, name):
        return getattr(self.t, name)


def _b16(*s):
    return OnGpu(torch.zeros(*s, dtype=torch.bfloat16))


def _i32(*s):
    return OnGpu(torch.zeros(*s, dtype=torch.int32))


def _host(t):
    return t.t


def _refused(call, args, name, change, error):
    """call(**args) with args[name] changed is refused, and the message names it."""
    with pytest.raises(error) as e:
        call(**dict(args, **{name: change(args[name])}))
    assert name.split(".")[-1] in str(e.value)


def _rope_args(m):
    return dict(q=_b16(m, 128), k=_b16(m, 64), pos=_i32(m), q_out=_b16(m, 128), k_out=_b16(m, 64), status=_i32(1),
                n_active=_i32(1), q_gain=_b16(64), k_gain=_b16(64), cos_sin=OnGpu(torch.zeros(8, 64)))


def _map(q_gain, k_gain, cos_sin):
    return lr.HeadMap(64, norm=True, q_gain=q_gain, k_gain=k_gain, rot_dim=64, cos_sin=cos_sin)


def _rope(q, k, pos, q_out, k_out, status, n_active, q_gain, k_gain, cos_sin):
    lr.qk_norm_rope(q, k, pos, _map(q_gain, k_gain, cos_sin), q_out, k_out, status, n_active=n_active, stream=1)


def _append_args(m):
    a = _rope_args(m)
    del a["k_out"]
    return dict(a, v=_b16(m, 64), rows=_i32(m), k_pool=_b16(32, 64), v_pool=_b16(32, 64))


def _append(q, k, v, pos, rows, q_out, status, n_active, q_gain, k_gain, cos_sin, k_pool, v_pool):
    lr.kv_append(k, v, pos, rows, _map(q_gain, k_gain, cos_sin), lr.PagedKV(k_pool, v_pool, 1, 64), status, q=q,
                 q_out=q_out, n_active=n_active, stream=1)


def _attend_args(m):
    return dict(q=_b16(m, 128), k_pool=_b16(32, 64), v_pool=_b16(32, 64), prefix_blocks=_i32(1), prefix_len=_i32(1),
                block_table=_i32(2, 1), lengths=_i32(2), out=_b16(m, 128), workspace=OnGpu(torch.zeros(1 << 16, dtype=torch.uint8)),
                status=_i32(1), q_start=_i32(3))


def _attend(q, k_pool, v_pool, prefix_blocks, prefix_len, block_table, lengths, out, workspace, status, q_start):
    lr.prefix_attention(q, 2, lr.PagedKV(k_pool, v_pool, 1, 64), prefix_blocks, prefix_len, block_table, lengths, out,
                        workspace, status, q_start=q_start, max_q=3, stream=1)


CALLS = [(_rope, _rope_args), (_append, _append_args), (_attend, _attend_args)]


@pytest.mark.parametrize("call,args", CALLS)
def test_a_tensor_on_the_host_is_refused(call, args):
    a = args(4)
    for name in a:
        _refused(call, a, name, _host, TypeError)
    call(**{k: _host(v) for k, v in args(0).items()})     # no rows: nothing is read


@pytest.mark.parametrize("call,args", CALLS)
@pytest.mark.parametrize("m", [0, 4])
def test_the_status_word_is_an_int32_on_the_device(call, args, m):
    a = args(m)
    for change in (lambda t: OnGpu(torch.zeros(1)), lambda t: OnGpu(torch.zeros(1, dtype=torch.int64))):
        _refused(call, a, "status", change, TypeError)
    _refused(call, a, "status", lambda t: _i32(0), ValueError)


@pytest.mark.parametrize("m", [0, 4])
def test_counts_have_an_element(m):
    _refused(_rope, _rope_args(m), "n_active", lambda t: _i32(0), ValueError)
    _refused(_append, _append_args(m), "n_active", lambda t: _i32(0), ValueError)
    _refused(_attend, _attend_args(m), "prefix_len", lambda t: _i32(0), ValueError)


def _context_args(m):
    a = _attend_args(m)
    for x in ("q", "out", "workspace", "status"):
        del a[x]
    return dict(a, pos=_i32(m), rows=_i32(m), n_active=_i32(1), q_gain=_b16(64), k_gain=_b16(64),
                cos_sin=OnGpu(torch.zeros(8, 64)))


def _context(k_pool, v_pool, prefix_blocks, prefix_len, block_table, lengths, q_start, pos, rows, n_active, q_gain, k_gain,
             cos_sin):
    return lr.Context(lr.PagedKV(k_pool, v_pool, 1, 64), _map(q_gain, k_gain, cos_sin), pos, rows, prefix_blocks,
                      prefix_len, block_table, lengths, q_start=q_start, max_q=3, n_active=n_active)


def _block():
    f = [lr.FactorPair(torch.zeros(64, i, dtype=torch.bfloat16), torch.zeros(o, 64, dtype=torch.bfloat16))
         for i, o in ((64, 128), (64, 64), (64, 64), (128, 64), (64, 64), (64, 64), (64, 64))]
    return lr.Block(64, 64, 2, 1, 64, f)


def test_the_block_refuses_a_context_on_the_host():
    blk, m = _block(), 4
    h, scratch = OnGpu(torch.zeros(m, 64)), OnGpu(torch.zeros(1, dtype=torch.uint8))

    def call(h=h, scratch=scratch, status=_i32(1), **ctx):
        lr.block_forward_cached(h, blk, _context(**ctx), scratch, status, stream=1)

    a = _context_args(m)
    assert lr.block_cached_scratch_bytes(m, blk, _context(**{k: _host(v) for k, v in a.items()})) > 0
    for name in a:
        _refused(call, a, name, _host, TypeError)
    for name in ("n_active", "prefix_len"):
        _refused(call, a, name, lambda t: _i32(0), ValueError)
    a.update(h=h, scratch=scratch, status=_i32(1))
    for name in ("h", "scratch", "status"):
        _refused(call, a, name, _host, TypeError)
    _refused(call, a, "status", lambda t: OnGpu(torch.zeros(1)), TypeError)
    for bad in (torch.zeros(m, 32), torch.zeros(64), torch.zeros(m, 64, 1)):
        _refused(call, a, "h", lambda t: OnGpu(bad), ValueError)
