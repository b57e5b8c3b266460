"""The calls over a context without the C extension: the same structures, refusals and results through ctypes."""

import os
import subprocess
import sys
import sysconfig

import pytest

torch = pytest.importorskip("torch")
import rank_decomposed_gb300 as lr  # noqa: E402
from rank_decomposed_gb300 import _marshal, build  # noqa: E402
from test_attention_abi import test_binding_refuses_wrong_tensors  # noqa: E402,F401
from test_attention_binding import *  # noqa: E402,F401,F403
from test_attention_binding import _context, _context_args, _host, _map  # noqa: E402

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(autouse=True)
def through_ctypes(monkeypatch):
    monkeypatch.setattr(lr, "_calls", _marshal)
    monkeypatch.setattr(lr, "_ready", False)


def _extension():
    return pytest.importorskip("rank_decomposed_gb300._calls")


def test_the_structures_are_those_of_the_extension(monkeypatch):
    ext = _extension()
    both = []
    a = {k: _host(v) for k, v in _context_args(4).items()}
    strided = torch.zeros(32, 192, dtype=torch.bfloat16)
    for calls in (ext, _marshal):
        monkeypatch.setattr(lr, "_calls", calls)
        monkeypatch.setattr(lr, "_ready", False)
        got = []
        for change in (dict(), dict(prefix_blocks=None, prefix_len=None), dict(q_start=None, n_active=None),
                       dict(k_pool=strided[:, :64], v_pool=strided[:, 64:128]), dict(q_gain=None, k_gain=None)):
            c = _context(**dict(a, **change))
            for c.scale in (None, 0.3):
                got.append(bytes(c.c(4, 2)))
            got += [bytes(c.heads.c()), bytes(c.cache.c())]
        got.append(bytes(lr.HeadMap(128).c()))
        got.append(bytes(lr.PagedKV(strided[:1, :100], strided[:1, 64:164], 1, 64, block_rows=1).c()))
        both.append(got)
    assert both[0] == both[1] and any(both[0][0])


def test_the_package_runs_without_the_extension():
    code = ("import sys; sys.modules['rank_decomposed_gb300._calls'] = None\n"
            "import torch, rank_decomposed_gb300 as lr\n"
            "b = torch.zeros(0, 64, dtype=torch.bfloat16)\n"
            "lr.qk_norm_rope(b, None, None, lr.HeadMap(64), b, None, None, stream=1)\n"
            "assert lr._calls.__name__.endswith('_marshal')\n")
    subprocess.run([sys.executable, "-c", code], check=True, cwd=ROOT)


def test_the_build_needs_no_python_headers(monkeypatch, tmp_path):
    if os.path.exists(os.path.join(sysconfig.get_paths()["include"], "Python.h")):
        assert build.calls_command() is not None
        assert _extension().__file__ == build.CALLS_LIB      # a name that other Pythons do not load
    monkeypatch.setattr(build.sysconfig, "get_paths", lambda: {"include": str(tmp_path)})
    assert build.calls_command() is None


@pytest.mark.gpu
@pytest.mark.parametrize("qs", [None, [30, 1, 200]])
def test_results_are_those_of_the_extension(monkeypatch, qs):
    from test_gpu_attention import Batch, close
    b = Batch(51, 8, 2, 64, 100, [90, 21, 210], qs=qs)
    out = b.run()
    assert int(b.status.item()) == 0
    close(out, *b.want())
    g = torch.Generator().manual_seed(1)
    q, k, v = (torch.randn(5, n * 64, generator=g).bfloat16().cuda() for n in (8, 2, 2))
    hm = _map((1 + torch.randn(64, generator=g) / 8).bfloat16().cuda(), None, torch.from_numpy(lr.rope_table(8, 64)).cuda())
    pos, rows = torch.arange(5).int().cuda(), (torch.arange(5).int() * 3).cuda()
    results = []
    for calls in (_marshal, _extension()):
        monkeypatch.setattr(lr, "_calls", calls)
        monkeypatch.setattr(lr, "_ready", False)
        qo, ko = torch.zeros_like(q), torch.zeros_like(k)
        kp, vp = (torch.zeros(16, 128, dtype=torch.bfloat16, device="cuda") for _ in "kv")
        lr.qk_norm_rope(q, k, pos, hm, qo, ko, b.status)
        lr.kv_append(k, v, pos, rows, hm, lr.PagedKV(kp, vp, 2, 64), b.status, q=q, q_out=qo)
        torch.cuda.synchronize()
        results.append((qo, ko, kp, vp))
    assert int(b.status.item()) == 0 and results[0][2].any()
    assert all(torch.equal(x, y) for x, y in zip(*results))
    assert torch.equal(results[0][2][rows.long()], results[0][1])
