"""CPU tests of the boundary of the 8-bit activation path: every entry point of awq_a8.h is exported,
and every argument error is reported before any HIP call (no compute call is made here)."""
import os
import re
import subprocess
import sys

import pytest
import torch

from tests.conftest import ROOT

HEADER = os.path.join(ROOT, "include", "awq_a8.h")
OK, INVALID, SHAPE, UNSUP, WS = 0, 1, 2, 3, 4
F32, BF16, I8, E4M3 = 0, 1, 2, 3
P = 1 << 20  # a fake aligned device address: never dereferenced on these paths


@pytest.fixture(scope="module")
def L():
    from post_weight_quantization_mean_amd import awq
    if not os.path.exists(awq._LIB_PATH):
        import __graft_entry__
        __graft_entry__.build()
    return awq.lib()


def test_declared_entry_points_are_exported(L):
    names = re.findall(r"AWQ_API\s+[\w\s\*]+?\b(awq_\w+)\s*\(", open(HEADER).read())
    assert sorted(names) == ["awq_act_mul", "awq_rmsnorm", "awq_w4a8", "awq_w4a8_weight", "awq_w4a8_weight_bytes",
                             "awq_w4a8_workspace_bytes"]
    for n in names:
        assert hasattr(L, n)


def rmsnorm(L, X=P, xt=BF16, M=4, K=256, ldx=256, R=P, rt=BF16, ldr=256, H=2 * P, ldh=256, gamma=P, gt=F32,
            eps=1e-6, Y=3 * P, yt=I8, ldy=256, scale=P):
    return L.awq_rmsnorm(X, xt, M, K, ldx, R, rt, ldr, H, ldh, gamma, gt, eps, Y, yt, ldy, scale, None)


@pytest.mark.parametrize("kw,status", [
    (dict(X=None), INVALID), (dict(gamma=None), INVALID), (dict(Y=None), INVALID), (dict(scale=None), INVALID),
    (dict(M=0), INVALID), (dict(K=0), INVALID), (dict(M=-1), INVALID), (dict(ldx=255), INVALID),
    (dict(ldr=255), INVALID), (dict(ldh=255), INVALID), (dict(ldy=255), INVALID),
    (dict(R=None), INVALID),  # a residual output without a residual
    (dict(xt=I8), UNSUP), (dict(rt=E4M3), UNSUP), (dict(gt=I8), UNSUP), (dict(yt=4), UNSUP), (dict(yt=-1), UNSUP),
    (dict(eps=0.0), INVALID), (dict(eps=-1.0), INVALID), (dict(eps=float("nan")), INVALID),
    (dict(eps=float("inf")), INVALID),
    (dict(X=P + 1), INVALID), (dict(gamma=P + 2), INVALID), (dict(scale=P + 2), INVALID), (dict(R=P + 1), INVALID),
    (dict(Y=3 * P + 2, yt=F32), INVALID),
    (dict(H=P, ldh=512), INVALID),  # in place over R with another row stride
    (dict(M=1 << 62, ldx=1 << 10), SHAPE),
])
def test_rmsnorm_argument_errors(L, kw, status):
    assert rmsnorm(L, **kw) == status


def act_mul(L, G=P, xt=BF16, M=4, K=256, ldg=512, U=P + 512, ldu=512, s=P, act=1, Y=3 * P, yt=E4M3, ldy=256, scale=P):
    return L.awq_act_mul(G, xt, M, K, ldg, U, ldu, s, act, Y, yt, ldy, scale, None)


@pytest.mark.parametrize("kw,status", [
    (dict(G=None), INVALID), (dict(Y=None), INVALID), (dict(scale=None), INVALID), (dict(M=0), INVALID),
    (dict(K=0), INVALID), (dict(ldg=255), INVALID), (dict(ldu=255), INVALID), (dict(ldy=255), INVALID),
    (dict(xt=I8), UNSUP), (dict(act=3), UNSUP), (dict(act=-1), UNSUP), (dict(yt=9), UNSUP), (dict(s=P + 2), INVALID),
    (dict(G=P + 1), INVALID), (dict(U=P + 1), INVALID),
    (dict(Y=P, yt=BF16), INVALID),   # over G with another row stride
    (dict(Y=P, ldy=512), INVALID),   # over G in another type
    (dict(Y=P + 512, ldy=512, yt=F32), INVALID),
    (dict(M=1 << 62, ldg=1 << 10), SHAPE),
])
def test_act_mul_argument_errors(L, kw, status):
    assert act_mul(L, **kw) == status


def test_weight_bytes(L):
    assert L.awq_w4a8_weight_bytes(16, 128) == 1024 + 256 + 256
    assert L.awq_w4a8_weight_bytes(17, 256) == 32 * 128 + 256 + 256
    assert L.awq_w4a8_weight_bytes(4096, 4096) == 4096 * 2048 + 4096 * 32 * 4 + 4096 * 4
    for n, k in [(0, 128), (16, 0), (16, 100), (-1, 128), (1 << 62, 128), (1 << 40, 1 << 40)]:
        assert L.awq_w4a8_weight_bytes(n, k) == 0


def weight(L, q=P, sc=P, z=P, N=32, K=256, group=128, wt=P, wb=1 << 20):
    return L.awq_w4a8_weight(q, sc, z, N, K, group, wt, wb, None)


@pytest.mark.parametrize("kw,status", [
    (dict(q=None), INVALID), (dict(sc=None), INVALID), (dict(z=None), INVALID), (dict(N=0), INVALID),
    (dict(K=0), INVALID), (dict(K=200), SHAPE), (dict(group=64), UNSUP), (dict(wt=None), WS), (dict(wb=100), WS),
    (dict(wt=P + 16), INVALID), (dict(q=P + 8), INVALID), (dict(sc=P + 1), INVALID), (dict(N=1 << 62), SHAPE),
])
def test_weight_argument_errors(L, kw, status):
    assert weight(L, **kw) == status


def w4a8(L, X=P, xt=I8, xs=P, M=4, K=256, ldx=256, wt=P, N=32, group=128, Y=P, yt=F32, ldy=32, ws=P, wsb=1 << 40):
    return L.awq_w4a8(X, xt, xs, M, K, ldx, wt, N, group, Y, yt, ldy, ws, wsb, None)


@pytest.mark.parametrize("kw,status", [
    (dict(X=None), INVALID), (dict(xs=None), INVALID), (dict(wt=None), INVALID), (dict(Y=None), INVALID),
    (dict(M=0), INVALID), (dict(N=0), INVALID), (dict(K=0), INVALID), (dict(K=200, ldx=208), SHAPE),
    (dict(ldx=240), INVALID), (dict(ldx=264), INVALID), (dict(X=P + 8), INVALID), (dict(wt=P + 64), INVALID),
    (dict(xs=P + 2), INVALID), (dict(ldy=31), INVALID), (dict(Y=P + 2), INVALID), (dict(xt=BF16), UNSUP),
    (dict(yt=I8), UNSUP), (dict(group=64), UNSUP), (dict(ldx=1 << 24), SHAPE), (dict(M=1 << 62, ldx=1 << 10), SHAPE),
])
def test_w4a8_argument_errors(L, kw, status):
    assert w4a8(L, **kw) == status


def test_workspace_bytes_of_rejected_sizes(L):
    for m, k, n in [(0, 256, 16), (4, 200, 16), (4, 256, 0), (1 << 62, 256, 16)]:
        assert L.awq_w4a8_workspace_bytes(m, k, n) == 0


def test_python_refusals_need_no_gpu():
    from post_weight_quantization_mean_amd import awq
    x, g = torch.zeros(2, 128), torch.ones(128)
    with pytest.raises(ValueError):
        awq.rmsnorm(x, g)  # not on a device
    with pytest.raises(ValueError):
        awq.act_mul(x)
    with pytest.raises(ValueError):
        awq.w4a8_weight(torch.zeros(2, 16, dtype=torch.int32), g, g)
    with pytest.raises(ValueError):
        awq.w4a8(awq.Act8(x.to(torch.int8), torch.ones(2)), awq.W4A8Weight(torch.zeros(8, dtype=torch.uint8), 2, 128))


@pytest.mark.parametrize("yt,status", [(BF16 | 0x100, WS), (F32 | 0x100, WS), (I8 | 0x100, UNSUP), (BF16 | 0x200, WS),
                                       (F32 | 0x200, WS), (BF16 | 0x300, UNSUP), (BF16 | 0x400, UNSUP), (-1, UNSUP), (-1 & ~0xff | BF16, UNSUP)])
def test_w4a8_sums_flag(L, yt, status):
    """Either flag goes with either result type (these calls get as far as the missing workspace), both or others with none."""
    assert w4a8(L, M=8260, ws=None, wsb=0, yt=yt) == status


@pytest.mark.parametrize("m,k,n", [(1 << 38, 128, 1 << 40), (1 << 37, 128, 1 << 40), (1 << 62, 128, 16), (1 << 29, 128, 16),
                                   (1 << 28, 128, 512), (1 << 28, 128, 257), (4, 128, (1 << 27) + 1), (1 << 61, 128, 1 << 61)])
def test_product_sizes_beyond_a_launch(L, m, k, n):
    """Products of sizes whose tile counts leave int64 (a count of 0 ended the process in a division) or a launch's
    threads are refused."""
    assert L.awq_w4a8_workspace_bytes(m, k, n) == 0
    assert w4a8(L, M=m, K=k, ldx=k, N=n, ldy=n) == SHAPE


def test_largest_product_sizes(L):
    assert L.awq_w4a8_workspace_bytes((1 << 29) - 1, 128, 256) == ((1 << 29) - 1) * 8 * 4
    assert L.awq_w4a8_workspace_bytes((1 << 28) - 1, 128, 512) == ((1 << 28) - 1) * 8 * 4
    assert L.awq_w4a8_weight_bytes(1 << 27, 128) == (1 << 27) * (64 + 4 + 4) and L.awq_w4a8_weight_bytes((1 << 27) + 1, 128) == 0
    assert weight(L, N=(1 << 27) + 1, K=128, wb=1 << 60) == SHAPE


def test_other_calls_need_no_native_binding():
    """Without _a8.so (absent, or built for another interpreter) the library still loads and serves what it served
    before; the calls that need the module say so, and run once it is there."""
    code = """
import sys, torch
name = "post_weight_quantization_mean_amd._a8"
sys.modules[name] = None  # the import system's mark of a module that cannot be imported
from post_weight_quantization_mean_amd import awq
assert awq.lib().awq_abi_version() == 8 and awq.search_workspace_bytes(64, 128, 128) > 0
assert awq.w4a8_weight_bytes(16, 128) == 1536
x, g = torch.zeros(2, 128), torch.ones(128)
for call in (lambda: awq.rmsnorm(x, g), lambda: awq.act_mul(x)):
    try:
        call()
    except ImportError as e:
        assert "_a8.so" in str(e)
    else:
        raise AssertionError("no ImportError")
del sys.modules[name]
try:
    awq.rmsnorm(x, g)
except ValueError as e:
    print("bound:", e)
"""
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "bound: X must be a 2-D device tensor" in r.stdout, r.stdout + r.stderr


def test_library_is_linked_though_the_binding_fails(tmp_path, monkeypatch):
    from post_weight_quantization_mean_amd import build
    monkeypatch.setattr(build, "PKG", str(tmp_path))
    monkeypatch.setattr(build, "LIB", str(tmp_path / "libawq.so"))
    monkeypatch.setattr(build, "SOURCES", ["fold.hip"])

    def fails():
        raise RuntimeError("g++ failed")
    monkeypatch.setattr(build, "build_binding", fails)
    with pytest.raises(RuntimeError, match=r"g\+\+ failed"):
        build.build()
    assert (tmp_path / "libawq.so").exists()


@pytest.mark.parametrize("kw", [
    dict(Y=2 * P, yt=BF16),                      # over H
    dict(Y=2 * P),                               # the same in codes
    dict(X=4 * P, Y=4 * P),                      # codes over X
    dict(X=4 * P, Y=4 * P, yt=F32),
    dict(X=4 * P, Y=4 * P, yt=BF16, ldy=512),    # X's type in another row stride
    dict(R=4 * P, Y=4 * P),                      # codes over R
    dict(X=4 * P, xt=F32, H=4 * P),              # H over X in another type
    dict(X=4 * P, H=4 * P, ldh=512),
    dict(gamma=4 * P, Y=4 * P), dict(gamma=4 * P, H=4 * P),
])
def test_rmsnorm_refuses_crossed_outputs(L, kw):
    assert rmsnorm(L, **kw) == INVALID


@pytest.mark.parametrize("kw", [dict(Y=P, X=P), dict(Y=6 * P, wt=6 * P), dict(Y=6 * P, xs=6 * P),
                                dict(M=8260, ws=2 * P, Y=2 * P), dict(M=8260, ws=2 * P, X=2 * P), dict(M=8260, ws=2 * P, wt=2 * P)])
def test_w4a8_refuses_outputs_over_operands(L, kw):
    assert w4a8(L, **{**dict(X=3 * P, xs=4 * P, wt=5 * P, Y=7 * P, ws=8 * P), **kw}) == INVALID
