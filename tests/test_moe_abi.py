"""CPU tests of the boundary of the router, the mixture of experts and the low-rank adapters: every entry point of their
headers is exported, and every argument error is reported before any HIP call (no compute call is made here)."""
import os
import re

import pytest
import torch

from tests.conftest import ROOT

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


@pytest.mark.parametrize("header,want", [
    ("awq_moe.h", ["awq_moe", "awq_moe_layer", "awq_moe_route", "awq_moe_workspace_bytes"]),
    ("awq_lora.h", ["awq_lora", "awq_lora_workspace_bytes"])])
def test_declared_entry_points_are_exported(L, header, want):
    names = re.findall(r"AWQ_API\s+[\w\s\*]+?\b(awq_\w+)\s*\(", open(os.path.join(ROOT, "include", header)).read())
    assert sorted(names) == want
    for n in names:
        assert hasattr(L, n)


def route(L, logits=P, lt=F32, M=4, E=16, ldl=16, k=4, score=0, renorm=1, ids=2 * P, w=3 * P):
    return L.awq_moe_route(logits, lt, M, E, ldl, k, score, renorm, ids, w, None)


@pytest.mark.parametrize("kw,status", [
    (dict(logits=None), INVALID), (dict(ids=None), INVALID), (dict(w=None), INVALID), (dict(M=0), INVALID),
    (dict(M=-1), INVALID), (dict(E=0), INVALID), (dict(k=0), INVALID), (dict(k=-1), INVALID), (dict(k=17), INVALID),
    (dict(ldl=15), INVALID), (dict(logits=P + 2), INVALID), (dict(ids=2 * P + 2), INVALID), (dict(w=3 * P + 1), INVALID),
    (dict(lt=I8), UNSUP), (dict(lt=-1), UNSUP), (dict(score=2), UNSUP), (dict(score=-1), UNSUP),
    (dict(E=1025, ldl=1025), SHAPE), (dict(E=64, ldl=64, k=33), SHAPE), (dict(M=(1 << 24) + 1), SHAPE),
    (dict(M=1 << 24, ldl=1 << 40), SHAPE), (dict(ids=P), INVALID), (dict(w=P), INVALID), (dict(w=2 * P), INVALID)])
def test_route_argument_errors(L, kw, status):
    assert route(L, **kw) == status


def moe(L, X=P, xt=BF16, xs=None, M=4, H=256, ldx=256, ids=2 * P, w=3 * P, k=2, gu=4 * P, down=5 * P, E=8, I=128, group=128,
        act=1, Y=6 * P, yt=BF16, ldy=256, ws=8 * P, wsb=1 << 40):
    return L.awq_moe(X, xt, xs, M, H, ldx, ids, w, k, gu, down, E, I, group, act, Y, yt, ldy, ws, wsb, None)


def layer(L, X=P, xt=BF16, xs=None, M=4, H=256, ldx=256, logits=2 * P, lt=F32, ldl=8, k=2, score=0, gu=4 * P, down=5 * P, E=8,
          I=128, group=128, act=1, Y=6 * P, yt=BF16, ldy=256, ws=8 * P, wsb=1 << 40):
    return L.awq_moe_layer(X, xt, xs, M, H, ldx, logits, lt, ldl, k, score, 1, gu, down, E, I, group, act, Y, yt, ldy, ws, wsb,
                           None)


BOTH = [
    (dict(X=None), INVALID), (dict(gu=None), INVALID), (dict(down=None), INVALID), (dict(Y=None), INVALID),
    (dict(M=0), INVALID), (dict(H=0), INVALID), (dict(I=0), INVALID), (dict(E=0), INVALID), (dict(k=0), INVALID),
    (dict(M=-5), INVALID), (dict(ldx=255), INVALID), (dict(ldy=255), INVALID), (dict(X=P + 8), INVALID),
    (dict(ldx=260), INVALID), (dict(gu=4 * P + 16), INVALID), (dict(down=5 * P + 128), INVALID), (dict(Y=6 * P + 1), INVALID),
    (dict(xt=I8), INVALID), (dict(xt=E4M3, xs=P + 2), INVALID), (dict(xt=4), UNSUP), (dict(yt=I8), UNSUP), (dict(act=2), UNSUP),
    (dict(act=-1), UNSUP), (dict(group=64), UNSUP), (dict(H=192, ldx=192, ldy=192), SHAPE), (dict(I=96), SHAPE),
    (dict(H=(1 << 20) + 128, ldx=1 << 21, ldy=1 << 21), SHAPE), (dict(I=(1 << 20) + 128), SHAPE),
    (dict(M=(1 << 24) + 1), SHAPE), (dict(M=1 << 24, ldy=1 << 40), SHAPE),
    (dict(ws=None), WS), (dict(wsb=100), WS), (dict(ws=8 * P + 16), INVALID), (dict(ws=P), INVALID), (dict(ws=4 * P), INVALID),
    (dict(ws=5 * P), INVALID), (dict(ws=6 * P), INVALID), (dict(ws=2 * P), INVALID), (dict(Y=P), INVALID), (dict(Y=4 * P), INVALID),
    (dict(Y=5 * P), INVALID), (dict(Y=2 * P), INVALID), (dict(xt=I8, xs=6 * P), INVALID)]


@pytest.mark.parametrize("kw,status", BOTH + [
    (dict(ids=None), INVALID), (dict(w=None), INVALID), (dict(ids=2 * P + 2), INVALID), (dict(w=3 * P + 2), INVALID),
    (dict(Y=3 * P), INVALID), (dict(E=1025), SHAPE), (dict(k=33), SHAPE)])
def test_moe_argument_errors(L, kw, status):
    assert moe(L, **kw) == status


@pytest.mark.parametrize("kw,status", BOTH + [
    (dict(logits=None), INVALID), (dict(lt=I8), UNSUP), (dict(score=2), UNSUP), (dict(k=9), INVALID), (dict(ldl=7), INVALID),
    (dict(logits=2 * P + 2), INVALID), (dict(E=1025, ldl=1025), SHAPE), (dict(E=64, ldl=64, k=33), SHAPE)])
def test_layer_argument_errors(L, kw, status):
    assert layer(L, **kw) == status


def test_moe_workspace(L):
    """The size covers a pass of at most 2048 pairs, and the routing of all tokens; 0 where the call refuses the sizes."""
    ws = L.awq_moe_workspace_bytes
    for M, k in ((1, 1), (4, 8), (256, 8), (2048, 1), (10000, 3)):
        pairs = min(M, 2048 // k) * k
        assert pairs * 128 * 6 + pairs * 256 * 4 + M * k * 8 <= ws(M, 16, k, 256, 128) <= pairs * 128 * 6 + pairs * 256 * 4 + M * k * 8 + 1024
    for bad in ((0, 16, 2, 256, 128), (4, 1025, 2, 256, 128), (4, 16, 33, 256, 128), (4, 16, 2, 200, 128), (4, 16, 2, 256, 64),
                (4, 16, 0, 256, 128), (1 << 40, 16, 2, 256, 128), (4, 1024, 2, 256, 1 << 20)):
        assert ws(*bad) == 0
    assert moe(L, wsb=ws(4, 8, 2, 256, 128) - 1) == WS


def lora(L, X=P, xt=BF16, xs=None, M=4, K=256, ldx=256, A=2 * P, B=3 * P, n=3, R=16, ranks=None, scale=None, ids=4 * P, base=5 * P,
         ldb=512, Y=6 * P, yt=BF16, ldy=512, N=512, ws=8 * P, wsb=1 << 40):
    return L.awq_lora(X, xt, xs, M, K, ldx, A, B, n, R, ranks, scale, ids, base, ldb, Y, yt, ldy, N, ws, wsb, None)


@pytest.mark.parametrize("kw,status", [
    (dict(X=None), INVALID), (dict(A=None), INVALID), (dict(B=None), INVALID), (dict(ids=None), INVALID),
    (dict(base=None), INVALID), (dict(Y=None), INVALID), (dict(M=0), INVALID), (dict(K=0), INVALID), (dict(N=0), INVALID),
    (dict(R=0), INVALID), (dict(n=0), INVALID), (dict(M=-3), INVALID), (dict(ldx=255), INVALID), (dict(ldb=511), INVALID),
    (dict(ldy=511), INVALID), (dict(xt=I8), INVALID), (dict(xt=I8, xs=P + 2), INVALID), (dict(xt=5), UNSUP), (dict(yt=E4M3), UNSUP),
    (dict(K=260, ldx=264), SHAPE), (dict(R=12), SHAPE), (dict(R=264), SHAPE), (dict(M=1 << 24), SHAPE),
    (dict(N=1 << 22, ldb=1 << 22, ldy=1 << 22), SHAPE), (dict(M=1 << 20, N=1 << 20, ldb=1 << 20, ldy=1 << 20), SHAPE),
    (dict(n=1 << 31), SHAPE), (dict(M=1 << 20, ldx=1 << 50), SHAPE), (dict(X=P + 8), INVALID), (dict(ldx=260), INVALID),
    (dict(A=2 * P + 8), INVALID), (dict(B=3 * P + 8), INVALID), (dict(ids=4 * P + 2), INVALID), (dict(ranks=P + 2), INVALID),
    (dict(scale=P + 2), INVALID), (dict(base=5 * P + 1), INVALID), (dict(ws=None), WS), (dict(wsb=4), WS),
    (dict(ws=8 * P + 8), INVALID), (dict(Y=5 * P, ldy=520), INVALID), (dict(Y=P), INVALID), (dict(Y=2 * P), INVALID),
    (dict(Y=3 * P), INVALID), (dict(Y=4 * P), INVALID), (dict(ws=P), INVALID), (dict(ws=5 * P), INVALID), (dict(ws=6 * P), INVALID),
    (dict(scale=6 * P), INVALID), (dict(ranks=8 * P), INVALID)])
def test_lora_argument_errors(L, kw, status):
    assert lora(L, **kw) == status


def test_lora_workspace(L):
    ws = L.awq_lora_workspace_bytes
    for M, K, N, R in ((1, 4096, 4096, 16), (48, 4096, 6144, 64), (256, 512, 100, 8), (257, 512, 100, 8), (4096, 14336, 4096, 256)):
        need = ws(M, K, N, R)
        assert need % (M * R * 4) == 0 and 1 <= need // (M * R * 4) <= 16
        assert lora(L, M=M, K=K, ldx=K, N=N, ldb=N, ldy=N, R=R, wsb=need - 1) == WS
    for bad in ((0, 256, 256, 16), (4, 257, 256, 16), (4, 256, 256, 20), (4, 256, 256, 512), (1 << 24, 256, 256, 16),
                (4, 256, 1 << 22, 16), (1 << 23, 256, 4096, 16)):
        assert ws(*bad) == 0


@pytest.mark.parametrize("E,k,H,I", [(4, 1, 512, 128), (64, 8, 2048, 1024), (9, 7, 256, 384), (40, 32, 128, 128)])
def test_moe_workspace_of_a_larger_batch_serves_a_smaller_one(L, E, k, H, I):
    sizes = [L.awq_moe_workspace_bytes(M, E, k, H, I) for M in range(1, 5000)]
    assert all(a <= b for a, b in zip(sizes, sizes[1:]))


@pytest.mark.parametrize("K,N,R", [(512, 100, 8), (1000, 64, 8), (4096, 14336, 16), (5120, 11008, 32), (28672, 4096, 256)])
def test_lora_workspace_of_a_larger_batch_serves_a_smaller_one(L, K, N, R):
    sizes = [L.awq_lora_workspace_bytes(M, K, N, R) for M in range(1, 9000)]
    assert all(a <= b for a, b in zip(sizes, sizes[1:]))
    assert L.awq_lora_workspace_bytes(1 << 20, K, N, R) <= ((1 << 20) + 8192) * R * 4  # no splits where the tokens fill the card


def test_python_refuses_host_tensors_and_unknown_names():
    from post_weight_quantization_mean_amd import awq
    x, l = torch.zeros(2, 128), torch.zeros(2, 8)
    q, s = torch.zeros(2, 16, 16, dtype=torch.int32), torch.zeros(2, 16, 1, dtype=torch.float16)
    with pytest.raises(ValueError):
        awq.moe_route(l, 2)
    with pytest.raises(ValueError):
        awq.moe_route(l, 2, score="tanh")
    with pytest.raises(ValueError):
        awq.moe_weight(q, s, s)
    with pytest.raises(ValueError):
        awq.moe_weight(q[0], s, s)
    with pytest.raises(ValueError):
        awq.moe_weight(torch.zeros(2, 12, 16, dtype=torch.int32), s[:, :12].contiguous(), s[:, :12].contiguous())
    w = awq.MoEWeight(torch.zeros(8, dtype=torch.uint8), 2, 16, 128)
    with pytest.raises(ValueError):
        awq.moe(x, l, w, w, "none", k=1)
    with pytest.raises(ValueError):
        awq.moe(x, l, w, w, k=1)
    with pytest.raises(TypeError):
        awq.moe((x,), l, w, w, k=1)
    a, b = torch.zeros(1, 8, 128, dtype=torch.bfloat16), torch.zeros(1, 16, 8, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        awq.lora(x, a, b, torch.zeros(2, dtype=torch.int32), torch.zeros(2, 16))
