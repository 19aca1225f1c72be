"""What mpe_select_experts, mpe_expert_importance and mpe_linear refuse, without
a device: every refusal comes before any device work."""
import ctypes
import struct

import pytest

P = 0x10000  # a 16-byte aligned address that nothing reads


@pytest.fixture(scope="module")
def mpe():
    from mixed_precision_expert_b200.build import build
    build()
    import mixed_precision_expert_b200 as m
    m.lib()
    return m


def select(mpe, E=64, k=4, score=0, groups=1, keep=1, gscore=1, renorm=1, scale=1.0, logits=P, typ=0, ld=None,
           T=4, bias=0, ids=1 << 30, w=1 << 31, args=True):
    c = struct.pack("=4Qq9if", logits, bias, ids, w, E if ld is None else ld, T, E, k, typ, score, groups, keep, gscore,
                    renorm, scale) if args else None
    return mpe.lib().mpe_select_experts(c, None)


@pytest.mark.parametrize("bad", [
    dict(E=0), dict(E=-5), dict(E=1025), dict(k=0), dict(k=-1), dict(k=33), dict(E=4, k=5), dict(score=2), dict(score=-1),
    dict(groups=0), dict(groups=-1), dict(groups=3), dict(groups=33, E=66), dict(keep=0), dict(keep=2), dict(gscore=2),
    dict(groups=16, keep=1, k=5), dict(typ=3), dict(typ=-1), dict(ld=63), dict(ld=-64), dict(ld=1 << 38),
    dict(T=-1), dict(T=(1 << 22) + 1), dict(logits=0), dict(ids=0), dict(w=0), dict(logits=P + 2),
    dict(logits=P + 1, typ=1), dict(ids=P + 2), dict(w=P + 1), dict(bias=P + 2), dict(args=False),
    # an output over something else
    dict(w=1 << 30), dict(w=(1 << 30) + 60), dict(ids=P), dict(w=P + 1020), dict(bias=1 << 30), dict(bias=(1 << 31) + 60)])
def test_select_refuses(mpe, bad):
    assert select(mpe, **bad) == -1
    assert b"mpe_select_experts" in mpe.lib().mpe_last_error_global()


def test_no_tokens_is_nothing_to_do(mpe):
    assert select(mpe, T=0, logits=0, ids=0, w=0) == 0
    assert mpe.lib().mpe_expert_importance(None, None) == -1
    assert linear(mpe, M=0, x=0, w=0, out=0) == 0


def importance(mpe, logits=P, typ=0, ld=64, T=1000, E=64, score=0, out=1 << 30, ws=1 << 31, nbytes=1 << 30):
    return mpe.lib().mpe_expert_importance(struct.pack("=4Qq4i", logits, out, ws, nbytes, ld, T, E, typ, score), None)


@pytest.mark.parametrize("bad", [
    dict(T=0), dict(T=-1), dict(E=0), dict(E=1025, ld=2000), dict(score=2), dict(typ=7), dict(ld=63), dict(logits=0),
    dict(out=0), dict(out=P + 2), dict(ws=0), dict(nbytes=16), dict(ws=P + 8), dict(logits=P + 2),
    dict(out=P), dict(ws=P), dict(ws=1 << 30), dict(out=(1 << 31) + 64)])
def test_importance_refuses(mpe, bad):
    assert importance(mpe, **bad) == -1
    assert b"mpe_expert_importance" in mpe.lib().mpe_last_error_global()


def test_importance_workspace(mpe):
    f = mpe.lib().mpe_expert_importance_workspace
    assert f(0, 64) == 0 and f(1, 64) == 0 and f(10, 0) == 0 and f(-1, 5) == 0 and f(10, 1025) == 0
    assert 0 < f(1000, 64) <= f(100000, 64) <= f(2 ** 31 - 1, 64) < 1 << 30


def linear(mpe, x=P, w=2 * P, bias=0, residual=0, out=1 << 40, ldx=64, ldw=64, ldr=128, ldo=128, M=4, N=128, K=64,
           typ=1, btyp=1, otyp=1, act=0, gated=0):
    return mpe.lib().mpe_linear(struct.pack("=5Q4q8i", x, w, bias, residual, out, ldx, ldw, ldr, ldo, M, N, K, typ,
                                            btyp, otyp, act, gated), None)


@pytest.mark.parametrize("bad", [
    dict(M=-1), dict(N=0), dict(N=-1), dict(K=0), dict(K=-8), dict(M=(1 << 30) + 1, ldo=128), dict(N=(1 << 30) + 1),
    dict(typ=0), dict(typ=3), dict(otyp=2), dict(otyp=5), dict(bias=P * 9, btyp=2), dict(act=-1), dict(act=5),
    dict(x=0), dict(w=0), dict(out=0), dict(ldx=56), dict(ldx=68), dict(ldw=66), dict(ldw=-64), dict(ldx=1 << 38),
    dict(ldo=127), dict(residual=1 << 41, ldr=100), dict(x=P + 8), dict(w=2 * P + 2), dict(out=(1 << 40) + 1),
    dict(residual=(1 << 41) + 1), dict(bias=P * 9 + 1), dict(otyp=0, out=(1 << 40) + 2), dict(bias=P * 9 + 2, btyp=0),
    # out over an input
    dict(out=P), dict(out=2 * P), dict(out=P + 16), dict(out=2 * P + 128 * 128 - 16), dict(bias=(1 << 40) + 128),
    dict(out=2 * P + 128 * 128 - 16, gated=1, N=64, ldo=64),
    dict(M=1, out=2 * P + 112, ldw=192), dict(M=1, out=2 * P + 256, ldw=192), dict(M=1, out=2 * P - 128),
    dict(M=1 << 30, ldo=1 << 37, out=1 << 30, x=1 << 40, w=1 << 45),
    # a residual over out that is not out
    dict(residual=(1 << 40) + 256), dict(residual=(1 << 40), ldr=136), dict(residual=(1 << 40) + 16)])
def test_linear_refuses(mpe, bad):
    assert linear(mpe, **bad) == -1
    assert b"mpe_linear" in mpe.lib().mpe_last_error_global()


@pytest.mark.parametrize("good", [
    dict(), dict(residual=1 << 40), dict(M=1, ldx=3, ldo=1, ldr=2), dict(M=1, residual=1 << 40, ldr=77),
    dict(out=P + 128, ldx=128, ldo=128, N=64, w=1 << 30),                      # columns of one buffer: x | out
    dict(x=P + 128, out=P, ldx=128, ldo=128, N=64, w=1 << 30),                 # out | x
    dict(residual=(1 << 40) + 256, ldo=256, ldr=256),                          # out | residual
    dict(M=1, out=2 * P + 128, ldw=192),                                       # a row beside w's columns
    dict(M=1, out=P + 128, w=1 << 30), dict(bias=P * 9), dict(bias=P * 9, btyp=0, otyp=0)])
def test_linear_takes(mpe, good):
    """Arguments that pass every check fail later, for want of a device."""
    import torch
    if torch.cuda.is_available():
        pytest.skip("would run on the device")
    assert linear(mpe, **good) == -5


def test_null_structs(mpe):
    assert mpe.lib().mpe_linear(None, None) == -1
    assert mpe.lib().mpe_global_status(None, 0) == -1


def test_binding_refuses_tensors_off_the_device():
    import torch

    import mixed_precision_expert_b200 as mpe
    l = torch.zeros(4, 64)
    x, w = torch.zeros(4, 64).bfloat16(), torch.zeros(128, 64).bfloat16()
    for call in (lambda: mpe.select_experts(l, 4), lambda: mpe.expert_importance(l), lambda: mpe.linear(x, w)):
        with pytest.raises(ValueError, match="CUDA device"):
            call()
