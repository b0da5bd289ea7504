"""moe_window_* on a machine without a GPU: workspace sizes, refusals, status codes."""
import ctypes

import pytest

import verify_weight_streaming_b200 as mr

P = ctypes.c_void_p
A = P(256)
BIG = 1 << 40


def test_workspace_bytes():
    assert mr.moe_window_workspace_bytes(1, 1, 8, 8) > 0
    assert mr.moe_window_workspace_bytes(16, 32, 4096, 2048) >= 512 * 4096 * 4
    for bad in ((0, 1, 8, 8), (1, 0, 8, 8), (1, 1, 0, 8), (1, 1, 8, 0), (17, 1, 8, 8), (1, 33, 8, 8),
                (1, 1, 1 << 21, 8), (1, 1, 8, 1 << 21)):
        assert mr.moe_window_workspace_bytes(*bad) == 0


def bf16(X=A, ldx=128, ids=A, wts=A, ldr=4, Wu=A, ldu=128, su=128 * 128, Wd=A, ldd=64, sd=64 * 128, Y=A, ldy=128, m=2,
         topk=4, experts=8, hidden=128, inter=64, base=0, dt=mr.MR_F32, flags=0, ws=A, size=BIG):
    return mr.lib.moe_window_bf16(X, ldx, ids, wts, ldr, Wu, ldu, su, Wd, ldd, sd, Y, ldy, m, topk, experts, hidden,
                                  inter, base, dt, flags, ws, size, None)


COMMON = [
    (dict(X=None), mr.MR_ERR_INVALID_ARG), (dict(ids=None), mr.MR_ERR_INVALID_ARG),
    (dict(wts=None), mr.MR_ERR_INVALID_ARG), (dict(Wu=None), mr.MR_ERR_INVALID_ARG),
    (dict(Wd=None), mr.MR_ERR_INVALID_ARG), (dict(Y=None), mr.MR_ERR_INVALID_ARG),
    (dict(ws=None), mr.MR_ERR_INVALID_ARG), (dict(m=0), mr.MR_ERR_INVALID_ARG), (dict(topk=0), mr.MR_ERR_INVALID_ARG),
    (dict(experts=0), mr.MR_ERR_INVALID_ARG), (dict(base=-1), mr.MR_ERR_INVALID_ARG),
    (dict(base=2 ** 31 - 4), mr.MR_ERR_INVALID_ARG), (dict(dt=mr.MR_F16), mr.MR_ERR_INVALID_ARG),
    (dict(flags=2), mr.MR_ERR_INVALID_ARG), (dict(ldx=120), mr.MR_ERR_INVALID_ARG),
    (dict(ldr=3), mr.MR_ERR_INVALID_ARG), (dict(ldy=127), mr.MR_ERR_INVALID_ARG),
    (dict(size=mr.moe_window_workspace_bytes(2, 4, 128, 64) - 1), mr.MR_ERR_INVALID_ARG),
    (dict(X=P(264)), mr.MR_ERR_MISALIGNED), (dict(ldx=132), mr.MR_ERR_MISALIGNED), (dict(ids=P(258)), mr.MR_ERR_MISALIGNED),
    (dict(wts=P(258)), mr.MR_ERR_MISALIGNED), (dict(Wu=P(264)), mr.MR_ERR_MISALIGNED),
    (dict(Wd=P(264)), mr.MR_ERR_MISALIGNED), (dict(Y=P(258)), mr.MR_ERR_MISALIGNED),
    (dict(Y=P(257), dt=mr.MR_BF16), mr.MR_ERR_MISALIGNED), (dict(ws=P(384)), mr.MR_ERR_MISALIGNED),
    (dict(m=17), mr.MR_ERR_UNSUPPORTED), (dict(topk=33, ldr=33), mr.MR_ERR_UNSUPPORTED),
]


@pytest.mark.parametrize("kw,code", COMMON + [
    (dict(hidden=0), mr.MR_ERR_INVALID_ARG), (dict(inter=0), mr.MR_ERR_INVALID_ARG),
    (dict(ldu=120), mr.MR_ERR_INVALID_ARG), (dict(ldd=56), mr.MR_ERR_INVALID_ARG), (dict(su=-8), mr.MR_ERR_INVALID_ARG),
    (dict(ldu=132), mr.MR_ERR_MISALIGNED), (dict(sd=60), mr.MR_ERR_MISALIGNED),
    (dict(hidden=124), mr.MR_ERR_MISALIGNED), (dict(inter=60), mr.MR_ERR_MISALIGNED),
    (dict(m=16, hidden=16384, ldx=16384, ldu=16384, ldy=16384), mr.MR_ERR_UNSUPPORTED),
    (dict(m=16, inter=16384, ldd=16384), mr.MR_ERR_UNSUPPORTED),
])
def test_bf16_refusals(kw, code):
    assert bf16(**kw) == code


def w4(X=A, ldx=128, ids=A, wts=A, ldr=4, Wu=A, ub=BIG, Wd=A, db=BIG, Y=A, ldy=128, m=2, topk=4, experts=8, hidden=128,
       inter=64, base=0, fmt=64, dt=mr.MR_F32, flags=0, ws=A, size=BIG):
    return mr.lib.moe_window_w4(X, ldx, ids, wts, ldr, Wu, ub, Wd, db, Y, ldy, m, topk, experts, hidden, inter, base,
                                fmt, dt, flags, ws, size, None)


@pytest.mark.parametrize("kw,code", COMMON + [
    (dict(fmt=128), mr.MR_ERR_INVALID_ARG), (dict(fmt=48), mr.MR_ERR_UNSUPPORTED), (dict(fmt=0), mr.MR_ERR_INVALID_ARG),
    (dict(fmt=64 | 0x400), mr.MR_ERR_INVALID_ARG), (dict(hidden=96, ldx=96, ldy=96), mr.MR_ERR_INVALID_ARG),
    (dict(inter=2 ** 31 - 8), mr.MR_ERR_UNSUPPORTED), (dict(inter=0), mr.MR_ERR_INVALID_ARG),
    (dict(ub=8 * mr.w4_packed_bytes(128, 128, 64, True) - 1), mr.MR_ERR_INVALID_ARG),
    (dict(db=8 * mr.w4_packed_bytes(128, 64, 64) - 1), mr.MR_ERR_INVALID_ARG),
])
def test_w4_refusals(kw, code):
    assert w4(**kw) == code


def test_documented_sizes_fit():
    torch = pytest.importorskip("torch")
    if torch.cuda.is_available():
        pytest.skip("only on a machine without a device: the stand-in pointers are never read there")
    big = dict(m=16, topk=32, ldr=32, hidden=4096, ldx=4096, ldy=4096, inter=2048)
    assert bf16(ldu=4096, ldd=2048, **big) == mr.MR_ERR_CUDA
    for fmt in (32, 32 | mr.MR_W4_ZEROS, 128):
        assert w4(fmt=fmt, **big) == mr.MR_ERR_CUDA


def test_binding_refusals():
    torch = pytest.importorskip("torch")
    bf = torch.bfloat16
    good = dict(X=torch.zeros(2, 128, dtype=bf), ids=torch.zeros(2, 4, dtype=torch.int32), weights=torch.zeros(2, 4),
                Wup=torch.zeros(8, 128, 128, dtype=bf), Wdown=torch.zeros(8, 128, 64, dtype=bf), Y=torch.zeros(2, 128),
                workspace=torch.zeros(1))
    for bad in (dict(ids=torch.zeros(3, 4, dtype=torch.int32)), dict(weights=torch.zeros(2, 5)),
                dict(weights=torch.zeros(4, 2).t()), dict(Y=torch.zeros(2, 120)), dict(Wup=torch.zeros(8, 64, 128, dtype=bf)),
                dict(Wdown=torch.zeros(8, 64, 64, dtype=bf)), dict(Wup=torch.zeros(8, 128, dtype=bf)),
                dict(Wdown=torch.zeros(8, 64, 128, dtype=bf).transpose(1, 2)), dict(X=torch.zeros(2, 128)),
                dict(ids=torch.zeros(2, 4, dtype=torch.int64)), dict(weights=torch.zeros(2, 4, dtype=bf)),
                dict(Wup=torch.zeros(8, 128, 128)), dict()):  # the last: not on a CUDA device
        with pytest.raises(ValueError):
            mr.moe_window_bf16(**dict(good, **bad))
