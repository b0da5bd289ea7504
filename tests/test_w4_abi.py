"""The 4-bit entry points on a machine without a GPU: sizes, refusals, status codes."""
import ctypes

import pytest

import verify_weight_streaming_b200 as mr

P = ctypes.c_void_p
A16 = P(256)
SMALL = P(258)
Z, F16 = mr.MR_W4_ZEROS, mr.MR_W4_SCALE_F16
OK_BYTES = 1 << 30


@pytest.mark.parametrize("n,k,fmt,paired,want", [
    (16, 128, 128, 0, 1024 + 32), (16, 128, 64, 0, 1024 + 64), (16, 128, 32 | Z, 0, 1024 + 128 + 64),
    (17, 128, 128 | F16, 0, 2 * 1056), (1, 32, 32, 0, 1152), (16, 160, 32, 0, 2 * 1152),
    (16, 128, 128, 1, 1056), (18, 128, 128, 1, 2 * 1056), (131072, 2560, 128, 0, 8192 * 20 * 1056),
    (0, 128, 128, 0, 0), (16, 100, 128, 0, 0), (16, 128, 16, 0, 0), (16, 128, 0, 0, 0), (17, 128, 128, 1, 0),
    (16, 128, 128 | 0x400, 0, 0),
])
def test_packed_bytes(n, k, fmt, paired, want):
    assert mr.lib.w4_packed_bytes(n, k, fmt, paired) == want


def pack(q=A16, s=A16, z=None, out=A16, size=OK_BYTES, count=1, n=32, k=128, fmt=128, paired=0):
    return mr.lib.w4_pack(q, s, z, out, size, count, n, k, fmt, paired, None)


@pytest.mark.parametrize("kw,code", [
    (dict(q=None), mr.MR_ERR_INVALID_ARG), (dict(s=None), mr.MR_ERR_INVALID_ARG),
    (dict(out=None), mr.MR_ERR_INVALID_ARG), (dict(count=0), mr.MR_ERR_INVALID_ARG),
    (dict(n=0), mr.MR_ERR_INVALID_ARG), (dict(k=0), mr.MR_ERR_INVALID_ARG), (dict(k=130), mr.MR_ERR_INVALID_ARG),
    (dict(fmt=0), mr.MR_ERR_INVALID_ARG), (dict(fmt=128 | 0x800), mr.MR_ERR_INVALID_ARG),
    (dict(fmt=16), mr.MR_ERR_UNSUPPORTED), (dict(fmt=255, k=255), mr.MR_ERR_UNSUPPORTED),
    (dict(fmt=128 | Z), mr.MR_ERR_INVALID_ARG), (dict(z=A16), mr.MR_ERR_INVALID_ARG),
    (dict(n=33, paired=1), mr.MR_ERR_INVALID_ARG), (dict(size=2 * 1056 - 1), mr.MR_ERR_INVALID_ARG),
    (dict(size=3 * 2 * 1056 - 1, count=3), mr.MR_ERR_INVALID_ARG),
    (dict(q=SMALL), mr.MR_ERR_MISALIGNED), (dict(s=P(257)), mr.MR_ERR_MISALIGNED),
    (dict(out=P(264)), mr.MR_ERR_MISALIGNED),
])
def test_pack_refusals(kw, code):
    assert pack(**kw) == code


def gemv(A=A16, lda=128, W=A16, size=OK_BYTES, C=A16, ldc=32, m=4, n=32, k=128, dt=mr.MR_BF16, fmt=128, flags=0):
    return mr.lib.mrgemv_w4(A, lda, W, size, C, ldc, m, n, k, dt, fmt, flags, None)


@pytest.mark.parametrize("kw,code", [
    (dict(A=None), mr.MR_ERR_INVALID_ARG), (dict(W=None), mr.MR_ERR_INVALID_ARG),
    (dict(C=None), mr.MR_ERR_INVALID_ARG), (dict(m=0), mr.MR_ERR_INVALID_ARG), (dict(n=0), mr.MR_ERR_INVALID_ARG),
    (dict(k=0), mr.MR_ERR_INVALID_ARG), (dict(lda=120), mr.MR_ERR_INVALID_ARG),
    (dict(ldc=31), mr.MR_ERR_INVALID_ARG), (dict(dt=mr.MR_F32), mr.MR_ERR_INVALID_ARG),
    (dict(dt=-1), mr.MR_ERR_INVALID_ARG), (dict(flags=mr.MR_GEMV_SIGMOID), mr.MR_ERR_INVALID_ARG),
    (dict(size=2 * 1056 - 1), mr.MR_ERR_INVALID_ARG), (dict(fmt=64 | Z, size=2 * 1056), mr.MR_ERR_INVALID_ARG),
    (dict(k=160, lda=160), mr.MR_ERR_INVALID_ARG), (dict(fmt=48, k=96), mr.MR_ERR_UNSUPPORTED),
    (dict(lda=132), mr.MR_ERR_MISALIGNED), (dict(A=SMALL), mr.MR_ERR_MISALIGNED),
    (dict(W=P(264)), mr.MR_ERR_MISALIGNED), (dict(C=SMALL), mr.MR_ERR_MISALIGNED),
    (dict(m=17), mr.MR_ERR_UNSUPPORTED), (dict(k=1 << 21, lda=1 << 21, size=1 << 40), mr.MR_ERR_UNSUPPORTED),
    (dict(m=16, k=16384, lda=16384), mr.MR_ERR_UNSUPPORTED),
])
def test_gemv_refusals(kw, code):
    assert gemv(**kw) == code


def test_widest_window_takes_k_4096_in_every_format():
    import torch
    if torch.cuda.is_available():
        pytest.skip("only on a machine without a device: the stand-in pointers are never read there")
    for fmt in (32, 32 | Z, 64 | Z | F16, 128):
        assert gemv(m=16, k=4096, lda=4096, fmt=fmt) == mr.MR_ERR_CUDA


def test_binding_refusals():
    torch = pytest.importorskip("torch")
    q = torch.zeros((16, 64), dtype=torch.uint8)
    s = torch.zeros((16, 1), dtype=torch.bfloat16)
    out = torch.zeros(1056, dtype=torch.uint8)
    for bad in (dict(q=q.to(torch.int32)), dict(s=s[:8]), dict(s=s.float()), dict(z=torch.zeros(16, 2, dtype=torch.uint8)),
                dict(z=torch.zeros(16, 1)), dict(q=torch.zeros((64, 16), dtype=torch.uint8).t()),
                dict(out=torch.zeros(1056))):
        args = dict(dict(q=q, s=s, z=None, out=out), **bad)
        with pytest.raises(ValueError):
            mr.w4_pack(args["q"], args["s"], args["z"], args["out"])
    with pytest.raises(ValueError):
        mr.mrgemv_w4(torch.zeros((2, 128), dtype=torch.bfloat16), out, torch.zeros((3, 16)), 128)
    a = torch.zeros((2, 128), dtype=torch.bfloat16)
    for c, packed in ((torch.zeros((2, 16)).half(), out), (torch.zeros((2, 16)), out.to(torch.int32)),
                      (torch.zeros((2, 16)), out)):  # the last: not on a CUDA device
        with pytest.raises(ValueError):
            mr.mrgemv_w4(a, packed, c, 128)
    with pytest.raises(ValueError):
        mr.w4_pack(q, s, None, out)
