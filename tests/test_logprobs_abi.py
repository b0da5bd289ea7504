"""token_logprobs on a machine without a GPU: refusals and status codes."""
import ctypes

import pytest

import verify_weight_streaming_b200 as mr

P = ctypes.c_void_p
A, ODD = P(256), P(258)


def call(x=A, ld=100, dt=mr.MR_F32, m=2, n=100, scale=1.0, tok=A, ldt=3, ntok=3, lp=A, ldp=3, lse=A, ent=A, topk=5, idx=A,
         tlp=A, ldo=5):
    return mr.lib.token_logprobs(x, ld, dt, m, n, scale, tok, ldt, ntok, lp, ldp, lse, ent, topk, idx, tlp, ldo, None)


@pytest.mark.parametrize("kw,code", [
    (dict(x=None), mr.MR_ERR_INVALID_ARG), (dict(m=0), mr.MR_ERR_INVALID_ARG), (dict(n=0), mr.MR_ERR_INVALID_ARG),
    (dict(dt=3), mr.MR_ERR_INVALID_ARG), (dict(dt=-1), mr.MR_ERR_INVALID_ARG), (dict(ld=99), mr.MR_ERR_INVALID_ARG),
    (dict(scale=0.0), mr.MR_ERR_INVALID_ARG), (dict(scale=-1.0), mr.MR_ERR_INVALID_ARG),
    (dict(scale=float("nan")), mr.MR_ERR_INVALID_ARG), (dict(scale=float("inf")), mr.MR_ERR_INVALID_ARG),
    (dict(tok=None), mr.MR_ERR_INVALID_ARG), (dict(lp=None), mr.MR_ERR_INVALID_ARG), (dict(ldt=2), mr.MR_ERR_INVALID_ARG),
    (dict(ldp=2), mr.MR_ERR_INVALID_ARG), (dict(ntok=-1), mr.MR_ERR_INVALID_ARG), (dict(topk=-1), mr.MR_ERR_INVALID_ARG),
    (dict(topk=101, ldo=101), mr.MR_ERR_INVALID_ARG), (dict(idx=None), mr.MR_ERR_INVALID_ARG),
    (dict(ldo=4), mr.MR_ERR_INVALID_ARG), (dict(topk=0), mr.MR_ERR_INVALID_ARG),
    (dict(ntok=0, tok=None, lp=None, lse=None, ent=None, topk=0, idx=None, tlp=None), mr.MR_ERR_INVALID_ARG),
    (dict(x=ODD), mr.MR_ERR_MISALIGNED), (dict(x=P(257), dt=mr.MR_BF16), mr.MR_ERR_MISALIGNED),
    (dict(tok=ODD), mr.MR_ERR_MISALIGNED), (dict(lp=ODD), mr.MR_ERR_MISALIGNED), (dict(lse=ODD), mr.MR_ERR_MISALIGNED),
    (dict(ent=ODD), mr.MR_ERR_MISALIGNED), (dict(idx=ODD), mr.MR_ERR_MISALIGNED), (dict(tlp=ODD), mr.MR_ERR_MISALIGNED),
    (dict(topk=33, ldo=33), mr.MR_ERR_UNSUPPORTED), (dict(ntok=257, ldt=257, ldp=257), mr.MR_ERR_UNSUPPORTED),
    (dict(n=2 ** 30 + 1, ld=2 ** 31), mr.MR_ERR_UNSUPPORTED),
])
def test_refusals(kw, code):
    assert call(**kw) == code


def test_valid_calls_without_device():
    import torch
    if torch.cuda.is_available():
        pytest.skip("only on a machine without a device: the stand-in pointers are never read there")
    assert call() == mr.MR_ERR_CUDA
    assert call(x=ODD, dt=mr.MR_F16, tlp=None) == mr.MR_ERR_CUDA
    assert call(ntok=0, tok=None, lp=None, topk=0, idx=None, tlp=None, ent=None) == mr.MR_ERR_CUDA


def test_binding_refusals():
    torch = pytest.importorskip("torch")
    x, tok, lp = torch.zeros(2, 50), torch.zeros(2, 3, dtype=torch.int32), torch.zeros(2, 3)
    idx, tlp = torch.zeros(2, 4, dtype=torch.int32), torch.zeros(2, 4)
    for bad in (dict(tokens=tok), dict(logprob=lp), dict(tokens=tok[:1], logprob=lp), dict(tokens=tok, logprob=lp[:, :2]),
                dict(lse=torch.zeros(3)), dict(entropy=torch.zeros(2, 1)), dict(lse=torch.zeros(4)[::2]),
                dict(top_logprob=tlp), dict(top_idx=idx[:1]), dict(top_idx=idx, top_logprob=tlp[:, :3])):
        with pytest.raises(ValueError):
            mr.token_logprobs(x, **bad)
    for bad in (dict(tokens=tok.long(), logprob=lp), dict(tokens=tok, logprob=lp.double()), dict(lse=torch.zeros(2).half()),
                dict(top_idx=idx.long()), dict(lse=torch.zeros(2))):  # the last: not on a CUDA device
        with pytest.raises(ValueError):
            mr.token_logprobs(x, **bad)
