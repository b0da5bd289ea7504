"""One row: the stride of a dimension of size one has no meaning, and torch may hold any number there."""
import numpy as np
import pytest

import w4_util
from gpu_util import host, need_gpu, torch

import verify_weight_streaming_b200 as mr

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    need_gpu()
    yield
    assert mr.mr_poll_errors() == 0


def restride(t, stride):
    """The same [1, n] row, its first stride another."""
    return t.as_strided(t.shape, (stride, 1))


@pytest.mark.parametrize("stride", [0, 1, 3])
def test_one_row_of_any_stride(stride):
    rng = np.random.default_rng(1)
    k, n, topk, inter = 256, 200, 4, 64
    odd = lambda t: restride(t, stride)  # noqa: E731
    a = torch.from_numpy(rng.standard_normal((1, k))).to(torch.bfloat16).cuda()
    packed, fmt = w4_util.pack(mr, w4_util.weight(2, (), n, k, 64, True))
    c0, c1 = torch.zeros((1, n), device="cuda"), torch.zeros((1, n), device="cuda")
    mr.mrgemv_w4(a, packed, c0, fmt)
    mr.mrgemv_w4(odd(a), packed, odd(c1), fmt)
    assert np.array_equal(host(c0), host(c1)) and host(c0).any()

    ids = torch.tensor([[1, 0, -1, 2]], dtype=torch.int32, device="cuda")
    wts = torch.from_numpy(rng.standard_normal((1, topk)).astype(np.float32)).cuda()
    up = torch.from_numpy(rng.standard_normal((3, 2 * inter, k)) / 16).to(torch.bfloat16).cuda()
    down = torch.from_numpy(rng.standard_normal((3, k, inter)) / 8).to(torch.bfloat16).cuda()
    ws = torch.zeros(mr.moe_window_workspace_bytes(1, topk, k, inter), dtype=torch.uint8, device="cuda")
    y0, y1 = torch.zeros((1, k), device="cuda"), torch.zeros((1, k), device="cuda")
    mr.moe_window_bf16(a, ids, wts, up, down, y0, ws)
    mr.moe_window_bf16(odd(a), ids, odd(wts), up, down, odd(y1), ws)
    assert np.array_equal(host(y0), host(y1)) and host(y0).any()
    mr.moe_window_bf16(a, odd(ids), wts, up, down, y1.zero_(), ws)
    assert np.array_equal(host(y0), host(y1))
    one = lambda t: t[:1].as_strided(t[:1].shape, (stride, *t.stride()[1:]))  # noqa: E731  (one expert)
    mr.moe_window_bf16(a, ids, wts, up[:1].clone(), down[:1].clone(), y0, ws)
    mr.moe_window_bf16(a, ids, wts, one(up), one(down), y1, ws)
    assert np.array_equal(host(y0), host(y1)) and host(y0).any()

    tokens, out = torch.tensor([[3, 7]], dtype=torch.int32, device="cuda"), []
    for f in (lambda t: t, odd):
        lp, tl, ti = torch.zeros((1, 2), device="cuda"), torch.zeros((1, 5), device="cuda"), torch.zeros(
            (1, 5), dtype=torch.int32, device="cuda")
        lse, ent = (torch.zeros(4, device="cuda")[:1].as_strided((1,), (1 if f is not odd else stride,)) for _ in range(2))
        mr.token_logprobs(f(c0), f(tokens), f(lp), lse=lse, entropy=ent, top_idx=ti, top_logprob=f(tl))
        mr.token_logprobs(f(c0), top_idx=f(ti))
        out.append([host(t).copy() for t in (lp, tl, ti, lse, ent)])
    for x, y in zip(*out):
        assert np.array_equal(x, y) and x.any()


def test_one_column_of_any_stride():
    c = torch.randn((3, 50), device="cuda")
    tokens = torch.tensor([[4, 9, 30]], dtype=torch.int32, device="cuda").t()  # [3, 1], strides (1, 3)
    got, want = torch.zeros((1, 3), device="cuda").t(), torch.zeros((3, 1), device="cuda")
    idx = torch.zeros((1, 3), dtype=torch.int32, device="cuda").t()
    mr.token_logprobs(c, tokens, got, top_idx=idx)
    mr.token_logprobs(c, tokens.contiguous(), want)
    assert np.array_equal(host(got), host(want)) and torch.equal(idx[:, 0].long(), c.argmax(1))
