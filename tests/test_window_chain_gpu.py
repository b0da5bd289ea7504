"""The operators of a verify window together: router, routed experts, 4-bit head, log probabilities.

One window of draft rows goes through router_gemv_topk -> moe_window -> cast_f32_bf16 -> mrgemv_w4 -> token_logprobs,
eagerly and captured in one CUDA graph that is replayed with new rows; every step is checked against 64 bits on
that step's own inputs, and the window's rows against the same rows alone.
"""
import numpy as np
import pytest

import w4_util
from gpu_util import host, need_gpu, torch

import verify_weight_streaming_b200 as mr

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
HIDDEN, INTER, EXPERTS, TOPK, VOCAB = 512, 256, 64, 6, 5004


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    need_gpu()
    yield
    assert mr.mr_poll_errors() == 0


# (A vocabulary whose rows of fp32 logits all start at the same address modulo 16: token_logprobs' sums depend on it.)
class Window:
    def __init__(self, m, group):
        rng = np.random.default_rng(7)
        self.m, self.group = m, group
        self.router = torch.from_numpy(rng.standard_normal((EXPERTS, HIDDEN)) / 22).to(torch.bfloat16).cuda()
        self.head64 = w4_util.weight(1, (), VOCAB, HIDDEN, 128, True)
        self.head, self.head_fmt = w4_util.pack(mr, self.head64)
        if group:
            self.up64, self.down64 = (w4_util.weight(2, (EXPERTS,), 2 * INTER, HIDDEN, group, False),
                                      w4_util.weight(3, (EXPERTS,), HIDDEN, INTER, group, False))
            (self.up, self.fmt), (self.down, _) = w4_util.pack(mr, self.up64, True), w4_util.pack(mr, self.down64)
            self.up64, self.down64 = w4_util.dense64(self.up64), w4_util.dense64(self.down64)
        else:
            self.up = torch.from_numpy(rng.standard_normal((EXPERTS, 2 * INTER, HIDDEN)) / 22).to(torch.bfloat16).cuda()
            self.down = torch.from_numpy(rng.standard_normal((EXPERTS, HIDDEN, INTER)) / 16).to(torch.bfloat16).cuda()
            self.up64, self.down64 = self.up.cpu().double().numpy(), self.down.cpu().double().numpy()
        new = lambda *shape, dtype=torch.float32: torch.zeros(shape, dtype=dtype, device="cuda")  # noqa: E731
        self.x = new(m, HIDDEN, dtype=torch.bfloat16)
        self.drafts = new(m, 1, dtype=torch.int32)
        self.ids, self.val = new(m, TOPK, dtype=torch.int32), new(m, TOPK)
        self.y, self.y16 = new(m, HIDDEN), new(m, HIDDEN, dtype=torch.bfloat16)
        self.logits = new(m, VOCAB)
        self.logprob, self.entropy, self.lse = new(m, 1), new(m), new(m)
        self.top_idx, self.top_logprob = new(m, 3, dtype=torch.int32), new(m, 3)
        self.route_ws = new(mr.router_gemv_topk_workspace_bytes(m, EXPERTS, False), dtype=torch.uint8)
        self.moe_ws = new(mr.moe_window_workspace_bytes(m, TOPK, HIDDEN, INTER), dtype=torch.uint8)

    def fill(self, seed):
        rng = np.random.default_rng(seed)
        self.x.copy_(torch.from_numpy(rng.standard_normal((self.m, HIDDEN))))
        self.drafts.copy_(torch.from_numpy(rng.integers(0, VOCAB, (self.m, 1))))

    def run(self):
        mr.router_gemv_topk(self.x, self.router, TOPK, self.ids, self.val, workspace=self.route_ws, flags=mr.MR_GEMV_PDL)
        if self.group:
            mr.moe_window_w4(self.x, self.ids, self.val, self.up, self.down, self.y, self.moe_ws, EXPERTS, INTER,
                             self.fmt, flags=mr.MR_MOE_SOFTMAX)
        else:
            mr.moe_window_bf16(self.x, self.ids, self.val, self.up, self.down, self.y, self.moe_ws,
                               flags=mr.MR_MOE_SOFTMAX)
        mr.cast_f32_bf16(self.y, self.y16)
        mr.mrgemv_w4(self.y16, self.head, self.logits, self.head_fmt, flags=mr.MR_GEMV_PDL)
        mr.token_logprobs(self.logits, self.drafts, self.logprob, lse=self.lse, entropy=self.entropy,
                          top_idx=self.top_idx, top_logprob=self.top_logprob)

    def results(self):
        return [host(t).copy() for t in (self.ids, self.y, self.logits, self.logprob, self.lse, self.entropy,
                                         self.top_idx, self.top_logprob)]

    def check(self):
        ids, y, logits, logprob, lse, entropy, top_idx, top_logprob = self.results()
        x, val = self.x.cpu().double().numpy(), self.val.cpu().double().numpy()
        router = x @ self.router.cpu().double().numpy().T
        assert np.array_equal(np.sort(ids, 1), np.sort(np.argsort(-router, 1)[:, :TOPK], 1))  # no near ties in these
        w = np.exp(val - val.max(1, keepdims=True))
        w /= w.sum(1, keepdims=True)
        for t in range(self.m):
            want, size = 0.0, 0.0
            for s, e in enumerate(ids[t]):
                g, u = np.split(self.up64[e] @ x[t], 2)
                h = g / (1 + np.exp(-g)) * u
                big = np.abs(self.up64[e]) @ np.abs(x[t])
                sens = np.abs(h) + 1.1 * big[:INTER] * np.abs(u) + np.abs(g) * big[INTER:]
                want = want + w[t, s] * (self.down64[e] @ h)
                size = size + w[t, s] * (np.abs(self.down64[e]) @ sens)
            assert (np.abs(y[t] - want) <= 600 * U * size).all()  # the layer's own test counts these roundings
        y16, head = self.y16.cpu().double().numpy(), w4_util.dense64(self.head64)
        assert (np.abs(logits - y16 @ head.T) <= (8 * 17 * 2 + 8) * U * (np.abs(y16) @ np.abs(head).T)).all()
        z = logits.astype(np.float64)
        top = z.max(1, keepdims=True)
        s = np.exp(z - top).sum(1, keepdims=True)
        logp = z - top - np.log(s)
        eps = 2.0 ** -20 + 200 * U + 16 * U * np.abs(z).max()
        assert np.allclose(lse, (top + np.log(s))[:, 0], rtol=0, atol=eps)
        assert np.allclose(logprob, np.take_along_axis(logp, self.drafts.cpu().numpy(), 1), rtol=0, atol=eps)
        assert np.allclose(entropy, -(np.exp(logp) * logp).sum(1), rtol=0, atol=32 * eps)
        order = np.argsort(-z, 1, kind="stable")[:, :3]
        assert np.array_equal(top_idx, order)
        assert np.allclose(top_logprob, np.take_along_axis(logp, order, 1), rtol=0, atol=eps)


@pytest.mark.parametrize("m,group", [(1, 0), (5, 128), (16, 0)])
def test_window(m, group):
    window = Window(m, group)
    window.fill(11)
    window.run()
    window.check()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        window.run()
    for seed in (12, 13):
        window.fill(seed)
        graph.replay()
        window.check()


@pytest.mark.parametrize("group", [0, 64])
def test_rows_of_a_window_have_the_bits_of_single_windows(group):
    window = Window(8, group)
    window.fill(21)
    window.run()
    whole = window.results()
    for row in (0, 3, 7):
        one = Window(1, group)
        one.x.copy_(window.x[row:row + 1])
        one.drafts.copy_(window.drafts[row:row + 1])
        one.run()
        for a, b in zip(one.results(), whole):
            assert np.array_equal(a.view(np.uint32), b[row:row + 1].view(np.uint32))


def test_on_another_stream_than_the_tensors_were_made_on():
    window = Window(4, 0)
    window.fill(31)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        for _ in range(3):
            window.run()
    side.synchronize()
    window.check()
