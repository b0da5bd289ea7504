"""A weight written two kernels before a product that reads it ahead (MR_GEMV_PDL), with an operator of the window between.

token_logprobs and mrgemv_w4 let the next kernel start only once their own predecessor has completed, so what that wrote is
there when the product requests its weight. Every pass writes another weight; the product has to have the bits of the
same product run alone afterwards.
"""
import numpy as np
import pytest

import w4_util
from gpu_util import host, need_gpu, torch

import verify_weight_streaming_b200 as mr

pytestmark = pytest.mark.gpu
N, K = 4864, 896


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    need_gpu()
    yield
    assert mr.mr_poll_errors() == 0


class Chain:
    def __init__(self, between):
        rng = np.random.default_rng(5)
        new = lambda *shape, dtype=torch.float32: torch.zeros(shape, dtype=dtype, device="cuda")  # noqa: E731
        self.between = between
        self.q, self.s, _ = (None if t is None else t.cuda() for t in w4_util.weight(1, (), N, K, 64, False))
        self.fmt = mr.w4_format(64, False, self.s.dtype)
        self.packed = new(mr.w4_packed_bytes(N, K, self.fmt), dtype=torch.uint8)
        self.other, _ = w4_util.pack(mr, w4_util.weight(2, (), 512, K, 64, False))
        self.w32, self.w16 = new(N, K), new(N, K, dtype=torch.bfloat16)
        self.a = torch.from_numpy(rng.standard_normal((3, K))).to(torch.bfloat16).cuda()
        self.logits = torch.from_numpy(rng.standard_normal((16, 30000)).astype(np.float32)).cuda()
        self.lse, self.top = new(16), new(16, 4, dtype=torch.int32)
        self.c4, self.c16, self.c0 = new(3, N), new(3, N), new(3, 512)

    def fill(self, seed):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        self.q.random_(0, 256, generator=gen)
        self.w32.normal_(generator=gen)

    def step(self):
        if self.between == "logprobs":
            mr.token_logprobs(self.logits, lse=self.lse, top_idx=self.top)
        else:
            mr.mrgemv_w4(self.a, self.other, self.c0, self.fmt, flags=mr.MR_GEMV_PDL)

    def run(self):
        mr.w4_pack(self.q, self.s, None, self.packed)
        self.step()
        mr.mrgemv_w4(self.a, self.packed, self.c4, self.fmt, flags=mr.MR_GEMV_PDL)
        mr.cast_f32_bf16(self.w32, self.w16)
        self.step()
        mr.mrgemv_bf16(self.a, self.w16, self.c16, flags=mr.MR_GEMV_PDL)

    def check(self):
        got = host(self.c4).copy(), host(self.c16).copy()
        packed, w16 = torch.empty_like(self.packed), self.w32.to(torch.bfloat16)
        mr.w4_pack(self.q, self.s, None, packed)
        torch.cuda.synchronize()
        mr.mrgemv_w4(self.a, packed, self.c4, self.fmt)
        mr.mrgemv_bf16(self.a, w16, self.c16)
        for a, b in zip(got, (self.c4, self.c16)):
            assert np.array_equal(a.view(np.uint32), host(b).view(np.uint32))


@pytest.mark.parametrize("between", ["logprobs", "product"])
def test_weight_written_two_kernels_before(between):
    chain = Chain(between)
    for seed in range(8):
        chain.fill(seed)
        torch.cuda.synchronize()
        chain.run()
        chain.check()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        chain.run()
    for seed in range(8, 24):
        chain.fill(seed)
        graph.replay()
        chain.check()
