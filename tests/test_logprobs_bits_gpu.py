"""A row's results have the same bits however many CTAs share it, with and without loads ahead.

With 148 SMs and top alternatives, a row of 131072 fp32 (8 pieces) goes to 8 CTAs alone, 4 among 100 rows, 2 among 200 and 1 among
400; rows of 50021 f16 (2 pieces) go to 2 CTAs alone and to 1 without loads ahead among 700; rows of 4096 fp32 are
one CTA's, with loads ahead alone and without among 2048.  Rows lie at multiples of 16 bytes: the sums depend on that.
"""
import numpy as np
import pytest

from gpu_util import host, need_gpu, torch

import verify_weight_streaming_b200 as mr

pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    need_gpu()
    yield
    assert mr.mr_poll_errors() == 0


def ask(x, tokens, topk):
    m, new = x.shape[0], lambda *shape, dtype=torch.float32: torch.zeros(shape, dtype=dtype, device="cuda")
    lp, lse, ent, ti, tl = (new(m, tokens.shape[1]), new(m), new(m), new(m, topk, dtype=torch.int32), new(m, topk))
    top = dict(top_idx=ti, top_logprob=tl) if topk else {}
    mr.token_logprobs(x, tokens, lp, scale=1.25, lse=lse, entropy=ent, **top)
    return [host(t).view(np.uint32) for t in (lp, lse[:, None], ent[:, None], ti, tl)]


@pytest.mark.parametrize("topk", [0, 6])
@pytest.mark.parametrize("n,dtype,counts", [(131072, "f32", (100, 200, 400)), (50021, "f16", (700,)),
                                            (40004, "bf16", (300, 700)), (4096, "f32", (2048,)), (151667, "bf16", (250, 500))])
def test_rows_alone_and_among_others(n, dtype, counts, topk):
    m, ld = max(counts), -(-n // 8) * 8
    gen = torch.Generator(device="cuda").manual_seed(n)
    x = torch.empty((m, ld), dtype=DT[dtype], device="cuda").normal_(0, 3, generator=gen)[:, :n]
    x[1, torch.rand(n, generator=gen, device="cuda") < 0.9] = -float("inf")
    x[2, 5:] = torch.finfo(DT[dtype]).min
    x[3] = 0.5
    x[4, n // 3] = float("nan")
    x[5, : n - 9] = -float("inf")
    x[6, n - 1] = float("inf")
    x[7] = x[7].abs() * 100 + 20000  # many equal ones in 16 bits
    tokens = torch.randint(0, n, (m, 2), generator=gen, device="cuda").to(torch.int32)
    rows = [0, 1, 2, 3, 4, 5, 6, 7, m // 2, min(counts) - 1]
    alone = [ask(x[r:r + 1], tokens[r:r + 1], topk) for r in rows]
    for among in [x[:9], *(x[:count] for count in counts)]:
        whole = ask(among, tokens[:len(among)], topk)
        for r, one in zip(rows, alone):
            if r < len(among):
                assert all(np.array_equal(a, b[r:r + 1]) for a, b in zip(one, whole)), (len(among), r)
