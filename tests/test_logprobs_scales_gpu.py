"""token_logprobs at the ends of its range of scales, and on logits far from zero, against 64 bits.

Tolerance.  u = 2^-24; z = scale * x, M the row's largest logit.  The kernel's d = c x log2 e - R has a constant off by 2u
relative and one rounding, so a difference of two d is off by 3u of itself: with p d^2 summed over a row below 160 (12^2
and its variance, n <= 2^18 within the last bits that count) that moves an entropy by less than 500 u.  R = c M log2 e is
rounded to r <= u |R|, at most 64 below 2^31 (beyond, the largest logit is subtracted first and r is 0): r is in every term, so it
cancels between log s and the mean but for their own roundings.  With eps = 2^-20 + (140 + n / 256) u for a sum
relative to itself (ex2.approx, the chains of additions),
 entropy: eps (2 + 2 (|mean d| + r)) + 500 u
 logprob: eps (1 + r) + 8 u (|value| + r)
 lse:     eps + 8 u (|c M| + |value|).
"""
import numpy as np
import pytest

from gpu_util import host, need_gpu, torch

import verify_weight_streaming_b200 as mr

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    need_gpu()
    yield
    assert mr.mr_poll_errors() == 0


def check(x, tokens, topk, scale):
    m, n = x.shape
    tokens = torch.tensor(tokens, dtype=torch.int32, device="cuda").reshape(m, -1)
    new = lambda *shape, dtype=torch.float32: torch.full(shape, 77, dtype=dtype, device="cuda")  # noqa: E731
    lp, lse, ent, ti, tl = (new(m, tokens.shape[1]), new(m), new(m), new(m, topk, dtype=torch.int32), new(m, topk))
    mr.token_logprobs(x, tokens, lp, scale=scale, lse=lse, entropy=ent, top_idx=ti, top_logprob=tl)
    x64 = x.cpu().double().numpy()
    order = np.argsort(-x64, axis=1, kind="stable")[:, :topk]
    z = x64 * float(np.float32(scale))
    top = z.max(axis=1, keepdims=True)
    e = np.exp(z - top)
    s = e.sum(axis=1, keepdims=True)
    mean = np.where(e > 0, e * np.where(e > 0, z - top, 0), 0).sum(axis=1) / s[:, 0]
    logp = z - top - np.log(s)
    eps = 2.0 ** -20 + (140 + n / 256) * U
    far = np.abs(top[:, 0]) * 1.4427
    r = np.where(far < 2.0 ** 31, np.minimum(U * far, 64.0), 0.0)
    assert np.array_equal(host(ti), order)

    def close(got, want, tol, name):
        with np.errstate(over="ignore"):  # beyond fp32: infinite
            got, want = host(got).astype(np.float64), np.float32(want).astype(np.float64)
        tol = np.broadcast_to(tol, want.shape)
        fine = np.isfinite(want)
        assert np.array_equal(got[~fine], want[~fine]), (name, got, want)
        assert not np.isnan(got).any(), (name, got, want)
        assert (np.abs(got[fine] - want[fine]) <= tol[fine] + U * np.abs(want[fine])).all(), (name, got, want)

    close(lse, (top + np.log(s))[:, 0], eps + 8 * U * (np.abs(top[:, 0]) + np.log(n)), "lse")
    close(ent, np.log(s[:, 0]) - mean, eps * (2 + 2 * (np.abs(mean) + r)) + 500 * U, "entropy")
    for got, at in ((lp, tokens.cpu().numpy()), (tl, order)):
        want = np.take_along_axis(logp, at, 1)
        size = np.where(np.isfinite(want), np.abs(want), 0)
        close(got, want, eps * (1 + r[:, None]) + 8 * U * (size + r[:, None]), "logprob")


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("n", [40, 131072, 262144])
@pytest.mark.parametrize("mask", ["inf", "lowest", "-1e30"])
def test_masked_rows_at_every_scale(dtype, n, mask):
    """Rows of which a mask leaves one logit, two, a piece, or every other one: whole warps see nothing but masked ones."""
    if dtype == "f16" and mask == "-1e30":
        mask = "-3e4"
    low = {"inf": -float("inf"), "lowest": torch.finfo(DT[dtype]).min}.get(mask) or float(mask)
    rng = np.random.default_rng(n)
    live = [[0], [n // 2], [n - 1], [n // 3, 2 * n // 3], [0, n - 1], list(range(n // 4, n // 4 + 9)),
            list(range(0, n // 16)), list(range(0, n, 2))]
    base = torch.from_numpy(rng.standard_normal((len(live), n))).to(DT[dtype]).cuda()
    x = torch.full_like(base, low)
    for r, at in enumerate(live):
        x[r, at] = base[r, at]
    x[4, [0, n - 1]] = 0.75  # two equal ones: entropy log 2
    tokens = [[at[0], at[-1]] for at in live]
    for scale in (1e-6, 1.0, 2e4, 5e4, 1e5, 1e6):
        check(x, tokens, 3, scale)


def test_close_logits_at_the_largest_scale():
    """Steps of 2^-20 around 1 at scale 1e6: about one nat each."""
    x = torch.full((3, 131072), -float("inf"), device="cuda")
    steps = torch.arange(12, device="cuda") * 2.0 ** -20
    x[0, 70000:70012] = 1.0 - steps
    x[1, ::11000] = 1.0 - steps
    x[2, :] = -5.0
    x[2, 3:15] = 1.0 + steps
    check(x, [[70003], [11000], [9]], 12, 1e6)


@pytest.mark.parametrize("dtype,scale", [("f32", 1.0), ("f32", 40.0), ("f32", 1e6), ("bf16", 1.0), ("bf16", 40.0),
                                         ("bf16", 1e6), ("f16", 1e6)])
def test_logits_far_from_zero(dtype, scale):
    """Largest products from 2^23 to 2^40: one logit well above the others, two equal ones, steps, all equal, both signs."""
    rng = np.random.default_rng(17)
    size = 2.0 ** rng.uniform(23, 40, 120) / scale
    size[:3] = 1.4971036e9 / scale, 1.4971036e9 * 1.0625 / scale, 1.86e9 / scale  # about 2^31 in units of log 2
    size = size[size < (6e4 if dtype == "f16" else 1e38)]
    n = 3001
    x = torch.zeros((6 * len(size), n), dtype=torch.float64)
    for i, v in enumerate(size):
        rows = x[6 * i:6 * i + 6]
        rows[0, 777] = v
        rows[1, 5], rows[1, 2999] = v, v
        rows[2] = v * (1 - torch.arange(n) / 4096.0)
        rows[3] = -v
        rows[4] = -2 * v
        rows[4, 2000] = -v
        rows[5] = -float("inf")
        rows[5, ::700] = -v
    check(x.to(DT[dtype]).cuda(), [[777, 5]] * len(x), 4, scale)
