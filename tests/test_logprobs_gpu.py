"""token_logprobs on the GPU against 64 bits.

Tolerance.  u = 2^-24.  The kernel forms d = c x log2 e - R with one rounding of
the product's constant (relative u) and one of R = c M log2 e (relative u, the same
in every term, so it cancels but for the final sum), then 2^d by ex2.approx (2
units of 2^-22 relative).  With A = max |c x| over the finite logits and the
largest gap D = max c (M - x) that still counts (2^d >= 2^-149, so D <= 104): a term
is off by at most 4u + 2^-21 + D u relative, the sum of n terms by no more than that
plus its own roundings, under (n / (256 * pieces) + 32) u per chain.  So
log s is within eps = 2^-20 + (140 + n / 256) u absolute, and
 lse, logprob: eps + 8 u (A + |value|)
 entropy:      its mean d is a ratio of sums off by eps relative each, its
               terms |d| 2^d at most: eps * (2 + 2 |mean d|) + 8 u (1 + A).
"""
import numpy as np
import pytest

from gpu_util import host, need_gpu, padded, torch

import verify_weight_streaming_b200 as mr

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    need_gpu()
    yield
    assert mr.mr_poll_errors() == 0


def ask(x, tokens, topk, scale=1.0):
    """Every output, with canaries around it."""
    m, ntok = x.shape[0], tokens.shape[1]
    lp, _ = padded(m + 1, ntok + 2, ntok + 2, torch.float32, 77.0)
    tl, _ = padded(m + 1, topk + 3, topk + 3, torch.float32, 77.0)
    ti, _ = padded(m + 1, topk + 3, topk + 3, torch.int32, -77)
    lse, ent = (torch.full((m + 1,), 77.0, device="cuda") for _ in range(2))
    mr.token_logprobs(x, tokens, lp[:m, :ntok], scale=scale, lse=lse[:m], entropy=ent[:m], top_idx=ti[:m, :topk],
                      top_logprob=tl[:m, :topk])
    lp, tl, ti, lse, ent = map(host, (lp, tl, ti, lse, ent))
    assert (lp[m] == 77).all() and (lp[:, ntok:] == 77).all() and (tl[m] == 77).all() and (tl[:, topk:] == 77).all()
    assert (ti[m] == -77).all() and (ti[:, topk:] == -77).all() and lse[m] == 77 and ent[m] == 77
    return lp[:m, :ntok], lse[:m], ent[:m], ti[:m, :topk], tl[:m, :topk]


def expect(x, tokens, topk, scale):
    z = x.cpu().double().numpy()
    order = np.argsort(-z, axis=1, kind="stable")[:, :topk]
    z = z * float(np.float32(scale))
    top = z.max(axis=1, keepdims=True)
    e = np.exp(z - top)
    s = e.sum(axis=1, keepdims=True)
    lse = top + np.log(s)
    with np.errstate(invalid="ignore"):
        d = np.where(e > 0, e * (z - top), 0).sum(axis=1) / s[:, 0]
    ent = np.log(s[:, 0]) - d
    tok = tokens.cpu().numpy()
    ok = (tok >= 0) & (tok < z.shape[1])
    # (z - max) - log s: beside a maximum of -3e38 even 64 bits would lose log s in z - lse
    logp = (z - top) - np.log(s)
    lp = np.where(ok, np.take_along_axis(logp, np.where(ok, tok, 0), 1), np.nan)
    big = np.where(np.isfinite(z), np.abs(z), 0).max(axis=1)
    return lp, lse[:, 0], ent, order, np.take_along_axis(logp, order, 1), d, big


def close(got, want, tol):
    got, want = got.astype(np.float64), np.asarray(want)
    assert np.array_equal(np.isnan(got), np.isnan(want)) and np.array_equal(np.isinf(got), np.isinf(want))
    fine = np.isfinite(want)
    assert (got[np.isinf(want)] == want[np.isinf(want)]).all()
    err = np.abs(got[fine] - want[fine])
    tol = np.broadcast_to(tol, want.shape)[fine]
    assert (err <= tol).all(), (float((err - tol).max()), float(err.max()))


def check(x, tokens, topk, scale=1.0):
    lp, lse, ent, ti, tl = ask(x, tokens, topk, scale)
    wlp, wlse, went, wti, wtl, d, big = expect(x, tokens, topk, scale)
    eps = 2.0 ** -20 + (140 + x.shape[1] / 256) * U
    assert np.array_equal(ti, wti)
    close(lse, wlse, eps + 8 * U * (big + np.abs(wlse)))
    for got, want in ((lp, wlp), (tl, wtl)):
        close(got, want, eps + 8 * U * (big[:, None] + np.where(np.isfinite(want), np.abs(want), 0)))
    close(ent, went, eps * (2 + 2 * np.abs(d)) + 8 * U * (1 + big))


def logits(seed, m, n, dtype, ld=None, offset=0, sigma=3.0):
    rng = np.random.default_rng(seed)
    ld = ld or n
    flat = torch.full((m * ld + offset,), float("nan"), dtype=DT[dtype], device="cuda")
    x = flat[offset:].view(m, ld)[:, :n]
    x.copy_(torch.from_numpy(rng.standard_normal((m, n)) * sigma))
    return x


def given(seed, m, n, count):
    return torch.from_numpy(np.random.default_rng(seed).integers(0, n, (m, count)).astype(np.int32)).cuda()


@pytest.mark.parametrize("m,n,dtype,topk,ntok,scale", [
    (1, 131072, "f32", 10, 1, 1.0), (16, 151667, "f32", 20, 2, 1.25), (306, 50021, "f16", 0, 1, 1.0),
    (64, 131072, "bf16", 5, 1, 0.7), (3, 262144, "f32", 32, 4, 1.0), (5, 1, "f32", 1, 1, 1.0), (5, 1, "bf16", 1, 3, 2.0),
    (4, 7, "f16", 7, 2, 1.0), (9, 33, "bf16", 32, 1, 1.0), (7, 512, "f32", 10, 2, 1.0), (2, 2049, "bf16", 32, 256, 1.0),
    (11, 16385, "f32", 3, 0, 1.0), (2, 32768 + 9, "bf16", 31, 1, 1.5), (3, 65536 * 4 + 1, "f16", 17, 1, 0.5),
    (2000, 40, "f32", 4, 1, 1.0), (2, 700001, "bf16", 32, 1, 1.0), (700, 9001, "bf16", 20, 1, 1.0),
    (640, 2048, "f32", 0, 1, 1.0), (620, 140000, "f16", 3, 1, 1.0),
])
def test_rows(m, n, dtype, topk, ntok, scale):
    check(logits(n, m, n, dtype), given(n + 1, m, n, ntok), topk, scale)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_rows_that_start_anywhere(dtype):
    for offset in range(1, 9):
        check(logits(offset, 5, 1003, dtype, ld=1003 + 7 + offset % 3, offset=offset), given(3, 5, 1003, 2), 12)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("n", [37, 5000, 100003])
def test_masked_rows(dtype, n):
    """-inf in most places, in all but one or two, and before the first 16 bytes end; padding tokens."""
    x = logits(n, 6, n, dtype)
    rng = np.random.default_rng(5)
    x[0, rng.random(n) < 0.95] = float("-inf")
    x[1] = float("-inf")
    x[1, n // 2] = 0.25
    x[2] = float("-inf")
    x[2, 0], x[2, n - 1] = -1.0, -1.0
    x[3, : n // 2] = float("-inf")
    x[4, n // 2:] = float("-inf")
    tokens = given(6, 6, n, 4)
    tokens[1, 0], tokens[2, 0], tokens[2, 1] = n // 2, 0, n - 1
    tokens[4, 1], tokens[4, 2], tokens[5, 0], tokens[5, 1] = -1, n, -(2 ** 31), 2 ** 31 - 1
    check(x, tokens, min(32, n))


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_masks_of_the_lowest_value(dtype):
    """finfo.min as the mask: beside ordinary logits it counts nothing, in every place it is an even row."""
    n = 3001
    low = torch.finfo(DT[dtype]).min
    x = logits(9, 3, n, dtype)
    x[0, 5:] = low
    x[1] = low
    x[2, ::2] = low
    lp, lse, ent, ti, tl = ask(x, given(1, 3, n, 2), 8)
    wlp, wlse, went, wti, wtl, d, big = expect(x, given(1, 3, n, 2), 8, 1.0)
    assert np.array_equal(ti, wti)
    eps = 2.0 ** -20 + (140 + n / 256) * U
    close(lse, wlse, eps + 8 * U * (np.abs(wlse) + np.where(np.abs(wlse) < 100, 20, 0)))
    close(ent, went, eps * (2 + 2 * np.abs(d)) + 8 * U * 21)
    close(lp[1], wlp[1], eps + 8 * U * 10)
    close(tl[1], wtl[1], eps + 8 * U * 10)
    fine = np.abs(wlp) < 1e3
    close(lp[fine], wlp[fine], eps + 8 * U * 40)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("n", [50, 70001])
def test_rows_without_a_defined_answer(dtype, n):
    inf, nan = float("inf"), float("nan")
    x = logits(3, 6, n, dtype)
    x[0] = -inf
    x[1, n - 2] = nan
    x[2, 7], x[2, n - 1] = inf, inf
    x[3] = inf
    x[4] = nan
    tokens = torch.tensor([[0, 7, n - 1]] * 6, dtype=torch.int32).cuda()
    lp, lse, ent, ti, tl = ask(x, tokens, 4)
    z = x.float().cpu().numpy()
    key = np.where(np.isnan(z), np.inf, z)  # a NaN ranks above +inf
    for r in range(6):
        want = sorted(range(n), key=lambda j: (0 if np.isnan(z[r, j]) else 1, -key[r, j], j))[:4]
        assert list(ti[r]) == want, r
    assert lse[0] == -inf and np.isnan(lp[0]).all() and np.isnan(ent[0]) and np.isnan(tl[0]).all()
    for r in (1, 4):
        assert np.isnan(lse[r]) and np.isnan(lp[r]).all() and np.isnan(ent[r]) and np.isnan(tl[r]).all()
    assert lse[2] == inf and lse[3] == inf and np.isnan(ent[[2, 3]]).all()
    assert lp[2, 0] == -inf and np.isnan(lp[2, 1]) and np.isnan(lp[2, 2]) and np.isnan(lp[3]).all()
    assert np.isnan(tl[2, :2]).all() and (tl[2, 2:] == -inf).all() and np.isnan(tl[3]).all()
    x5 = x[5:6].clone()
    check(x5, tokens[5:6], 4)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("n", [40, 3000, 140001])
def test_ties_go_to_the_lower_index(dtype, n):
    rng = np.random.default_rng(n)
    x = logits(1, 7, n, dtype)
    x[0] = 1.5
    x[1] = torch.from_numpy(rng.choice([-1.0, 0.0, 2.0], n)).cuda()
    x[2] = torch.from_numpy(np.where(rng.random(n) < 0.5, 0.0, -0.0)).cuda()
    x[3] = torch.arange(n, device="cuda") // 7 / 64.0          # rising: every step brings a new best
    x[4] = -(torch.arange(n, device="cuda") // 5) / 64.0
    x[5, : n // 2] = 9.0
    x[6] = 0.0
    x[6, n - 1] = 3.0
    lp, lse, ent, ti, tl = ask(x, given(2, 7, n, 1), 32)
    z = x.double().cpu().numpy()
    assert np.array_equal(ti, np.argsort(-z, axis=1, kind="stable")[:, :32])


def test_large_values_keep_their_differences():
    x = logits(4, 2, 1000, "f32") + 30000.0
    check(x.contiguous(), given(5, 2, 1000, 3), 10)
    check((x - 60000.0).contiguous(), given(5, 2, 1000, 3), 10, scale=0.01)


def test_huge_logits_do_not_overflow():
    x = torch.full((2, 300), -3.0e38, device="cuda")
    x[0, 5], x[0, 9] = 3.0e38, 3.0e38
    x[1, 4] = 3.3e38
    lp, lse, ent, ti, tl = ask(x, torch.tensor([[5, 0], [4, 0]], dtype=torch.int32).cuda(), 3)
    assert np.allclose(lp[:, 0], [-np.log(2.0), 0.0], rtol=0, atol=4 * U) and (lp[:, 1] == -np.inf).all()
    assert np.allclose(ent, [np.log(2.0), 0.0], rtol=0, atol=4 * U) and list(ti[0]) == [5, 9, 0]


def test_a_masked_token_of_the_lowest_value_keeps_its_log_probability():
    low = torch.finfo(torch.float32).min
    x = logits(14, 2, 2000, "f32")
    x[:, 100:] = low
    lp, lse, _, _, _ = ask(x, torch.tensor([[150, 3], [1999, 7]], dtype=torch.int32).cuda(), 2)
    assert np.allclose(lp[:, 0], low, rtol=8 * U, atol=0) and np.isfinite(lp).all() and np.isfinite(lse).all()


def test_a_row_has_the_same_bits_alone():
    x = logits(6, 9, 40004, "bf16")
    tokens = given(7, 9, 40004, 2)
    whole = ask(x, tokens, 6)
    for r in (0, 4, 8):
        for a, b in zip(ask(x[r:r + 1], tokens[r:r + 1], 6), whole):
            assert np.array_equal(a.view(np.uint32), b[r:r + 1].view(np.uint32))


def test_each_output_alone():
    x, tokens = logits(8, 4, 3000, "f32"), given(9, 4, 3000, 2)
    lp, lse, ent, ti, tl = ask(x, tokens, 5)
    one = torch.zeros(4, device="cuda")
    mr.token_logprobs(x, lse=one)
    assert np.array_equal(host(one), lse)
    mr.token_logprobs(x, entropy=one)
    assert np.array_equal(host(one), ent)
    two = torch.zeros((4, 2), device="cuda")
    mr.token_logprobs(x, tokens, two)
    assert np.array_equal(host(two), lp)
    idx = torch.zeros((4, 5), dtype=torch.int32, device="cuda")
    mr.token_logprobs(x, top_idx=idx)
    assert np.array_equal(host(idx), ti)


def test_captured_and_replayed():
    x, tokens = logits(10, 3, 33000, "f32"), given(11, 3, 33000, 1)
    lse, lp = torch.zeros(3, device="cuda"), torch.zeros((3, 1), device="cuda")
    idx = torch.zeros((3, 4), dtype=torch.int32, device="cuda")
    mr.token_logprobs(x, tokens, lp, lse=lse, top_idx=idx)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        mr.token_logprobs(x, tokens, lp, lse=lse, top_idx=idx)
    x.copy_(logits(12, 3, 33000, "f32"))
    graph.replay()
    wlp, wlse, _, wti, _, _, big = expect(x, tokens, 4, 1.0)
    assert np.array_equal(host(idx), wti)
    close(host(lse), wlse, 2.0 ** -20 + 300 * U + 8 * U * (big + np.abs(wlse)))
