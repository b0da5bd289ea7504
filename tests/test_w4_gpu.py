"""mrgemv_w4 and w4_pack on the GPU against the product in 64 bits.

Tolerance.  The values (q - z) are exact in 16 bits and so is every product in
fp32.  A group's sum is at most 8 matrix instructions of 16 products and an
accumulator each; every one of those 17 addends may lose less than one unit
of 2^-23 of the largest when it is aligned, so a group is within
8 * 17 * 2^-23 of its sum of absolute products.  The scaled group sums are added
one rounding (2^-24) each, then the four quarters of k: at most
(groups + 4) * 2^-24 more.
"""
import numpy as np
import pytest

import w4_util
from gpu_util import host, need_gpu, padded, torch

import verify_weight_streaming_b200 as mr

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    need_gpu()
    yield
    assert mr.mr_poll_errors() == 0


def acts(seed, m, k, dtype="bf16"):
    rng = np.random.default_rng(seed)
    return torch.from_numpy(rng.standard_normal((m, k))).to(w4_util.DTYPES[dtype]).cuda()


def product(a, packed, fmt, n, flags=0):
    """C with canaries around it, checked."""
    m = a.shape[0]
    buf, _ = padded(m + 1, n + 5, n + 5, torch.float32, 77.0)
    mr.mrgemv_w4(a, packed, buf[:m, :n], fmt, flags=flags)
    h = host(buf)
    assert (h[m] == 77.0).all() and (h[:, n:] == 77.0).all()
    return h[:m, :n]


def check(c, a, w, group):
    a64, w64 = a.cpu().double().numpy(), w4_util.dense64(w)
    k = a64.shape[1]
    tol = (8 * 17 * 2.0 ** -23 + (k // group + 4) * 2.0 ** -24) * (np.abs(a64) @ np.abs(w64).T)
    err = np.abs(c - a64 @ w64.T)
    assert (err <= tol).all(), float((err - tol).max())


@pytest.mark.parametrize("m,n,k,group,zeros,act,scales", [
    (1, 512, 2560, 128, False, "bf16", "bf16"), (8, 4864, 896, 64, True, "bf16", "f16"),
    (16, 6144, 2560, 32, True, "f16", "f16"), (9, 1000, 4096, 128, True, "f16", "bf16"),
    (1, 1, 32, 32, False, "bf16", "bf16"), (16, 15, 32, 32, True, "f16", "f16"), (3, 17, 160, 32, True, "bf16", "bf16"),
    (7, 33, 64, 64, False, "f16", "bf16"), (5, 600, 192, 64, True, "bf16", "f16"), (2, 16, 128, 128, False, "bf16", "f16"),
    (16, 5000, 384, 128, False, "f16", "f16"), (4, 40000, 256, 128, False, "bf16", "bf16"),
    (1, 128, 11264, 128, False, "bf16", "bf16"), (3, 80000, 128, 32, True, "bf16", "f16"),
    (16, 90001, 160, 32, False, "f16", "bf16"),
])
def test_product(m, n, k, group, zeros, act, scales):
    w = w4_util.weight(n * 7 + k, (), n, k, group, zeros, scales)
    packed, fmt = w4_util.pack(mr, w)
    a = acts(m, m, k, act)
    check(product(a, packed, fmt, n), a, w, group)


@pytest.mark.parametrize("group,zeros", [(32, True), (64, False), (128, True)])
def test_small_integers_are_exact(group, zeros):
    """Integer activations and power-of-two scales: every partial sum is exact, so any misplaced value shows."""
    m, n, k = 11, 70, 5 * 128 + group
    w = w4_util.weight(5, (), n, k, group, zeros, "f16", pow2=True)
    packed, fmt = w4_util.pack(mr, w)
    a = torch.from_numpy(np.random.default_rng(6).integers(-3, 4, (m, k)).astype(np.float32)).to(torch.bfloat16).cuda()
    want = a.cpu().double().numpy() @ w4_util.dense64(w).T
    assert np.array_equal(product(a, packed, fmt, n), want)


@pytest.mark.parametrize("act,group", [("bf16", 128), ("f16", 32)])
def test_rows_have_the_same_bits_for_every_m(act, group):
    n, k = 777, 2560
    w = w4_util.weight(8, (), n, k, group, True)
    packed, fmt = w4_util.pack(mr, w)
    a = acts(9, 16, k, act)
    whole = product(a, packed, fmt, n).view(np.uint32)
    for m in range(1, 16):
        assert np.array_equal(product(a[:m], packed, fmt, n).view(np.uint32), whole[:m]), m
    order = np.random.default_rng(3).permutation(16)
    assert np.array_equal(product(a[order], packed, fmt, n).view(np.uint32), whole[order])
    assert np.array_equal(product(a[5:6], packed, fmt, n).view(np.uint32), whole[5:6])


@pytest.mark.parametrize("m,k,group", [(2, 640, 128), (11, 224, 32)])
def test_columns_have_the_same_bits_in_a_wide_and_a_narrow_weight(m, k, group):
    """A wide weight's tiles go to one warp each, a narrow one's to four."""
    n = 96000
    w = w4_util.weight(61, (), n, k, group, True)
    packed, fmt = w4_util.pack(mr, w)
    a = acts(62, m, k)
    wide = product(a, packed, fmt, n).view(np.uint32)
    for first, rows in ((0, 512), (48000, 4096), (95984, 16)):
        at = mr.w4_packed_bytes(first, k, fmt) if first else 0
        part = packed[at:at + mr.w4_packed_bytes(rows, k, fmt)]
        assert np.array_equal(product(a, part, fmt, rows).view(np.uint32), wide[:, first:first + rows])


def test_strides_and_programmatic_launch():
    m, n, k = 6, 500, 640
    w = w4_util.weight(21, (), n, k, 128, False)
    packed, fmt = w4_util.pack(mr, w)
    buf, a = padded(m, k, k + 24, torch.bfloat16, float("nan"))
    a.copy_(acts(22, m, k))
    got = product(a, packed, fmt, n)
    check(got, a, w, 128)
    assert np.array_equal(got.view(np.uint32), product(a.contiguous(), packed, fmt, n, mr.MR_GEMV_PDL).view(np.uint32))


def test_infinities_and_nan_stay_in_their_row_and_column():
    m, n, k = 9, 40, 256
    q, s, z = w4_util.weight(31, (), n, k, 128, True)
    s[7, 1] = float("nan")
    packed, fmt = w4_util.pack(mr, (q, s, z))
    a = acts(32, m, k)
    a[3, 100] = float("nan")
    a[8, 0] = float("inf")
    c = product(a, packed, fmt, n)
    fine = np.ones((m, n), bool)
    fine[[3, 8]] = False
    fine[:, 7] = False
    assert np.isfinite(c[fine]).all() and np.isnan(c[3]).all() and np.isnan(c[:, 7]).all()
    assert not np.isfinite(c[8]).any()


def test_captured_and_replayed_with_new_inputs():
    m, n, k = 4, 900, 512
    w = w4_util.weight(41, (), n, k, 64, True)
    packed, fmt = w4_util.pack(mr, w)
    a, c = acts(42, m, k), torch.zeros((m, n), dtype=torch.float32, device="cuda")
    mr.mrgemv_w4(a, packed, c, fmt)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        mr.mrgemv_w4(a, packed, c, fmt, flags=mr.MR_GEMV_PDL)
        mr.mrgemv_w4(a, packed, c, fmt, flags=mr.MR_GEMV_PDL)
    a.copy_(acts(43, m, k))
    c.zero_()
    graph.replay()
    check(host(c), a, w, 64)


def test_pack_of_several_weights_and_of_paired_halves():
    """Three weights packed at once are the three packed alone; paired halves are the rows put in tile order."""
    w = w4_util.weight(51, (3,), 44, 96, 32, True)
    packed, fmt = w4_util.pack(mr, w)
    each = [w4_util.pack(mr, tuple(t[i] for t in w))[0] for i in range(3)]
    assert torch.equal(packed, torch.cat(each))
    paired, _ = w4_util.pack(mr, w, paired=True)
    order = [r for tile in range(3) for r in [*range(8 * tile, 8 * tile + 8), *range(22 + 8 * tile, 30 + 8 * tile)]]
    rows = torch.tensor([r if (r < 22 if i % 16 < 8 else r < 44) else -1 for i, r in enumerate(order)])
    fill = (torch.full_like(w[0][:, :1], 0x88), torch.zeros_like(w[1][:, :1]), torch.full_like(w[2][:, :1], 8))
    at = torch.where(rows < 0, torch.full_like(rows, 44), rows)
    same = tuple(torch.cat((t, f), dim=1)[:, at] for t, f in zip(w, fill))
    assert torch.equal(paired, w4_util.pack(mr, same)[0])
