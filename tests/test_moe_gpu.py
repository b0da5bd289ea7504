"""moe_window_bf16 / moe_window_w4 on the GPU against the layer in 64 bits.

Tolerance.  u = 2^-24.  A sum of k products on the tensor core loses less than
8 * 17 * 2^-23 of its absolute sum inside a block of 128, and one u for each
block or group and each part of k after it: tau(k) = 8 * 17 * 2u +
(4 * ceil(k / 128) + 8) u.  Let Sg, Su be the absolute sums behind the gate and
up values.  |silu'| <= 1.1, so the activation is off by at most
dh = tau (1.1 Sg |up| + |silu(gate)| Su) + 16 u |h| (expf within 2 ulp, and the
few operations around it), its products being second order.  The down
projection carries |Wd| dh and adds tau(inter) |Wd| |h| with 16 u for the
pieces; the weighted sum adds (topk + 8) u of its own absolute terms (a softmax's
weights are off by no more than 8 u plus topk u).  A bf16 result adds its
rounding, half a step: a value in [1, 2) has steps of 2^-7 (7 stored bits), so at
most 2^-8 of the value and of its error.
"""
import numpy as np
import pytest

import w4_util
from gpu_util import host, need_gpu, padded, torch

import verify_weight_streaming_b200 as mr

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    need_gpu()
    yield
    assert mr.mr_poll_errors() == 0


class Experts:
    """Seeded weights of `count` experts, their float64 values and the call on them."""

    def __init__(self, seed, count, hidden, inter, group=0, zeros=False, pad=0):
        self.count, self.hidden, self.inter, self.group = count, hidden, inter, group
        if group:
            up = w4_util.weight(seed, (count,), 2 * inter, hidden, group, zeros)
            down = w4_util.weight(seed + 1, (count,), hidden, inter, group, zeros)
            self.up64, self.down64 = w4_util.dense64(up), w4_util.dense64(down)
            (self.up, self.fmt), (self.down, _) = w4_util.pack(mr, up, paired=True), w4_util.pack(mr, down)
        else:
            rng = np.random.default_rng(seed)
            def one(rows, cols):
                buf = torch.full((count, rows + pad, cols + pad), float("nan"), dtype=torch.bfloat16)
                buf[:, :rows, :cols] = torch.from_numpy(rng.standard_normal((count, rows, cols)) / np.sqrt(cols))
                return buf.cuda()[:, :rows, :cols]
            self.up, self.down = one(2 * inter, hidden), one(hidden, inter)
            self.up64, self.down64 = self.up.cpu().double().numpy(), self.down.cpu().double().numpy()

    def __call__(self, x, ids, wts, out=torch.float32, base=0, flags=0, workspace=None):
        m, topk = ids.shape
        if workspace is None:
            size = mr.moe_window_workspace_bytes(m, topk, self.hidden, self.inter)
            workspace = torch.full((size,), 0xFF, dtype=torch.uint8, device="cuda")  # NaN everywhere
        buf, _ = padded(m + 1, self.hidden + 3, self.hidden + 3, out, 77.0)
        y = buf[:m, :self.hidden]
        if self.group:
            mr.moe_window_w4(x, ids, wts, self.up, self.down, y, workspace, self.count, self.inter, self.fmt,
                             expert_base=base, flags=flags)
        else:
            mr.moe_window_bf16(x, ids, wts, self.up, self.down, y, workspace, expert_base=base, flags=flags)
        h = host(buf.float())
        assert (h[m] == 77.0).all() and (h[:, self.hidden:] == 77.0).all()
        return h[:m, :self.hidden]

    def expect(self, x, ids, wts, base=0, flags=0):
        """(y, bound on its error) in 64 bits."""
        x, ids, wts = x.cpu().double().numpy(), ids.cpu().numpy(), wts.cpu().double().numpy()
        y, tol = np.zeros((len(x), self.hidden)), np.zeros((len(x), self.hidden))
        tau = lambda k: 8 * 17 * 2 * U + (4 * -(-k // 128) + 8) * U  # noqa: E731
        for t in range(len(x)):
            w = wts[t].copy()
            if flags & mr.MR_MOE_SOFTMAX:
                live = ids[t] >= 0
                w = np.where(live, np.exp(w - (w[live].max() if live.any() else 0)), 0)
                w = w / (w.sum() or 1)
            for s, e in enumerate(ids[t] - base):
                if ids[t, s] < 0 or not 0 <= e < self.count:
                    continue
                up, down = self.up64[e], self.down64[e]
                pre, absum = up @ x[t], np.abs(up) @ np.abs(x[t])
                gate, lift = pre[:self.inter], pre[self.inter:]
                act = gate / (1 + np.exp(-gate))
                h = act * lift
                dh = tau(self.hidden) * (1.1 * absum[:self.inter] * np.abs(lift) + np.abs(act) * absum[self.inter:])
                dh = dh + 16 * U * np.abs(h)
                one, size = down @ h, np.abs(down) @ np.abs(h)
                y[t] += w[s] * one
                tol[t] += abs(w[s]) * (np.abs(down) @ dh + (tau(self.inter) + 16 * U + (2 * len(ids[t]) + 16) * U) * size)
        return y, tol


def rows(seed, m, hidden, ld=None):
    buf = torch.full((m, ld or hidden), float("nan"), dtype=torch.bfloat16)
    buf[:, :hidden] = torch.from_numpy(np.random.default_rng(seed).standard_normal((m, hidden)))
    return buf.cuda()[:, :hidden]


def choices(seed, m, topk, total):
    rng = np.random.default_rng(seed)
    ids = np.stack([rng.permutation(total)[:topk] for _ in range(m)]).astype(np.int32)
    return torch.from_numpy(ids).cuda(), torch.from_numpy(rng.standard_normal((m, topk)).astype(np.float32)).cuda()


def check(got, want, tol, out=torch.float32):
    if out == torch.bfloat16:
        tol = tol + (np.abs(want) + tol) * 2.0 ** -8
    err = np.abs(got - want)
    assert (err <= tol).all(), float((err - tol).max())


@pytest.mark.parametrize("m,topk,count,hidden,inter,group,zeros,out", [
    (1, 10, 32, 2560, 640, 0, False, "f32"), (16, 10, 32, 2560, 640, 0, False, "bf16"),
    (8, 10, 32, 2560, 640, 128, False, "f32"), (5, 4, 16, 1024, 512, 32, True, "bf16"),
    (16, 2, 8, 896, 256, 64, True, "f32"), (16, 4, 4, 512, 128, 0, False, "f32"),
    (1, 1, 1, 8, 8, 0, False, "f32"), (2, 3, 5, 24, 40, 0, False, "bf16"), (3, 2, 4, 136, 264, 0, False, "f32"),
    (1, 1, 2, 32, 32, 32, True, "f32"), (16, 32, 40, 64, 96, 32, False, "f32"), (7, 6, 9, 160, 64, 32, True, "f32"),
    (12, 1, 1, 256, 2048, 0, False, "f32"), (9, 2, 3, 4096, 128, 0, False, "f32"), (16, 3, 3, 128, 2048, 128, True, "f32"),
    (16, 8, 1500, 32, 32, 32, True, "f32"), (16, 32, 1100, 64, 40, 0, False, "f32"), (10, 2, 2, 264, 72, 0, False, "bf16"),
])
@pytest.mark.parametrize("softmax", [False, True])
def test_layer(m, topk, count, hidden, inter, group, zeros, out, softmax):
    ex = Experts(hidden + inter, count, hidden, inter, group, zeros)
    x, (ids, wts) = rows(1, m, hidden), choices(2, m, topk, count)
    flags = mr.MR_MOE_SOFTMAX if softmax else 0
    dtype = torch.float32 if out == "f32" else torch.bfloat16
    want, tol = ex.expect(x, ids, wts, flags=flags)
    check(ex(x, ids, wts, dtype, flags=flags), want, tol, dtype)


@pytest.mark.parametrize("group", [0, 64])
def test_strides(group):
    ex = Experts(11, 6, 256, 128, group, pad=0 if group else 8)
    x = rows(12, 4, 256, 280)
    ids, wts = choices(13, 4, 6, 6)
    wide_i, wide_w = torch.full((4, 9), -5, dtype=torch.int32, device="cuda"), torch.full((4, 9), float("nan"), device="cuda")
    wide_i[:, :6], wide_w[:, :6] = ids, wts
    want, tol = ex.expect(x, ids, wts)
    check(ex(x, wide_i[:, :6], wide_w[:, :6]), want, tol)


@pytest.mark.parametrize("group", [0, 32])
@pytest.mark.parametrize("softmax", [False, True])
def test_empty_foreign_and_repeated_entries(group, softmax):
    """-1, experts of another device, ids past every expert, an expert twice in a row, a row with nothing."""
    ex = Experts(21, 5, 256, 96, group)
    ids = torch.tensor([[7, -1, 8, 11], [-1, -1, -1, -1], [9, 9, 9, 9], [0, 6, 12, 2 ** 31 - 1], [-(2 ** 31), 11, 7, 7],
                        [100, 3, -7, 8]], dtype=torch.int32).cuda()
    wts = choices(22, 6, 4, 8)[1]
    wts[ids < 0] = float("nan")
    x = rows(23, 6, 256)
    flags = mr.MR_MOE_SOFTMAX if softmax else 0
    want, tol = ex.expect(x, ids, wts, base=7, flags=flags)
    got = ex(x, ids, wts, base=7, flags=flags)
    check(got, want, tol)
    assert (got[[1, 3]] == 0).all()


@pytest.mark.parametrize("m", [1, 16])
def test_every_row_and_choice_on_one_expert(m):
    """More than 8 rows of one expert, and one expert 32 times in a row."""
    for group in (0, 128):
        ex = Experts(31, 3, 128, 128, group)
        ids = torch.full((m, 32), 2, dtype=torch.int32, device="cuda")
        wts, x = choices(32, m, 32, 32)[1], rows(33, m, 128)
        want, tol = ex.expect(x, ids, wts)
        check(ex(x, ids, wts), want, tol)


@pytest.mark.parametrize("group", [0, 128])
def test_rows_have_the_same_bits_alone_and_together(group):
    ex = Experts(41, 6, 640, 384, group)
    x, (ids, wts) = rows(42, 16, 640), choices(43, 16, 3, 6)
    whole = ex(x, ids, wts, flags=mr.MR_MOE_SOFTMAX).view(np.uint32)
    for m in (1, 2, 5, 9, 15):
        assert np.array_equal(ex(x[:m], ids[:m], wts[:m], flags=mr.MR_MOE_SOFTMAX).view(np.uint32), whole[:m])
    order = torch.from_numpy(np.random.default_rng(4).permutation(16)).cuda()
    got = ex(x[order].contiguous(), ids[order].contiguous(), wts[order].contiguous(), flags=mr.MR_MOE_SOFTMAX)
    assert np.array_equal(got.view(np.uint32), whole[order.cpu().numpy()])


@pytest.mark.parametrize("group", [0, 64])
def test_few_and_many_experts_give_a_row_the_same_bits(group):
    """One row's experts are summed by four warps a tile, 16 rows' many by one."""
    ex = Experts(45, 200, 320, 512, group)
    x, (ids, wts) = rows(46, 16, 320), choices(47, 16, 8, 200)
    whole = ex(x, ids, wts).view(np.uint32)
    for r in (0, 7, 15):
        assert np.array_equal(ex(x[r:r + 1], ids[r:r + 1], wts[r:r + 1]).view(np.uint32), whole[r:r + 1])
    want, tol = ex.expect(x, ids, wts)
    check(whole.view(np.float32), want, tol)


@pytest.mark.parametrize("group", [0, 128])
def test_shards_add_up_to_the_whole(group):
    """Experts split over three devices' calls: the parts' sum is the whole, softmax over all entries in each."""
    ex = Experts(51, 9, 256, 128, group)
    x, (ids, wts) = rows(52, 4, 256), choices(53, 4, 5, 9)
    want, tol = ex.expect(x, ids, wts, flags=mr.MR_MOE_SOFTMAX)
    total = 0.0
    for at in range(0, 9, 3):
        part = object.__new__(Experts)
        part.__dict__.update(ex.__dict__, count=3)
        if group:
            nu, nd = ex.up.numel() // 9, ex.down.numel() // 9
            part.up, part.down = ex.up[at * nu:(at + 3) * nu], ex.down[at * nd:(at + 3) * nd]
        else:
            part.up, part.down = ex.up[at:at + 3], ex.down[at:at + 3]
        total = total + part(x, ids, wts, base=at, flags=mr.MR_MOE_SOFTMAX).astype(np.float64)
    check(total, want, tol)


def test_not_finite_activations_stay_in_their_row():
    for group in (0, 64):
        ex = Experts(61, 4, 128, 64, group)
        x, (ids, wts) = rows(62, 6, 128), choices(63, 6, 2, 4)
        x[1, 5], x[4, 0] = float("nan"), float("inf")
        y = ex(x, ids, wts)
        fine = [0, 2, 3, 5]
        assert np.isnan(y[1]).all() and not np.isfinite(y[4]).any()
        want, tol = ex.expect(x[fine], ids[fine], wts[fine])
        check(y[fine], want, tol)


@pytest.mark.parametrize("group", [0, 32])
def test_captured_calls_share_a_workspace(group):
    """Two layers in one graph on one workspace, replayed with new inputs, no host work between."""
    ex = Experts(71, 8, 256, 128, group)
    x, (ids, wts) = rows(72, 3, 256), choices(73, 3, 4, 8)
    size = mr.moe_window_workspace_bytes(3, 4, 256, 128)
    ws = torch.full((size,), 0xFF, dtype=torch.uint8, device="cuda")
    y1, y2 = (torch.zeros((3, 256), dtype=torch.bfloat16, device="cuda") for _ in range(2))

    def call(a, b):
        if group:
            mr.moe_window_w4(a, ids, wts, ex.up, ex.down, b, ws, 8, 128, ex.fmt, flags=mr.MR_MOE_SOFTMAX)
        else:
            mr.moe_window_bf16(a, ids, wts, ex.up, ex.down, b, ws, flags=mr.MR_MOE_SOFTMAX)

    call(x, y1)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(x, y1)
        call(y1, y2)
    for seed in (74, 75):
        x.copy_(rows(seed, 3, 256))
        ids.copy_(choices(seed, 3, 4, 8)[0])
        graph.replay()
        torch.cuda.synchronize()
        want, tol = ex.expect(x, ids, wts, flags=mr.MR_MOE_SOFTMAX)
        check(host(y1.float()), want, tol, torch.bfloat16)
        want, tol = ex.expect(y1, ids, wts, flags=mr.MR_MOE_SOFTMAX)
        check(host(y2.float()), want, tol, torch.bfloat16)


def test_two_streams_at_once():
    ex = Experts(81, 16, 512, 256)
    data = [(rows(82 + i, 8, 512), *choices(92 + i, 8, 4, 16)) for i in range(2)]
    torch.cuda.synchronize()
    size = mr.moe_window_workspace_bytes(8, 4, 512, 256)
    streams = [torch.cuda.Stream() for _ in range(2)]
    ws = [torch.zeros(size, dtype=torch.uint8, device="cuda") for _ in range(2)]
    ys = [torch.zeros((8, 512), device="cuda") for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(5):
        for i, st in enumerate(streams):
            x, ids, wts = data[i]
            mr.moe_window_bf16(x, ids, wts, ex.up, ex.down, ys[i], ws[i], stream=st)
    torch.cuda.synchronize()
    for i in range(2):
        want, tol = ex.expect(*data[i])
        check(host(ys[i]), want, tol)
