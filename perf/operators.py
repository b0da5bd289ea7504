"""Cases that time the verify window's model operators, in plain torch and through the library.

  w4        mrgemv_w4: multi-row product with a 4-bit weight and group scales
  moe       moe_window_bf16 / moe_window_w4: the routed experts of a few tokens
  logprobs  token_logprobs: log probabilities of given tokens, entropy, top alternatives
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
FLOATS = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def listed():
    return [
        # one decoded token against a router-sized weight: the call's latency is all there is
        dict(name="w4 512x2560 m1", op="w4", m=1, n=512, k=2560, group=128, zeros=False, act="bf16", scales="bf16"),
        # a verify window of 8 drafts against an FFN weight with zero points
        dict(name="w4 4864x896 m8", op="w4", m=8, n=4864, k=896, group=64, zeros=True, act="bf16", scales="f16"),
        # the widest window against a wide projection, small groups
        dict(name="w4 6144x2560 m16", op="w4", m=16, n=6144, k=2560, group=32, zeros=True, act="f16", scales="f16"),
        # the output head over a large vocabulary, a window of 4
        dict(name="w4 131072x2560 m4", op="w4", m=4, n=131072, k=2560, group=128, zeros=False, act="bf16",
             scales="bf16"),
        # one decoded token through the routed experts
        dict(name="moe bf16 m1", op="moe", m=1, topk=10, total=512, experts=512, base=0, hidden=2560, inter=640,
             group=0, zeros=False, softmax=True, out="f32"),
        # the widest window: 160 choices among 512 experts
        dict(name="moe bf16 m16", op="moe", m=16, topk=10, total=512, experts=512, base=0, hidden=2560, inter=640,
             group=0, zeros=False, softmax=True, out="bf16"),
        # a window of 8 with experts held in 4 bits
        dict(name="moe w4 m8", op="moe", m=8, topk=10, total=512, experts=512, base=0, hidden=2560, inter=640,
             group=128, zeros=False, softmax=True, out="f32"),
        # a device that holds 200 of the 512 experts: most choices are another device's
        dict(name="moe w4 shard m5", op="moe", m=5, topk=10, total=512, experts=200, base=131, hidden=2560, inter=640,
             group=32, zeros=True, softmax=False, out="bf16"),
        # one sampled token with its ten best alternatives
        dict(name="logprobs 1x131072", op="logprobs", m=1, n=131072, tokens=1, top=10, dtype="f32", scale=1.0,
             masked=0.0),
        # a verify window over a vocabulary of odd size, grammar-masked, with a temperature
        dict(name="logprobs 16x151667", op="logprobs", m=16, n=151667, tokens=2, top=20, dtype="f32", scale=1.25,
             masked=0.3),
        # scoring a prompt chunk: rows of odd length that start anywhere
        dict(name="logprobs 306x50021 f16", op="logprobs", m=306, n=50021, tokens=1, top=0, dtype="f16", scale=1.0,
             masked=0.0),
        # scoring the longest prompt chunk
        dict(name="logprobs 2048x131072 bf16", op="logprobs", m=2048, n=131072, tokens=1, top=5, dtype="bf16",
             scale=1.0, masked=0.0),
    ]


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(("w4", "moe", "logprobs"))
    if op == "w4":
        group = rng.choice((32, 64, 128))
        k = max(1, _log(rng, 128, 4096) // group) * group
        n = min(_log(rng, 64, 131072), 131072 * 2560 // k)
        return dict(op=op, m=rng.randint(1, 16), n=n, k=k, group=group, zeros=rng.random() < 0.5,
                    act=rng.choice(("bf16", "f16")), scales=rng.choice(("bf16", "f16")))
    if op == "moe":
        group = rng.choice((0, 32, 64, 128))
        step = group or 8
        hidden = max(1, _log(rng, 256, 4096) // step) * step
        inter = max(1, _log(rng, 128, 1024) // step) * step
        total = min(_log(rng, 8, 512), 512 * 2560 * 640 // (hidden * inter))
        experts = total if rng.random() < 0.7 else rng.randint(1, total)
        return dict(op=op, m=rng.randint(1, 16), topk=rng.randint(1, min(10, total)), total=total, experts=experts,
                    base=rng.randint(0, total - experts), hidden=hidden, inter=inter, group=group,
                    zeros=bool(group) and rng.random() < 0.5, softmax=rng.random() < 0.5,
                    out=rng.choice(("f32", "bf16")))
    n = _log(rng, 512, 262144)
    return dict(op=op, m=_log(rng, 1, max(1, min(2048, 2048 * 131072 // n))), n=n, tokens=rng.randint(1, 4),
                top=rng.randint(0, 32), dtype=rng.choice(("f32", "bf16", "f16")) if n <= 131072 else "bf16",
                scale=rng.choice((1.0, 1.25, 0.7)), masked=rng.choice((0.0, 0.3)))


# ---- inputs ---------------------------------------------------------------


def _nibbles(gen, shape):
    """4-bit values of a quantised normal weight, two to a byte (the even column in the low half)."""
    out = torch.empty(shape, dtype=torch.uint8, device=DEV)
    flat = out.view(-1)
    for at in range(0, flat.numel(), 1 << 27):
        part = flat[at:at + (1 << 27)]
        half = [torch.randn(part.shape, generator=gen, device=DEV, dtype=torch.float16).mul_(2.3).add_(7.7).round_()
                .clamp_(0, 15).to(torch.uint8) for _ in range(2)]
        part.copy_(half[0] | (half[1] << 4))
    return out


def _scales(gen, shape, k, dtype):
    return (torch.rand(shape, generator=gen, device=DEV) * 0.2 + 0.3).div_(math.sqrt(k)).to(dtype)


def _zeros(gen, shape):
    return torch.randint(5, 11, shape, generator=gen, device=DEV, dtype=torch.uint8)


def _weight4(gen, lead, n, k, case, dtype):
    g = k // case["group"]
    return (_nibbles(gen, (*lead, n, k // 2)), _scales(gen, (*lead, n, g), k, dtype),
            _zeros(gen, (*lead, n, g)) if case["zeros"] else None)


def _inputs(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    if case["op"] == "w4":
        a = torch.randn((case["m"], case["k"]), generator=gen, device=DEV).to(FLOATS[case["act"]])
        return dict(a=a, w=_weight4(gen, (), case["n"], case["k"], case, FLOATS[case["scales"]]))
    if case["op"] == "moe":
        m, hidden, inter, experts = case["m"], case["hidden"], case["inter"], case["experts"]
        x = torch.randn((m, hidden), generator=gen, device=DEV).to(torch.bfloat16)
        logits = torch.randn((m, case["total"]), generator=gen, device=DEV)
        val, ids = torch.topk(logits, case["topk"], dim=1)
        if not case["softmax"]:
            val = torch.rand(val.shape, generator=gen, device=DEV)
        state = dict(x=x, ids=ids.to(torch.int32), val=val.contiguous())
        if case["group"]:
            state["up"] = _weight4(gen, (experts,), 2 * inter, hidden, case, torch.bfloat16)
            state["down"] = _weight4(gen, (experts,), hidden, inter, case, torch.bfloat16)
        else:
            state["up"] = torch.empty((experts, 2 * inter, hidden), dtype=torch.bfloat16, device=DEV)
            state["up"].normal_(0, 1 / math.sqrt(hidden), generator=gen)
            state["down"] = torch.empty((experts, hidden, inter), dtype=torch.bfloat16, device=DEV)
            state["down"].normal_(0, 1 / math.sqrt(inter), generator=gen)
        return state
    m, n = case["m"], case["n"]
    logits = torch.empty((m, n), dtype=FLOATS[case["dtype"]], device=DEV).normal_(0, 3, generator=gen)
    tokens = torch.randint(0, n, (m, case["tokens"]), generator=gen, device=DEV)
    if case["masked"]:
        logits.masked_fill_(torch.rand((m, n), generator=gen, device=DEV) < case["masked"], float("-inf"))
    logits.scatter_(1, tokens, torch.full((m, case["tokens"]), 11.0, dtype=logits.dtype, device=DEV))
    return dict(logits=logits, tokens=tokens.to(torch.int32))


def prepare(case, seed):
    state = dict(_inputs(case, seed), case=case)
    if own:
        import verify_weight_streaming_b200 as mr
        state["mr"] = mr

        def pack(w, paired):
            q, scales, zeros = w
            fmt = mr.w4_format(case["group"], zeros is not None, scales.dtype)
            count = q.shape[0] if q.dim() == 3 else 1
            size = count * mr.w4_packed_bytes(q.shape[-2], 2 * q.shape[-1], fmt, paired)
            packed = torch.empty(size, dtype=torch.uint8, device=DEV)
            mr.w4_pack(q, scales, zeros, packed, paired=paired)
            return packed, fmt

        if case["op"] == "w4":
            state["packed"], state["fmt"] = pack(state["w"], False)
            state["c"] = torch.empty((case["m"], case["n"]), dtype=torch.float32, device=DEV)
        elif case["op"] == "moe":
            if case["group"]:
                state["packed_up"], state["fmt"] = pack(state["up"], True)
                state["packed_down"], _ = pack(state["down"], False)
            state["y"] = torch.empty((case["m"], case["hidden"]), dtype=FLOATS[case["out"]], device=DEV)
            size = mr.moe_window_workspace_bytes(case["m"], case["topk"], case["hidden"], case["inter"])
            state["workspace"] = torch.zeros(size, dtype=torch.uint8, device=DEV)
        else:
            m, top = case["m"], case["top"]
            state["logprob"] = torch.empty((m, case["tokens"]), dtype=torch.float32, device=DEV)
            state["lse"] = torch.empty(m, dtype=torch.float32, device=DEV)
            state["entropy"] = torch.empty(m, dtype=torch.float32, device=DEV)
            state["top_idx"] = torch.empty((m, top), dtype=torch.int32, device=DEV)
            state["top_logprob"] = torch.empty((m, top), dtype=torch.float32, device=DEV)
    return state


# ---- plain forms ----------------------------------------------------------


def _dequant(w):
    """(q - z) * s in 32 bits, for [..., n, k/2] bytes, [..., n, groups] scales and zero points."""
    q, scales, zeros = w
    v = torch.stack((q & 15, q >> 4), dim=-1).reshape(*scales.shape, -1).float()
    z = 8.0 if zeros is None else zeros.float().unsqueeze(-1)
    return ((v - z) * scales.float().unsqueeze(-1)).flatten(-2)


def _plain_w4(state):
    return state["a"].float() @ _dequant(state["w"]).t()


def _plain_moe(state):
    case, x, ids = state["case"], state["x"], state["ids"].long()
    m, topk = ids.shape
    local = ids - case["base"]
    held = (ids >= 0) & (local >= 0) & (local < case["experts"])
    at = torch.where(held, local, torch.zeros_like(local)).reshape(-1)
    if case["group"]:
        up = _dequant([None if t is None else t[at] for t in state["up"]])
        down = _dequant([None if t is None else t[at] for t in state["down"]])
    else:
        up, down = state["up"][at].float(), state["down"][at].float()
    rows = x.float().unsqueeze(1).expand(m, topk, -1).reshape(m * topk, -1, 1)
    gate, lift = (up @ rows).squeeze(-1).chunk(2, dim=1)
    h = gate / (1 + torch.exp(-gate)) * lift
    parts = (down @ h.unsqueeze(-1)).reshape(m, topk, -1)
    share = state["val"]
    if case["softmax"]:
        e = torch.exp(share - share.amax(dim=1, keepdim=True))
        share = e / e.sum(dim=1, keepdim=True)
    share = torch.where(held, share, torch.zeros_like(share))
    return (parts * share.unsqueeze(-1)).sum(dim=1).to(FLOATS[case["out"]])


def _plain_logprobs(state):
    case, logits = state["case"], state["logits"]
    z = logits.float() * case["scale"]
    top_z = z.amax(dim=1, keepdim=True)
    e = torch.exp(z - top_z)
    total = e.sum(dim=1, keepdim=True)
    lse = top_z + torch.log(total)
    logprob = torch.gather(z, 1, state["tokens"].long()) - lse
    mean = torch.where(e > 0, (z - top_z) * e, torch.zeros_like(z)).sum(dim=1) / total.squeeze(1)
    entropy = torch.log(total.squeeze(1)) - mean
    # unique integer keys: the value's order in the high half, the lower index above in the low half
    top = case["top"]
    if top:
        bits = (logits.float() + 0.0).view(torch.int32).long()
        order = torch.where(bits < 0, -(bits & 0x7FFFFFFF), bits)
        keys = order * (1 << 32) + (0xFFFFFFFF - torch.arange(z.shape[1], device=z.device))
        best = torch.topk(keys, top, dim=1).values
        top_idx = 0xFFFFFFFF - (best & 0xFFFFFFFF)
    else:
        top_idx = torch.empty((z.shape[0], 0), dtype=torch.int64, device=z.device)
    top_logprob = torch.gather(z, 1, top_idx) - lse
    return dict(logprob=logprob, lse=lse.squeeze(1), entropy=entropy, top_idx=top_idx.to(torch.int32),
                top_logprob=top_logprob)


def run(state):
    case = state["case"]
    if not own:
        return {"w4": _plain_w4, "moe": _plain_moe, "logprobs": _plain_logprobs}[case["op"]](state)
    mr = state["mr"]
    if case["op"] == "w4":
        mr.mrgemv_w4(state["a"], state["packed"], state["c"], state["fmt"])
        return state["c"]
    if case["op"] == "moe":
        flags = mr.MR_MOE_SOFTMAX if case["softmax"] else 0
        if case["group"]:
            mr.moe_window_w4(state["x"], state["ids"], state["val"], state["packed_up"], state["packed_down"],
                             state["y"], state["workspace"], case["experts"], case["inter"], state["fmt"],
                             expert_base=case["base"], flags=flags)
        else:
            mr.moe_window_bf16(state["x"], state["ids"], state["val"], state["up"], state["down"], state["y"],
                               state["workspace"], expert_base=case["base"], flags=flags)
        return state["y"]
    mr.token_logprobs(state["logits"], state["tokens"], state["logprob"], scale=case["scale"], lse=state["lse"],
                      entropy=state["entropy"], top_idx=state["top_idx"], top_logprob=state["top_logprob"])
    return {name: state[name] for name in ("logprob", "lse", "entropy", "top_idx", "top_logprob")}


# ---- what a pass cannot do without ----------------------------------------


def _bytes4(rows, k, case):
    per_group = 2 + (1 if case["zeros"] else 0)
    return rows * (k / 2 + k / case["group"] * per_group)


def work(case):
    m = case["m"]
    if case["op"] == "w4":
        n, k = case["n"], case["k"]
        return dict(bytes=_bytes4(n, k, case) + m * k * 2 + m * n * 4, flops=2.0 * m * n * k)
    if case["op"] == "moe":
        hidden, inter = case["hidden"], case["inter"]
        # choices of a row are distinct: the expected number of held experts that any row picks
        used = case["experts"] * (1 - (1 - case["topk"] / case["total"]) ** m)
        if case["group"]:
            expert = _bytes4(2 * inter, hidden, case) + _bytes4(hidden, inter, case)
        else:
            expert = 3 * hidden * inter * 2
        held = m * case["topk"] * case["experts"] / case["total"]
        out = m * hidden * (4 if case["out"] == "f32" else 2)
        return dict(bytes=used * expert + m * hidden * 2 + m * case["topk"] * 8 + out,
                    flops=held * 6.0 * hidden * inter)
    size = 4 if case["dtype"] == "f32" else 2
    small = m * (8 * case["tokens"] + 8 + 8 * case["top"])
    return dict(bytes=m * case["n"] * size + small, flops=5.0 * m * case["n"])


# ---- the definition in 64 bits --------------------------------------------


def _rows64(w, rows, group):
    """Rows of a 4-bit weight in 64 bits, element by element."""
    q, scales, zeros = w
    cols = torch.arange(2 * q.shape[-1], device=q.device)
    v = (q[rows][:, cols // 2].to(torch.int64) >> (4 * (cols % 2))) & 15
    z = 8 if zeros is None else zeros[rows][:, cols // group].to(torch.int64)
    return (v - z).double() * scales[rows][:, cols // group].double()


def _expert64(w, e, group):
    if not group:
        return w[e].double()
    one = [None if t is None else t[e] for t in w]
    return _rows64(one, slice(None), group)


def exact(case, seed):
    state = _inputs(case, seed)
    if case["op"] == "w4":
        a = state["a"].double()
        out = [a @ _rows64(state["w"], slice(at, at + 8192), case["group"]).T for at in range(0, case["n"], 8192)]
        return torch.cat(out, dim=1)
    if case["op"] == "moe":
        ids, val = state["ids"].cpu().numpy(), state["val"].double().cpu().numpy()
        y = torch.zeros((case["m"], case["hidden"]), dtype=torch.float64, device=DEV)
        for t in range(case["m"]):
            w = val[t]
            if case["softmax"]:
                w = np.exp(w - w.max())
                w = w / w.sum()
            for s in range(case["topk"]):
                e = int(ids[t, s]) - case["base"]
                if not 0 <= e < case["experts"]:
                    continue
                both = _expert64(state["up"], e, case["group"]) @ state["x"][t].double()
                gate, lift = both[:case["inter"]], both[case["inter"]:]
                y[t] += float(w[s]) * (_expert64(state["down"], e, case["group"]) @ (gate * torch.sigmoid(gate) * lift))
        return y
    rows = []
    for r in range(case["m"]):
        z = state["logits"][r].double()
        order = torch.sort(z, descending=True, stable=True).indices[:case["top"]]
        z = z * case["scale"]
        p = torch.exp(z - z.max())
        lse = z.max() + torch.log(p.sum())
        logp = z - lse
        entropy = -torch.where(p > 0, (p / p.sum()) * logp, torch.zeros_like(p)).sum()
        rows.append((logp[state["tokens"][r].long()], lse, entropy, order.to(torch.int32), logp[order]))
    names = ("logprob", "lse", "entropy", "top_idx", "top_logprob")
    return {name: torch.stack([row[i] for row in rows]) for i, name in enumerate(names)}
