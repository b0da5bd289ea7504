"""4-bit weights for the tests: seeded values, and what they stand for in 64 bits."""
import numpy as np

from gpu_util import torch

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16}


def weight(seed, lead, n, k, group, zeros, scale_dtype="bf16", pow2=False):
    """(q, scales, zeros) on the CPU: q uint8 [*lead, n, k/2], the even column in the low half."""
    rng = np.random.default_rng(seed)
    q = rng.integers(0, 16, (*lead, n, k), dtype=np.uint8)
    s = rng.uniform(0.3, 1.0, (*lead, n, k // group)) / np.sqrt(k)
    if pow2:
        s = 2.0 ** rng.integers(-3, 3, (*lead, n, k // group))
    z = rng.integers(0, 16, (*lead, n, k // group), dtype=np.uint8) if zeros else None
    packed = q[..., 0::2] | (q[..., 1::2] << 4)
    return (torch.from_numpy(np.ascontiguousarray(packed)), torch.from_numpy(s).to(DTYPES[scale_dtype]),
            None if z is None else torch.from_numpy(z))


def dense64(w):
    """The weight in float64, [*lead, n, k]."""
    q, s, z = w
    qn = q.cpu().numpy()
    v = np.stack((qn & 15, qn >> 4), axis=-1).reshape(*qn.shape[:-1], -1).astype(np.float64)
    s64 = s.cpu().double().numpy()
    group = v.shape[-1] // s64.shape[-1]
    z64 = 8.0 if z is None else np.repeat(z.cpu().numpy().astype(np.float64), group, axis=-1)
    return (v - z64) * np.repeat(s64, group, axis=-1)


def pack(mr, w, paired=False):
    """(packed CUDA tensor, format) of a weight."""
    q, s, z = (None if t is None else t.cuda() for t in w)
    group = 2 * q.shape[-1] // s.shape[-1]
    fmt = mr.w4_format(group, z is not None, s.dtype)
    count = q.shape[0] if q.dim() == 3 else 1
    out = torch.full((count * mr.w4_packed_bytes(q.shape[-2], 2 * q.shape[-1], fmt, paired),), 0xA5,
                     dtype=torch.uint8, device="cuda")
    mr.w4_pack(q, s, z, out, paired=paired)
    return out, fmt
