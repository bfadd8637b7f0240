"""Shared inputs for the decoding-step tests: seeded NumPy arrays and device copies in the layouts
of include/svdq_serve.h.  (Not a test module.)"""
from __future__ import annotations

import numpy as np
import torch

from oracle.numerics import bf16_to_bits, round_bf16


def bf16_values(rng, *shape, scale=1.0):
    """Exact bf16 values (float64) of normal draws."""
    return round_bf16(rng.standard_normal(shape) * scale)


def to_dev_bf16(values) -> torch.Tensor:
    bits = bf16_to_bits(values)
    return torch.from_numpy(bits.view(np.int16)).view(torch.bfloat16).cuda()


def to_dev(a, dtype=None) -> torch.Tensor:
    t = torch.from_numpy(np.ascontiguousarray(a))
    return (t if dtype is None else t.to(dtype)).cuda()


def host64(t: torch.Tensor) -> np.ndarray:
    return t.float().cpu().numpy().astype(np.float64)


def host_bits(t: torch.Tensor) -> np.ndarray:
    return t.contiguous().cpu().view(torch.int16).numpy().view(np.uint16)


def random_cache(rng, num, heads, bs, dim):
    """(k_codes, k_scale, v_codes, v_scale) with codes c [num, heads, bs, dim] and fp32 scales."""
    def one():
        c = np.clip(np.rint(rng.standard_normal((num, heads, bs, dim)) * 40), -127, 127).astype(np.int64)
        s = (np.exp(0.4 * rng.standard_normal((num, heads))) / 40).astype(np.float32)
        return c, s
    kc, ks = one()
    vc, vs = one()
    return kc, ks, vc, vs


def dev_cache(kc, ks, vc, vs):
    """The device arrays of a cache given as codes c."""
    from bit_post_quantized_amd import serve
    return serve.BlockCache(to_dev((kc + 128).astype(np.uint8)),
                            to_dev(np.ascontiguousarray(np.swapaxes(vc + 128, 2, 3)).astype(np.uint8)),
                            to_dev(ks), to_dev(vs))


def host_cache(cache):
    """(k codes c, k scale, v codes c, v scale) of a device cache, V's tokens before channels."""
    return (cache.k_codes.cpu().numpy().astype(np.int64) - 128, cache.k_scale.cpu().numpy(),
            np.swapaxes(cache.v_codes.cpu().numpy().astype(np.int64) - 128, 2, 3),
            cache.v_scale.cpu().numpy())
