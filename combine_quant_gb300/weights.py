"""Weight preparation for the quantised expert products, done once when weights
are loaded (torch operations on the weights' device; no part of a call).

``quantize_mx``: fp8 codes with one power-of-two scale per 32 of the last axis,
for ``expert_matmul`` with mx types. ``quantize_w4``: 4-bit codes with group
scales, for ``expert_matmul_w4``.
"""
from __future__ import annotations

from typing import Optional

import torch

_FP8 = {False: (torch.float8_e4m3fn, 448.0), True: (torch.float8_e5m2, 57344.0)}


def quantize_mx(w: torch.Tensor, e5m2: bool = False) -> tuple[torch.Tensor, torch.Tensor]:
    """Codes uint8 [..., k] and e8m0 scales uint8 [..., Align2(k / 32)] (value
    2^(s - 127), pad column 0), by the rule of dispatch mode 5: per block of 32 the
    smallest power of two that brings max(|w|, 1e-4) within the fp8 range."""
    k = w.shape[-1]
    if k % 32 != 0:
        raise ValueError(f"the last axis must be a multiple of 32, got {k}")
    dtype, largest = _FP8[bool(e5m2)]
    b = w.float().reshape(*w.shape[:-1], k // 32, 32)
    m, e = torch.frexp(b.abs().amax(-1).clamp(min=1e-4) / largest)
    e = torch.where(m > 0.5, e, e - 1).clamp(-127, 127)  # ceil(log2(q)), q = m 2^e, m in [0.5, 1)
    codes = torch.ldexp(b, -e[..., None]).clamp(-largest, largest).to(dtype).view(torch.uint8)
    scales = torch.zeros(*w.shape[:-1], (k // 32 + 1) // 2 * 2, dtype=torch.uint8, device=w.device)
    scales[..., : k // 32] = (e + 127).to(torch.uint8)
    return codes.reshape(w.shape), scales


def quantize_w4(w: torch.Tensor, group: int = 128, zeros: bool = False
                ) -> tuple[torch.Tensor, torch.Tensor, Optional[torch.Tensor]]:
    """Codes uint8 [..., k / 2] (element j in the low half of byte j / 2 when j is
    even), scales [..., k / group] in w's type, and with ``zeros`` the zero points
    uint8 [..., k / group], else None (the codes' zero is 8). w ~ (q - z) * s,
    round to nearest; symmetric groups span max|w| with codes 0.5 to 15.5 around 8,
    groups with a zero point their least to their largest value (and 0)."""
    k = w.shape[-1]
    if w.dtype not in (torch.bfloat16, torch.float16):
        raise ValueError(f"w must be bf16 or fp16, got {w.dtype}")
    if group not in (32, 64, 128) or k % group != 0:
        raise ValueError(f"group must be 32, 64 or 128 and divide {k}, got {group}")
    b = w.float().reshape(*w.shape[:-1], k // group, group)
    tiny = torch.finfo(w.dtype).tiny
    if zeros:
        lo, hi = b.amin(-1).clamp(max=0.0), b.amax(-1).clamp(min=0.0)
        s = ((hi - lo) / 15).clamp(min=tiny).to(w.dtype)
        z = torch.round(-lo / s.float()).clamp(0, 15)
    else:
        s = (b.abs().amax(-1) / 7.5).clamp(min=tiny).to(w.dtype)
        z = torch.full_like(s, 8.0, dtype=torch.float32)
    q = torch.round(b / s.float()[..., None] + z[..., None]).clamp(0, 15).to(torch.uint8)
    q = q.reshape(*w.shape[:-1], k // 2, 2)
    return q[..., 0] | (q[..., 1] << 4), s, z.to(torch.uint8) if zeros else None
