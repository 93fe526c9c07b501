"""Microscaled operands from their definition, in 64 bits and apart from the library."""
import math

import torch

import xnor_popcount_gemm_gb300 as bt

#: code: mantissa bits, smallest normal exponent, largest exponent, largest value
FORMAT = {bt.BT_CODE_E4M3: (3, -6, 8, 448.0), bt.BT_CODE_E2M1: (1, 0, 2, 6.0)}


def table(code):
    """The format's values from 0 on, by code."""
    mant, emin, _, vmax = FORMAT[code]
    v, c = [0.0], 0
    while v[-1] < vmax:
        c += 1
        e, m = c >> mant, c & ((1 << mant) - 1)
        v.append(math.ldexp(m, emin - mant) if e == 0 else math.ldexp((1 << mant) + m, emin + e - 1 - mant))
    return torch.tensor(v, dtype=torch.float64)


def quantized(x, code):
    """x [R, K] (CPU): its values in 64 bits, the codes without their signs [R, blocks * 32], the scales' bytes."""
    mant, emin, emax, vmax = FORMAT[code]
    R, K = x.shape
    v = torch.nn.functional.pad(x.double(), (0, -K % 32)).view(R, -1, 32)
    bad = ~torch.isfinite(v).all(dim=2, keepdim=True)
    v = torch.where(bad, torch.zeros_like(v), v)
    top = v.abs().amax(dim=2, keepdim=True)
    e = torch.where(top > 0, torch.frexp(top)[1] - 1 - emax, torch.full_like(top, -127, dtype=torch.int32)).clamp(min=-127)
    scale = torch.ldexp(torch.ones_like(top), e)
    t = table(code)
    a = (v / scale).abs().clamp(max=vmax)
    lo = (torch.searchsorted(t, a.contiguous(), right=True) - 1).clamp(max=len(t) - 2)
    mid = (t[lo] + t[lo + 1]) / 2
    i = torch.where(a < mid, lo, torch.where(a > mid, lo + 1, lo + lo % 2))      # ties: the even code
    values = torch.where(bad, torch.full_like(v, math.nan), t[i] * torch.sign(v) * scale)
    scales = torch.where(bad, torch.full_like(e, 255), e + 127)
    i = torch.where(bad, torch.zeros_like(i), i)
    return values.view(R, -1)[:, :K], i.view(R, -1), scales.view(R, -1)


def scale_at(R, blocks, K, code):
    """Byte of every (row, block) among an operand's scales."""
    row = bt.bt_mx_row_bytes(K, code)
    atoms = row // (64 if code == bt.BT_CODE_E2M1 else 128)
    r, b = torch.arange(R).view(-1, 1), torch.arange(blocks).view(1, -1)
    return ((r // 128) * atoms + b // 4) * 512 + (r % 32) * 16 + (r // 32 % 4) * 4 + b % 4


def unpacked(q):
    """(magnitude codes, signs, scales' bytes) of MxRows, from the documented layout, up to the end of its rows."""
    c = q.codes.cpu().long()
    if q.code == bt.BT_CODE_E2M1:
        c = torch.stack([c & 15, c >> 4], dim=2).view(c.shape[0], -1)
        mag, sign = c & 7, c >> 3
    else:
        mag, sign = c & 127, c >> 7
    R, K = q.shape
    s = q.scales.cpu().long()[scale_at(R, c.shape[1] // 32, K, q.code)]
    return mag, sign, s
