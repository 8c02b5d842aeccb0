"""Packed rows of experts for the dense products' tests: groups with gaps, rows that belong
to nobody, and the 64-bit products of a group."""
from __future__ import annotations

import torch

from lm_util import U32, matvec_ref


def groups(counts, align=1, tail=0):
    """(offsets, counts) int32 on the GPU and the rows of the buffer, `tail` rows behind the last group."""
    offsets = [0]
    for c in counts:
        offsets.append(offsets[-1] + -(-c // align) * align)
    return (torch.tensor(offsets, dtype=torch.int32).cuda(),
            torch.tensor(counts, dtype=torch.int32).cuda(), offsets[-1] + tail)


def randn(g, dtype, *shape, scale=1.0):
    return (torch.randn(*shape, generator=g) * scale).to(dtype).cuda()


def owned(offsets, counts, rows):
    """Whether a row belongs to an expert."""
    mine = torch.zeros(rows, dtype=torch.bool)
    for o, c in zip(offsets.tolist(), counts.tolist()):
        mine[o:o + c] = True
    return mine.cuda()


def product(x, w, swiglu):
    """(v, error of binary32 sums) of rows x [r, K] with w [n, K], wherever they are.  A sum of K
    products in chains of 16 or more, each addition off by at most an ulp (truncation
    included): K / 16 * 2 half ulps, which matvec_ref's K / 8 + 64 cover."""
    return matvec_ref(x, w.double(), swiglu)


def codes_bound(v, err):
    """Error of e4m3 codes times their scale against v: half a step (2^-4 relative, or half the
    subnormal spacing 2^-9 of a scale), the scale's own error (its group's largest), and four
    binary32 roundings."""
    group = v.reshape(v.shape[0], -1, 128)
    e = err.reshape(group.shape)
    scale = (group.abs().amax(2, keepdim=True).clamp(min=1e-4) + e.amax(2, keepdim=True)) / 448.0
    off = e.amax(2, keepdim=True) / 448.0 + 4 * U32 * scale
    # a code of magnitude q <= 448 times the scale's error
    bound = (group.abs() + e) * 2.0 ** -4 + scale * 2.0 ** -10 + e + 448.0 * off * 2.0 ** -4
    bound = bound + (group.abs() / scale) * off
    return bound.reshape(v.shape), (scale - e.amax(2, keepdim=True) / 448.0).squeeze(2), off.squeeze(2)
