"""Plain references of the generation operators, in 64 bits on the CPU, and the
rounding bounds their tests use.  A rounding is off by at most half a step:
2^-8 of the value in bf16, 2^-24 in float32, 2^-4 in e4m3 (2^-10 absolute below
its normal range)."""
import math

import numpy as np
import torch

BF16_HALF = 2.0 ** -8
F32_HALF = 2.0 ** -24


def randn(*shape, seed, scale=1.0):
    """bf16 N(0, scale^2) on the CPU."""
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * scale).to(torch.bfloat16)


def paged(B, capacity, page, Hkv, D, seed, spare=3, poison=True):
    """K and V pages (CPU, bf16) and a page table in random order; pages that no
    sequence holds are NaN."""
    each = -(-capacity // page)
    total = B * each + spare
    k, v = randn(total, page, Hkv, D, seed=seed), randn(total, page, Hkv, D, seed=seed + 1)
    order = torch.randperm(total, generator=torch.Generator().manual_seed(seed + 2))
    table = order[: B * each].to(torch.int32).view(B, each)
    if poison:
        k[order[B * each:].long()] = float("nan")
        v[order[B * each:].long()] = float("nan")
    return k, v, table


def poison_past(k, v, table, lens, page):
    """NaN in every row of a sequence's pages past its length; table entries past its last page are wild."""
    for b, n in enumerate(lens):
        n = max(int(n), 0)
        for p in range(table.shape[1]):
            first = n - p * page
            if first <= 0:
                k[table[b, p].long()] = float("nan")
                v[table[b, p].long()] = float("nan")
                table[b, p] = (-1, 1 << 30)[p & 1]
            elif first < page:
                k[table[b, p].long(), first:] = float("nan")
                v[table[b, p].long(), first:] = float("nan")


def gather(pages, table_row, n, page):
    """[n, Hkv, D] float64 rows of one sequence."""
    at = torch.arange(n)
    return pages[table_row[at // page].long(), at % page].double()


def decode_f64(q, k, v, table, lens, page, scale, skip=None):
    """(o, bound): attention of q [B, Hq, D] over each sequence's first lens[b]
    tokens in float64, and how far a float32 computation whose weights are the
    sum of two bf16 values may be off.  skip[b]: tokens that are not attended.

    With d = (D + 8) 2^-24 max_j scale sum|q k_j| + 2^-20 the error of a score
    in exp's argument (a float32 dot product of D terms, its scaling and the
    running maximum's subtraction) and of exp2, every weight is off by a factor
    of at most e^(2 d) with the sum's; a weight loses 2^-8 of what its own
    rounding by 2^-8 left, and the output is rounded once:
    |error| <= 2^-8 |o| + (2^-16 + 4 d) sum_j p_j |v_j|."""
    B, Hq, D = q.shape
    Hkv = k.shape[2]
    o, bound = torch.zeros(B, Hq, D, dtype=torch.float64), torch.zeros(B, Hq, D, dtype=torch.float64)
    for b in range(B):
        n = max(int(lens[b]), 0)
        keep = torch.ones(n, dtype=torch.bool)
        if skip is not None and skip[b]:
            keep[list(skip[b])] = False
        if not bool(keep.any()):
            continue
        safe = table[b].clamp(0, k.shape[0] - 1)
        kk, vv = gather(k, safe, n, page)[keep], gather(v, safe, n, page)[keep]
        for h in range(Hq):
            kh, vh, qh = kk[:, h // (Hq // Hkv)], vv[:, h // (Hq // Hkv)], q[b, h].double()
            p = torch.softmax(kh @ qh * scale, 0)
            o[b, h] = p @ vh
            d = (D + 8) * F32_HALF * float((kh.abs() @ qh.abs()).max()) * scale + 2.0 ** -20
            bound[b, h] = BF16_HALF * o[b, h].abs() + (BF16_HALF ** 2 + 4 * d) * (p @ vh.abs()) + 1e-30
    return o, bound


def rope_freqs(rot, theta=10000.0, kind="none", factor=1.0, original_len=1, low=1.0, high=32.0):
    """Radians per position, as Python floats (the same double operations as the definition's)."""
    base = theta * math.pow(factor, rot / (rot - 2.0)) if kind == "ntk" else theta
    out = []
    for i in range(rot // 2):
        f = math.pow(base, -2.0 * i / rot)
        if kind == "linear":
            f = f / factor
        if kind == "by_parts":
            turns = original_len * f / 6.283185307179586
            keep = min(max((turns - low) / (high - low), 0.0), 1.0)
            f = (1.0 - keep) * (f / factor) + keep * f
        out.append(f)
    return out


def rope_table_wide(positions, freqs, amplitude=1.0):
    """cos, sin in float64 of angles multiplied out in extended precision (at
    least 64 significant bits here and on Arm), reduced by whole turns there."""
    wide = np.longdouble
    two_pi = wide(2) * (wide(math.pi) + wide(1.2246467991473532e-16))
    angle = np.asarray(positions, dtype=wide)[:, None] * np.asarray(freqs, dtype=wide)[None]
    angle = angle - np.rint(angle / two_pi) * two_pi
    return amplitude * np.cos(angle).astype(np.float64), amplitude * np.sin(angle).astype(np.float64)


def add_norm_f64(x, residual, w, eps):
    """h (bf16, CPU) and y (float64) of rows x [T, C]."""
    h = x if residual is None else (x.double() + residual.double()).to(torch.bfloat16)
    y = h.double()
    y = y / torch.sqrt(y.square().mean(-1, keepdim=True) + float(np.float32(eps)))
    return h, y if w is None else y * w.double()
