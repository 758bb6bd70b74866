"""Plain references of the operators on caches in 4 bits and of eviction, on the
CPU: what a row is stored as, what it stands for, attention over it with its
rounding bound, and which tokens stay."""
import torch

from generate_ref import BF16_HALF, F32_HALF, paged

F16_HALF = 2.0 ** -11
NAN_SCALE = 0xFF


def scale_values():
    """What the 256 scale bytes stand for, float64."""
    byte = torch.arange(256)
    e, m = byte >> 3, byte & 7
    s = torch.where(e == 0, m * 2, (8 + m) << e).double() * 2.0 ** -18
    s[0xD8:] = float("nan")
    return s


def store(rows):
    """codes [.., D / 2] and scales [.., D / 16] uint8 of bf16 rows [.., D]."""
    x = rows.double().unflatten(-1, (-1, 16))
    top = x.abs().amax(-1)
    table = scale_values()[:0xD8]
    # the nearest scale to top / 7: compared as 7 s against top, which is exact
    i = torch.searchsorted(7 * table, top.nan_to_num(0.0).contiguous()).clamp(1, 0xD7)
    down, up = top - 7 * table[i - 1], 7 * table[i] - top
    i = i - ((down < up) | ((down == up) & (i % 2 == 1))).long()
    bad = ~top.isfinite()
    i[bad] = NAN_SCALE
    s = table[i.clamp(max=0xD7)]
    code = torch.where((s > 0)[..., None], torch.sign(x) * torch.floor(x.abs() / s.clamp(min=2.0 ** -20)[..., None] + 0.5), 0.0)
    code = code.clamp(-8, 7)
    code[bad] = 0.0
    code = (code + 8).to(torch.uint8).flatten(-2)
    return code[..., 0::2] | (code[..., 1::2] << 4), i.to(torch.uint8)


def values(codes, scales):
    """What they stand for, float64 [.., D]."""
    c = torch.stack((codes & 15, codes >> 4), -1).flatten(-2).double() - 8
    return (c.unflatten(-1, (-1, 16)) * scale_values()[scales.long()][..., None]).flatten(-2)


class Pages:
    """A cache of either kind: K and V pages (poisoned past the lengths), its page table; bits 16 or 4."""

    def __init__(self, bits, B, capacity, page, Hkv, D, seed, poison=True):
        self.bits, self.page = bits, page
        self.k, self.v, self.table = paged(B, capacity, page, Hkv, D, seed, poison=poison)

    def hold(self):
        """Fixes what the pages hold: .held (the tensors of the cache) and .kv (float64 values of K and V)."""
        if self.bits == 16:
            self.held, self.kv = [self.k, self.v], [self.k.double(), self.v.double()]
        else:
            (kc, ks), (vc, vs) = store(self.k), store(self.v)
            self.held, self.kv = [kc, vc, ks, vs], [values(kc, ks), values(vc, vs)]
        return self

    def cuda(self, h3, lens):
        self.dheld, self.dtable = [t.cuda() for t in self.held], self.table.cuda()
        self.dlen = torch.tensor(list(lens), dtype=torch.int32, device="cuda")
        return (h3.PagedKV if self.bits == 16 else h3.PagedKV4)(*self.dheld, self.dtable, self.dlen)


def attend(q, kv, table, lens, page, scale, skip=None, bits=4):
    """(o, bound, weights, weights_bound) of q [B, Hq, D] over each sequence's first lens[b] tokens in float64, and how far a
    computation with float32 sums may be off.

    d bounds the error of a score in exp's argument: a float32 dot product of D terms, its scaling and the subtraction of
    what it is taken against, exp2, and the queries' channels below 2^-20 of the largest in binary16 (2^-30 of it each).
    A softmax weight is then off by a factor of at most e^(2 d).  The second product takes weights of 11 bits
    (a cache in 4 bits: half a step 2^-11, and 2^-32 of the largest one where they fall out of binary16's range) or of 16
    bits (2^-16); the output is rounded once.  A token's weight is a float32 sum over the heads."""
    B, Hq, D = q.shape
    k, v = kv
    Hkv = k.shape[2]
    room = table.shape[1] * page
    o, bound = torch.zeros(B, Hq, D, dtype=torch.float64), torch.zeros(B, Hq, D, dtype=torch.float64)
    w, w_bound = torch.zeros(B, room, dtype=torch.float64), torch.zeros(B, room, dtype=torch.float64)
    half = F16_HALF if bits == 4 else BF16_HALF ** 2
    for b in range(B):
        n = min(max(int(lens[b]), 0), room)
        at = torch.arange(n)
        at = at[[j for j in range(n) if not (skip and j in skip[b])]] if skip and skip[b] else at
        if not len(at):
            continue
        rows = table[b].clamp(0, k.shape[0] - 1)[at // page].long()
        kk, vv = k[rows, at % page], v[rows, at % page]
        for h in range(Hq):
            kh, vh, qh = kk[:, h // (Hq // Hkv)], vv[:, h // (Hq // Hkv)], q[b, h].double()
            p = torch.softmax(kh @ qh * scale, 0)
            o[b, h] = p @ vh
            d = ((D + 8) * F32_HALF * float((kh.abs() @ qh.abs()).max()) +
                 2.0 ** -30 * float(qh.abs().max()) * float(kh.abs().sum(-1).max())) * scale + 2.0 ** -20
            tail = len(at) * 2.0 ** -32 * vh.abs().amax(0) if bits == 4 else 0.0
            bound[b, h] = BF16_HALF * o[b, h].abs() + (half + 4 * d) * (p @ vh.abs()) + tail + 1e-30
            w[b, at] += p
            w_bound[b, at] += (4 * d + Hq * F32_HALF) * p
    return o, bound, w, w_bound + 1e-30


def evict(held, table, lens, page, weights, keep, recent):
    """held (copied), weights (copied) and lengths after an eviction, by the definition."""
    held, weights, out = [t.clone() for t in held], weights.clone(), []
    room = table.shape[1] * page
    for b, n in enumerate(lens):
        n = min(max(int(n), 0), room)
        out.append(min(n, keep))
        if n <= keep:
            continue
        front, old = keep - recent, n - recent
        w = weights[b, :n].clone()
        key = [(0 if x != x else 1, -x) for x in w[:old].tolist()]  # a NaN first
        stay = set(sorted(range(old), key=key.__getitem__)[:front])
        gaps = [j for j in range(front) if j not in stay]
        moves = list(zip(sorted(j for j in stay if j >= front), gaps)) + [(old + i, front + i) for i in range(recent)]
        before = [t.clone() for t in held]
        for src, dst in moves:
            a, z = int(table[b, src // page]), int(table[b, dst // page])
            weights[b, dst] = w[src]
            if 0 <= a < held[0].shape[0] and 0 <= z < held[0].shape[0]:
                for t, t0 in zip(held, before):
                    t[z, dst % page] = t0[a, src % page]
        weights[b, keep:n] = 0.0
    return held, weights, torch.tensor(out, dtype=torch.int32)
