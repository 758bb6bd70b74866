"""Cases of the operators that keep a generation's cache small: the rotated append to a paged cache in 4 bits, the
reading of cached tokens as contiguous rows, the attention of one new token over the 4-bit cache, the same attention
with each cached token's weight added up, and the eviction of the tokens that were attended to least.

`run` computes them in their plain form, elementary torch operations in float32 (float64 where a product and a sum are
rounded once, or where values lie next to a border), or, where `own` is true, through the framework's entry points.

Of 16 neighbouring channels a 4-bit row holds one scale s, a byte whose bits moved up by 7 are a binary16, and codes c:
each channel stands for (c - 8) s."""
import math

import torch

own = False

BF16, F16, F32, F64, I32, U8 = torch.bfloat16, torch.float16, torch.float32, torch.float64, torch.int32, torch.uint8
EPS = 1e-6
SCALE_MAX = 3840.0   # the largest scale
GROUP = 16           # channels that share one


def listed():
    return [
        # the new token of each request in a batch: norm, rotation of 96 of 128 channels, codes and scales
        dict(name="append_token", op="append", B=8, S=1, Hq=24, Hkv=8, D=128, page=16, rot=96, norm=True,
             interleaved=False, start=1000, ragged=False),
        # prompts of unlike length, padded to the longest, interleaved pairs, no norm
        dict(name="append_prompts", op="append", B=4, S=2048, Hq=16, Hkv=4, D=128, page=16, rot=128, norm=False,
             interleaved=True, start=100, ragged=True),
        # a long clip's rows into an empty cache
        dict(name="append_clip", op="append", B=1, S=32760, Hq=24, Hkv=24, D=128, page=64, rot=96, norm=True,
             interleaved=False, start=0, ragged=False),
        # what a few requests hold so far, before their prompts' next part; pages that are no power of two
        dict(name="read_prompts", op="read", B=4, S=1021, Hkv=2, D=64, page=24, low=0, high=1021, bits=16),
        # a long clip's cached rows, for the prefill of the next one
        dict(name="read_clip", op="read", B=1, S=32760, Hkv=24, D=128, page=64, low=32760, high=32760, bits=4),
        # a single stream of generation right after a short prompt: launch and wait times count
        dict(name="decode_one_short", op="decode", bits=4, weights=False, B=1, Hq=16, Hkv=4, D=128, page=16, low=37, high=37),
        # a serving batch with four query heads to a key-value head, caches of unlike lengths
        dict(name="decode_batch_gqa", op="decode", bits=4, weights=False, B=16, Hq=16, Hkv=4, D=128, page=16, low=4096,
             high=8192),
        # one token against a packed clip's whole cache, as many key-value heads as query heads
        dict(name="decode_clip", op="decode", bits=4, weights=False, B=1, Hq=24, Hkv=24, D=128, page=64, low=104448,
             high=104448),
        # the serving batch on a 16-bit cache, with what each token was attended to
        dict(name="weights_batch", op="decode", bits=16, weights=True, B=16, Hq=16, Hkv=4, D=128, page=16, low=4096, high=8192),
        # a few long requests on a 4-bit cache, with what each token was attended to
        dict(name="weights_long", op="decode", bits=4, weights=True, B=4, Hq=24, Hkv=8, D=128, page=32, low=16380, high=32760),
        # a serving batch's 16-bit caches, some of them still short, back to 4096 tokens
        dict(name="evict_batch", op="evict", bits=16, B=16, Hkv=4, D=128, page=16, low=3900, high=4352, keep=4096, recent=256),
        # a packed clip's 4-bit cache down to a shorter clip's length, the last frame kept
        dict(name="evict_clip", op="evict", bits=4, B=1, Hkv=24, D=128, page=64, low=104448, high=104448, keep=32760, recent=1536),
    ]


HEADS = [(4, 4), (12, 12), (24, 24), (16, 4), (16, 2), (24, 8), (20, 4), (8, 1), (32, 1)]
PAGES = [16, 24, 32, 64, 128]


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["append", "read", "decode", "decode", "evict"])
    (Hq, Hkv), D, page = rng.choice(HEADS), rng.choice([64, 128, 128, 256]), rng.choice(PAGES)
    if op == "append":
        tokens = _log(rng, 1, max(1, min(32760, int(1.0e9 / ((Hq + 2 * Hkv) * D * 4)))))
        B = min(tokens, _log(rng, 1, 64))
        return dict(op=op, B=B, S=tokens // B, Hq=Hq, Hkv=Hkv, D=D, page=page, rot=rng.choice([D, D // 2, 3 * D // 4, D // 2 + 2]),
                    norm=rng.random() < 0.5, interleaved=rng.random() < 0.5, start=_log(rng, 1, 4000) - 1,
                    ragged=rng.random() < 0.5)
    bits, B = rng.choice([4, 16]), _log(rng, 1, 64)
    most = max(2, min(104448, int((5e8 if bits == 4 else 1.2e9) / (B * Hkv * D * 4))))  # tokens of one sequence
    if op == "read":
        high = _log(rng, 1, min(most, 32760))
        return dict(op=op, B=B, S=high, Hkv=Hkv, D=D, page=page, low=rng.choice([0, high // 2, high]), high=high, bits=bits)
    if op == "decode":
        high = _log(rng, 1, most)
        return dict(op=op, bits=bits, weights=bits == 16 or rng.random() < 0.4, B=B, Hq=Hq, Hkv=Hkv, D=D, page=page,
                    low=rng.choice([0, high // 2, high]), high=high)
    high = _log(rng, 2, most)
    keep = rng.randint(1, high - 1)
    return dict(op=op, bits=bits, B=B, Hkv=Hkv, D=D, page=page, low=rng.choice([0, keep, high]), high=high, keep=keep,
                recent=rng.choice([0, keep // 8, keep // 2, min(keep, 64)]))


# ---------------------------------------------------------------- inputs

def _randn(*shape, g):
    return torch.randn(*shape, generator=g, device="cuda", dtype=BF16)


def _lengths(case, g):
    """Cache lengths of a case: the longest is there, the others are spread."""
    n = torch.randint(case["low"], case["high"] + 1, (case["B"],), generator=g, device="cuda", dtype=I32)
    n[-1:] = case["high"]
    return n


def _table(B, capacity, page, g):
    """The pages of B sequences of up to `capacity` tokens, in no order, with a few that nobody holds."""
    each = -(-max(capacity, 1) // page)
    total = B * each + 3
    return torch.randperm(total, generator=g, device="cuda")[: B * each].to(I32).view(B, each), total


def _store(rows, bits, g):
    """What a cache holds of rows [.., D] in bf16: (themselves,), or (codes, scales)."""
    return (rows,) if bits == 16 else _in_4_bits(rows)


def _pages(case, g):
    """K's and V's pages and the page table."""
    table, total = _table(case["B"], case["high"], case["page"], g)
    shape = (total, case["page"], case["Hkv"], case["D"])
    k = _randn(*shape, g=g)
    k += 0.5 * _randn(*shape[2:], g=g)  # an offset of each head: some keys stand out
    return _store(k, case["bits"], g), _store(_randn(*shape, g=g), case["bits"], g), table


def _cache(s):
    import video_dit_dense_gb300 as h3
    if len(s["k"]) == 1:
        return h3.PagedKV(s["k"][0], s["v"][0], s["table"], s["kv_len"])
    return h3.PagedKV4(s["k"][0], s["v"][0], s["k"][1], s["v"][1], s["table"], s["kv_len"])


def _prepare_append(case, g):
    B, S, Hq, Hkv, D, rot = (case[n] for n in ("B", "S", "Hq", "Hkv", "D", "rot"))
    start = torch.randint(case["start"] // 2, case["start"] + 1, (B,), generator=g, device="cuda", dtype=I32)
    table, total = _table(B, case["start"] + S, case["page"], g)
    at = torch.arange(case["start"] + S, device="cuda", dtype=F64)[:, None]
    angle = at * 10000.0 ** (torch.arange(rot // 2, device="cuda", dtype=F64) * (-2.0 / rot))
    qkv = _randn(B, S, (Hq + 2 * Hkv) * D, g=g)  # one projection's output
    q, k, v = (t.unflatten(-1, (-1, D)) for t in qkv.split([Hq * D, Hkv * D, Hkv * D], dim=-1))
    shape = (total, case["page"], Hkv)
    s = dict(q=q, k_new=k, v_new=v, table=table, kv_len=start, cos=angle.cos().to(F32), sin=angle.sin().to(F32),
             k=tuple(torch.zeros(*shape, D // n, device="cuda", dtype=U8) for n in (2, GROUP)),
             v=tuple(torch.zeros(*shape, D // n, device="cuda", dtype=U8) for n in (2, GROUP)),
             q_out=torch.zeros(B, S, Hq, D, device="cuda", dtype=BF16), k_out=torch.zeros(B, S, Hkv, D, device="cuda", dtype=BF16),
             v_out=torch.zeros(B, S, Hkv, D, device="cuda", dtype=BF16), len_out=torch.zeros_like(start), wq=None, wk=None,
             new_len=None)
    if case["norm"]:
        s["wq"] = torch.rand(D, generator=g, device="cuda") + 0.5
        s["wk"] = torch.rand(D, generator=g, device="cuda") + 0.5
    if case["ragged"]:
        s["new_len"] = torch.randint(0, S + 1, (B,), generator=g, device="cuda", dtype=I32)
        s["new_len"][-1:] = S
    if own:
        s["cache"] = _cache(s)
        s["grown"] = s["cache"].with_lengths(s["len_out"])
    return s


def _prepare_read(case, g):
    k, v, table = _pages(case, g)
    s = dict(k=k, v=v, table=table, kv_len=_lengths(case, g))
    s["k_out"], s["v_out"] = (torch.zeros(case["B"], case["S"], case["Hkv"], case["D"], device="cuda", dtype=BF16) for _ in range(2))
    if own:
        s["cache"] = _cache(s)
    return s


def _prepare_decode(case, g):
    k, v, table = _pages(case, g)
    s = dict(k=k, v=v, table=table, kv_len=_lengths(case, g), q=_randn(case["B"], 1, case["Hq"], case["D"], g=g))
    s["o"] = torch.empty_like(s["q"])
    s["weights"] = None
    if case["weights"]:  # what earlier tokens attended to
        s["weights"] = torch.rand(case["B"], table.shape[1] * case["page"], generator=g, device="cuda") * 0.01
    if own:
        import video_dit_dense_gb300 as h3
        s["cache"] = _cache(s)
        make = h3.paged_decode_weights_workspace if case["weights"] else h3.paged_decode_q4_workspace
        s["workspace"] = make(s["q"], s["cache"])
    return s


def _prepare_evict(case, g):
    k, v, table = _pages(case, g)
    # sums of softmax weights: a few tokens have most of it, and some have none
    sums = torch.randn(case["B"], table.shape[1] * case["page"], generator=g, device="cuda").mul(2.0).exp()
    sums[torch.rand(sums.shape, generator=g, device="cuda") < 0.02] = 0.0
    s = dict(k=k, v=v, table=table, kv_len=_lengths(case, g), sums=sums, weights=sums.clone())
    s["len_out"] = torch.zeros_like(s["kv_len"])
    if own:
        import video_dit_dense_gb300 as h3
        s["cache"] = _cache(s)
        s["workspace"] = h3.paged_evict_workspace(s["cache"], case["keep"], case["recent"])
    return s


def prepare(case, seed):
    g = torch.Generator("cuda").manual_seed(seed)
    make = dict(append=_prepare_append, read=_prepare_read, decode=_prepare_decode, evict=_prepare_evict)[case["op"]]
    return dict(case=case, **make(case, g))


# ---------------------------------------------------------------- one pass

def run(state):
    return dict(append=_append, read=_read, decode=_decode, evict=_evict)[state["case"]["op"]](state)


def _in_4_bits(rows):
    """Codes [.., D / 2], the even channel in the lower half of a byte, and scales [.., D / 16] of rows [.., D]."""
    x = rows.to(F32).unflatten(-1, (-1, GROUP))
    top = x.abs().amax(-1)
    t = (top / torch.full_like(top, 7.0)).clamp(max=SCALE_MAX)                  # by a plain number it would be a product
    step = torch.exp2((torch.frexp(t)[1] - 1).clamp(min=-14).to(F32) - 3.0)     # of three bits behind the leading one
    s = (t / step).round() * step
    bits = s.to(F16).view(torch.int16).bitwise_right_shift(7).to(U8)
    r = x / torch.where(s == 0, 1.0, s)[..., None]
    c = ((r.abs() + 0.5).floor().copysign(r).clamp(-8, 7) * (s != 0)[..., None] + 8).to(U8).flatten(-2)
    return c[..., 0::2] | (c[..., 1::2] << 4), bits


def _values(codes, scales):
    """What codes [.., D / 2] and scales [.., D / 16] stand for, in float32."""
    s = (scales.to(torch.int16) << 7).view(F16).to(F32)
    c = torch.stack((codes & 15, codes >> 4), -1).flatten(-2).to(F32) - 8.0
    return (c.unflatten(-1, (-1, GROUP)) * s[..., None]).flatten(-2)


def _rows(held, rows, at):
    """Rows of pages (themselves, or codes and scales) in float32."""
    return held[0][rows, at].to(F32) if len(held) == 1 else _values(held[0][rows, at], held[1][rows, at])


def _normed(x, w, case):
    """bf16((x r) w) in float32, r = 1 / sqrt(mean(x^2) + EPS), with the sum of squares in the order that the framework
    documents: 16 channels in order (two groups of 8), then pairs of such sums, neighbours first from far to near."""
    D, rot = case["D"], case["rot"]
    lanes, turning = D // 16, rot // 16
    lane = torch.arange(lanes, device="cuda")
    if case["interleaved"]:
        first, second = lane, lane + lanes
    else:
        first, second = torch.where(lane < turning, lane, lane + lanes), lane + turning
    groups = x.to(F32).square().unflatten(-1, (-1, 8))                          # exact: 8 bits squared
    mine = torch.cat((groups[..., first, :], groups[..., second, :]), -1)       # [.., lanes, 16]
    total = mine[..., 0]
    for e in range(1, 16):
        total = total + mine[..., e]
    while total.shape[-1] > 1:
        total = total[..., : total.shape[-1] // 2] + total[..., total.shape[-1] // 2:]
    r = 1.0 / (total * (1.0 / D) + EPS).sqrt()
    return ((x.to(F32) * r) * w).to(BF16).to(F32)


def _rotated(x, w, cos, sin, case):
    """x [B, S, H, D] with the norm (weights w or None) and the rotation of its first channels, in float32: one product is
    rounded, the other goes into the sum as it is."""
    x = x.to(F32) if w is None else _normed(x, w, case)
    rot = case["rot"]
    a, b = (x[..., 0:rot:2], x[..., 1:rot:2]) if case["interleaved"] else (x[..., : rot // 2], x[..., rot // 2: rot])
    y = (a.to(F64) * cos.to(F64) - (b * sin).to(F64)).to(F32), (b.to(F64) * cos.to(F64) + (a * sin).to(F64)).to(F32)
    turned = torch.stack(y, -1).flatten(-2) if case["interleaved"] else torch.cat(y, -1)
    return torch.cat((turned, x[..., rot:]), -1)


def _append(s):
    c = s["case"]
    if own:
        import video_dit_dense_gb300 as h3
        h3.h3attn_qk_norm_rope_append_q4(s["q"], s["k_new"], s["v_new"], s["q_out"], s["cache"], s["wq"], s["wk"], s["cos"],
                                         s["sin"], c["rot"], EPS, interleaved=c["interleaved"], new_len=s["new_len"],
                                         len_out=s["len_out"])
        # the new tokens as the cache holds them
        h3.h3attn_paged_read(s["grown"], s["k_out"], s["v_out"], first=s["kv_len"])
        return s["q_out"], s["k_out"], s["v_out"], s["len_out"]
    S, page = c["S"], c["page"]
    i = torch.arange(S, device="cuda")
    at = s["kv_len"][:, None].long() + i                                    # [B, S]: the token's place and position
    count = torch.full_like(s["kv_len"], S) if s["new_len"] is None else s["new_len"]
    new = (i < count[:, None])[..., None, None]
    cos, sin = s["cos"][at][:, :, None], s["sin"][at][:, :, None]
    row = s["table"].gather(1, at // page).long()
    k = _rotated(s["k_new"], s["wk"], cos, sin, c).to(BF16)
    out = []
    for held, rows, before in ((s["k"], k, s["k_out"]), (s["v"], s["v_new"], s["v_out"])):
        # what is past a sequence's new tokens stays as it is
        for there, fresh in zip(held, _in_4_bits(rows)):
            there[row, at % page] = torch.where(new, fresh, there[row, at % page])
        out.append(torch.where(new, _rows(held, row, at % page).to(BF16), before))
    q_out = torch.where(new, _rotated(s["q"], s["wq"], cos, sin, c).to(BF16), s["q_out"])
    return q_out, out[0], out[1], s["kv_len"] + count


def _read(s):
    c = s["case"]
    if own:
        import video_dit_dense_gb300 as h3
        return h3.h3attn_paged_read(s["cache"], s["k_out"], s["v_out"])
    at = torch.arange(c["S"], device="cuda")
    pages = s["table"][:, at // c["page"]].long()
    there = (at < s["kv_len"][:, None])[..., None, None]
    return tuple(torch.where(there, _rows(s[n], pages, at % c["page"]).to(BF16), s[n + "_out"]) for n in ("k", "v"))


def _decode(s):
    c = s["case"]
    if own:
        import video_dit_dense_gb300 as h3
        if c["weights"]:
            h3.h3attn_paged_decode_weights(s["q"], s["o"], s["cache"], s["weights"], s["workspace"])
        else:
            h3.h3attn_paged_decode_q4(s["q"], s["o"], s["cache"], workspace=s["workspace"])
        return s["o"], s["weights"]
    B, Hq, Hkv, D, page, most = c["B"], c["Hq"], c["Hkv"], c["D"], c["page"], c["high"]
    at = torch.arange(most, device="cuda")
    pages = s["table"][:, at // page].long()                                # [B, L]
    k = _rows(s["k"], pages, at % page)                                     # [B, L, Hkv, D]
    q = s["q"].to(F32).view(B, Hkv, Hq // Hkv, D)
    score = q @ k.permute(0, 2, 3, 1) / math.sqrt(D)                        # [B, Hkv, G, L]
    del k
    score = score.masked_fill(at >= s["kv_len"][:, None, None, None], -math.inf)
    top = score.amax(-1, keepdim=True)
    p = (score - top.masked_fill(top == -math.inf, 0.0)).exp()
    del score
    total = p.sum(-1, keepdim=True)
    total = total.masked_fill(total == 0, 1.0)
    v = _rows(s["v"], pages, at % page).permute(0, 2, 1, 3)                 # [B, Hkv, L, D]
    o = (p @ v) / total
    if c["weights"]:
        s["weights"][:, :most] += (p / total).sum((1, 2))
    return o.to(BF16).view(B, 1, Hq, D), s["weights"]


def _evict(s):
    c = s["case"]
    keep, recent, page = c["keep"], c["recent"], c["page"]
    s["weights"].copy_(s["sums"])  # what the steps since the last eviction have left there
    if own:
        import video_dit_dense_gb300 as h3
        h3.h3attn_paged_evict(s["cache"], s["weights"], keep, recent, s["len_out"], s["workspace"])
        return s["k"], s["v"], s["weights"], s["len_out"]
    n, most = s["kv_len"][:, None].long(), c["high"]
    j, front, long = torch.arange(most, device="cuda"), keep - recent, n > keep
    old = j < n - recent
    # of the older tokens the `front` heaviest, the first ones among equal ones
    order = s["weights"][:, :most].masked_fill(~old, -math.inf).sort(dim=-1, descending=True, stable=True)[1]
    rank = torch.empty_like(order).scatter_(1, order, j.expand_as(order))
    kept = old & (rank < front)
    # the i-th that is kept behind the border goes to the i-th gap in front of it
    mover, gap = kept & (j >= front), ~kept & (j < front)
    places = torch.where(mover, mover.cumsum(-1) - 1, most)
    movers = torch.zeros(c["B"], most + 1, dtype=torch.long, device="cuda").scatter_(1, places, j.expand_as(places))
    source = torch.where(gap, movers.gather(1, (gap.cumsum(-1) - 1).clamp(min=0)), j)[:, :keep]
    source = torch.where(j[:keep] < front, source, n - keep + j[:keep])       # the last ones in their order
    source = torch.where(long, source, j[:keep])
    row, to_row = s["table"].gather(1, source // page).long(), s["table"][:, j[:keep] // page].long()
    for held in s["k"] + s["v"]:
        held[to_row, j[:keep] % page] = held[row, source % page]
    moved = s["weights"].gather(1, source)
    s["weights"][:, :most].masked_fill_(long & (j >= keep) & (j < n), 0.0)
    s["weights"][:, :keep] = moved
    return s["k"], s["v"], s["weights"], s["kv_len"].clamp(max=keep)


# ---------------------------------------------------------------- what a pass cannot do without

def _row_bytes(case):
    """Of a token's key and value rows in the cache."""
    D = case["D"]
    return case["Hkv"] * (4 * D if case.get("bits", 4) == 16 else D + D // 8)


def work(case):
    op, B, Hkv, D = (case[n] for n in ("op", "B", "Hkv", "D"))
    if op == "append":
        S, Hq = case["S"], case["Hq"]
        tokens = ((B - 1) * S / 2 + S) if case["ragged"] else B * S
        # rows in, q and the cache's rows out, and those read back
        return dict(bytes=tokens * ((Hq + 2 * Hkv) * D * 2 + Hq * D * 2 + 2 * _row_bytes(case) + 2 * Hkv * D * 2 + case["rot"] * 4),
                    flops=tokens * (Hq + 2 * Hkv) * D * (7 if case["norm"] else 3))
    # lengths are spread evenly between low and high, and the last is high
    lengths = [case["low"] + (case["high"] - case["low"]) * (i + 0.5) / B for i in range(B - 1)] + [case["high"]]
    keys = sum(lengths)
    if op == "read":
        return dict(bytes=keys * (_row_bytes(case) + Hkv * D * 4), flops=keys * Hkv * D * 2)
    if op == "decode":
        Hq = case["Hq"]
        more = 8 if case["weights"] else 0
        return dict(bytes=keys * (_row_bytes(case) + more) + 2 * B * Hq * D * 2 + keys / case["page"] * 4, flops=4 * keys * Hq * D)
    keep, recent, moved = case["keep"], case["recent"], 0
    for n in lengths:
        if n > keep:  # of the older tokens an equal share is kept behind the border and in front of it
            moved += min(recent, n) + (n - keep) * (keep - recent) / max(n - recent, 1)
    return dict(bytes=8 * keys + moved * 2 * _row_bytes(case), flops=keys * 8)


# ---------------------------------------------------------------- the definitions, in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    return dict(append=_exact_append, read=_exact_read, decode=_exact_decode, evict=_exact_evict)[case["op"]](s, case)


def _scales_64(byte):
    """(8 + m) 2^(e - 18) of a byte with e above and m in its lower three bits; m 2^-17 where e is 0."""
    e, m = byte.long() >> 3, byte.long() & 7
    return torch.where(e == 0, m * 2, (8 + m) << e).to(F64) * 2.0 ** -18


def _values_64(held, rows, at):
    if len(held) == 1:
        return held[0][rows, at].to(F64)
    codes, s = held[0][rows, at].to(I32), _scales_64(held[1][rows, at])
    out = torch.empty(*codes.shape[:-1], 2 * codes.shape[-1], device="cuda", dtype=F64)
    out[..., 0::2], out[..., 1::2] = (codes % 16 - 8).to(F64), (torch.div(codes, 16, rounding_mode="floor") - 8).to(F64)
    return out * s.repeat_interleave(GROUP, -1)


def _held_64(x):
    """What the cache holds of rows x (bf16 values in float64)."""
    top = x.unflatten(-1, (-1, GROUP)).abs().amax(-1)
    all_scales = _scales_64(torch.arange(0xD8, device="cuda", dtype=U8))       # in order
    i = torch.searchsorted(7.0 * all_scales, top.contiguous()).clamp(1, len(all_scales) - 1)
    below, above = top - 7.0 * all_scales[i - 1], 7.0 * all_scales[i] - top
    i = i - ((below < above) | ((below == above) & (i % 2 == 1))).long()       # of two equally near ones the even byte
    s = all_scales[i].repeat_interleave(GROUP, -1)
    code = torch.where(s > 0, torch.sign(x) * torch.floor(x.abs() / s.clamp(min=2.0 ** -20) + 0.5), 0.0)
    return code.clamp(-8.0, 7.0) * s


def _exact_append(s, case):
    half, D = case["rot"] // 2, case["D"]
    first = torch.arange(half, device="cuda") * (2 if case["interleaved"] else 1)
    second = first + (1 if case["interleaved"] else half)

    def turn(x, w, at):
        x = x.to(F64)
        if w is not None:
            x = (x / (x.square().sum(-1, keepdim=True) / D + EPS).sqrt() * w.to(F64)).to(BF16).to(F64)
        z = torch.complex(x[..., first], x[..., second]) * torch.complex(s["cos"][at].to(F64), s["sin"][at].to(F64))[:, None]
        x = x.clone()
        x[..., first], x[..., second] = z.real, z.imag
        return x

    q_out, k_out, v_out, ends = s["q_out"].to(F64), s["k_out"].to(F64), s["v_out"].to(F64), []
    for b, n0 in enumerate(s["kv_len"].tolist()):
        n = case["S"] if s["new_len"] is None else int(s["new_len"][b])
        at = torch.arange(n0, n0 + n, device="cuda")
        q_out[b, :n] = turn(s["q"][b, :n], s["wq"], at)
        k_out[b, :n] = _held_64(turn(s["k_new"][b, :n], s["wk"], at).to(BF16).to(F64))
        v_out[b, :n] = _held_64(s["v_new"][b, :n].to(F64))
        ends.append(n0 + n)
    return q_out, k_out, v_out, torch.tensor(ends, dtype=I32, device="cuda")


def _exact_read(s, case):
    outs = s["k_out"].to(F64), s["v_out"].to(F64)
    for b, n in enumerate(s["kv_len"].tolist()):
        at = torch.arange(n, device="cuda")
        rows = s["table"][b].long()[torch.div(at, case["page"], rounding_mode="floor")]
        for out, name in zip(outs, ("k", "v")):
            out[b, :n] = _values_64(s[name], rows, at.remainder(case["page"]))
    return outs


def _exact_decode(s, case):
    B, Hq, Hkv, D, page = (case[n] for n in ("B", "Hq", "Hkv", "D", "page"))
    o = torch.zeros(B, 1, Hq, D, device="cuda", dtype=F64)
    weights = s["weights"].to(F64) if case["weights"] else None
    for b, n in enumerate(s["kv_len"].tolist()):
        if n == 0:
            continue
        at = torch.arange(n, device="cuda")
        rows = s["table"][b].long()[torch.div(at, page, rounding_mode="floor")]
        for h in range(Hkv):
            def one(held):
                return _values_64(tuple(t[:, :, h] for t in held), rows, at.remainder(page))
            heads = slice(h * (Hq // Hkv), (h + 1) * (Hq // Hkv))
            p = torch.softmax(s["q"][b, 0, heads].to(F64) @ one(s["k"]).T / D ** 0.5, -1)
            o[b, 0, heads] = p @ one(s["v"])
            if weights is not None:
                weights[b, :n] += p.sum(0)
    return o, weights


def _exact_evict(s, case):
    keep, recent, page = case["keep"], case["recent"], case["page"]
    weights, ends = s["sums"].to(F64), []
    for b, n in enumerate(s["kv_len"].tolist()):
        ends.append(min(n, keep))
        if n <= keep:
            continue
        front, w = keep - recent, weights[b, :n].clone()
        # by weight from above, then by place
        order = sorted(range(n - recent), key=w[: n - recent].neg().tolist().__getitem__)[:front]
        stay = set(order)
        gaps = [j for j in range(front) if j not in stay]
        goes = dict(zip(sorted(j for j in order if j >= front), gaps))
        goes.update({n - recent + i: front + i for i in range(recent)})
        src, dst = torch.tensor(list(goes), device="cuda"), torch.tensor(list(goes.values()), device="cuda")
        if len(goes):
            a, z = s["table"][b].long()[src // page], s["table"][b].long()[dst // page]
            for held in s["k"] + s["v"]:
                held[z, dst % page] = held[a, src % page]
            weights[b, dst] = w[src]
        weights[b, keep:n] = 0.0
    def plain(held):
        return tuple(t.to(F64) if t.dtype == BF16 else t for t in held)
    return plain(s["k"]), plain(s["v"]), weights, torch.tensor(ends, dtype=I32, device="cuda")
