"""Cases of the operators that take one step of generation through a transformer block: the sum with the
residual stream and its RMS norm, rotary tables, the rotated append to a paged key-value cache, and the attention of
one new token over that cache.

`run` computes them in their plain form, elementary torch operations in float32 (float64 for the angles), or, where
`own` is true, through the framework's entry points."""
import math

import torch

own = False

BF16, F32, F64, I32 = torch.bfloat16, torch.float32, torch.float64, torch.int32
E4M3, E8M0 = torch.float8_e4m3fn, torch.float8_e8m0fnu
E4M3_MAX = 448.0
EPS = 1e-6


def listed():
    return [
        # a single stream of generation right after a short prompt: launch and wait times count
        dict(name="decode_one_short", op="decode", B=1, Hq=16, Hkv=4, D=128, page=16, low=37, high=37),
        # a serving batch with four query heads to a key-value head, caches of unlike lengths
        dict(name="decode_batch_gqa", op="decode", B=16, Hq=16, Hkv=4, D=128, page=16, low=4096, high=8192),
        # many short requests of a small model, some of them new and still without keys; pages that are no power of two
        dict(name="decode_many_d64", op="decode", B=64, Hq=16, Hkv=2, D=64, page=24, low=0, high=2048),
        # one token against a packed clip's whole cache, as many key-value heads as query heads
        dict(name="decode_clip", op="decode", B=1, Hq=24, Hkv=24, D=128, page=64, low=104448, high=104448),
        # the new token of each request in a batch: norm, rotation of 96 of 128 channels, append
        dict(name="append_token", op="append", B=8, S=1, Hq=24, Hkv=8, D=128, page=16, rot=96, norm=True,
             interleaved=False, start=1000, ragged=False),
        # prompts of unlike length, padded to the longest, interleaved pairs, no norm
        dict(name="append_prompts", op="append", B=4, S=2048, Hq=16, Hkv=4, D=128, page=16, rot=128, norm=False,
             interleaved=True, start=100, ragged=True),
        # a long clip's rows into an empty cache
        dict(name="append_clip", op="append", B=1, S=32760, Hq=24, Hkv=24, D=128, page=64, rot=96, norm=True,
             interleaved=False, start=0, ragged=False),
        # the rotary rows of one frame's tokens, at given positions
        dict(name="table_frame", op="table", N=1536, rot=96, kind="none", factor=1.0, given=True),
        # a whole table for half a million positions, stretched by parts from 32760
        dict(name="table_long", op="table", N=524291, rot=128, kind="by_parts", factor=16.0, given=False),
        # one token of one request between two layers
        dict(name="norm_token", op="norm", T=1, C=5120, residual=True, out="bf16"),
        # a prompt before a product in 8 bits with a power-of-two scale for each 32 channels
        dict(name="norm_prompt_mx", op="norm", T=4099, C=4096, residual=True, out="mx"),
        # a long clip's hidden rows before a product in 8 bits with one scale a row
        dict(name="norm_clip_rows", op="norm", T=32760, C=5120, residual=True, out="row"),
    ]


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["decode", "append", "table", "norm"])
    if op == "decode":
        Hq, Hkv = rng.choice([(4, 4), (12, 12), (24, 24), (16, 4), (16, 2), (24, 8), (20, 4), (8, 1), (32, 1)])
        D = rng.choice([64, 128, 128, 256])
        B, page = _log(rng, 1, 64), rng.choice([16, 24, 32, 64, 128])
        most = max(1, min(104448, int(1.2e9 / (B * Hkv * D * 4))))
        high = _log(rng, 1, most)
        return dict(op=op, B=B, Hq=Hq, Hkv=Hkv, D=D, page=page, low=rng.choice([0, high // 2, high]), high=high)
    if op == "append":
        Hq, Hkv = rng.choice([(4, 4), (12, 12), (24, 24), (16, 4), (16, 2), (24, 8), (20, 4), (8, 1), (32, 1)])
        D = rng.choice([64, 128, 128, 256])
        tokens = _log(rng, 1, max(1, min(32760, int(1.0e9 / ((Hq + 2 * Hkv) * D * 4)))))
        B = min(tokens, _log(rng, 1, 64))
        return dict(op=op, B=B, S=tokens // B, Hq=Hq, Hkv=Hkv, D=D, page=rng.choice([16, 24, 32, 64, 128]),
                    rot=rng.choice([D, D // 2, 3 * D // 4, D // 2 + 2]), norm=rng.random() < 0.5,
                    interleaved=rng.random() < 0.5, start=_log(rng, 1, 4000) - 1, ragged=rng.random() < 0.5)
    if op == "table":
        kind = rng.choice(["none", "linear", "ntk", "by_parts"])
        return dict(op=op, N=_log(rng, 1, 524291), rot=rng.choice([32, 64, 96, 128, 46]), kind=kind,
                    factor=1.0 if kind == "none" else rng.choice([2.0, 4.0, 16.0]), given=rng.random() < 0.5)
    out = rng.choice(["bf16", "row", "mx"])
    C = 32 * rng.randint(4, 256) + (0 if out == "mx" else 8 * rng.randint(0, 3))
    return dict(op=op, T=_log(rng, 1, max(1, min(32760, int(1.1e9 / (7 * C))))), C=min(C, 8192), residual=rng.random() < 0.8,
                out=out)


# ---------------------------------------------------------------- inputs

def _lengths(case, g):
    """Cache lengths of a decode case: the longest is there, the others are spread."""
    n = torch.randint(case["low"], case["high"] + 1, (case["B"],), generator=g, device="cuda", dtype=I32)
    n[-1:] = case["high"]
    return n


def _pages(B, capacity, page, Hkv, D, g):
    """A cache of B sequences of up to `capacity` tokens, its pages in no order, with a few that nobody holds."""
    each = -(-capacity // page)
    total = B * each + 3
    k = torch.randn(total, page, Hkv, D, generator=g, device="cuda", dtype=BF16)
    v = torch.randn(total, page, Hkv, D, generator=g, device="cuda", dtype=BF16)
    table = torch.randperm(total, generator=g, device="cuda")[: B * each].to(I32).view(B, each)
    return k, v, table


def _prepare_decode(case, g):
    B, Hq, Hkv, D = (case[n] for n in ("B", "Hq", "Hkv", "D"))
    k, v, table = _pages(B, case["high"], case["page"], Hkv, D, g)
    k += 0.5 * torch.randn(Hkv, D, generator=g, device="cuda").to(BF16)  # an offset of each head: some keys stand out
    s = dict(k=k, v=v, table=table, kv_len=_lengths(case, g),
             q=torch.randn(B, 1, Hq, D, generator=g, device="cuda", dtype=BF16))
    s["o"] = torch.empty_like(s["q"])
    if own:
        import video_dit_dense_gb300 as h3
        s["cache"] = h3.PagedKV(k, v, table, s["kv_len"])
        s["workspace"] = h3.paged_decode_workspace(s["q"], s["cache"])
    return s


def _prepare_append(case, g):
    B, S, Hq, Hkv, D, rot = (case[n] for n in ("B", "S", "Hq", "Hkv", "D", "rot"))
    start = torch.randint(case["start"] // 2, case["start"] + 1, (B,), generator=g, device="cuda", dtype=I32)
    k_pages, v_pages, table = _pages(B, case["start"] + S, case["page"], Hkv, D, g)
    at = torch.arange(case["start"] + S, device="cuda", dtype=F64)[:, None]
    angle = at * 10000.0 ** (torch.arange(rot // 2, device="cuda", dtype=F64) * (-2.0 / rot))
    qkv = torch.randn(B, S, (Hq + 2 * Hkv) * D, generator=g, device="cuda", dtype=BF16)  # one projection's output
    q, k, v = (t.unflatten(-1, (-1, D)) for t in qkv.split([Hq * D, Hkv * D, Hkv * D], dim=-1))
    s = dict(q=q, k=k, v=v, k_pages=k_pages, v_pages=v_pages, table=table, kv_len=start,
             cos=angle.cos().to(F32), sin=angle.sin().to(F32), q_out=torch.zeros(B, S, Hq, D, device="cuda", dtype=BF16),
             len_out=torch.zeros_like(start), wq=None, wk=None, new_len=None)
    if case["norm"]:
        s["wq"] = torch.rand(D, generator=g, device="cuda") + 0.5
        s["wk"] = torch.rand(D, generator=g, device="cuda") + 0.5
    if case["ragged"]:
        s["new_len"] = torch.randint(0, S + 1, (B,), generator=g, device="cuda", dtype=I32)
        s["new_len"][-1:] = S
    if own:
        import video_dit_dense_gb300 as h3
        s["cache"] = h3.PagedKV(k_pages, v_pages, table, start)
    return s


def _prepare_table(case, g):
    N, rot = case["N"], case["rot"]
    s = dict(pos=None, first=0, cos=torch.empty(N, rot // 2, device="cuda"), sin=torch.empty(N, rot // 2, device="cuda"))
    if case["given"]:
        s["pos"] = torch.randint(0, 1 << 20, (N,), generator=g, device="cuda", dtype=I32)
    else:
        s["first"] = int(torch.randint(0, 4096, (1,), generator=g, device="cuda"))
    if own:
        import video_dit_dense_gb300 as h3
        s["scaling"] = None if case["kind"] == "none" else h3.RopeScaling(case["kind"], case["factor"], 32760, 1.0, 32.0,
                                                                          _amplitude(case))
    return s


def _prepare_norm(case, g):
    T, C = case["T"], case["C"]
    x = torch.randn(T, C, generator=g, device="cuda", dtype=BF16)
    s = dict(x=x, residual=None, h=None, w=torch.rand(C, generator=g, device="cuda") + 0.5, scale=None)
    if case["residual"]:
        # a residual stream has grown over the layers, and a few of its channels stand far out
        s["residual"] = torch.randn(T, C, generator=g, device="cuda", dtype=BF16) * 4
        s["residual"][:, torch.randint(0, C, (4,), generator=g, device="cuda")] *= 16
        s["h"] = torch.empty_like(x)
    s["y"] = torch.empty(T, C, device="cuda", dtype=BF16 if case["out"] == "bf16" else E4M3)
    if case["out"] == "row":
        s["scale"] = torch.empty(T, device="cuda")
    elif case["out"] == "mx":
        s["scale"] = torch.empty(T, C // 32, device="cuda", dtype=E8M0)
    return s


def prepare(case, seed):
    g = torch.Generator("cuda").manual_seed(seed)
    make = dict(decode=_prepare_decode, append=_prepare_append, table=_prepare_table, norm=_prepare_norm)[case["op"]]
    return dict(case=case, **make(case, g))


# ---------------------------------------------------------------- one pass

def run(state):
    return dict(decode=_decode, append=_append, table=_table, norm=_norm)[state["case"]["op"]](state)


def _decode(s):
    if own:
        import video_dit_dense_gb300 as h3
        return h3.h3attn_paged_decode(s["q"], s["o"], s["cache"], workspace=s["workspace"])
    c = s["case"]
    B, Hq, Hkv, D, page, most = c["B"], c["Hq"], c["Hkv"], c["D"], c["page"], c["high"]
    at = torch.arange(most, device="cuda")
    pages = s["table"][:, at // page].long()                                # [B, L]
    k = s["k"][pages, at % page].to(F32)                                    # [B, L, Hkv, D]
    q = s["q"].to(F32).view(B, Hkv, Hq // Hkv, D)
    score = q @ k.permute(0, 2, 3, 1) / math.sqrt(D)                        # [B, Hkv, G, L]
    del k
    score = score.masked_fill(at >= s["kv_len"][:, None, None, None], -math.inf)
    top = score.amax(-1, keepdim=True) if most else score.new_zeros(B, Hkv, Hq // Hkv, 1)
    p = (score - top.masked_fill(top == -math.inf, 0.0)).exp()
    total = p.sum(-1, keepdim=True)
    v = s["v"][pages, at % page].to(F32).permute(0, 2, 1, 3)                # [B, Hkv, L, D]
    o = (p @ v) / total.masked_fill(total == 0, 1.0)
    return o.to(BF16).view(B, 1, Hq, D)


def _rotated(x, w, cos, sin, case):
    """x [B, S, H, D] with the norm (weights w or None) and the rotation of its first channels, in float32."""
    x = x.to(F32)
    if w is not None:
        x = (x * (x.square().mean(-1, keepdim=True) + EPS).rsqrt() * w).to(BF16).to(F32)
    rot = case["rot"]
    if case["interleaved"]:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        turned = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
    else:
        a, b = x[..., : rot // 2], x[..., rot // 2: rot]
        turned = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
    return torch.cat((turned, x[..., rot:]), -1)


def _append(s):
    c = s["case"]
    if own:
        import video_dit_dense_gb300 as h3
        h3.h3attn_qk_norm_rope_append(s["q"], s["k"], s["v"], s["q_out"], s["cache"], s["wq"], s["wk"], s["cos"], s["sin"],
                                      c["rot"], EPS, interleaved=c["interleaved"], new_len=s["new_len"],
                                      len_out=s["len_out"])
        return s["q_out"], s["k_pages"], s["v_pages"], s["len_out"]
    B, S, page = c["B"], c["S"], c["page"]
    i = torch.arange(S, device="cuda")
    at = s["kv_len"][:, None].long() + i                                    # [B, S]: the token's place and position
    count = torch.full_like(s["kv_len"], S) if s["new_len"] is None else s["new_len"]
    new = (i < count[:, None])[..., None, None]
    cos, sin = s["cos"][at][:, :, None], s["sin"][at][:, :, None]
    row = s["table"].gather(1, at // page).long()
    k = _rotated(s["k"], s["wk"], cos, sin, c).to(BF16)
    # what is past a sequence's new tokens stays as it is
    s["k_pages"][row, at % page] = torch.where(new, k, s["k_pages"][row, at % page])
    s["v_pages"][row, at % page] = torch.where(new, s["v"], s["v_pages"][row, at % page])
    q_out = torch.where(new, _rotated(s["q"], s["wq"], cos, sin, c).to(BF16), s["q_out"])
    return q_out, s["k_pages"], s["v_pages"], s["kv_len"] + count


def _amplitude(case):
    """Stretching by parts sharpens the scores by this factor, on the queries' and on the keys' side."""
    return 0.1 * math.log(case["factor"]) + 1.0 if case["kind"] == "by_parts" else 1.0


def _frequencies(case):
    """Radians a position, [rot / 2] in float64."""
    rot, kind, f = case["rot"], case["kind"], case["factor"]
    theta = 10000.0 * f ** (rot / (rot - 2.0)) if kind == "ntk" else 10000.0
    freq = theta ** (torch.arange(rot // 2, device="cuda", dtype=F64) * (-2.0 / rot))
    if kind == "linear":
        return freq / f
    if kind == "by_parts":
        turns = 32760 * freq / (2 * math.pi)
        keep = ((turns - 1.0) / (32.0 - 1.0)).clamp(0.0, 1.0)
        return (1 - keep) * (freq / f) + keep * freq
    return freq


def _table(s):
    c = s["case"]
    if own:
        import video_dit_dense_gb300 as h3
        return h3.h3attn_rope_table(s["cos"], s["sin"], c["rot"], 10000.0, s["scaling"], s["pos"], s["first"])
    at = s["pos"] if s["pos"] is not None else torch.arange(s["first"], s["first"] + c["N"], device="cuda")
    angle = at.to(F64)[:, None] * _frequencies(c)
    return (angle.cos() * _amplitude(c)).to(F32), (angle.sin() * _amplitude(c)).to(F32)


def _norm(s):
    c = s["case"]
    if own:
        import video_dit_dense_gb300 as h3
        h3.h3attn_add_rmsnorm(s["x"], s["residual"], s["h"], s["y"], s["w"], EPS, s["scale"])
        return s["h"], s["y"], s["scale"]
    h = s["x"] if s["residual"] is None else (s["x"].to(F32) + s["residual"].to(F32)).to(BF16)
    y = h.to(F32)
    y = y * (y.square().mean(-1, keepdim=True) + EPS).rsqrt() * s["w"]
    h = None if s["residual"] is None else h
    if c["out"] == "bf16":
        return h, y.to(BF16), None
    if c["out"] == "row":
        scale = y.abs().amax(-1) / E4M3_MAX
        scale = scale.masked_fill(scale == 0, 1.0)
        return h, (y / scale[:, None]).clamp(-E4M3_MAX, E4M3_MAX).to(E4M3), scale
    y = y.unflatten(-1, (-1, 32))
    part, power = torch.frexp(y.abs().amax(-1) / E4M3_MAX)      # amax / 448 = part * 2^power with 0.5 <= part < 1
    power = torch.where(part == 0.5, power - 1, power).masked_fill(part == 0, 0)  # the least power of two that is not below
    scale = torch.exp2(power.to(F32))
    return h, (y / scale[..., None]).to(E4M3).flatten(-2), scale.to(E8M0)


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    op = case["op"]
    if op == "decode":
        B, Hq, Hkv, D = (case[n] for n in ("B", "Hq", "Hkv", "D"))
        # lengths are spread evenly between low and high, and the last is high
        keys = (B - 1) * (case["low"] + case["high"]) / 2 + case["high"]
        return dict(bytes=keys * Hkv * D * 4 + 2 * B * Hq * D * 2 + keys / case["page"] * 4, flops=4 * keys * Hq * D)
    if op == "append":
        B, S, Hq, Hkv, D = (case[n] for n in ("B", "S", "Hq", "Hkv", "D"))
        tokens = ((B - 1) * S / 2 + S) if case["ragged"] else B * S
        rows = tokens * (Hq + 2 * Hkv)
        return dict(bytes=rows * D * 4 + tokens * case["rot"] * 4, flops=rows * D * (7 if case["norm"] else 3))
    if op == "table":
        return dict(bytes=case["N"] * (case["rot"] * 4 + (4 if case["given"] else 0)), flops=case["N"] * case["rot"] * 20)
    T, C, out = case["T"], case["C"], case["out"]
    each = (2 + (4 if case["residual"] else 0) + (2 if out == "bf16" else 1)) * C + dict(bf16=0, row=4, mx=C // 32)[out]
    return dict(bytes=T * each + 4 * C, flops=T * C * 6)


# ---------------------------------------------------------------- the definitions, in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    return dict(decode=_exact_decode, append=_exact_append, table=_exact_table, norm=_exact_norm)[case["op"]](s, case)


def _exact_decode(s, case):
    B, Hq, Hkv, D, page = (case[n] for n in ("B", "Hq", "Hkv", "D", "page"))
    o = torch.zeros(B, 1, Hq, D, device="cuda", dtype=F64)
    for b, n in enumerate(s["kv_len"].tolist()):
        if n == 0:
            continue
        mine = s["table"][b, : -(-n // page)].long()
        for h in range(Hkv):
            keys = s["k"][mine, :, h].reshape(-1, D)[:n].to(F64)
            values = s["v"][mine, :, h].reshape(-1, D)[:n].to(F64)
            heads = slice(h * (Hq // Hkv), (h + 1) * (Hq // Hkv))
            o[b, 0, heads] = torch.softmax(s["q"][b, 0, heads].to(F64) @ keys.T / D ** 0.5, -1) @ values
    return o


def _exact_append(s, case):
    page, half, D = case["page"], case["rot"] // 2, case["D"]
    q_out, k_pages, v_pages = s["q_out"].to(F64), s["k_pages"].to(F64), s["v_pages"].to(F64)
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

    ends = []
    for b, n0 in enumerate(s["kv_len"].tolist()):
        n = case["S"] if s["new_len"] is None else int(s["new_len"][b])
        at = torch.arange(n0, n0 + n, device="cuda")
        rows = s["table"][b].long()[torch.div(at, page, rounding_mode="floor")], at.remainder(page)
        q_out[b, :n] = turn(s["q"][b, :n], s["wq"], at)
        k_pages[rows] = turn(s["k"][b, :n], s["wk"], at)
        v_pages[rows] = s["v"][b, :n].to(F64)
        ends.append(n0 + n)
    return q_out, k_pages, v_pages, torch.tensor(ends, dtype=I32, device="cuda")


def _exact_table(s, case):
    rot, f, kind = case["rot"], case["factor"], case["kind"]
    theta = 10000.0 * (f ** (rot / (rot - 2.0)) if kind == "ntk" else 1.0)
    freq = []
    for i in range(rot // 2):
        w = math.pow(theta, -2.0 * i / rot)
        turns = 32760 * w / (2 * math.pi)
        share = dict(none=1.0, ntk=1.0, linear=0.0, by_parts=min(1.0, max(0.0, (turns - 1.0) / 31.0)))[kind]
        freq.append(w * share + w / f * (1.0 - share))
    at = torch.arange(case["N"], device="cuda") + s["first"] if s["pos"] is None else s["pos"]
    m = 1.0 + 0.1 * math.log(f) if kind == "by_parts" else 1.0
    z = torch.polar(torch.full((case["N"], rot // 2), m, device="cuda", dtype=F64),
                    torch.outer(at.to(F64), torch.tensor(freq, device="cuda", dtype=F64)))
    return z.real.contiguous(), z.imag.contiguous()


def _exact_norm(s, case):
    h = s["x"].to(F64)
    if s["residual"] is not None:
        h = (h + s["residual"].to(F64)).to(BF16).to(F64)  # the stream is kept in bf16, and its norm is that of what is kept
    y = h / torch.linalg.vector_norm(h, dim=-1, keepdim=True).square().div(case["C"]).add(EPS).sqrt() * s["w"].to(F64)
    h = None if s["residual"] is None else h
    if case["out"] == "bf16":
        return h, y, None
    grouped = y if case["out"] == "row" else y.view(case["T"], -1, 32)
    scale = grouped.abs().max(-1, keepdim=True).values / E4M3_MAX
    if case["out"] == "mx":
        scale = torch.pow(2.0, torch.ceil(torch.log2(scale)))
    scale = torch.where(scale > 0, scale, torch.ones_like(scale))
    # the values that the 8 bits stand for, beside their scales
    return h, (grouped / scale).to(F32).to(E4M3).to(F64).view_as(y), scale.squeeze(-1)
