"""The append where a warp takes several turns over the heads of its tokens: large
calls, which the small cases beside these never are.  Chosen by the launcher's own
rule so that a warp walks from query over key to value heads, with 1, 2 and 4
heads of a token at a time and with a last part that is shorter than the others.
Sampled tokens are compared bit for bit with the reference, all rows bit for bit
with the same tokens appended in calls of one turn, and rows that nobody appended
have to stay."""
import numpy as np
import pytest
import torch

from test_gpu_append import bits, reference

UNROLL, WARPS_PER_SM = 2, 32


def plan(tokens, Hq, Hkv, D, sms):
    """(heads of a token at a time, turns of a warp, parts, heads of the last part) as the launcher takes them."""
    heads, rows = Hq + 2 * Hkv, 512 // D
    log2 = min(2 if heads >= 48 else 1 if heads >= 16 else 0, 1 if rows == 2 else 2)
    batch = UNROLL << log2
    most = -(-heads // batch)
    warps = -(-tokens // (rows >> log2))
    waves = warps / (sms * WARPS_PER_SM)
    least, best, turns = float("inf"), most, most
    while turns >= 1:
        cost = max(waves * -(-most // turns) + 0.5, 1.0) * (turns + 0.5)
        if cost < least:
            least, best = cost, turns
        turns = min(turns - 1, 32)
    parts = -(-heads // (best * batch))
    return 1 << log2, best, parts, heads - (parts - 1) * best * batch


def tokens_for(want, Hq, Hkv, D):
    """The fewest tokens whose plan is wanted."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    n = 1024
    while n < 80000:
        if want(*plan(n, Hq, Hkv, D, sms)):
            return n
        n += 97
    raise AssertionError("no size has this plan")


def test_sizes_of_every_plan():
    """With 152 SMs: the shapes below reach several turns, in one part and in several, with a short last one."""
    for Hq, Hkv, D in ((6, 2, 64), (16, 4, 128), (24, 24, 128), (24, 24, 64), (12, 12, 256)):
        plans = [plan(n, Hq, Hkv, D, 152) for n in range(1024, 80000, 97)]
        assert any(t >= 2 and parts == 1 for _, t, parts, _ in plans), (Hq, Hkv, D)
    assert {plan(50000, Hq, Hkv, 64, 152)[0] for Hq, Hkv in ((6, 2), (16, 4), (24, 24))} == {1, 2, 4}
    for Hq, Hkv, D in ((32, 1, 128), (7, 7, 64), (9, 3, 256)):
        assert any(t >= 2 and parts >= 2 and last < t * UNROLL * h
                   for h, t, parts, last in (plan(n, Hq, Hkv, D, 152) for n in range(1024, 80000, 97))), (Hq, Hkv, D)


class Big:
    """Two sequences of unlike lengths in one padded batch, pages of 24 tokens, on the GPU."""

    def __init__(self, tokens, Hq, Hkv, D, rot, interleaved, norm, ragged, seed=0):
        S = -(-tokens // 2)
        self.S, self.Hq, self.Hkv, self.D, self.rot, self.interleaved = S, Hq, Hkv, D, rot, interleaved
        g = torch.Generator("cuda").manual_seed(seed)
        qkv = torch.randn(2, S, (Hq + 2 * Hkv) * D, generator=g, device="cuda").to(torch.bfloat16)
        self.src = [t.unflatten(-1, (-1, D)) for t in qkv.split([Hq * D, Hkv * D, Hkv * D], dim=-1)]
        self.start, self.new = [5, 31], [S, S - S // 3 if ragged else S]
        self.kv_len = torch.tensor(self.start, dtype=torch.int32, device="cuda")
        self.new_len = torch.tensor(self.new, dtype=torch.int32, device="cuda") if ragged else None
        self.page, each = 24, -(-(S + 31) // 24)
        order = torch.randperm(2 * each + 3, generator=torch.Generator().manual_seed(seed))
        self.table = order[:2 * each].to(torch.int32).view(2, each).cuda()
        self.pages = 2 * each + 3
        rows = S + 31
        angle = torch.arange(rows, device="cuda")[:, None].double() * 10000.0 ** (torch.arange(rot // 2, device="cuda") * (-2.0 / rot))
        self.cos, self.sin = angle.cos().float(), angle.sin().float()
        self.wq = self.wk = None
        if norm:
            self.wq, self.wk = (torch.rand(D, generator=g, device="cuda") + 0.5 for _ in range(2))

    def outputs(self):
        d = dict(dtype=torch.bfloat16, device="cuda")
        return (torch.full((2, self.S, self.Hq, self.D), 3.0, **d), torch.full((self.pages, self.page, self.Hkv, self.D), 5.0, **d),
                torch.full((self.pages, self.page, self.Hkv, self.D), 7.0, **d))

    def call(self, h3, src, q_out, k_pages, v_pages, table, kv_len, new_len, len_out=None):
        cache = h3.PagedKV(k_pages, v_pages, table, kv_len)
        h3.h3attn_qk_norm_rope_append(*src, q_out, cache, self.wq, self.wk, self.cos, self.sin, self.rot, 1e-6, self.interleaved,
                                      None, new_len, len_out)

    def in_small_calls(self, h3):
        """The same tokens, at most 512 a call."""
        q_out, k_pages, v_pages = self.outputs()
        sms = torch.cuda.get_device_properties(0).multi_processor_count
        assert plan(512, self.Hq, self.Hkv, self.D, sms)[1] == 1
        for b in range(2):
            for s in range(0, self.new[b], 512):
                e = min(s + 512, self.new[b])
                self.call(h3, [t[b:b + 1, s:e] for t in self.src], q_out[b:b + 1, s:e], k_pages, v_pages, self.table[b:b + 1],
                          torch.tensor([self.start[b] + s], dtype=torch.int32, device="cuda"), None)
        return q_out, k_pages, v_pages

    def check_sampled(self, q_out, k_pages, v_pages):
        """Against the reference, every head of a few dozen tokens."""
        cpu = dict(w=None if self.wq is None else (self.wq.cpu(), self.wk.cpu()), cos=self.cos.cpu(), sin=self.sin.cpu())
        for b in range(2):
            at = np.unique(np.concatenate([np.arange(9), np.linspace(0, self.new[b] - 1, 23).astype(int),
                                           np.arange(self.new[b] - 9, self.new[b])]))
            places = at + self.start[b]
            where = self.table[b].cpu()[places // self.page].long(), torch.from_numpy(places % self.page)
            src = [t[b].cpu()[at] for t in self.src]
            for i, got in ((0, q_out[b].cpu()[at]), (1, k_pages[where[0].cuda(), where[1].cuda()])):
                want = reference(src[i], None if cpu["w"] is None else cpu["w"][i], cpu["cos"], cpu["sin"], places, self.rot,
                                 self.interleaved, 1e-6)
                assert np.array_equal(bits(got), want), (b, "qk"[i])
            assert np.array_equal(bits(v_pages[where[0].cuda(), where[1].cuda()]), bits(src[2])), (b, "v")


def same(a, b):
    return all(torch.equal(x.view(torch.int16), y.view(torch.int16)) for x, y in zip(a, b))


@pytest.mark.gpu
@pytest.mark.parametrize("D,rot,interleaved", [(64, 48, False), (64, 34, False), (64, 64, True), (128, 96, False), (128, 66, False),
                                               (128, 66, True), (256, 192, False), (256, 130, False), (256, 256, True)])
@pytest.mark.parametrize("Hq,Hkv,ragged,norm", [(6, 2, True, True), (16, 4, False, False), (16, 4, True, True), (24, 24, True, True)])
def test_several_turns(h3, Hq, Hkv, ragged, norm, D, rot, interleaved):
    if D == 256 and Hkv == 24:
        Hq = Hkv = 12
    tokens = tokens_for(lambda h, turns, parts, last: turns >= 2 and (parts >= 2 or Hq < 12), Hq, Hkv, D)
    c = Big(tokens, Hq, Hkv, D, rot, interleaved, norm, ragged, seed=tokens)
    outs, lens = c.outputs(), torch.full((2,), -1, dtype=torch.int32, device="cuda")
    c.call(h3, c.src, *outs, c.table, c.kv_len, c.new_len, lens)
    assert h3.h3attn_check_device_status() == 0
    assert lens.tolist() == [s + n for s, n in zip(c.start, c.new)]
    c.check_sampled(*outs)
    assert same(outs, c.in_small_calls(h3))


@pytest.mark.gpu
@pytest.mark.parametrize("Hq,Hkv,D,rot", [(24, 24, 128, 96), (24, 24, 64, 34), (16, 4, 128, 96), (6, 2, 64, 48), (12, 12, 256, 130)])
def test_every_head_of_a_token_in_one_warp(h3, Hq, Hkv, D, rot):
    """So many tokens that the heads are not cut: the most turns there are."""
    tokens = tokens_for(lambda h, turns, parts, last: parts == 1 and turns >= 2, Hq, Hkv, D)
    c = Big(tokens, Hq, Hkv, D, rot, False, True, True, seed=3)
    outs = c.outputs()
    c.call(h3, c.src, *outs, c.table, c.kv_len, c.new_len)
    c.check_sampled(*outs)
    assert same(outs, c.in_small_calls(h3))


@pytest.mark.gpu
@pytest.mark.parametrize("Hq,Hkv,D,rot", [(32, 1, 128, 96), (7, 7, 64, 34), (9, 3, 256, 130)])
def test_a_short_last_part(h3, Hq, Hkv, D, rot):
    tokens = tokens_for(lambda h, turns, parts, last: turns >= 2 and parts >= 2 and last < turns * UNROLL * h, Hq, Hkv, D)
    c = Big(tokens, Hq, Hkv, D, rot, False, True, True, seed=4)
    outs = c.outputs()
    c.call(h3, c.src, *outs, c.table, c.kv_len, c.new_len)
    c.check_sampled(*outs)
    assert same(outs, c.in_small_calls(h3))


@pytest.mark.gpu
@pytest.mark.parametrize("Hq,Hkv,D,rot,interleaved", [(24, 24, 128, 96, False), (16, 4, 64, 34, False), (16, 4, 128, 128, True)])
def test_queries_in_place(h3, Hq, Hkv, D, rot, interleaved):
    tokens = tokens_for(lambda h, turns, parts, last: turns >= 2, Hq, Hkv, D)
    c = Big(tokens, Hq, Hkv, D, rot, interleaved, True, True, seed=5)
    c.src = [t.contiguous() for t in c.src]
    before = c.src[0].clone()
    outs = c.outputs()
    c.call(h3, c.src, *outs, c.table, c.kv_len, c.new_len)
    other = c.outputs()
    c.call(h3, c.src, c.src[0], *other[1:], c.table, c.kv_len, c.new_len)
    outs[0][1, c.new[1]:] = before[1, c.new[1]:]          # padding keeps what it was
    assert same(outs, (c.src[0], *other[1:]))


@pytest.mark.gpu
def test_no_queries(h3):
    """Keys and values alone: the walk begins with the key heads."""
    tokens = tokens_for(lambda h, turns, parts, last: turns >= 2, 0, 24, 128)
    c = Big(tokens, 0, 24, 128, 96, False, True, False, seed=6)
    c.src[0], c.wq = None, None
    _, k_pages, v_pages = c.outputs()
    c.call(h3, c.src, None, k_pages, v_pages, c.table, c.kv_len, None)
    both = Big(tokens, 0, 24, 128, 96, False, True, False, seed=6)
    places = torch.arange(c.S, device="cuda")
    for b in range(2):
        at = places + c.start[b]
        k = both.src[1][b:b + 1].contiguous()
        want = torch.empty_like(k)
        h3.h3attn_qk_norm_rope_out(None, k, None, want, None, c.wk, c.cos[c.start[b]:].contiguous(),
                                   c.sin[c.start[b]:].contiguous(), 96, 1e-6)
        where = c.table[b][at // c.page].long(), at % c.page
        assert torch.equal(k_pages[where].view(torch.int16), want[0].view(torch.int16))
        assert torch.equal(v_pages[where].view(torch.int16), both.src[2][b].view(torch.int16))
