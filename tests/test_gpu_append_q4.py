"""The append to a cache in 4 bits: codes and scales bit for bit those of the
rows that the bf16 append stores, in every layout, at ties, outside the scales'
range, with rows that are not there, and nothing written beside them."""
import pytest
import torch

from cache4_ref import store
from generate_ref import randn


class Step:
    """New tokens of B sequences, both caches, filled with a pattern."""

    def __init__(self, B, S, Hq, Hkv, D, page, start, seed=0, scale=1.0, capacity=None):
        self.B, self.S, self.page = B, S, page
        capacity = max(start) + S if capacity is None else capacity
        each = -(-capacity // page)
        self.total = B * each + 2
        self.table = torch.randperm(self.total, generator=torch.Generator().manual_seed(seed))[: B * each].int().view(B, each)
        self.qkv = randn(B, S, Hq + 2 * Hkv, D, seed=seed + 1, scale=scale)
        self.Hq, self.Hkv, self.D, self.start = Hq, Hkv, D, list(start)

    def run(self, h3, rot=96, norm=True, interleaved=False, new_len=None, pos=None, rows=None, fill=0x5A):
        Hq, Hkv, D = self.Hq, self.Hkv, self.D
        dev = self.qkv.cuda()
        q, k, v = dev.split([Hq, Hkv, Hkv], dim=2)
        g = torch.Generator().manual_seed(9)
        wq, wk = ((torch.rand(D, generator=g) + 0.5).cuda() if norm else None for _ in range(2))
        rows = max(self.start) + self.S if rows is None else rows
        cos, sin = torch.empty(rows, rot // 2, device="cuda"), torch.empty(rows, rot // 2, device="cuda")
        if rot:
            h3.h3attn_rope_table(cos, sin, rot)
        lens = torch.tensor(self.start, dtype=torch.int32, device="cuda")
        new = None if new_len is None else torch.tensor(new_len, dtype=torch.int32, device="cuda")
        shape = (self.total, self.page, Hkv)
        self.pages = [torch.full((*shape, D), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
        self.q4 = [torch.full((*shape, D // n), fill, dtype=torch.uint8, device="cuda") for n in (2, 2, 16, 16)]
        table = self.table.cuda()
        outs = []
        for kind in (16, 4):
            cache = h3.PagedKV(*self.pages, table, lens) if kind == 16 else h3.PagedKV4(*self.q4, table, lens)
            q_out = torch.full((self.B, self.S, Hq, D), 3.0, dtype=torch.bfloat16, device="cuda") if Hq else None
            end = torch.full_like(lens, -7)
            call = h3.h3attn_qk_norm_rope_append if kind == 16 else h3.h3attn_qk_norm_rope_append_q4
            assert call(q if Hq else None, k, v, q_out, cache, wq if Hq else None, wk, cos if rot else None, sin if rot else None,
                        rot, 1e-6, interleaved, pos, new, end) is q_out
            outs.append((q_out, end))
        torch.cuda.synchronize()
        (q16, e16), (q4, e4) = outs
        assert torch.equal(e16, e4) and (q16 is None or torch.equal(q16.view(torch.int16), q4.view(torch.int16)))
        return self

    def check(self, written, fill=0x5A):
        """written: (b, place) of the tokens that were stored."""
        want = [torch.full(t.shape, fill, dtype=torch.uint8) for t in self.q4]
        for b, j in written:
            row = (int(self.table[b, j // self.page]), j % self.page)
            for i in range(2):
                want[i][row], want[2 + i][row] = store(self.pages[i][row].cpu())
        for name, got, ref in zip(("k codes", "v codes", "k scales", "v scales"), self.q4, want):
            assert torch.equal(got.cpu(), ref), name


def all_of(start, S):
    return [(b, n + s) for b, n in enumerate(start) for s in range(S)]


@pytest.mark.gpu
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("Hq,Hkv", [(4, 2), (24, 8), (1, 1), (0, 3), (8, 1)])
@pytest.mark.parametrize("rot_of,interleaved", [(1, False), (0.75, False), (0.5, True), (0, False), ("+2", False), ("+2", True),
                                                ("odd", False)])
def test_layouts(h3, D, Hq, Hkv, rot_of, interleaved):
    rot = D // 2 + 2 if rot_of == "+2" else D // 2 + 16 if rot_of == "odd" else int(D * rot_of)
    s = Step(2, 5, Hq, Hkv, D, 16, [3, 30], seed=D + Hq).run(h3, rot, interleaved=interleaved)
    s.check(all_of([3, 30], 5))
    assert h3.h3attn_check_device_status() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("size", [1e-30, 2.0 ** -19, 2e-5, 3e-4, 1e-2, 60.0, 2e4, 1e6, 1e37])
def test_sizes_of_values(h3, size):
    Step(1, 40, 2, 2, 128, 24, [0], seed=3, scale=size).run(h3, 0, norm=False).check(all_of([0], 40))


@pytest.mark.gpu
def test_ties_of_scales_and_codes(h3):
    """Maxima 7 m with m half way between two scales, and values half way between two codes."""
    s = Step(1, 64, 1, 1, 64, 16, [0], seed=4)
    x = torch.zeros(64, 64)
    for i in range(64):
        s_of = (8 + i % 8 + (0.5 if i % 3 == 0 else 0)) * 2.0 ** (i // 8 - 12)
        x[i] = (torch.arange(64) % 16 - 7.5) * (8 + i % 8) * 2.0 ** (i // 8 - 12)
        x[i, ::16] = 7 * s_of
    s.qkv = x.to(torch.bfloat16).view(1, 64, 1, 64).repeat(1, 1, 3, 1)
    s.run(h3, 0, norm=False).check(all_of([0], 64))


@pytest.mark.gpu
def test_not_finite_stays_in_its_group(h3):
    s = Step(1, 6, 1, 2, 128, 16, [0], seed=5)
    s.qkv[0, 1, 2, 5] = float("nan")
    s.qkv[0, 2, 1, 100] = float("inf")
    s.qkv[0, 3, 3, 127] = -float("inf")
    s.qkv[0, 4, 4, :] = -0.0
    s.run(h3, 0, norm=False).check(all_of([0], 6))


@pytest.mark.gpu
def test_padding_bad_pages_and_positions(h3):
    """Tokens that are not new, that have no page, or whose position has no table row."""
    s = Step(4, 7, 2, 2, 128, 4, [0, 5, 2, -3], seed=6, capacity=16)
    s.table[1, 2] = -1                                     # places 8 to 11 of sequence 1
    s.table[2, 0] = s.total
    s.run(h3, 96, new_len=[7, 6, 0, 100], rows=9)
    assert h3.h3attn_check_device_status() == h3.H3ATTN_ERR_INVALID_ARG
    written = [(0, j) for j in range(7)] + [(1, j) for j in (5, 6, 7)] + [(3, j) for j in range(7)]
    s.check(written)


@pytest.mark.gpu
def test_capacity_positions_and_many_tokens(h3):
    s = Step(1, 6, 2, 1, 64, 8, [4], seed=7, capacity=8).run(h3, 64)     # two places beyond the capacity
    assert h3.h3attn_check_device_status() == h3.H3ATTN_ERR_INVALID_ARG
    s.check([(0, j) for j in range(4, 8)])
    pos = torch.tensor([[5, 0, 3], [1, 1, 2]], dtype=torch.int32, device="cuda")
    Step(2, 3, 2, 2, 128, 8, [4, 1], seed=8).run(h3, 96, pos=pos).check(all_of([4, 1], 3))
    Step(3, 700, 8, 4, 128, 24, [0, 100, 17], seed=9).run(h3, 96).check(all_of([0, 100, 17], 700))
    assert h3.h3attn_check_device_status() == 0


@pytest.mark.gpu
def test_codes_past_32_bits(h3):
    """Pages that begin past 2^31 bytes of codes."""
    page, Hkv, D = 64, 16, 256
    pages = (1 << 32) // (page * Hkv * D) * 2 + 3
    dev = dict(dtype=torch.uint8, device="cuda")
    held = [torch.empty(pages, page, Hkv, D // n, **dev) for n in (2, 2, 16, 16)]
    table = torch.tensor([[pages - 1, pages - 2]], dtype=torch.int32, device="cuda")
    lens = torch.tensor([60], dtype=torch.int32, device="cuda")
    kv = randn(2, 1, 9, Hkv, D, seed=2)
    cache = h3.PagedKV4(*held, table, lens)
    end = torch.empty_like(lens)
    h3.h3attn_qk_norm_rope_append_q4(None, kv[0].cuda(), kv[1].cuda(), None, cache, None, None, None, None, 0, len_out=end)
    for i in range(2):
        codes, scales = store(kv[i, 0])
        assert torch.equal(held[i][pages - 1, 60:].cpu(), codes[:4]) and torch.equal(held[i][pages - 2, :5].cpu(), codes[4:])
        assert torch.equal(held[2 + i][pages - 1, 60:].cpu(), scales[:4])
    out = torch.zeros(2, 1, 9, Hkv, D, dtype=torch.bfloat16, device="cuda")
    h3.h3attn_paged_read(cache.with_lengths(end), out[0], out[1], first=lens)
    from cache4_ref import values
    assert torch.equal(out.double().cpu()[0, 0], values(*store(kv[0, 0])))
    assert torch.equal(out.double().cpu()[1, 0], values(*store(kv[1, 0])))
