"""GPU parity of the decode attention over a cache in 4 bits, and of the tokens'
weights over both caches, against float64 with the bounds that their roundings
allow (cache4_ref.attend): lengths around tiles and pages, empty sequences,
poisoned rows and pages, group sizes, split and unsplit."""
import pytest
import torch

from cache4_ref import Pages, attend
from generate_ref import poison_past, randn


class Case:
    def __init__(self, lens, Hq, Hkv, D, page, capacity=None, seed=0, peak=0.0, poison=True, scale=None, bits=4, q_scale=1.0):
        B = len(lens)
        self.lens, self.page, self.bits = list(lens), page, bits
        capacity = max([1] + [n for n in lens]) if capacity is None else capacity
        self.p = Pages(bits, B, capacity, page, Hkv, D, seed)
        self.q = randn(B, Hq, D, seed=seed + 7, scale=q_scale)
        self.scale = D ** -0.5 if scale is None else scale
        if peak:
            self.p.k += peak * randn(Hkv, D, seed=seed + 8)
        if poison:
            poison_past(self.p.k, self.p.v, self.p.table, lens, page)

    def cuda(self, h3):
        self.cache = self.p.hold().cuda(h3, self.lens)
        self.dq = self.q.cuda()
        room = self.p.table.shape[1] * self.page
        self.before = torch.rand(len(self.lens), room, generator=torch.Generator().manual_seed(5))
        return self

    def reference(self, skip=None):
        return attend(self.q, self.p.kv, self.p.table, self.lens, self.page, self.scale, skip, self.bits)

    def run(self, h3, split=True, stream=None):
        ws = h3.paged_decode_q4_workspace(self.dq, self.cache) if split else None
        if ws is not None:
            ws.fill_(0xFF)  # NaN in every float: contents on entry do not matter
        o = torch.full_like(self.dq, float("nan"))
        if stream is not None:
            stream.wait_stream(torch.cuda.current_stream())
        assert h3.h3attn_paged_decode_q4(self.dq, o, self.cache, self.scale, ws, stream) is o
        torch.cuda.synchronize()
        return o

    def run_weights(self, h3, stream=None):
        ws = h3.paged_decode_weights_workspace(self.dq, self.cache)
        ws.fill_(0xFF)
        o, w = torch.full_like(self.dq, float("nan")), self.before.cuda()
        if stream is not None:
            stream.wait_stream(torch.cuda.current_stream())
        assert h3.h3attn_paged_decode_weights(self.dq, o, self.cache, w, ws, self.scale, stream) is o
        torch.cuda.synchronize()
        return o, w


def close(got, ref, bound, what=""):
    err = (got.cpu().double() - ref).abs()
    assert bool((err <= bound).all()), f"{what}: {float((err / bound.clamp(min=1e-300)).nan_to_num(nan=1e9).max())} bounds"


def close_weights(c, w, ref, bound, what=""):
    """Added to what was there, one float32 rounding; where no token is, untouched."""
    before = c.before.double()
    close(w, before + ref, torch.where(ref > 0, bound + (before + ref) * 2.0 ** -24, 0.0), what + " weights")


def check(h3, c, what=""):
    c.cuda(h3)
    o, bound, w, w_bound = c.reference()
    if c.bits == 4:
        for split in (True, False):
            close(c.run(h3, split), o, bound, f"{what} split={split}")
    got, weights = c.run_weights(h3)
    close(got, o, bound, what + " with weights")
    close_weights(c, weights, w, w_bound, what)
    assert h3.h3attn_check_device_status() == 0


HEADS = [(1, 1), (4, 4), (16, 4), (8, 1), (9, 1), (16, 1), (17, 1), (40, 2), (24, 24), (6, 3), (14, 2)]
MANY_HEADS = [(32, 1), (31, 1), (34, 2), (48, 1), (64, 1), (96, 3), (128, 4)]


@pytest.mark.gpu
@pytest.mark.parametrize("bits", [4, 16])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("Hq,Hkv", HEADS)
def test_heads_and_head_dims(h3, bits, Hq, Hkv, D):
    check(h3, Case([150, 0, 33, 1], Hq, Hkv, D, 16, capacity=1040, seed=D + Hq, bits=bits))


@pytest.mark.gpu
@pytest.mark.parametrize("bits", [4, 16])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("Hq,Hkv", MANY_HEADS)
@pytest.mark.parametrize("capacity", [264, 5000])
def test_more_heads_than_a_tile(h3, bits, capacity, Hq, Hkv, D):
    check(h3, Case([1, 0, 15, 16, 17, 32, 33, 47, 49, 64, 65, 130, 263], Hq, Hkv, D, 8, capacity=capacity, seed=D + Hq, bits=bits))


@pytest.mark.gpu
@pytest.mark.parametrize("bits", [4, 16])
@pytest.mark.parametrize("page", [1, 3, 16, 24, 64, 1000])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_lengths_around_tiles_and_pages(h3, bits, page, D):
    check(h3, Case([0, 1, 2, 15, 16, 17, 31, 32, 33, 47, 48, 63, 64, 65, 127, 128, 129, 255, 257, 500], 4, 2, D, page, capacity=1100,
                   seed=page, bits=bits))


@pytest.mark.gpu
@pytest.mark.parametrize("bits", [4, 16])
@pytest.mark.parametrize("Hq,Hkv,D", [(2, 1, 128), (24, 24, 128), (16, 2, 64), (10, 1, 256), (16, 4, 128), (32, 1, 128)])
@pytest.mark.parametrize("n", [1025, 9001])
def test_one_long_sequence(h3, bits, n, Hq, Hkv, D):
    check(h3, Case([n], Hq, Hkv, D, 16, seed=n, bits=bits))


@pytest.mark.gpu
@pytest.mark.parametrize("bits", [4, 16])
def test_unlike_lengths(h3, bits):
    check(h3, Case([5000, 1, 0, 7, 2500, 40, 0, 0, 16, 999, 0], 8, 2, 128, 24, seed=5, bits=bits))


@pytest.mark.gpu
@pytest.mark.parametrize("bits", [4, 16])
def test_all_empty(h3, bits):
    c = Case([0, 0, 0], 4, 2, 128, 16, capacity=8000, bits=bits).cuda(h3)
    o, w = c.run_weights(h3)
    assert bool((o == 0).all()) and torch.equal(w.cpu(), c.before)
    if bits == 4:
        for split in (True, False):
            assert bool((c.run(h3, split) == 0).all())


@pytest.mark.gpu
@pytest.mark.parametrize("bits", [4, 16])
def test_lengths_outside_the_capacity(h3, bits):
    """Below zero: no key.  Above the capacity: the capacity."""
    c = Case([40, -5, 48, 48], 4, 2, 128, 16, capacity=48, poison=False, bits=bits)
    c.lens = [40, -5, 1000, 2 ** 31 - 1]
    check(h3, c)


@pytest.mark.gpu
@pytest.mark.parametrize("bits", [4, 16])
@pytest.mark.parametrize("peak,scale,q_scale", [(3.0, None, 1.0), (0.0, 4.0, 1.0), (0.0, 1e-3, 1.0), (0.0, 1e5, 1e-6), (0.0, 1e-9, 3e7)])
def test_peaky_and_flat_softmax(h3, bits, peak, scale, q_scale):
    check(h3, Case([1700, 90], 8, 4, 128, 16, peak=peak, scale=scale, seed=4, bits=bits, q_scale=q_scale))


@pytest.mark.gpu
@pytest.mark.parametrize("size", [1e-6, 2.0 ** -12, 1e-2, 1e3, 2e4])
def test_sizes_of_rows(h3, size):
    """Rows over the whole range of the scales."""
    c = Case([700, 33], 8, 2, 128, 16, capacity=3000, seed=14, poison=False, scale=0.09 / max(size, 1e-2))
    c.p.k, c.p.v = c.p.k * size, c.p.v * size
    check(h3, c)


@pytest.mark.gpu
def test_queries_of_unlike_channels(h3):
    """Channels of one query row 2^22 apart, rows of zeros."""
    c = Case([300, 40], 8, 2, 128, 16, capacity=3000, seed=15)
    c.q[:, :, ::3] *= 2.0 ** -22
    c.q[0, 2] = 0.0
    check(h3, c)


@pytest.mark.gpu
@pytest.mark.parametrize("bits", [4, 16])
@pytest.mark.parametrize("B", [33, 512, 513, 700])
def test_many_sequences(h3, bits, B):
    check(h3, Case([(37 * b) % 90 for b in range(B)], 4, 2, 64, 16, capacity=2600, seed=B, bits=bits))


@pytest.mark.gpu
@pytest.mark.parametrize("bits", [4, 16])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Hq,Hkv", [(4, 2), (32, 1)])
def test_bad_pages_are_not_attended(h3, bits, Hq, Hkv, D):
    c = Case([100, 40, 64, 3000], Hq, Hkv, D, 16, capacity=3200, seed=9, bits=bits)
    c.p.table[0, 2] = -1
    c.p.table[0, 6] = c.p.k.shape[0]
    c.p.table[1, 0] = c.p.table[1, 1] = c.p.table[1, 2] = 2 ** 31 - 1   # nothing is left of this one
    c.p.table[3, 50] = c.p.table[3, 51] = -5
    skip = [set(range(32, 48)) | set(range(96, 100)), set(range(40)), set(), set(range(800, 832))]
    c.cuda(h3)
    o, bound, w, w_bound = c.reference(skip)
    runs = [lambda: c.run(h3, True), lambda: c.run(h3, False)] if bits == 4 else []
    for run in runs:
        close(run(), o, bound)
        assert h3.h3attn_check_device_status() == h3.H3ATTN_ERR_INVALID_ARG
        assert h3.h3attn_check_device_status() == 0
    got, weights = c.run_weights(h3)
    assert h3.h3attn_check_device_status() == h3.H3ATTN_ERR_INVALID_ARG
    close(got, o, bound)
    close_weights(c, weights, w, w_bound)
    assert bool((got[1] == 0).all())


@pytest.mark.gpu
@pytest.mark.parametrize("bits", [4, 16])
def test_nan_in_an_attended_row_stays_in_its_sequence(h3, bits):
    c = Case([50, 60], 4, 2, 128, 16, capacity=3000, seed=2, bits=bits)
    c.p.k[c.p.table[0, 1].long(), 3, 0, 5] = float("nan")
    c.cuda(h3)
    o, w = c.run_weights(h3)
    for got in [o] + ([c.run(h3)] if bits == 4 else []):
        got = got.float()
        assert bool(got[0, :2].isnan().all()) and bool(got[0, 2:].isfinite().all()) and bool(got[1].isfinite().all())
    assert bool(w[0, :50].isnan().all()) and bool(w[0, 50:].isfinite().all()) and bool(w[1].isfinite().all())


@pytest.mark.gpu
def test_nan_in_a_value_row(h3):
    c = Case([50, 3100], 4, 2, 128, 16, seed=2)
    c.p.v[c.p.table[1, 100].long(), 3, 1, 5] = float("inf")
    c.cuda(h3)
    o = c.run(h3).float()
    assert bool(o[1, 2:, :16].isnan().all()) and bool(o[1, 2:, 16:].isfinite().all())
    assert bool(o[1, :2].isfinite().all()) and bool(o[0].isfinite().all())


@pytest.mark.gpu
@pytest.mark.parametrize("bits", [4, 16])
def test_repeatable(h3, bits):
    c = Case([4000, 100, 2900], 8, 2, 128, 16, seed=3, bits=bits).cuda(h3)
    first = c.run_weights(h3)
    for _ in range(3):
        again = c.run_weights(h3)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])
    if bits == 4:
        assert torch.equal(c.run(h3), first[0])   # the weights do not change the output


@pytest.mark.gpu
def test_bf16_output_with_weights_is_the_decodes(h3):
    for Hq, Hkv, D in ((16, 4, 128), (24, 24, 64), (32, 1, 128), (10, 1, 256)):
        c = Case([1500, 40, 3, 0], Hq, Hkv, D, 16, seed=3, bits=16).cuda(h3)
        o = torch.empty_like(c.dq)
        h3.h3attn_paged_decode(c.dq, o, c.cache, c.scale, h3.paged_decode_workspace(c.dq, c.cache))
        assert torch.equal(o, c.run_weights(h3)[0])


@pytest.mark.gpu
@pytest.mark.parametrize("bits", [4, 16])
def test_weights_sum_to_the_heads(h3, bits):
    c = Case([4100, 77], 16, 4, 128, 16, seed=13, bits=bits).cuda(h3)
    c.before.zero_()
    _, w = c.run_weights(h3)
    assert torch.allclose(w.double().sum(1).cpu(), torch.tensor([16.0, 16.0], dtype=torch.float64), rtol=1e-5)


@pytest.mark.gpu
@pytest.mark.parametrize("bits", [4, 16])
def test_stream_guards_and_small_workspaces(h3, bits):
    c = Case([3100, 31], 8, 2, 128, 16, seed=8, bits=bits).cuda(h3)
    o, bound, w, w_bound = c.reference()
    got, weights = c.run_weights(h3, torch.cuda.Stream())
    close(got, o, bound)
    close_weights(c, weights, w, w_bound)
    need = h3.h3attn_paged_decode_weights_workspace_size(c.cache, 8)
    ws = torch.full((need + 4096,), 0xFF, dtype=torch.uint8, device="cuda")
    buf = torch.full((4, 8, 128), 9.0, dtype=torch.bfloat16, device="cuda")
    h3.h3attn_paged_decode_weights(c.dq, buf[1:3], c.cache, c.before.cuda(), ws, c.scale)
    torch.cuda.synchronize()
    close(buf[1:3], o, bound)
    assert bool((buf[0] == 9).all()) and bool((buf[3] == 9).all()) and bool((ws[need:] == 0xFF).all())
    for bad in (None, ws[:need - 16]):
        with pytest.raises(h3.H3AttnError):
            h3.h3attn_paged_decode_weights(c.dq, buf[1:3], c.cache, c.before.cuda(), bad)


@pytest.mark.gpu
@pytest.mark.parametrize("bits", [4, 16])
def test_graph_replays_with_new_lengths(h3, bits):
    c = Case([500, 2900, 100], 8, 2, 128, 16, poison=False, seed=12, bits=bits).cuda(h3)
    ws = h3.paged_decode_weights_workspace(c.dq, c.cache)
    o, w = torch.empty_like(c.dq), c.before.cuda()
    h3.h3attn_paged_decode_weights(c.dq, o, c.cache, w, ws)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        h3.h3attn_paged_decode_weights(c.dq, o, c.cache, w, ws)
    for lens in ([1, 2900, 333], [0, 0, 0], [900, 0, 17]):
        c.lens = lens
        c.q = randn(3, 8, 128, seed=sum(lens))
        c.p.dlen.copy_(torch.tensor(lens, dtype=torch.int32))
        c.dq.copy_(c.q)
        w.copy_(c.before)
        graph.replay()
        torch.cuda.synchronize()
        want, bound, wt, wt_bound = c.reference()
        close(o, want, bound, str(lens))
        close_weights(c, w, wt, wt_bound, str(lens))


@pytest.mark.gpu
def test_pages_past_32_bits(h3):
    """Pages that begin past 2^32 bytes of the codes."""
    page, Hkv, D, n = 64, 8, 128, 200
    pages = (1 << 32) // (page * Hkv * D // 2) + 9
    c = Case([n], 16, Hkv, D, page, seed=1, poison=False)
    c.p.hold()
    far = torch.arange(pages - 4, pages, dtype=torch.int32)
    held = []
    for t in c.p.held:
        big = torch.empty(pages, *t.shape[1:], dtype=torch.uint8, device="cuda")
        big[far.long().cuda()] = t[c.p.table[0].long()].cuda()
        held.append(big)
    cache = h3.PagedKV4(*held, far[None].cuda(), torch.tensor([n], dtype=torch.int32, device="cuda"))
    dq = c.q.cuda()
    o = torch.empty_like(dq)
    h3.h3attn_paged_decode_q4(dq, o, cache, workspace=h3.paged_decode_q4_workspace(dq, cache))
    torch.cuda.synchronize()
    close(o, *c.reference()[:2])


@pytest.mark.gpu
@pytest.mark.parametrize("n,rest", [(17 * 32, 40), (33 * 32, 2000), (200 * 32, 0), (16 * 32, 600), (2432 * 4, 31)])
def test_sequences_that_end_where_another_begins(h3, n, rest):
    check(h3, Case([n, rest, 1, n // 2, 7, rest, n], 4, 1, 128, 16, seed=n))


@pytest.mark.gpu
@pytest.mark.parametrize("lens", [[2000], [8000], [5413, 5400], [2000, 1, 0, 1999], [333] * 12])
@pytest.mark.parametrize("Hq,Hkv,D", [(16, 4, 128), (8, 1, 128), (32, 1, 128), (24, 8, 64), (4, 2, 256)])
def test_few_tiles_a_warp(h3, lens, Hq, Hkv, D):
    check(h3, Case(lens, Hq, Hkv, D, 32, seed=len(lens) + D))


@pytest.mark.gpu
def test_refusals(h3):
    c = Case([20, 30], 4, 2, 64, 16).cuda(h3)
    q, w = c.dq, c.before.cuda()
    ws = h3.paged_decode_weights_workspace(q, c.cache)
    kv16 = Case([20, 30], 4, 2, 64, 16, bits=16).cuda(h3).cache
    h3.h3attn_paged_decode_q4(q, torch.empty_like(q), c.cache)
    for bad in ((q[0], q.clone(), c.cache), (q, q, c.cache), (q, q.float(), c.cache), (q, q[:, :2].clone(), c.cache),
                (q.cpu(), q.clone(), c.cache), (q, q.clone(), None), (q[:1], q[:1].clone(), c.cache), (q, q.clone(), kv16),
                (q[:, :3].clone(), q[:, :3].clone(), c.cache), (q, q.clone(), c.cache, -1.0), (q, q.clone(), c.cache, float("nan"))):
        with pytest.raises(h3.H3AttnError):
            h3.h3attn_paged_decode_q4(*bad)
    with pytest.raises(h3.H3AttnError):
        h3.h3attn_paged_decode(q, q.clone(), c.cache)
    for weights, space in ((w.double(), ws), (w[:1], ws), (w[:, :16].clone(), ws), (w.cpu(), ws), (w, ws.cpu()), (w.t().contiguous().t(), ws),
                           (w, w.view(torch.uint8)), (ws[:w.numel() * 4].view(torch.float32).view(w.shape), ws)):
        with pytest.raises(h3.H3AttnError):
            h3.h3attn_paged_decode_weights(q, q.clone(), c.cache, weights, space)
    with pytest.raises(h3.H3AttnError):
        h3.h3attn_paged_decode_weights(q, q.clone(), None, w, ws)


@pytest.mark.gpu
@pytest.mark.parametrize("bits", [4, 16])
@pytest.mark.parametrize("lens,Hq,Hkv,D", [([300, 0, 5000, 1, 256, 257, 900], 6, 2, 128), ([0, 0, 3], 33, 1, 64),
                                           ([255, 256, 257, 512, 513] * 9, 5, 1, 64), ([1], 40, 40, 64)])
def test_tables_with_more_room_than_tokens(h3, bits, lens, Hq, Hkv, D):
    """Weights are added up of the tokens that are there, wherever the tables would end."""
    check(h3, Case(lens, Hq, Hkv, D, 16, capacity=9000, seed=len(lens), bits=bits))


@pytest.mark.gpu
@pytest.mark.parametrize("bits", [4, 16])
def test_more_tokens_than_threads_that_add_weights(h3, bits):
    """41 sequences of 32 times 256 tokens, split; and 600 of up to ten times 256, each by one CTA, with four that add."""
    check(h3, Case([8000] * 41, 2, 1, 64, 64, seed=1, bits=bits))
    check(h3, Case([2600 if b % 200 == 7 else (37 * b) % 90 for b in range(600)], 2, 1, 64, 16, seed=2, bits=bits))
