"""GPU parity of the paged decode attention against float64, with the bound that
its roundings allow (see generate_ref.decode_f64): lengths around tiles and
pages, empty sequences, poisoned rows and pages past the lengths, group sizes
of every column-tile count, split and unsplit."""
import pytest
import torch

from generate_ref import decode_f64, paged, poison_past, randn


class Case:
    def __init__(self, lens, Hq, Hkv, D, page, capacity=None, seed=0, peak=0.0, poison=True, scale=None):
        B = len(lens)
        self.lens, self.page = list(lens), page
        capacity = max([1] + [n for n in lens]) if capacity is None else capacity
        self.k, self.v, self.table = paged(B, capacity, page, Hkv, D, seed)
        self.q = randn(B, Hq, D, seed=seed + 7)
        self.scale = D ** -0.5 if scale is None else scale
        if peak:
            self.k += peak * randn(Hkv, D, seed=seed + 8)
        if poison:
            poison_past(self.k, self.v, self.table, lens, page)

    def cuda(self, h3):
        self.dlen = torch.tensor(self.lens, dtype=torch.int32, device="cuda")
        self.dk, self.dv, self.dt, self.dq = self.k.cuda(), self.v.cuda(), self.table.cuda(), self.q.cuda()
        self.cache = h3.PagedKV(self.dk, self.dv, self.dt, self.dlen)
        return self

    def reference(self, skip=None):
        cap = self.table.shape[1] * self.page
        return decode_f64(self.q, self.k, self.v, self.table, [min(n, cap) for n in self.lens], self.page, self.scale, skip)

    def run(self, h3, split=True, stream=None):
        ws = h3.paged_decode_workspace(self.dq, self.cache) if split else None
        if ws is not None:
            ws.fill_(0xFF)  # NaN in every float: contents on entry do not matter
        o = torch.full_like(self.dq, float("nan"))
        if stream is not None:
            stream.wait_stream(torch.cuda.current_stream())
        assert h3.h3attn_paged_decode(self.dq, o, self.cache, self.scale, ws, stream) is o
        torch.cuda.synchronize()
        return o


def close(o, ref, bound, what=""):
    err = (o.cpu().double() - ref).abs()
    assert bool((err <= bound).all()), f"{what}: {float((err / bound.clamp(min=1e-300)).nan_to_num(nan=1e9).max())} bounds"


def check(h3, c, what=""):
    c.cuda(h3)
    ref, bound = c.reference()
    for split in (True, False):
        close(c.run(h3, split), ref, bound, f"{what} split={split}")
    assert h3.h3attn_check_device_status() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (4, 4), (16, 4), (8, 1), (9, 1), (16, 1), (17, 1), (40, 2), (24, 24), (6, 3), (14, 2)])
def test_heads_and_head_dims(h3, Hq, Hkv, D):
    check(h3, Case([150, 0, 33, 1], Hq, Hkv, D, 16, capacity=1040, seed=D + Hq))


@pytest.mark.gpu
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("Hq,Hkv", [(32, 1), (31, 1), (34, 2), (48, 1), (64, 1), (96, 3), (128, 4), (256, 8)])
@pytest.mark.parametrize("capacity", [264, 3000])
def test_more_heads_than_a_tile(h3, capacity, Hq, Hkv, D):
    """Several tiles of query heads to a key-value head, in one launch and in two: odd and even numbers of token tiles,
    and sequences that end at every place of a pair of them."""
    check(h3, Case([1, 0, 15, 16, 17, 32, 33, 47, 49, 64, 65, 130, 263], Hq, Hkv, D, 8, capacity=capacity, seed=D + Hq))


@pytest.mark.gpu
@pytest.mark.parametrize("D", [128, 256])
def test_more_heads_than_a_tile_with_bad_pages(h3, D):
    c = Case([100, 40, 1500], 32, 1, D, 16, capacity=1600, seed=D)
    c.table[0, 1] = -1
    c.table[1, 0] = c.table[1, 1] = c.table[1, 2] = c.k.shape[0]
    c.table[2, 50] = 2 ** 31 - 1
    ref, bound = c.reference([set(range(16, 32)), set(range(40)), set(range(800, 816))])
    c.cuda(h3)
    for split in (True, False):
        o = c.run(h3, split)
        assert h3.h3attn_check_device_status() == h3.H3ATTN_ERR_INVALID_ARG
        close(o, ref, bound, f"split={split}")
        assert bool((o[1] == 0).all())


@pytest.mark.gpu
@pytest.mark.parametrize("page", [1, 3, 16, 24, 64, 1000])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_lengths_around_tiles_and_pages(h3, page, D):
    check(h3, Case([0, 1, 2, 15, 16, 17, 31, 32, 33, 47, 48, 63, 64, 65, 127, 128, 129, 255, 257, 500], 4, 2, D, page, capacity=1100,
                   seed=page))


@pytest.mark.gpu
@pytest.mark.parametrize("Hq,Hkv,D", [(2, 1, 128), (24, 24, 128), (16, 2, 64), (10, 1, 256), (16, 4, 128)])
@pytest.mark.parametrize("n", [1025, 9001])
def test_one_long_sequence(h3, n, Hq, Hkv, D):
    check(h3, Case([n], Hq, Hkv, D, 16, seed=n))


@pytest.mark.gpu
def test_unlike_lengths(h3):
    check(h3, Case([3000, 1, 0, 7, 2500, 40, 0, 0, 16, 999, 0], 8, 2, 128, 24, seed=5))


@pytest.mark.gpu
def test_all_empty(h3):
    c = Case([0, 0, 0], 4, 2, 128, 16, capacity=4000).cuda(h3)
    for split in (True, False):
        assert bool((c.run(h3, split) == 0).all())


@pytest.mark.gpu
def test_lengths_outside_the_capacity(h3):
    """Below zero: no key.  Above the capacity: the capacity."""
    c = Case([40, -5, 48, 48], 4, 2, 128, 16, capacity=48, poison=False)
    c.lens = [40, -5, 1000, 2 ** 31 - 1]
    check(h3, c)


@pytest.mark.gpu
@pytest.mark.parametrize("peak,scale", [(3.0, None), (0.0, 4.0), (0.0, 1e-3)])
def test_peaky_and_flat_softmax(h3, peak, scale):
    check(h3, Case([700, 90], 8, 4, 128, 16, peak=peak, scale=scale, seed=4))


@pytest.mark.gpu
@pytest.mark.parametrize("B", [33, 512, 513, 700])
def test_many_sequences(h3, B):
    """Up to 512 sequences are split over the GPU, more are walked one a CTA."""
    lens = [(37 * b) % 90 for b in range(B)]
    c = Case(lens, 4, 2, 64, 16, capacity=520, seed=B).cuda(h3)
    assert (h3.paged_decode_workspace(c.dq, c.cache) is None) == (B > 512)
    check(h3, c)


@pytest.mark.gpu
def test_short_caches_take_no_workspace(h3):
    """A cache without room for more than four tiles a warp is walked whole, with and without a workspace."""
    for capacity, splits in ((128, False), (144, True)):
        c = Case([100, 128, 1], 4, 4, 128, 16, capacity=capacity, seed=capacity).cuda(h3)
        assert (h3.h3attn_paged_decode_workspace_size(c.cache, 4) > 0) == splits
        o = torch.empty_like(c.dq)
        h3.h3attn_paged_decode(c.dq, o, c.cache, workspace=torch.empty(1 << 20, dtype=torch.uint8, device="cuda"))
        torch.cuda.synchronize()
        close(o, *c.reference())


@pytest.mark.gpu
@pytest.mark.parametrize("D", [64, 128])
def test_bad_pages_are_not_attended(h3, D):
    c = Case([100, 40, 64], 4, 2, D, 16, capacity=600, seed=9)
    c.table[0, 2] = -1
    c.table[0, 6] = c.k.shape[0]
    c.table[1, 0] = c.table[1, 1] = c.table[1, 2] = 2 ** 31 - 1   # nothing is left of this one
    ref, bound = c.reference([set(range(32, 48)) | set(range(96, 100)), set(range(40)), set()])
    c.cuda(h3)
    for split in (True, False):
        o = c.run(h3, split)
        assert h3.h3attn_check_device_status() == h3.H3ATTN_ERR_INVALID_ARG
        assert h3.h3attn_check_device_status() == 0
        close(o, ref, bound)
        assert bool((o[1] == 0).all())


@pytest.mark.gpu
def test_nan_in_an_attended_row_stays_in_its_sequence(h3):
    c = Case([50, 60], 4, 2, 128, 16, capacity=400, seed=2)
    c.k[c.table[0, 1].long(), 3, 0, 5] = float("nan")
    c.cuda(h3)
    o = c.run(h3).float()
    assert bool(o[0, :2].isnan().all()) and bool(o[0, 2:].isfinite().all()) and bool(o[1].isfinite().all())


@pytest.mark.gpu
def test_repeatable(h3):
    """The parts are joined in a fixed order."""
    c = Case([4000, 100, 2900], 8, 2, 128, 16, seed=3).cuda(h3)
    first = c.run(h3)
    for _ in range(3):
        assert torch.equal(first, c.run(h3))


@pytest.mark.gpu
def test_shared_pages(h3):
    """Two sequences with a common prefix."""
    c = Case([64, 80], 4, 2, 128, 16, capacity=400, poison=False, seed=6)
    c.table[1, :4] = c.table[0, :4]
    check(h3, c)


@pytest.mark.gpu
def test_stream_workspace_and_guards(h3):
    """On another stream; a workspace larger than needed; one shared by two calls in turn; rows around o stay."""
    c = Case([800, 31], 8, 2, 128, 16, seed=8).cuda(h3)
    ref, bound = c.reference()
    close(c.run(h3, stream=torch.cuda.Stream()), ref, bound)
    other = Case([5, 1300, 64], 16, 2, 64, 24, seed=18).cuda(h3)
    need = [h3.h3attn_paged_decode_workspace_size(x.cache, x.q.shape[1]) for x in (c, other)]
    ws = torch.full((max(need) + 4096,), 0xFF, dtype=torch.uint8, device="cuda")
    buf = torch.full((4, 8, 128), 9.0, dtype=torch.bfloat16, device="cuda")
    o2 = torch.empty_like(other.dq)
    for _ in range(2):
        h3.h3attn_paged_decode(c.dq, buf[1:3], c.cache, workspace=ws)
        h3.h3attn_paged_decode(other.dq, o2, other.cache, workspace=ws)
    torch.cuda.synchronize()
    close(buf[1:3], ref, bound)
    close(o2, *other.reference())
    assert bool((buf[0] == 9).all()) and bool((buf[3] == 9).all())
    assert bool((ws[max(need):] == 0xFF).all())
    with pytest.raises(h3.H3AttnError):
        h3.h3attn_paged_decode(c.dq, buf[1:3], c.cache, workspace=ws[:need[0] - 16])


@pytest.mark.gpu
def test_graph_replays_with_new_lengths(h3):
    """Lengths, pages and queries are read by the replay, not by the capture."""
    c = Case([500, 900, 100], 8, 2, 128, 16, poison=False, seed=12).cuda(h3)
    ws = h3.paged_decode_workspace(c.dq, c.cache)
    o = torch.empty_like(c.dq)
    h3.h3attn_paged_decode(c.dq, o, c.cache, workspace=ws)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        h3.h3attn_paged_decode(c.dq, o, c.cache, workspace=ws)
    for lens in ([1, 900, 333], [0, 0, 0], [900, 0, 17]):
        c.lens = lens
        c.q = randn(3, 8, 128, seed=sum(lens))
        c.dlen.copy_(torch.tensor(lens, dtype=torch.int32))
        c.dq.copy_(c.q)
        graph.replay()
        torch.cuda.synchronize()
        close(o, *c.reference(), what=str(lens))


@pytest.mark.gpu
def test_pages_past_32_bits(h3):
    """Pages that begin past 2^31 elements of the cache."""
    page, Hkv, D, n = 64, 8, 128, 200
    pages = (1 << 31) // (page * Hkv * D) + 9
    c = Case([n], 16, Hkv, D, page, seed=1, poison=False)
    dk = torch.empty(pages, page, Hkv, D, dtype=torch.bfloat16, device="cuda")
    dv = torch.empty_like(dk)
    far = torch.arange(pages - 4, pages, dtype=torch.int32)
    dk[far.long().cuda()] = c.k[c.table[0].long()].cuda()
    dv[far.long().cuda()] = c.v[c.table[0].long()].cuda()
    cache = h3.PagedKV(dk, dv, far[None].cuda(), torch.tensor([n], dtype=torch.int32, device="cuda"))
    dq = c.q.cuda()
    o = torch.empty_like(dq)
    h3.h3attn_paged_decode(dq, o, cache, workspace=h3.paged_decode_workspace(dq, cache))
    torch.cuda.synchronize()
    close(o, *c.reference())


@pytest.mark.gpu
@pytest.mark.parametrize("n,rest", [(17 * 32, 40), (33 * 32, 2000), (200 * 32, 0), (16 * 32, 600), (2432 * 4, 31)])
def test_sequences_that_end_where_another_begins(h3, n, rest):
    """One unit head, so as many ranges as there are SMs: sequences over more and fewer of them than are joined at a
    time, whose last range another sequence begins in."""
    check(h3, Case([n, rest, 1, n // 2, 7, rest, n], 4, 1, 128, 16, seed=n))


@pytest.mark.gpu
def test_workspaces_that_hold_anything(h3):
    """Zeros, ones, small numbers, what another geometry's call left, and its own call's: each gives the same output."""
    c = Case([3000, 5, 2100], 8, 2, 128, 16, seed=30).cuda(h3)
    other = Case([900, 4000], 4, 4, 64, 24, seed=31).cuda(h3)
    need = max(h3.h3attn_paged_decode_workspace_size(x.cache, x.q.shape[1]) for x in (c, other))
    ws = torch.zeros(need, dtype=torch.uint8, device="cuda")
    want = c.run(h3)
    o, o2 = torch.empty_like(c.dq), torch.empty_like(other.dq)
    for fill in (0, 1, 255, None, "small", "self"):
        if fill == "small":
            ws[:need // 8 * 8].view(torch.int64).copy_(torch.arange(need // 8))
        elif fill is None:
            h3.h3attn_paged_decode(other.dq, o2, other.cache, workspace=ws)
        elif fill != "self":
            ws.fill_(fill)
        o.fill_(float("nan"))
        h3.h3attn_paged_decode(c.dq, o, c.cache, workspace=ws)
        assert torch.equal(o, want), fill


@pytest.mark.gpu
@pytest.mark.parametrize("lens", [[2000], [8000], [5413, 5400], [2000, 1, 0, 1999], [333] * 12])
@pytest.mark.parametrize("Hq,Hkv,D", [(16, 4, 128), (8, 1, 128), (32, 1, 128), (24, 8, 64), (4, 2, 256)])
def test_few_tiles_a_warp(h3, lens, Hq, Hkv, D):
    """Around the sizes from which on all SMs take part."""
    check(h3, Case(lens, Hq, Hkv, D, 32, seed=len(lens) + D))
