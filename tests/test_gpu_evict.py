"""Eviction from caches of either kind against the definition, bit for bit:
row sizes, ties and special weights, how many are kept and recent, pages that end
anywhere, bad pages, sequences that stay, replays."""
import pytest
import torch

from cache4_ref import Pages, evict


def weights_of(kind, shape, seed):
    g = torch.Generator().manual_seed(seed)
    w = torch.randn(shape, generator=g).mul(2).exp()
    if kind == "ties":
        w = torch.randint(0, 4, shape, generator=g).float()
    elif kind == "same":
        w = torch.full(shape, 0.25)
    elif kind == "special":
        w[torch.rand(shape, generator=g) < 0.2] = 0.0
        w[torch.rand(shape, generator=g) < 0.1] = -0.0
        w[torch.rand(shape, generator=g) < 0.1] = float("nan")
        w[torch.rand(shape, generator=g) < 0.05] = float("inf")
        w[torch.rand(shape, generator=g) < 0.1] *= -1
        w[torch.rand(shape, generator=g) < 0.05] = 1e-42
    elif kind == "rising":
        w = torch.arange(shape[1]).float().expand(shape).clone()
    elif kind == "falling":
        w = -torch.arange(shape[1]).float().expand(shape).clone()
    return w


def bits_of(t):
    return t.view(torch.int16) if t.dtype == torch.bfloat16 else t.view(torch.int32) if t.dtype == torch.float32 else t


class Case:
    def __init__(self, h3, bits, lens, keep, recent, Hkv=2, D=64, page=16, capacity=None, kind="plain", seed=0, bad=()):
        capacity = max([1] + list(lens)) if capacity is None else capacity
        self.p = Pages(bits, len(lens), capacity, page, Hkv, D, seed)
        for b, i, value in bad:
            self.p.table[b, i] = value
        self.cache = self.p.hold().cuda(h3, lens)
        self.lens, self.keep, self.recent, self.page = list(lens), keep, recent, page
        self.w = weights_of(kind, (len(lens), self.p.table.shape[1] * page), seed + 1)
        self.dw = self.w.cuda()
        self.out = torch.full((len(lens),), -9, dtype=torch.int32, device="cuda")
        self.ws = h3.paged_evict_workspace(self.cache, keep, recent)
        if self.ws is not None:
            self.ws.fill_(0xFF)

    def run(self, h3, stream=None):
        if stream is not None:
            stream.wait_stream(torch.cuda.current_stream())
        assert h3.h3attn_paged_evict(self.cache, self.dw, self.keep, self.recent, self.out, self.ws, stream) is self.out
        torch.cuda.synchronize()

    def compare(self):
        held, w, out = evict(self.p.held, self.p.table, self.lens, self.page, self.w, self.keep, self.recent)
        assert torch.equal(self.out.cpu(), out)
        assert torch.equal(bits_of(self.dw.cpu()), bits_of(w)), "weights"
        for i, (got, want) in enumerate(zip(self.p.dheld, held)):
            assert torch.equal(bits_of(got.cpu()), bits_of(want)), f"tensor {i}"


def check(h3, *args, **kw):
    c = Case(h3, *args, **kw)
    c.run(h3)
    assert h3.h3attn_check_device_status() == 0
    c.compare()


@pytest.mark.gpu
@pytest.mark.parametrize("bits", [4, 16])
@pytest.mark.parametrize("Hkv,D", [(1, 64), (2, 64), (3, 64), (1, 128), (5, 128), (24, 128), (1, 256), (7, 256)])
@pytest.mark.parametrize("page", [1, 16, 24])
def test_row_sizes(h3, bits, Hkv, D, page):
    check(h3, bits, [300, 0, 100, 64, 65], 64, 10, Hkv, D, page, seed=Hkv)


@pytest.mark.gpu
@pytest.mark.parametrize("bits", [4, 16])
@pytest.mark.parametrize("kind", ["plain", "ties", "same", "special", "rising", "falling"])
@pytest.mark.parametrize("keep,recent", [(1, 0), (1, 1), (64, 0), (64, 64), (100, 99), (512, 32), (700, 300), (999, 0), (999, 500)])
def test_weights_and_budgets(h3, bits, kind, keep, recent):
    check(h3, bits, [1000, 513, 999, 3, 700], keep, recent, kind=kind, seed=keep)


@pytest.mark.gpu
@pytest.mark.parametrize("n,keep,recent", [(4097, 4096, 512), (5000, 100, 50), (9000, 8999, 3000), (20000, 15000, 100), (40001, 9000, 4000),
                                           (8100, 8000, 5000), (30000, 20000, 9000), (30000, 29950, 9000),
                                           (70000, 69999, 1)])
@pytest.mark.parametrize("kind", ["plain", "ties", "special"])
def test_long_sequences(h3, n, keep, recent, kind):
    """One CTA and clusters of several; recent ones that overlap where they go."""
    check(h3, 4, [n, n // 2], keep, recent, 1, 64, 64, kind=kind, seed=n)


@pytest.mark.gpu
def test_room_that_is_not_used(h3):
    """Short sequences in wide tables, lengths outside the capacity, a budget above it."""
    check(h3, 4, [50, 7, 0, -4], 10, 4, capacity=20000)
    c = Case(h3, 16, [100, 100], 40, 8, capacity=100)
    c.lens = [10 ** 6, 2 ** 31 - 1]
    c.p.dlen.copy_(torch.tensor(c.lens, dtype=torch.int32))
    c.run(h3)
    c.compare()
    check(h3, 16, [100, 40], 5000, 8)
    check(h3, 16, [100, 40], 2 ** 31 - 1, 2 ** 31 - 1)


@pytest.mark.gpu
@pytest.mark.parametrize("B", [1, 100, 600])
def test_many_sequences(h3, B):
    check(h3, 4, [(97 * b) % 200 for b in range(B)], 60, 20, 1, 64, 16, capacity=200, kind="ties", seed=B)


@pytest.mark.gpu
@pytest.mark.parametrize("bits", [4, 16])
def test_bad_pages_are_reported_and_skipped(h3, bits):
    c = Case(h3, bits, [200, 150], 64, 16, bad=[(0, 8, -1), (0, 1, 2 ** 31 - 1), (1, 9, 10 ** 6)], seed=3)
    c.run(h3)
    assert h3.h3attn_check_device_status() == h3.H3ATTN_ERR_INVALID_ARG
    c.compare()


@pytest.mark.gpu
def test_again_and_on_another_stream(h3):
    """A second eviction after the first, on the lengths that it left, does nothing."""
    c = Case(h3, 16, [300, 290, 20], 256, 32, seed=7)
    c.run(h3, torch.cuda.Stream())
    c.compare()
    held, w = [t.clone() for t in c.p.dheld], c.dw.clone()
    out = torch.empty_like(c.out)
    h3.h3attn_paged_evict(c.cache.with_lengths(c.out), c.dw, 256, 32, out, c.ws)
    assert torch.equal(out, c.out) and torch.equal(w, c.dw) and all(torch.equal(bits_of(a), bits_of(b)) for a, b in zip(held, c.p.dheld))


@pytest.mark.gpu
def test_graph_replays(h3):
    c = Case(h3, 4, [300, 100, 260], 128, 32, capacity=5000, seed=8)
    held = [t.clone() for t in c.p.dheld]
    c.run(h3)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        h3.h3attn_paged_evict(c.cache, c.dw, 128, 32, c.out, c.ws)
    for seed, lens in ((1, [129, 128, 300]), (2, [5, 200, 270])):
        c.lens = lens
        c.p.dlen.copy_(torch.tensor(lens, dtype=torch.int32))
        c.w = weights_of("ties", c.w.shape, seed)
        c.dw.copy_(c.w)
        for t, t0 in zip(c.p.dheld, held):
            t.copy_(t0)
        graph.replay()
        torch.cuda.synchronize()
        c.compare()


@pytest.mark.gpu
def test_rows_past_32_bits(h3):
    """Pages that begin past 2^32 bytes."""
    page, Hkv, D = 64, 8, 128
    pages = (1 << 32) // (page * Hkv * D * 2) + 9
    c = Case(h3, 16, [500], 200, 40, Hkv, D, page, seed=1)
    far = torch.arange(pages - 8, pages)
    big = [torch.empty(pages, page, Hkv, D, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    for t, t0 in zip(big, c.p.held):
        t[far.cuda()] = t0[c.p.table[0].long()].cuda()
    cache = h3.PagedKV(*big, far.int()[None].cuda(), c.p.dlen)
    h3.h3attn_paged_evict(cache, c.dw, 200, 40, c.out, c.ws)
    held, w, _ = evict(c.p.held, c.p.table, [500], page, c.w, 200, 40)
    assert torch.equal(bits_of(c.dw.cpu()), bits_of(w))
    for t, want in zip(big, held):
        assert torch.equal(bits_of(t[far.cuda()].cpu()), bits_of(want[c.p.table[0].long()]))


@pytest.mark.gpu
def test_refusals(h3):
    c = Case(h3, 4, [30, 20], 16, 4)
    w, out, ws = c.dw, c.out, c.ws

    def call(cache=c.cache, weights=w, keep=16, recent=4, len_out=out, workspace=ws):
        h3.h3attn_paged_evict(cache, weights, keep, recent, len_out, workspace)
    call()
    for bad in (dict(keep=0), dict(recent=17), dict(recent=-1), dict(weights=w[:1]), dict(weights=w.double()), dict(weights=w[:, :5].clone()),
                dict(len_out=out[:1]), dict(len_out=out.long()), dict(len_out=c.p.dlen), dict(workspace=None), dict(workspace=ws[:16]),
                dict(workspace=ws.cpu()), dict(cache=None), dict(weights=w.cpu()), dict(keep=2 ** 31),
                dict(workspace=w.view(torch.uint8))):
        with pytest.raises(h3.H3AttnError):
            call(**bad)
    with pytest.raises(h3.H3AttnError):
        h3.paged_evict_workspace(c.cache, 0, 0)


@pytest.mark.gpu
@pytest.mark.parametrize("n", [700001, 900001])
@pytest.mark.parametrize("kind", ["plain", "ties"])
def test_as_many_weights_as_shared_memory_holds_and_more(h3, kind, n):
    """A cluster's shared memory nearly full, and a sequence whose weights are read anew in each pass; the tokens numbered
    in their rows."""
    keep, recent, page = 500000, 1000, 64
    pages = -(-n // page)
    held = [torch.zeros(pages, page, 1, 64 // m, dtype=torch.uint8, device="cuda") for m in (2, 2, 16, 16)]
    table = torch.randperm(pages, generator=torch.Generator().manual_seed(3)).int()
    token = torch.arange(pages * page, device="cuda").view(pages, page)[torch.argsort(table).cuda()]  # of each row
    held[0].view(torch.int64)[..., 0, 0] = token
    held[2].view(torch.int32)[..., 0, 0] = token.int()
    cache = h3.PagedKV4(*held, table[None].cuda(), torch.tensor([n], dtype=torch.int32, device="cuda"))
    w = weights_of(kind, (1, pages * page), 5).cuda()
    before, out = w.clone(), torch.zeros(1, dtype=torch.int32, device="cuda")
    h3.h3attn_paged_evict(cache, w, keep, recent, out, h3.paged_evict_workspace(cache, keep, recent))
    assert out.tolist() == [keep] and h3.h3attn_check_device_status() == 0
    place = torch.arange(keep, device="cuda")
    row = table.cuda().long()[place // page], place % page
    front, old = keep - recent, n - recent
    stay = torch.sort(before[0, :old], descending=True, stable=True)[1][:front].sort()[0]
    gaps = torch.ones(front, dtype=torch.bool, device="cuda").index_fill_(0, stay[stay < front], False).nonzero()[:, 0]
    want = torch.arange(keep, device="cuda")
    want[gaps] = stay[stay >= front]
    want[front:] = torch.arange(old, n, device="cuda")
    assert torch.equal(held[0].view(torch.int64)[..., 0, 0][row], want)
    assert torch.equal(held[2].view(torch.int32)[..., 0, 0][row], want.int())
    assert torch.equal(w[0, :keep], before[0, want]) and bool((w[0, keep:n] == 0).all()) and torch.equal(w[0, n:], before[0, n:])


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["plain", "ties", "special"])
@pytest.mark.parametrize("keep,recent", [(3000, 300), (8193, 5000), (1, 0)])
def test_unlike_lengths_in_wide_tables(h3, kind, keep, recent):
    """Sequences of one call that take one CTA of their cluster, some, and all."""
    check(h3, 4, [5000, 8192, 8193, 20000, 33000, 3000], keep, recent, 1, 64, 64, capacity=70000, kind=kind, seed=keep)


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["plain", "ties"])
@pytest.mark.parametrize("room", [400000, 810000, 900001])
@pytest.mark.parametrize("n", [3000, 20000, 150000])
def test_pages_for_the_tokens_in_a_very_wide_table(h3, n, room, kind):
    """As above where the weights of all the room lie in shared memory, and where they would not; no page behind the tokens."""
    keep, recent, page = 2000, 64, 64
    pages, wide = -(-n // page), -(-room // page)
    held = [torch.zeros(pages, page, 1, 64 // m, dtype=torch.uint8, device="cuda") for m in (2, 2, 16, 16)]
    held[0].view(torch.int64)[..., 0, 0] = torch.arange(pages * page, device="cuda").view(pages, page)
    table = torch.full((1, wide), -1, dtype=torch.int32)
    table[0, :pages] = torch.arange(pages)
    cache = h3.PagedKV4(*held, table.cuda(), torch.tensor([n], dtype=torch.int32, device="cuda"))
    w = weights_of(kind, (1, wide * page), n).cuda()
    before, out = w.clone(), torch.zeros(1, dtype=torch.int32, device="cuda")
    h3.h3attn_paged_evict(cache, w, keep, recent, out, h3.paged_evict_workspace(cache, keep, recent))
    assert out.tolist() == [keep] and h3.h3attn_check_device_status() == 0
    front, old = keep - recent, n - recent
    stay = torch.sort(before[0, :old], descending=True, stable=True)[1][:front].sort()[0]
    want = torch.arange(keep, device="cuda")
    want[torch.ones(front, dtype=torch.bool, device="cuda").index_fill_(0, stay[stay < front], False).nonzero()[:, 0]] = stay[stay >= front]
    want[front:] = torch.arange(old, n, device="cuda")
    assert torch.equal(held[0].view(torch.int64).view(-1, 4)[:keep, 0], want)
    assert torch.equal(w[0, :keep], before[0, want]) and bool((w[0, keep:n] == 0).all()) and torch.equal(w[0, n:], before[0, n:])
