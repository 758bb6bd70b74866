"""Decode with weights and eviction of two caches on two streams at once: outputs,
weights, pages and lengths bit for bit those of each run alone, which are the
definition's for the weights that they had."""
import pytest
import torch

from cache4_ref import Pages, evict
from generate_ref import randn
from test_gpu_evict import bits_of

LENS, PAGE, KEEP, RECENT, HQ, HKV, D = [3000, 700, 601, 90], 16, 600, 40, 8, 2, 128


class Calls:
    """Three decodes whose weights add up, then the eviction by them, on copies of one cache."""

    def __init__(self, h3, bits, seed):
        self.h3, self.p = h3, Pages(bits, len(LENS), max(LENS), PAGE, HKV, D, seed, poison=False).hold()
        self.room = self.p.table.shape[1] * PAGE
        self.q = [randn(len(LENS), HQ, D, seed=seed + 9 + i).cuda() for i in range(3)]
        self.fresh()
        self.ws = h3.paged_decode_weights_workspace(self.q[0], self.cache)
        self.ws_evict = h3.paged_evict_workspace(self.cache, KEEP, RECENT)

    def fresh(self):
        self.cache = self.p.cuda(self.h3, LENS)
        self.o = [torch.full_like(q, float("nan")) for q in self.q]
        self.w = torch.zeros(len(LENS), self.room, device="cuda")
        self.out = torch.full((len(LENS),), -9, dtype=torch.int32, device="cuda")
        self.added = torch.empty_like(self.w)

    def decode(self, i):
        self.h3.h3attn_paged_decode_weights(self.q[i], self.o[i], self.cache, self.w, self.ws)

    def evict(self):
        self.added.copy_(self.w)
        self.h3.h3attn_paged_evict(self.cache, self.w, KEEP, RECENT, self.out, self.ws_evict)

    def results(self):
        return [bits_of(t).cpu() for t in (*self.o, self.added, *self.p.dheld, self.w, self.out)]


@pytest.mark.gpu
@pytest.mark.parametrize("bits", [4, 16])
def test_two_streams(h3, bits):
    cases = [Calls(h3, bits, seed) for seed in (1, 2)]
    alone = []
    for c in cases:
        for i in range(3):
            c.decode(i)
        c.evict()
        torch.cuda.synchronize()
        held, w, out = evict(c.p.held, c.p.table, LENS, PAGE, c.added.cpu(), KEEP, RECENT)
        assert torch.equal(c.out.cpu(), out) and torch.equal(bits_of(c.w.cpu()), bits_of(w))
        for got, want in zip(c.p.dheld, held):
            assert torch.equal(bits_of(got.cpu()), bits_of(want))
        alone.append(c.results())
    streams = [torch.cuda.Stream() for _ in cases]
    for turn in range(5):
        for c in cases:
            c.fresh()
        torch.cuda.synchronize()
        steps = [lambda c, i=i: c.decode(i) for i in range(3)] + [lambda c: c.evict()]
        for step in steps:
            for c, stream in zip(cases, streams):
                with torch.cuda.stream(stream):
                    step(c)
        torch.cuda.synchronize()
        for c, want in zip(cases, alone):
            assert all(torch.equal(a, b) for a, b in zip(c.results(), want)), f"turn {turn}"
    assert h3.h3attn_check_device_status() == 0
