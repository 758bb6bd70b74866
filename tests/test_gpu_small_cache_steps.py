"""Steps of a bounded generation, each of them whole: the weights that a step leaves
are taken from the same append and decode on copies, which repeat bit for bit, and what
the eviction makes of them and of the pages is the definition's bit for bit.  The step that
README shows, which evicts at every token, and one that evicts once in several."""
import pytest
import torch

from cache4_ref import Pages, evict
from generate_ref import randn
from test_gpu_evict import bits_of
from test_gpu_small_cache_loop import readme_step


class Loop:
    def __init__(self, h3, bits, begin, keep, recent, room, Hq=8, Hkv=2, D=128, page=16):
        self.h3, self.keep, self.recent, self.page, self.Hq, self.Hkv, self.D = h3, keep, recent, page, Hq, Hkv, D
        B = len(begin)
        self.B, self.bits, self.begin = B, bits, list(begin)
        p = self.p = Pages(bits, B, room, page, Hkv, D, 1, poison=False).hold()
        self.cache = p.cuda(h3, begin)
        self.lens, self.after = p.dlen, torch.zeros_like(p.dlen)
        d = dict(dtype=torch.bfloat16, device="cuda")
        self.qkv = torch.zeros(B, 1, (Hq + 2 * Hkv) * D, **d)
        self.q, self.k, self.v = (t.unflatten(-1, (-1, D)) for t in self.qkv.split([Hq * D, Hkv * D, Hkv * D], -1))
        self.q1, self.o = torch.empty(B, 1, Hq, D, **d), torch.empty(B, 1, Hq, D, **d)
        self.wq, self.wk = (torch.rand(2, D, generator=torch.Generator().manual_seed(3)) + 0.5).cuda().unbind()
        self.cos, self.sin = torch.empty(400, 48, device="cuda"), torch.empty(400, 48, device="cuda")
        h3.h3attn_rope_table(self.cos, self.sin, 96)
        self.pos = torch.tensor(begin, dtype=torch.int32, device="cuda")[:, None].clone()
        self.weights = torch.zeros(B, p.table.shape[1] * page, device="cuda")

    def append(self, cache, q1, pos, after):
        call = self.h3.h3attn_qk_norm_rope_append_q4 if self.bits == 4 else self.h3.h3attn_qk_norm_rope_append
        call(self.q, self.k, self.v, q1, cache, self.wq, self.wk, self.cos, self.sin, 96, pos=pos, len_out=after)

    def copies(self):
        """The same step up to its eviction, on copies: (pages, weights, o, lengths)."""
        h3, held, w = self.h3, [t.clone() for t in self.p.dheld], self.weights.clone()
        cache = (h3.PagedKV4 if self.bits == 4 else h3.PagedKV)(*held, self.p.dtable, self.lens.clone())
        q1, o, after = torch.empty_like(self.q1), torch.empty_like(self.o), torch.zeros_like(self.after)
        self.append(cache, q1, self.pos.clone(), after)
        grown = cache.with_lengths(after)
        h3.h3attn_paged_decode_weights(q1, o, grown, w, h3.paged_decode_weights_workspace(q1, grown))
        return [t.cpu() for t in held], w.cpu(), o.cpu(), after.tolist()

    def compare(self, held, w, o, lens, what):
        assert torch.equal(bits_of(self.o.cpu()), bits_of(o)), what
        assert torch.equal(bits_of(self.weights.cpu()), bits_of(w)), what
        assert all(torch.equal(bits_of(a.cpu()), bits_of(b)) for a, b in zip(self.p.dheld, held)), what
        assert self.lens.tolist() == list(lens), what


@pytest.mark.gpu
@pytest.mark.parametrize("graph", [False, True])
@pytest.mark.parametrize("keep,recent", [(48, 8), (40, 0), (33, 33), (200, 150)])
def test_the_readme_step(h3, graph, keep, recent):
    loop = Loop(h3, 4, [keep - 5, 0, keep], keep, recent, keep + 1)
    c = loop.cache
    names = dict(h3=h3, k_codes=c.k_codes, v_codes=c.v_codes, k_scales=c.k_scales, v_scales=c.v_scales, page_table=loop.p.dtable,
                 lens=loop.lens, after=loop.after, keep=keep, recent=recent, q=loop.q, k=loop.k, v=loop.v, q1=loop.q1, o=loop.o,
                 wq=loop.wq, wk=loop.wk, cos=loop.cos, sin=loop.sin, pos=loop.pos, weights=loop.weights)
    exec(readme_step(), names)
    run = names["bounded_step"]
    if graph:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            names["bounded_step"]()
        run = g.replay
    evicted = 0
    for t in range(24):
        loop.qkv.copy_(randn(*loop.qkv.shape, seed=100 + t))
        held, w, o, lens = loop.copies()
        run()
        torch.cuda.synchronize()
        evicted += sum(n > keep for n in lens)
        loop.compare(*evict(held, loop.p.table, lens, loop.page, w, keep, recent)[:2], o, [min(n, keep) for n in lens], f"step {t}")
    assert evicted == 24 + 24 - 5 + max(24 - keep, 0)
    assert h3.h3attn_check_device_status() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("bits", [4, 16])
@pytest.mark.parametrize("every,keep,recent", [(8, 48, 8), (8, 48, 48), (32, 40, 36)])
def test_evictions_once_in_several_steps(h3, bits, every, keep, recent):
    """Tables with room for keep + every tokens; lengths go from one array to the other and back."""
    loop = Loop(h3, bits, [keep - 5, 0, keep], keep, recent, keep + every)
    lens, after = loop.cache.kv_len, loop.after
    ws = h3.paged_decode_weights_workspace(loop.q1, loop.cache)
    ws_evict = h3.paged_evict_workspace(loop.cache, keep, recent)
    evicted = 0
    for t in range(3 * every):
        loop.qkv.copy_(randn(*loop.qkv.shape, seed=100 + t))
        loop.lens = lens
        held, w, o, want = loop.copies()
        loop.append(loop.cache.with_lengths(lens), loop.q1, loop.pos, after)
        grown = loop.cache.with_lengths(after)
        h3.h3attn_paged_decode_weights(loop.q1, loop.o, grown, loop.weights, ws)
        if t % every == every - 1:
            h3.h3attn_paged_evict(grown, loop.weights, keep, recent, lens, ws_evict)
            evicted += sum(n - keep for n in want if n > keep)
            held, w, _ = evict(held, loop.p.table, want, loop.page, w, keep, recent)
            want = [min(n, keep) for n in want]
        else:
            lens, after = after, lens
        loop.pos.add_(1)
        torch.cuda.synchronize()
        loop.lens = lens
        loop.compare(held, w, o, want, f"step {t}")
    assert evicted == 2 * 3 * every - 5 + max(3 * every - keep, 0)
    assert h3.h3attn_check_device_status() == 0
