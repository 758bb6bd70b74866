"""The 4-bit cache, the tokens' weights and the eviction together: the bounded step
as README shows it, run from there, token by token, eagerly and replayed; and a prompt
that goes through the cache into a prefill."""
import os
import re
import textwrap

import pytest
import torch

from cache4_ref import Pages, attend, evict, store, values
from generate_ref import randn

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def readme_step():
    with open(os.path.join(ROOT, "README.md")) as f:
        blocks = [textwrap.dedent(b) for b in re.findall(r"```python\n(.*?)```", f.read(), re.S)]
    return next(b for b in blocks if "h3attn_paged_evict" in b)


@pytest.mark.gpu
@pytest.mark.parametrize("graph", [False, True])
def test_the_readme_step(h3, graph):
    B, Hq, Hkv, D, page, keep, recent, tokens = 3, 8, 2, 128, 16, 48, 8, 40
    begin = [40, 0, 48]
    p = Pages(4, B, keep + 1, page, Hkv, D, 1, poison=False).hold()
    small = p.cuda(h3, begin)
    lens = p.dlen
    d = dict(dtype=torch.bfloat16, device="cuda")
    qkv = torch.zeros(B, 1, (Hq + 2 * Hkv) * D, **d)
    q, k, v = (t.unflatten(-1, (-1, D)) for t in qkv.split([Hq * D, Hkv * D, Hkv * D], -1))
    names = dict(h3=h3, k_codes=small.k_codes, v_codes=small.v_codes, k_scales=small.k_scales, v_scales=small.v_scales,
                 page_table=p.dtable, lens=lens, after=torch.zeros_like(lens), keep=keep, recent=recent, q=q, k=k, v=v,
                 q1=torch.empty(B, 1, Hq, D, **d), o=torch.empty(B, 1, Hq, D, **d), wq=torch.ones(D, device="cuda"),
                 wk=torch.ones(D, device="cuda"), cos=torch.empty(200, 48, device="cuda"), sin=torch.empty(200, 48, device="cuda"),
                 pos=torch.tensor(begin, dtype=torch.int32, device="cuda")[:, None].clone(),
                 weights=torch.zeros(B, p.table.shape[1] * page, device="cuda"))
    h3.h3attn_rope_table(names["cos"], names["sin"], 96)
    exec(readme_step(), names)
    run = names["bounded_step"]
    if graph:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            names["bounded_step"]()
        run = g.replay
    want_lens = list(begin)
    for t in range(tokens):
        qkv.copy_(randn(B, 1, qkv.shape[-1], seed=100 + t))
        before, w_before = [x.cpu() for x in p.dheld], names["weights"].cpu()
        run()
        torch.cuda.synchronize()
        # the appended rows, as the bf16 append would round them
        rows = [torch.zeros(B, 1, Hkv, D, **d) for _ in range(2)]
        q2 = torch.empty_like(names["q1"])
        pages = [torch.zeros(B, 1, Hkv, D, **d) for _ in range(2)]
        each = h3.PagedKV(*pages, torch.arange(B, dtype=torch.int32, device="cuda")[:, None].contiguous(), torch.zeros_like(lens))
        h3.h3attn_qk_norm_rope_append(q, k, v, q2, each, names["wq"], names["wk"], names["cos"], names["sin"], 96,
                                      pos=names["pos"] - 1)
        assert torch.equal(q2, names["q1"])
        for b, n in enumerate(want_lens):
            at = int(p.table[b, n // page]), n % page
            for i in range(2):
                before[i][at], before[2 + i][at] = store(pages[i][b, 0].cpu())
        want_lens = [n + 1 for n in want_lens]
        # attention over what was there, and the weights that it leaves
        kv = [values(before[i], before[2 + i]) for i in range(2)]
        o, bound, w, w_bound = attend(names["q1"].cpu()[:, 0], kv, p.table, want_lens, page, D ** -0.5)
        assert bool(((names["o"].cpu()[:, 0].double() - o).abs() <= bound).all()), t
        # what stays: by the weights as the step has them, within their bound of the reference's
        total = w_before.double() + w
        got = names["weights"].cpu().double()
        held = [x.cpu() for x in p.dheld]
        for b, n in enumerate(want_lens):
            off = w_bound[b].sum() + total[b].sum() * 2.0 ** -22   # and each sum rounded to float32, here and in the step
            if n <= keep:
                assert bool(((got[b, :n] - total[b, :n]).abs() <= w_bound[b, :n] + total[b, :n] * 2.0 ** -22).all())
                assert all(torch.equal(x[p.table[b].long()], y[p.table[b].long()]) for x, y in zip(held, before))
            else:
                assert n == keep + 1
                old = total[b, :n - recent]
                assert float(old.sum() - old.min() + total[b, n - recent:n].sum()) == pytest.approx(float(got[b, :keep].sum()), abs=float(off))
                order = old.sort().values
                if float(order[1] - order[0]) > 2 * float(off):   # one token is clearly the lightest: the whole step is known
                    one, _, _ = evict(before, p.table[b:b + 1], [n], page, total[b:b + 1].float(), keep, recent)
                    assert all(torch.equal(x[p.table[b].long()], y[p.table[b].long()]) for x, y in zip(held, one))
        want_lens = [min(n, keep) for n in want_lens]
        assert lens.tolist() == want_lens
        assert names["pos"].flatten().tolist() == [n + t + 1 for n in begin]
    assert h3.h3attn_check_device_status() == 0


@pytest.mark.gpu
def test_a_prompt_through_the_cache_into_a_prefill(h3):
    """A prompt's first part is appended in 4 bits and read back; the second part's queries attend it in one prefill, the
    same as its tokens one by one in the decode."""
    B, S, Hq, Hkv, D, page, more = 2, 150, 8, 2, 128, 24, 5
    p = Pages(4, B, S, page, Hkv, D, 3).hold()
    cache = p.cuda(h3, [0, 0])
    k, v = randn(B, S, Hkv, D, seed=4).cuda(), randn(B, S, Hkv, D, seed=5).cuda()
    new = torch.tensor([S, 97], dtype=torch.int32, device="cuda")
    after = torch.empty_like(new)
    h3.h3attn_qk_norm_rope_append_q4(None, k, v, None, cache, None, None, None, None, 0, new_len=new, len_out=after)
    grown = cache.with_lengths(after)
    rows = [torch.zeros(B, S, Hkv, D, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    h3.h3attn_paged_read(grown, *rows)
    q = randn(B, more, Hq, D, seed=6).cuda()
    o = torch.empty_like(q)
    h3.h3attn_prefill(q, *rows, o, mask=h3.Mask(kv_len=after))
    one = torch.empty(B, Hq, D, dtype=torch.bfloat16, device="cuda")
    for i in range(more):
        h3.h3attn_paged_decode_q4(q[:, i].contiguous(), one, grown, workspace=h3.paged_decode_q4_workspace(one, grown))
        # both within their bounds of the exact output: bf16 rounding of it, and of P in the prefill (2^-8 of the weights)
        ref, bound, _, _ = attend(q[:, i].cpu(), [values(*(t.cpu() for t in (p.dheld[j], p.dheld[2 + j]))) for j in range(2)], p.table,
                                  after.tolist(), page, D ** -0.5)
        assert bool(((one.cpu().double() - ref).abs() <= bound).all())
        vmax = rows[1].abs().amax().item()
        assert float((o[:, i].cpu().double() - ref).abs().max()) <= 2.0 ** -7 * vmax
    assert h3.h3attn_check_device_status() == 0


@pytest.mark.gpu
def test_two_calls_at_once(h3):
    """Two streams, each with its own workspaces."""
    cases = []
    for seed in (1, 2):
        p = Pages(4, 2, 3000, 16, 2, 128, seed, poison=False).hold()
        cache = p.cuda(h3, [3000, 700])
        q = randn(2, 8, 128, seed=seed + 9).cuda()
        w = torch.zeros(2, p.table.shape[1] * 16, device="cuda")
        cases.append((p, cache, q, w, torch.empty_like(q), h3.paged_decode_weights_workspace(q, cache), h3.paged_evict_workspace(cache, 600, 40),
                      torch.zeros(2, dtype=torch.int32, device="cuda"), torch.cuda.Stream()))
    torch.cuda.synchronize()
    for p, cache, q, w, o, ws, we, out, stream in cases:
        h3.h3attn_paged_decode_weights(q, o, cache, w, ws, stream=stream)
        h3.h3attn_paged_evict(cache, w, 600, 40, out, we, stream=stream)
    torch.cuda.synchronize()
    for p, cache, q, w, o, ws, we, out, stream in cases:
        ref, bound, _, _ = attend(q.cpu(), p.kv, p.table, [3000, 700], 16, 128 ** -0.5)
        assert bool(((o.cpu().double() - ref).abs() <= bound).all())
        assert out.tolist() == [600, 600]
