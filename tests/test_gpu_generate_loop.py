"""The generation step as README shows it, run from there: token by token, eagerly
and replayed from a graph, it appends each token behind the one before and attends
all of them."""
import os
import re
import textwrap

import pytest
import torch

from generate_ref import decode_f64, randn

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def readme_step():
    with open(os.path.join(ROOT, "README.md")) as f:
        blocks = [textwrap.dedent(b) for b in re.findall(r"```python\n(.*?)```", f.read(), re.S)]
    return next(b for b in blocks if "h3attn_paged_decode" in b)


@pytest.mark.gpu
@pytest.mark.parametrize("graph", [False, True])
def test_the_readme_step(h3, graph):
    B, Hq, Hkv, D, C, page, tokens = 3, 8, 2, 128, 512, 16, 40
    begin = [0, 15, 290]
    each = -(-(max(begin) + tokens) // page)
    order = torch.randperm(B * each, generator=torch.Generator().manual_seed(1)).to(torch.int32).view(B, each)
    k_pages, v_pages = (torch.full((B * each, page, Hkv, D), float("nan"), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    prompt_k, prompt_v = randn(B, max(begin), Hkv, D, seed=2), randn(B, max(begin), Hkv, D, seed=3)
    for b, n in enumerate(begin):
        at = torch.arange(n)
        where = order[b][at // page].long().cuda(), (at % page).cuda()
        k_pages[where], v_pages[where] = prompt_k[b, :n].cuda(), prompt_v[b, :n].cuda()
    lens = torch.tensor(begin, dtype=torch.int32, device="cuda")
    d = dict(dtype=torch.bfloat16, device="cuda")
    qkv = torch.zeros(B, 1, (Hq + 2 * Hkv) * D, **d)
    q, k, v = (t.unflatten(-1, (-1, D)) for t in qkv.split([Hq * D, Hkv * D, Hkv * D], -1))
    x = randn(B, C, seed=4).cuda()
    names = dict(h3=h3, cache=h3.PagedKV(k_pages, v_pages, order.cuda(), lens), lens=lens, after=torch.zeros_like(lens),
                 x=x, residual=x.clone(), h=torch.empty_like(x), y=torch.empty_like(x), w=torch.ones(C, device="cuda"),
                 q=q, k=k, v=v, q1=torch.empty(B, 1, Hq, D, **d), o=torch.empty(B, 1, Hq, D, **d),
                 wq=torch.ones(D, device="cuda"), wk=torch.ones(D, device="cuda"),
                 cos=torch.empty(each * page, 48, device="cuda"), sin=torch.empty(each * page, 48, device="cuda"))
    h3.h3attn_rope_table(names["cos"], names["sin"], 96)
    exec(readme_step(), names)
    run = names.get("step")
    if graph:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            names["step"]()
        run = g.replay
    for t in range(tokens):
        qkv.copy_(randn(B, 1, qkv.shape[-1], seed=100 + t))
        run()
        torch.cuda.synchronize()
        assert lens.tolist() == [n + t + 1 for n in begin]
        for b, n in enumerate(begin):                                 # the token's own row, behind the one before
            at = n + t
            assert torch.equal(v_pages[order[b, at // page].item(), at % page], v[b, 0])
        if t % 13 == 0 or t == tokens - 1:
            o, bound = decode_f64(names["q1"].cpu()[:, 0], k_pages.cpu(), v_pages.cpu(), order, lens.tolist(), page, D ** -0.5)
            assert bool(((names["o"].cpu()[:, 0].double() - o).abs() <= bound).all()), t
    assert h3.h3attn_check_device_status() == 0
