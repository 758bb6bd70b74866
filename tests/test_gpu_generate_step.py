"""The generation operators together, as a block that generates calls them: the
prompt's rows are appended and attended by the prefill, then tokens follow one
by one through norm, projection, append and decode.  Each token's attention has
to be that of the causal prefill over the whole sequence."""
import pytest
import torch

from generate_ref import BF16_HALF, randn


@pytest.mark.gpu
@pytest.mark.parametrize("graph", [False, True])
def test_tokens_one_by_one_are_the_causal_prefill(h3, graph):
    B, Hq, Hkv, D, C, page, rot = 3, 8, 2, 128, 512, 16, 96
    prompt, new, S = [40, 17, 1], 6, 48
    x = randn(B, S, C, seed=1).cuda()
    res = randn(B, S, C, seed=2).cuda()
    w_norm = torch.rand(C, generator=torch.Generator().manual_seed(3)).cuda() + 0.5
    w_qkv = (randn(C, (Hq + 2 * Hkv) * D, seed=4) * C ** -0.5).cuda()
    wq = torch.rand(D, generator=torch.Generator().manual_seed(5)).cuda() + 0.5
    wk = torch.rand(D, generator=torch.Generator().manual_seed(6)).cuda() + 0.5
    cos, sin = torch.empty(S, rot // 2, device="cuda"), torch.empty(S, rot // 2, device="cuda")
    h3.h3attn_rope_table(cos, sin, rot, scaling=h3.RopeScaling("by_parts", 4.0, 16, amplitude=1.1))

    def project(xs, rs):
        """norm and projection of [B, n, C] rows -> q, k, v slices, and the stream"""
        n = xs.shape[1]
        flat_h = torch.empty(B * n, C, dtype=torch.bfloat16, device="cuda")
        y = torch.empty_like(flat_h)
        h3.h3attn_add_rmsnorm(xs.reshape(-1, C), rs.reshape(-1, C), flat_h, y, w_norm)
        qkv = (y @ w_qkv).view(B, n, -1)
        return [t.unflatten(-1, (-1, D)) for t in qkv.split([Hq * D, Hkv * D, Hkv * D], -1)]

    # all rows at once through the contiguous calls
    q, k, v = project(x, res)
    qf, kf, vf = q.contiguous(), k.contiguous(), v.contiguous()
    h3.h3attn_qk_norm_rope(qf, kf, wq, wk, cos, sin, rot)
    full = torch.empty_like(qf)
    h3.h3attn_prefill(qf, kf, vf, full, causal=True)

    # the prompts in one padded batch, then a token at a time
    each = -(-S // page)
    table = torch.randperm(B * each, generator=torch.Generator().manual_seed(7)).to(torch.int32).view(B, each).cuda()
    pages = torch.full((2, B * each, page, Hkv, D), float("nan"), dtype=torch.bfloat16, device="cuda")
    lens = torch.zeros(B, dtype=torch.int32, device="cuda")
    after = torch.empty_like(lens)
    cache = h3.PagedKV(pages[0], pages[1], table, lens)
    grown = cache.with_lengths(after)
    P = max(prompt)
    q, k, v = (t[:, :P] for t in (q, k, v))
    q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    q_out = torch.zeros(B, P, Hq, D, dtype=torch.bfloat16, device="cuda")
    h3.h3attn_qk_norm_rope_append(q, k, v, q_out, cache, wq, wk, cos, sin, rot,
                                  new_len=torch.tensor(prompt, dtype=torch.int32, device="cuda"), len_out=after)
    assert after.tolist() == prompt
    for b in range(B):
        assert torch.equal(q_out[b, :prompt[b]], qf[b, :prompt[b]]) and bool((q_out[b, prompt[b]:] == 0).all())

    xs, rs = torch.empty(B, 1, C, dtype=torch.bfloat16, device="cuda"), torch.empty(B, 1, C, dtype=torch.bfloat16, device="cuda")
    q1 = torch.empty(B, 1, Hq, D, dtype=torch.bfloat16, device="cuda")
    o1 = torch.empty_like(q1)
    ws = h3.paged_decode_workspace(q1, grown)
    y1, h1 = torch.empty(B, C, dtype=torch.bfloat16, device="cuda"), torch.empty(B, C, dtype=torch.bfloat16, device="cuda")
    qkv1 = torch.empty(B, (Hq + 2 * Hkv) * D, dtype=torch.bfloat16, device="cuda")

    def step():
        lens.copy_(after)
        h3.h3attn_add_rmsnorm(xs.view(B, C), rs.view(B, C), h1, y1, w_norm)
        torch.mm(y1, w_qkv, out=qkv1)
        a, b, c = (t.unflatten(-1, (-1, D)) for t in qkv1.view(B, 1, -1).split([Hq * D, Hkv * D, Hkv * D], -1))
        h3.h3attn_qk_norm_rope_append(a, b, c, q1, cache, wq, wk, cos, sin, rot, len_out=after)
        h3.h3attn_paged_decode(q1, o1, grown, workspace=ws)

    run = step
    if graph:
        kept = after.clone()
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):  # the product's library sets itself up before the capture
            torch.mm(y1, w_qkv, out=qkv1)
        torch.cuda.current_stream().wait_stream(s)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            step()
        after.copy_(kept)
        run = g.replay
    for t in range(new):
        at = [n + t for n in prompt]
        xs.copy_(torch.stack([x[b, i:i + 1] for b, i in enumerate(at)]))
        rs.copy_(torch.stack([res[b, i:i + 1] for b, i in enumerate(at)]))
        run()
        torch.cuda.synchronize()
        assert after.tolist() == [i + 1 for i in at]
        for b, i in enumerate(at):
            # The library's product of one row may round a sum of C terms the other way than that of many rows, by one bf16
            # step of its inputs to the norm: both attentions round their weights and outputs to bf16 besides.
            ref = full[b, i].float()
            scale = vf[b, :i + 1].float().abs().amax()
            assert bool(((o1[b, 0].float() - ref).abs() <= 16 * BF16_HALF * scale).all()), (t, b)
    assert h3.h3attn_check_device_status() == 0
