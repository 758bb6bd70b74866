"""Empty batches and steps through the Python binding: tensors without elements
are taken, and what has rows still gets them."""
import pytest
import torch


def step(h3, B, S, kv_len=5):
    d = dict(dtype=torch.bfloat16, device="cuda")
    pages, more = torch.full((4, 16, 2, 64), 3.0, **d), torch.full((4, 16, 2, 64), 3.0, **d)
    table = torch.arange(4, dtype=torch.int32, device="cuda")[:2 * B].view(B, 2)
    cache = h3.PagedKV(pages, more, table, torch.full((B,), kv_len, dtype=torch.int32, device="cuda"))
    q, k = torch.ones(B, S, 4, 64, **d), torch.ones(B, S, 2, 64, **d)
    w, cos = torch.ones(64, device="cuda"), torch.ones(32, 32, device="cuda")
    return cache, (q, k, k.clone(), torch.empty_like(q), cache, w, w, cos, cos.clone(), 64)


@pytest.mark.gpu
@pytest.mark.parametrize("B,S", [(2, 0), (0, 3), (0, 0)])
def test_append_of_no_tokens(h3, B, S):
    cache, args = step(h3, B, S)
    assert h3.h3attn_qk_norm_rope_append(*args) is args[3]
    torch.cuda.synchronize()
    assert bool((cache.k_pages == 3).all()) and bool((cache.v_pages == 3).all())
    assert h3.h3attn_check_device_status() == 0


@pytest.mark.gpu
def test_an_empty_slice_of_a_step(h3):
    cache, args = step(h3, 2, 3)
    q, k, v, o = (t[:, :0] for t in args[:4])
    h3.h3attn_qk_norm_rope_append(q, k, v, o.contiguous(), *args[4:])
    torch.cuda.synchronize()
    assert bool((cache.k_pages == 3).all())


@pytest.mark.gpu
def test_the_others_of_no_rows(h3):
    cache, args = step(h3, 0, 1)
    q = args[0]
    o = torch.empty_like(q)
    assert h3.paged_decode_workspace(q, cache) is None
    assert h3.h3attn_paged_decode(q, o, cache) is o
    x = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda")
    h3.h3attn_add_rmsnorm(x, x.clone(), x.clone(), x.clone())
    cos = torch.empty(0, 32, device="cuda")
    h3.h3attn_rope_table(cos, cos.clone(), 64)


@pytest.mark.gpu
def test_a_step_without_tokens_leaves_the_lengths_in_len_out(h3):
    """What decode takes next: the lengths as append counts them, not what the buffer held before."""
    cache, args = step(h3, 2, 0)
    cache.kv_len.copy_(torch.tensor([17, -4], dtype=torch.int32))
    out, new = torch.full((3,), 1000, dtype=torch.int32, device="cuda"), torch.tensor([2, -1], dtype=torch.int32, device="cuda")
    for new_len in (None, new):
        out.fill_(1000)
        h3.h3attn_qk_norm_rope_append(*args, new_len=new_len, len_out=out[:2])
        assert out.tolist() == [17, 0, 1000]
    cache.kv_len[0] = 40                                   # above the capacity of 32
    h3.h3attn_qk_norm_rope_append(None, *args[1:3], None, cache, None, None, None, None, 0, len_out=out[:2])
    assert out.tolist() == [32, 0, 1000]
    assert bool((cache.k_pages == 3).all()) and h3.h3attn_check_device_status() == 0
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        h3.h3attn_qk_norm_rope_append(*args, len_out=out[:2])
    cache.kv_len.copy_(torch.tensor([3, 9], dtype=torch.int32))
    graph.replay()
    torch.cuda.synchronize()
    assert out.tolist() == [3, 9, 1000]
    cache, args = step(h3, 0, 0)
    h3.h3attn_qk_norm_rope_append(*args, len_out=out[:0])
    assert h3.h3attn_check_device_status() == 0
