"""What the Python binding of the generation operators refuses on CUDA tensors,
and the strides, streams and argument forms that it takes."""
import os
import subprocess
import sys

import pytest
import torch

from generate_ref import randn


@pytest.fixture
def t():
    """Tensors of one step: B 2, S 1, 4 query and 2 key-value heads of 64."""
    d = dict(dtype=torch.bfloat16, device="cuda")
    pages = torch.zeros(8, 16, 2, 64, **d)
    return dict(q=torch.zeros(2, 1, 4, 64, **d), k=torch.zeros(2, 1, 2, 64, **d), pages=pages, more=torch.zeros_like(pages),
                table=torch.arange(4, dtype=torch.int32, device="cuda").view(2, 2),
                lens=torch.zeros(2, dtype=torch.int32, device="cuda"), cos=torch.zeros(16, 32, device="cuda"),
                w=torch.ones(64, device="cuda"), x=torch.zeros(4, 64, **d))


def cache(h3, t):
    return h3.PagedKV(t["pages"], t["more"], t["table"], t["lens"])


@pytest.mark.gpu
def test_paged_kv_refuses(h3, t):
    for change in (dict(pages=t["pages"].float()), dict(pages=t["pages"].transpose(1, 2)), dict(more=t["more"][:4]),
                   dict(table=t["table"].long()), dict(lens=t["lens"][:1]), dict(lens=t["lens"].cpu()), dict(table=t["table"][0]),
                   dict(pages=t["pages"].clone().requires_grad_())):
        with pytest.raises(h3.H3AttnError):
            cache(h3, {**t, **change})


@pytest.mark.gpu
def test_append_refuses(h3, t):
    c = cache(h3, t)

    def call(q=t["q"], k=t["k"], v=t["k"].clone(), o=t["q"].clone(), c=c, wq=t["w"], cos=t["cos"], rot=64, **more):
        h3.h3attn_qk_norm_rope_append(q, k, v, o, c, wq, t["w"], cos, t["cos"].clone(), rot, **more)
    call()
    for bad in (dict(q=None), dict(o=None), dict(q=t["q"].float()), dict(k=t["k"][:1]), dict(v=t["k"].cpu()), dict(o=t["q"][..., :32]),
                dict(wq=t["w"][:32]), dict(wq=t["w"].double()), dict(cos=None), dict(cos=t["cos"][:, :16]), dict(rot=63), dict(rot=130),
                dict(c=None), dict(c=t["pages"]), dict(pos=t["lens"]), dict(new_len=t["lens"].long()),
                dict(len_out=t["lens"]),                       # over kv_len itself
                dict(k=t["k"].expand(2, 1, 2, 64).clone().requires_grad_()), dict(eps=float("nan")),
                dict(q=torch.zeros(2, 1, 64, 4, dtype=torch.bfloat16, device="cuda").transpose(2, 3)),  # heads not behind one another
                dict(q=t["q"][:1].expand(2, 1, 4, 64))):       # the same token twice
        with pytest.raises(h3.H3AttnError):
            call(**bad)
    torch.cuda.synchronize()
    assert h3.h3attn_check_device_status() == 0


@pytest.mark.gpu
def test_decode_refuses(h3, t):
    c, q = cache(h3, t), t["q"]
    h3.h3attn_paged_decode(q, torch.empty_like(q), c)
    for bad in ((q[0], q.clone(), c), (q, q, c), (q, q.float(), c), (q, q[:, :, :2].clone(), c), (q.cpu(), q.clone(), c),
                (q, q.clone(), None), (q[:1], q[:1].clone(), c), (q.expand(2, 1, 4, 64).transpose(0, 1), q.clone(), c),
                (torch.cat((q, q), 1), torch.cat((q, q), 1), c), (q[:, :, :3].clone(), q[:, :, :3].clone(), c)):
        with pytest.raises(h3.H3AttnError):
            h3.h3attn_paged_decode(*bad)
    with pytest.raises(h3.H3AttnError):
        h3.h3attn_paged_decode(q, torch.empty_like(q), c, workspace=torch.empty(16))
    with pytest.raises(TypeError):
        h3.h3attn_paged_decode(q, torch.empty_like(q), c, scale="half")


@pytest.mark.gpu
def test_add_rmsnorm_and_table_refuse(h3, t):
    x, y8 = t["x"], torch.zeros(4, 64, device="cuda").to(torch.float8_e4m3fn)
    s = torch.zeros(4, device="cuda")
    for bad in ((x.float(), None, None, x), (x, x, None, x.clone()), (x, None, x.clone(), x.clone()), (x, None, None, x[:2]),
                (x, None, None, x.clone(), t["w"][:8]), (x, None, None, x.clone(), None, 1e-6, s), (x, None, None, y8),
                (x, None, None, y8, None, 1e-6, s[:2]), (x, None, None, y8, None, 1e-6, s.double()),
                (x, None, None, y8, None, 1e-6, torch.zeros(4, 3, dtype=torch.uint8, device="cuda")),
                (x.t(), None, None, x.t().clone()), (x[0], None, None, x[0].clone()), (x, None, None, x.clone(), None, -1.0)):
        with pytest.raises(h3.H3AttnError):
            h3.h3attn_add_rmsnorm(*bad)
    cos, sin = t["cos"], t["cos"].clone()
    for bad in ((cos, sin, 62), (cos, sin[:8], 64), (cos, cos, 64), (cos.double(), sin.double(), 64), (cos, sin, 64, 0.5),
                (cos, sin, 64, 1e4, None, t["lens"]), (cos, sin, 64, 1e4, None, None, -1),
                (cos, sin, 64, 1e4, h3.RopeScaling("linear", 0.5)), (cos.t().contiguous().t(), sin, 64)):
        with pytest.raises(h3.H3AttnError):
            h3.h3attn_rope_table(*bad)


@pytest.mark.gpu
def test_stream_arguments(h3, t):
    """None, a torch stream and a handle."""
    x = randn(4, 64, seed=1).cuda()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    outs = [torch.zeros_like(x) for _ in range(4)]
    h3.h3attn_add_rmsnorm(x, None, None, outs[0])
    h3.h3attn_add_rmsnorm(x, None, None, outs[1], stream=s)
    h3.h3attn_add_rmsnorm(x, None, None, outs[2], stream=s.cuda_stream)
    with torch.cuda.stream(s):
        h3.h3attn_add_rmsnorm(x, None, None, outs[3])
    torch.cuda.synchronize()
    assert all(torch.equal(o, outs[0]) for o in outs)
    with pytest.raises(AttributeError):
        h3.h3attn_add_rmsnorm(x, None, None, outs[0], stream="default")


@pytest.mark.gpu
def test_token_strides(h3):
    """Wider than the heads, one token a sequence, one sequence, one head: the rows arrive."""
    for B, S, H in ((2, 5, 3), (2, 1, 3), (1, 5, 3), (1, 1, 3), (2, 5, 1)):
        wide = randn(B, S, H * 64 + 72, seed=B + S + H).cuda()
        k, v = wide[..., 8:8 + H * 64].unflatten(-1, (H, 64)), randn(B, S, H, 64, seed=9).cuda()
        pages, more = (torch.zeros(B, 16, H, 64, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        c = h3.PagedKV(pages, more, torch.arange(B, dtype=torch.int32, device="cuda")[:, None].contiguous(),
                       torch.zeros(B, dtype=torch.int32, device="cuda"))
        h3.h3attn_qk_norm_rope_append(None, k, v, None, c, None, None, None, None, 0)
        assert torch.equal(pages[:, :S], k) and torch.equal(more[:, :S], v)


@pytest.mark.gpu
def test_two_streams_at_once(h3):
    """Calls on two streams with workspaces of their own do not touch one another's."""
    from test_gpu_decode import Case, close
    cases = [Case([4000, 900, 33], 8, 2, 128, 16, seed=50 + i).cuda(h3) for i in range(2)]
    streams = [torch.cuda.Stream() for _ in cases]
    ws = [h3.paged_decode_workspace(c.dq, c.cache) for c in cases]
    outs = [[torch.empty_like(c.dq) for _ in range(20)] for c in cases]
    torch.cuda.synchronize()
    for k in range(20):
        for c, s, w, o in zip(cases, streams, ws, outs):
            h3.h3attn_paged_decode(c.dq, o[k], c.cache, workspace=w, stream=s)
    torch.cuda.synchronize()
    for c, o in zip(cases, outs):
        close(o[0], *c.reference())
        assert all(torch.equal(o[0], x) for x in o)


FIRST_CALLS = """
import torch
import video_dit_dense_gb300 as h3
d = dict(dtype=torch.bfloat16, device="cuda")
g = torch.Generator("cuda").manual_seed(1)
x, y, h = torch.randn(2, 512, generator=g, **d), torch.empty(2, 512, **d), torch.empty(2, 512, **d)
q, k = torch.randn(2, 1, 8, 64, generator=g, **d), torch.randn(2, 1, 2, 64, generator=g, **d)
pages, more = torch.randn(80, 16, 2, 64, generator=g, **d), torch.randn(80, 16, 2, 64, generator=g, **d)
cos, sin = torch.empty(640, 32, device="cuda"), torch.empty(640, 32, device="cuda")
lens = torch.tensor([600, 37], dtype=torch.int32, device="cuda")
after, q1, o = torch.empty_like(lens), torch.empty_like(q), torch.empty_like(q)
table = torch.arange(80, dtype=torch.int32, device="cuda").view(2, 40)
cache = h3.PagedKV(pages, more, table, lens)
grown = cache.with_lengths(after)
ws = h3.paged_decode_workspace(q, grown)
assert ws is not None
outs = (h, y, cos, sin, q1, after, o)

def step():
    h3.h3attn_add_rmsnorm(x, x, h, y)
    h3.h3attn_rope_table(cos, sin, 64)
    h3.h3attn_qk_norm_rope_append(q, k, k, q1, cache, None, None, cos, sin, 64, len_out=after)
    h3.h3attn_paged_decode(q1, o, grown, workspace=ws)

torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    step()
for t in outs:
    t.zero_()
graph.replay()
torch.cuda.synchronize()
got = [t.clone() for t in outs]
step()
torch.cuda.synchronize()
assert all(torch.equal(a, b) for a, b in zip(got, outs)) and after.tolist() == [601, 38] and bool((o != 0).any())
assert h3.h3attn_check_device_status() == 0
print("replayed")
"""


@pytest.mark.gpu
def test_the_first_calls_of_a_process_may_be_captured(h3):
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", FIRST_CALLS], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "replayed" in r.stdout, r.stderr[-2000:]


@pytest.mark.gpu
def test_threads_at_once(h3):
    """Calls of several host threads, each on a stream and with a workspace of its own."""
    import threading
    from test_gpu_decode import Case, close
    cases = [Case([3000, 40, 700], 32 if i % 2 else 8, 2 if i % 2 else 1, 128, 16, seed=70 + i).cuda(h3) for i in range(4)]
    refs = [c.reference() for c in cases]
    outs, errors = [None] * len(cases), []
    torch.cuda.synchronize()

    def work(i):
        try:
            s, c = torch.cuda.Stream(), cases[i]
            with torch.cuda.stream(s):
                ws = h3.paged_decode_workspace(c.dq, c.cache)
                outs[i] = [torch.empty_like(c.dq) for _ in range(50)]
                for o in outs[i]:
                    h3.h3attn_paged_decode(c.dq, o, c.cache, workspace=ws)
            s.synchronize()
        except Exception as e:  # reported by the test's own thread
            errors.append(e)
    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(cases))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors
    for (ref, bound), o in zip(refs, outs):
        close(o[0], ref, bound)
        assert all(torch.equal(o[0], x) for x in o)
