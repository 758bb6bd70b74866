"""GPU parity of the rotary tables against angles multiplied out in extended
precision: far positions, every scaling, given positions, odd sizes."""
import numpy as np
import pytest
import torch

from generate_ref import rope_freqs, rope_table_wide

# The angle, at most an eighth of a turn (pi / 4) from a quadrant's border, is rounded to float32 once (2^-24 of it), the
# sine or cosine is within an ulp (2^-24 below 1), and its product with the amplitude is rounded once: 3 * 2^-24, and one
# in reserve for the double frequencies' own product.
BOUND = 4 * 2.0 ** -24


def run(h3, N, rot, scaling=None, pos=None, first=0, theta=10000.0):
    cos = torch.full((N, rot // 2), float("nan"), device="cuda")
    sin = torch.full((N, rot // 2), float("nan"), device="cuda")
    out = h3.h3attn_rope_table(cos, sin, rot, theta, scaling, None if pos is None else pos.cuda(), first)
    assert out[0] is cos and out[1] is sin
    return cos.cpu().double().numpy(), sin.cpu().double().numpy()


def close(got, ref, amplitude=1.0):
    for g, r in zip(got, ref):
        assert np.abs(g - r).max() <= BOUND * amplitude, np.abs(g - r).max() / BOUND


@pytest.mark.gpu
@pytest.mark.parametrize("rot", [2, 4, 6, 46, 64, 96, 128, 250, 256])
@pytest.mark.parametrize("first,N", [(0, 1), (0, 131), (1 << 20, 77), ((1 << 31) - 33, 33)])
def test_positions_near_and_far(h3, rot, first, N):
    close(run(h3, N, rot, first=first), rope_table_wide(np.arange(first, first + N), rope_freqs(rot)))


@pytest.mark.gpu
@pytest.mark.parametrize("kind,factor", [("none", 1.0), ("linear", 4.0), ("ntk", 8.0), ("by_parts", 16.0), ("by_parts", 1.0)])
@pytest.mark.parametrize("rot", [4, 96, 128])
def test_scalings(h3, rot, kind, factor):
    s = h3.RopeScaling(kind, factor, 4096, 1.0, 32.0, 1.25)
    freqs = rope_freqs(rot, 500000.0, kind, factor, 4096)
    close(run(h3, 300, rot, s, first=60000, theta=500000.0), rope_table_wide(np.arange(60000, 60300), freqs, 1.25), 1.25)


@pytest.mark.gpu
def test_given_positions(h3):
    """Any int32, in any order, negative ones and repeated ones too."""
    pos = torch.tensor([5, 5, 0, -1, -77, 2 ** 31 - 1, -2 ** 31, 12345], dtype=torch.int32)
    close(run(h3, 8, 96, pos=pos), rope_table_wide(pos.numpy(), rope_freqs(96)))


@pytest.mark.gpu
def test_the_table_serves_the_fused_norm(h3):
    """The fused norm and rotation reads the table as it is: cos^2 + sin^2 = 1, so a row's rotated pairs keep their norm."""
    cos, sin = torch.empty(40, 48, device="cuda"), torch.empty(40, 48, device="cuda")
    h3.h3attn_rope_table(cos, sin, 96)
    q = torch.randn(1, 40, 2, 128, generator=torch.Generator().manual_seed(1)).bfloat16().cuda()
    w = torch.ones(128, device="cuda")
    turned = torch.empty_like(q)
    straight = torch.empty_like(q)
    h3.h3attn_qk_norm_rope_out(q, None, turned, None, w, None, cos, sin, 96)
    h3.h3attn_qk_norm_rope_out(q, None, straight, None, w, None, None, None, 0)
    a, b = (t.float()[..., :48].square() + t.float()[..., 48:96].square() for t in (turned, straight))
    # two outputs each rounded by 2^-8 of itself: their squares' sum by 2 * 2^-8 and its square
    assert bool(((a - b).abs() <= (2 * 2.0 ** -8 + 2.0 ** -15) * b + 1e-30).all())


@pytest.mark.gpu
def test_stream_graph_and_guards(h3):
    N, rot = 33, 46
    buf = torch.full((2, N + 2, rot // 2 + 1), 7.0, device="cuda")
    pos = torch.arange(N, dtype=torch.int32, device="cuda")
    cos, sin = torch.empty(N, rot // 2, device="cuda"), torch.empty(N, rot // 2, device="cuda")
    flat = torch.full((N * (rot // 2) + 8,), 7.0, device="cuda")
    h3.h3attn_rope_table(flat[4:-4].view(N, rot // 2), sin, rot)
    assert bool((flat[:4] == 7).all()) and bool((flat[-4:] == 7).all())
    assert bool((buf == 7).all())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        h3.h3attn_rope_table(cos, sin, rot, pos=pos)
    pos.add_(100)
    graph.replay()
    torch.cuda.synchronize()
    close((cos.cpu().double().numpy(), sin.cpu().double().numpy()),
          rope_table_wide(np.arange(100, 100 + N), rope_freqs(rot)))
