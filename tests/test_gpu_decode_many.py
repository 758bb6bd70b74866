"""Decode attention of more sequences than are split over the GPU, with lengths that
are unlike, in one call and in parts that are split."""
import pytest
import torch

from test_gpu_decode import Case, close


def lengths(B):
    """Short ones, empty ones, and a few that are much longer than the others, at the ends too."""
    lens = [(37 * b) % 90 if b % 7 else 0 for b in range(B)]
    lens[0], lens[B // 2], lens[511], lens[-1] = 1100, 1203, 777, 1199
    return lens


@pytest.mark.gpu
@pytest.mark.parametrize("Hq,Hkv,D", [(4, 1, 64), (17, 1, 128), (2, 2, 256)])
@pytest.mark.parametrize("B", [512, 513, 700])
def test_unlike_lengths(h3, B, Hq, Hkv, D):
    c = Case(lengths(B), Hq, Hkv, D, 16, capacity=1204, seed=B + D, poison=False).cuda(h3)
    assert (h3.paged_decode_workspace(c.dq, c.cache) is None) == (B > 512)
    ref, bound = c.reference()
    close(c.run(h3), ref, bound, "one call")
    o = torch.full_like(c.dq, float("nan"))
    for b in range(0, B, 512):                       # in parts of up to 512, in one workspace
        e = min(b + 512, B)
        part = h3.PagedKV(c.dk, c.dv, c.dt[b:e], c.dlen[b:e])
        h3.h3attn_paged_decode(c.dq[b:e], o[b:e], part, c.scale, h3.paged_decode_workspace(c.dq[b:e], part))
    close(o, ref, bound, "in parts")
    assert h3.h3attn_check_device_status() == 0
