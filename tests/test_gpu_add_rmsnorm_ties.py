"""Row scales of the residual add + RMSNorm: y / s to 8 bits where the quotient is
known exactly.  The norm's factor is the same in y and in s, so y / s is
448 h w / max |h w|.  With a maximum of 7 * 2^j that is 64 h w / 2^j, a float32
without rounding; half of the values below lie exactly between two e4m3 values,
where any error decides the side."""
import pytest
import torch


def rows(T, C, seed):
    """h [T, C] (bf16 values) and the quotients, both exact: multiples of a 32nd of a power of two, and 7 * 2^j in a
    channel of each row."""
    g = torch.Generator().manual_seed(seed)
    m = torch.randint(16, 32, (T, C), generator=g)                         # five bits: the odd ones are ties
    e = torch.randint(-6, 5, (T, C), generator=g)                          # 2^-6, e4m3's least normal, and up
    q = m.double() / 16 * torch.exp2(e.double() + 4) * (1 - 2 * torch.randint(0, 2, (T, C), generator=g))
    q = q.clamp(-448, 448)
    q[torch.arange(T), torch.randint(0, C, (T,), generator=g)] = 448.0
    j = torch.randint(-20, 20, (T, 1), generator=g)
    return (q / 64 * torch.exp2(j.double())), q


@pytest.mark.gpu
@pytest.mark.parametrize("T,C", [(1, 8), (5, 40), (33, 520), (9, 1024), (600, 1000), (4, 4096), (2049, 4096), (3, 6144), (2051, 8192),
                                 (2049, 2056), (2, 16384)])
def test_quotients_that_lie_between_two_values(h3, T, C):
    h, q = rows(T, C, T + C)
    want = q.float().to(torch.float8_e4m3fn).view(torch.uint8)
    g = torch.Generator().manual_seed(C)
    power = torch.exp2(torch.randint(-3, 4, (C,), generator=g).double())   # weights that round nothing
    y, s = torch.empty(T, C, dtype=torch.float8_e4m3fn, device="cuda"), torch.empty(T, device="cuda")
    for w in (None, power):
        x = (h if w is None else h / w).to(torch.bfloat16)
        assert torch.equal(x.double() if w is None else x.double() * w, h)
        dx, dw = x.cuda(), None if w is None else w.float().cuda()
        for residual in (None, dx / 2):
            y.view(torch.uint8).fill_(0x7F)
            h3.h3attn_add_rmsnorm(dx if residual is None else dx / 2, residual, None if residual is None else torch.empty_like(dx),
                                  y, dw, 1e-6, s)
            off = y.cpu().view(torch.uint8) != want
            assert not bool(off.any()), f"{int(off.sum())} of {off.numel()} on the wrong side, w={w is not None}"
            top = h.abs().amax(-1) / (x.double().square().mean(-1) + float(torch.tensor(1e-6))).sqrt()
            # the sum of squares' error halved, the root, the product and the quotient: as y_rel in test_gpu_add_rmsnorm
            assert bool(((s.cpu().double() * 448 / top - 1).abs() <= (C / 64 + 16) * 2.0 ** -24).all())


@pytest.mark.gpu
def test_rows_next_to_the_ends_of_the_range(h3):
    """Where the quotient cannot be taken that way: scales that are held at 2^-126, maxima below float32's normal range."""
    C = 256
    x = torch.zeros(5, C, dtype=torch.bfloat16)
    x[0] = 2.0 ** -130
    x[1] = 2.0 ** -100
    x[2, 7] = 2.0 ** -133
    x[3] = 2.0 ** 60
    w = torch.full((C,), 2.0 ** -10)
    w[1] = 2.0 ** -12
    y, s = torch.empty(5, C, dtype=torch.float8_e4m3fn, device="cuda"), torch.empty(5, device="cuda")
    h3.h3attn_add_rmsnorm(x.cuda(), None, None, y, w.cuda(), 1.0, s)
    v = x.double() / (x.double().square().mean(-1, keepdim=True) + 1).sqrt() * w.double()
    scale = (v.abs().amax(-1) / 448).clamp(min=2.0 ** -126)
    # 256 squares of 2^60 are 2^128, past float32's range: such a row is written as zeros, and as a row of zeros its scale is 1
    v[3], scale[3:] = 0.0, 1.0
    assert bool(((s.cpu().double() / scale - 1).abs() <= 32 * 2.0 ** -24).all())
    got = y.cpu().float().double() * s.cpu().double()[:, None]
    # half a step of e4m3, at least that of its subnormals; below float32's normal range h w itself loses up to 2^-150, twice
    bound = torch.maximum(2.0 ** -4 * v.abs(), 2.0 ** -10 * scale[:, None]) * (1 + 2.0 ** -10) + 2.0 ** -149
    assert bool(((got - v).abs() <= bound).all())
