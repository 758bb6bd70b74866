"""GPU parity of the residual add + RMSNorm against its definition in 64 bits:
the stream h bit for bit, y and the e4m3 values with their scales within their
roundings, at sizes of every thread layout, with rows that are zero, tiny or not
finite, in place, captured, and on another stream."""
import numpy as np
import pytest
import torch

from generate_ref import BF16_HALF, add_norm_f64, randn

# y = (h w) r in float32: the sum of squares of C terms is off by at most (C / 32 + 16) halves of 2^-24 (each of at
# least 32 threads adds its own in turn, then a tree), r by half of that and the root, the quotient and two products
# add one rounding each.
def y_rel(C):
    return (C / 64 + 16) * 2.0 ** -24


FORMATS = ("bf16", "row", "mx_u8", "mx_e8m0")


def call(h3, x, residual, w, fmt, eps=1e-6, stream=None, h=None, y=None):
    T, C = x.shape
    if residual is not None and h is None:
        h = torch.full_like(x, float("nan"))
    scale = None
    if fmt == "bf16":
        y = torch.full_like(x, float("nan")) if y is None else y
    else:
        y = torch.zeros(T, C, dtype=torch.uint8, device="cuda").fill_(0x7F).view(torch.float8_e4m3fn)
        scale = (torch.full((T,), float("nan"), device="cuda") if fmt == "row" else
                 torch.full((T, C // 32), 255, dtype=torch.uint8, device="cuda"))
        if fmt == "mx_e8m0":
            scale = scale.view(torch.float8_e8m0fnu)
    out = h3.h3attn_add_rmsnorm(x, residual, h, y, w, eps, scale, stream)
    assert out is y
    return h, y, scale


def same_bits(a, b):
    return torch.equal(a.cpu().view(torch.int16), b.cpu().view(torch.int16))


def check(fmt, h, y, scale, h_ref, y_ref, what):
    T, C = y_ref.shape
    if h is not None:
        assert same_bits(h, h_ref), f"{what}: h"
    rel = y_rel(C)
    if fmt == "bf16":
        got = y.cpu().double()
        bound = (BF16_HALF + 2 * rel) * y_ref.abs() + 1e-38
        assert bool(((got - y_ref).abs() <= bound).all()), f"{what}: y off by {float(((got - y_ref).abs() / bound).max())} bounds"
        return
    got = y.cpu().view(torch.uint8)
    assert not bool(((got & 0x7F) == 0x7F).any()), f"{what}: NaN"
    got = got.view(torch.float8_e4m3fn).float().double()
    if fmt == "row":
        s = scale.cpu().double()
        amax = y_ref.abs().amax(-1)
        want = torch.where(amax > 0, (amax / 448).clamp(min=2.0 ** -126), torch.ones_like(amax))
        assert bool(((s - want).abs() <= 2 * (rel + 2.0 ** -23) * want).all()), f"{what}: scales"
        s = s[:, None].expand(T, C)
    else:
        e = scale.view(torch.uint8).cpu().double() - 127
        amax = y_ref.view(T, -1, 32).abs().amax(-1)
        for slack in (1 - 2 * rel, 1 + 2 * rel):  # where 448 * 2^n is within the error of the maximum, either is right
            want = torch.where(amax > 0, torch.ceil(torch.log2(amax * slack / 448)).clamp(min=-126), torch.zeros_like(amax))
            off = e != want
            e_ok = ~off if slack < 1 else e_ok | ~off
        assert bool(e_ok.all()), f"{what}: exponents"
        s = torch.exp2(e)[..., None].expand(T, C // 32, 32).reshape(T, C)
    bound = torch.maximum(2.0 ** -4 * y_ref.abs(), 2.0 ** -10 * s) * (1 + 2.0 ** -10)
    err = (got * s - y_ref).abs()
    assert bool((err <= bound).all()), f"{what}: e4m3 off by {float((err / bound).max())} bounds"


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("T,C", [(1, 8), (3, 40), (5, 512), (17, 520), (2, 1024), (9, 1536), (4, 2056), (7, 4096), (3, 5120),
                                 (2, 8192), (3, 8200), (2, 16384), (1, 32), (65, 64), (1000, 96)])
def test_against_definition(h3, T, C, fmt):
    if fmt.startswith("mx"):
        C = -(-C // 32) * 32
    x, res = randn(T, C, seed=T + C), randn(T, C, seed=T + C + 1, scale=4.0)
    w = torch.rand(C, generator=torch.Generator().manual_seed(C)) + 0.5
    for residual in (res, None):
        for weight in (w, None):
            h, y, scale = call(h3, x.cuda(), None if residual is None else residual.cuda(),
                               None if weight is None else weight.cuda(), fmt)
            h_ref, y_ref = add_norm_f64(x, residual, weight, 1e-6)
            check(fmt, h, y, scale, h_ref, y_ref, f"T={T} C={C} {fmt} residual={residual is not None}")


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", FORMATS)
def test_zero_tiny_and_huge_rows(h3, fmt):
    C = 256
    x = randn(6, C, seed=3)
    x[0] = 0.0
    x[1] = 2.0 ** -60            # eps decides: y = x * 1000
    x[2] = randn(1, C, seed=4, scale=2.0 ** 40)[0]
    x[3, :] = 0.0
    x[3, 77] = 5.0               # one channel holds everything; the other groups are zero
    x[4] = 2.0 ** -130           # below bf16's normal range
    h, y, scale = call(h3, x.cuda(), torch.zeros_like(x).cuda(), None, fmt)
    h_ref, y_ref = add_norm_f64(x, torch.zeros_like(x), None, 1e-6)
    check(fmt, h, y, scale, h_ref, y_ref, fmt)
    if fmt == "row":
        assert float(scale[0]) == 1.0
    elif fmt != "bf16":
        assert bool((scale[0].view(torch.uint8) == 127).all())


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", FORMATS)
def test_a_row_that_is_not_finite_stays_by_itself(h3, fmt):
    C = 1056
    x, w = randn(5, C, seed=8), torch.ones(C)
    x[1, 40] = float("nan")
    x[3, 41] = float("inf")
    h, y, scale = call(h3, x.cuda(), torch.zeros_like(x).cuda(), w.cuda(), fmt)
    y64 = y.cpu().float()
    assert bool(torch.isnan(y64[1]).all()) if fmt == "bf16" else bool(torch.isnan(y64[1, 40]))
    assert bool(torch.isnan(y64[3, 41]))                      # inf * 0
    assert bool((y64[3, :41] == 0).all())
    rows = [0, 2, 4]
    h_ref, y_ref = add_norm_f64(x[rows], torch.zeros(3, C).bfloat16(), w, 1e-6)
    check(fmt, h[rows], y.view(torch.uint8)[rows].view(y.dtype) if fmt != "bf16" else y[rows],
          None if scale is None else scale.view(torch.uint8)[rows] if fmt.startswith("mx") else scale[rows], h_ref, y_ref, fmt)


@pytest.mark.gpu
def test_in_place(h3):
    T, C = 37, 1160
    x, res = randn(T, C, seed=1), randn(T, C, seed=2)
    h_ref, y_ref = add_norm_f64(x, res, None, 1e-6)
    dx, dr = x.cuda(), res.cuda()
    h, y, _ = call(h3, dx, dr, None, "bf16", h=dr)            # the stream in place
    check("bf16", h, y, None, h_ref, y_ref, "h over residual")
    dx, dr = x.cuda(), res.cuda()
    h, y, _ = call(h3, dx, dr, None, "bf16", h=dr, y=dx)      # and the normed rows over x
    check("bf16", h, y, None, h_ref, y_ref, "h over residual, y over x")
    dx, dr = x.cuda(), res.cuda()
    h, y, _ = call(h3, dx, dr, None, "bf16", h=dx, y=dr)
    check("bf16", h, y, None, h_ref, y_ref, "h over x, y over residual")


@pytest.mark.gpu
def test_chain_stream_and_graph(h3):
    """Calls that read what the one before wrote, on another stream and replayed from a graph with new inputs."""
    T, C = 300, 1536
    x, res = randn(T, C, seed=11), randn(T, C, seed=12)
    w = (torch.rand(C, generator=torch.Generator().manual_seed(5)) + 0.5)
    dx, dr, dw = x.cuda(), res.cuda(), w.cuda()
    h1, y1, h2, y2 = (torch.empty_like(dx) for _ in range(4))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())

    def chain(stream):
        h3.h3attn_add_rmsnorm(dx, dr, h1, y1, dw, 1e-6, stream=stream)
        h3.h3attn_add_rmsnorm(y1, h1, h2, y2, None, 1e-6, stream=stream)

    def verify(x, res):
        torch.cuda.synchronize()
        h_ref, y_ref = add_norm_f64(x, res, w, 1e-6)
        check("bf16", h1, y1, None, h_ref, y_ref, "first")
        h_ref, y_ref = add_norm_f64(y1.cpu(), h1.cpu(), None, 1e-6)
        check("bf16", h2, y2, None, h_ref, y_ref, "second")
    with torch.cuda.stream(s):
        chain(s)
    verify(x, res)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        chain(None)
    for seed in (21, 22):
        x, res = randn(T, C, seed=seed), randn(T, C, seed=seed + 50)
        dx.copy_(x)
        dr.copy_(res)
        graph.replay()
        verify(x, res)


@pytest.mark.gpu
def test_rows_past_32_bits(h3):
    """More than 2^31 elements: the last rows are right."""
    C = 8192
    T = (1 << 31) // C + 5
    x = torch.zeros(T, C, dtype=torch.bfloat16, device="cuda")
    x[-7:] = randn(7, C, seed=2).cuda()
    y = torch.empty(T, C, dtype=torch.float8_e4m3fn, device="cuda")
    scale = torch.empty(T, device="cuda")
    h3.h3attn_add_rmsnorm(x, None, None, y, None, 1e-6, scale)
    _, y_ref = add_norm_f64(x[-7:].cpu(), None, None, 1e-6)
    check("row", None, y.view(torch.uint8)[-7:].view(torch.float8_e4m3fn), scale[-7:], None, y_ref, "last rows")
    assert bool((scale[:-7] == 1).all())


@pytest.mark.gpu
def test_guards_around_the_outputs(h3):
    """Nothing but the T rows is written."""
    T, C = 5, 1032
    x = randn(T, C, seed=6).cuda()
    buf = torch.full((T + 2, C), 3.0, dtype=torch.bfloat16, device="cuda")
    h3.h3attn_add_rmsnorm(x, None, None, buf[1:-1], None)
    assert bool((buf[0] == 3).all()) and bool((buf[-1] == 3).all())
    h3.h3attn_add_rmsnorm(x[:0], None, None, buf[:0], None)
    assert np.isfinite(float(buf[1:-1].float().abs().sum()))


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("T,C", [(2049, 520), (2048, 1016), (2051, 1032), (2049, 2048), (2050, 2080), (2049, 4096), (2049, 4104),
                                 (2051, 8192), (2049, 8200)])
def test_many_rows(h3, T, C, fmt):
    """Enough rows for the layouts of large batches, an odd number of them: the first, the last and some between, a row
    that is not finite beside others, and nothing behind the last one."""
    if fmt.startswith("mx"):
        C = -(-C // 32) * 32
    x, res = randn(T, C, seed=T + C), randn(T, C, seed=T + C + 1, scale=4.0)
    x[700, 3] = float("nan")
    w = torch.rand(C, generator=torch.Generator().manual_seed(C)) + 0.5
    rows = torch.cat((torch.arange(4), torch.tensor([699, 701]), torch.arange(900, T - 9, 37), torch.arange(T - 9, T)))
    for residual in (None, res):
        for weight in (w, None):
            h, y, scale = call(h3, x.cuda(), None if residual is None else residual.cuda(),
                               None if weight is None else weight.cuda(), fmt)
            h_ref, y_ref = add_norm_f64(x[rows], None if residual is None else residual[rows], weight, 1e-6)
            at = rows.cuda()
            check(fmt, None if h is None else h[at], y[at] if fmt == "bf16" else y.view(torch.uint8)[at].view(y.dtype),
                  None if scale is None else scale[at] if fmt == "row" else scale.view(torch.uint8)[at], h_ref, y_ref,
                  f"T={T} C={C} {fmt} residual={residual is not None}")
            assert bool(y[700, 3].float().isnan())
    if fmt == "bf16":
        buf = torch.full((T + 1, C), 3.0, dtype=torch.bfloat16, device="cuda")
        h3.h3attn_add_rmsnorm(x.cuda(), None, None, buf[:T], None)
        assert bool((buf[T] == 3).all())
        own = x.cuda()
        h3.h3attn_add_rmsnorm(own, None, None, own, None)  # in place
        assert same_bits(own[rows.cuda()], buf[:T][rows.cuda()])


@pytest.mark.gpu
def test_guards_behind_scaled_rows(h3):
    T, C = 2049, 1056
    x = randn(T, C, seed=16).cuda()
    y = torch.full((T + 1, C), 0x55, dtype=torch.uint8, device="cuda")
    s, e = torch.full((T + 1,), 3.0, device="cuda"), torch.full((T + 1, C // 32), 9, dtype=torch.uint8, device="cuda")
    for scale in (s, e):
        h3.h3attn_add_rmsnorm(x, None, None, y[:T].view(torch.float8_e4m3fn), None, y_scale=scale[:T])
        assert bool((y[T] == 0x55).all())
    assert float(s[T]) == 3.0 and bool((e[T] == 9).all())
