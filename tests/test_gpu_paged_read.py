"""Reading a paged cache of either kind back: every bit, rows that the cache
does not hold left alone, starts, strides of pages, bad pages."""
import pytest
import torch

from cache4_ref import Pages
from generate_ref import poison_past


def check(h3, bits, lens, S, Hkv, D, page, first=None, seed=0, capacity=None, bad=(), only=None):
    B = len(lens)
    capacity = max([1] + [n for n in lens]) if capacity is None else capacity
    p = Pages(bits, B, capacity, page, Hkv, D, seed)
    poison_past(p.k, p.v, p.table, lens, page)
    for b, i, value in bad:
        p.table[b, i] = value
    cache = p.hold().cuda(h3, lens)
    outs = [torch.full((B + 1, S, Hkv, D), 5.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    start = None if first is None else torch.tensor(first, dtype=torch.int32, device="cuda")
    args = [o[:B] if only in (None, i) else None for i, o in enumerate(outs)]
    got = h3.h3attn_paged_read(cache, *args, first=start)
    assert got[0] is args[0] and got[1] is args[1]
    torch.cuda.synchronize()
    status = h3.h3attn_check_device_status()
    room, missed = p.table.shape[1] * page, False
    for i, out in enumerate(outs):
        want = torch.full((B + 1, S, Hkv, D), 5.0, dtype=torch.float64)
        for b, n in enumerate(lens):
            for s in range(S if only in (None, i) else 0):
                j = (first[b] if first else 0) + s
                if 0 <= j < min(n, room):
                    pg = int(p.table[b, j // page])
                    if 0 <= pg < p.k.shape[0]:
                        want[b, s] = p.kv[i][pg, j % page]
                    else:
                        missed = True
        assert torch.equal(out.cpu().double().nan_to_num(nan=1e9), want.nan_to_num(nan=1e9))
    assert status == (h3.H3ATTN_ERR_INVALID_ARG if missed else 0)


@pytest.mark.gpu
@pytest.mark.parametrize("bits", [4, 16])
@pytest.mark.parametrize("Hkv,D", [(1, 64), (2, 64), (3, 64), (1, 128), (5, 128), (24, 128), (1, 256), (4, 256)])
@pytest.mark.parametrize("page", [1, 16, 24])
def test_shapes(h3, bits, Hkv, D, page):
    check(h3, bits, [0, 1, 37, 20], 37, Hkv, D, page, seed=D + Hkv)


@pytest.mark.gpu
@pytest.mark.parametrize("bits", [4, 16])
def test_starts_and_lengths(h3, bits):
    check(h3, bits, [50, 20, 9, 31], 12, 2, 128, 16, first=[45, 0, 9, -3])
    check(h3, bits, [50, 20], 1, 2, 128, 16, first=[49, 2 ** 31 - 1])
    check(h3, bits, [300, -5], 40, 2, 64, 16, capacity=32)          # a length above the capacity, and one below zero
    check(h3, bits, [40], 64, 4, 128, 16, only=0)
    check(h3, bits, [40], 64, 4, 128, 16, only=1)


@pytest.mark.gpu
@pytest.mark.parametrize("bits", [4, 16])
def test_bad_pages_are_left_out(h3, bits):
    check(h3, bits, [40, 33], 40, 2, 128, 8, bad=[(0, 1, -1), (0, 3, 2 ** 31 - 1), (1, 0, 2 ** 20)])


@pytest.mark.gpu
@pytest.mark.parametrize("bits", [4, 16])
def test_every_scale_and_code(h3, bits):
    if bits == 16:
        return check(h3, bits, [700], 700, 3, 256, 64)
    p = Pages(4, 1, 256, 64, 1, 64, 0, poison=False).hold()
    codes = torch.arange(256, dtype=torch.uint8).repeat(256, 1)[:, :32].clone()
    for j in range(256):
        codes[j] = (torch.arange(32) * 7 + j) % 256
    scales = torch.arange(256, dtype=torch.uint8)[:, None].repeat(1, 4)
    p.table = torch.arange(4, dtype=torch.int32)[None]
    for i in range(2):
        p.held[i][:4] = codes.view(4, 64, 1, 32)
        p.held[2 + i][:4] = scales.view(4, 64, 1, 4)
    cache = p.cuda(h3, [256])
    out = [torch.zeros(1, 256, 1, 64, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    h3.h3attn_paged_read(cache, *out)
    from cache4_ref import values
    want = values(codes, scales)
    for o in out:
        assert torch.equal(o[0, :, 0].cpu().double().nan_to_num(nan=1e9), want.nan_to_num(nan=1e9))


@pytest.mark.gpu
def test_refusals(h3):
    p = Pages(4, 2, 32, 16, 2, 64, 0).hold()
    cache = p.cuda(h3, [3, 4])
    k = torch.zeros(2, 5, 2, 64, dtype=torch.bfloat16, device="cuda")
    for bad in ((cache, None, None), (cache, k, k), (cache, k[:1], None), (cache, k.float(), None), (cache, k[:, :, :1], None),
                (None, k, None), (cache, k.cpu(), None), (cache, k, k[:, :4].clone()), (cache, k.transpose(0, 1), None),
                (cache, k, None, p.dlen[:1]), (cache, k, None, p.dlen.long()), (p.dheld[0], k, None)):
        with pytest.raises(h3.H3AttnError):
            h3.h3attn_paged_read(*bad)
    h3.h3attn_paged_read(cache, k[:, :0], None)


@pytest.mark.gpu
@pytest.mark.parametrize("bits", [4, 16])
@pytest.mark.parametrize("Hkv,D", [(1, 64), (1, 128), (2, 64), (3, 64), (1, 256), (2, 128)])
def test_many_tokens_of_short_rows(h3, bits, Hkv, D):
    """Several tokens of a lane at a time: sequences that end at every place among them, starts, bad pages."""
    lens = [0, 1, 2, 3, 4, 5, 4999, 5003, 5002, 5000, 17, 5001]
    p = Pages(bits, len(lens), 5003, 24, Hkv, D, 3, poison=False)
    p.table[7, 3] = -1
    cache = p.hold().cuda(h3, lens)
    first = torch.tensor([0, 0, 0, 1, 0, 2, -3, 5, 0, 1, 0, 0], dtype=torch.int32)
    outs = [torch.full((len(lens), 5003, Hkv, D), 5.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    h3.h3attn_paged_read(cache, *outs, first=first.cuda())
    assert h3.h3attn_check_device_status() == h3.H3ATTN_ERR_INVALID_ARG
    for out, kv in zip(outs, p.kv):
        want = torch.full(out.shape, 5.0, dtype=torch.bfloat16)
        for b, n in enumerate(lens):
            s = torch.arange(5003)
            j = s + int(first[b])
            ok = (j >= 0) & (j < n)
            ok[ok.clone()] &= p.table[b][j[ok] // 24] >= 0
            want[b, s[ok]] = kv[p.table[b][j[ok] // 24].long(), j[ok] % 24].to(torch.bfloat16)
        assert torch.equal(out.cpu(), want)
