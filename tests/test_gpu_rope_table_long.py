"""Rotary tables of more rows than the grid takes at once, on another stream, and
against the exact frequencies.

test_gpu_rope_table compares with the double-precision frequencies, which the host
works out as its reference does.  A frequency theta^(-2 i / rot) itself is rounded to
double there: its exponent, off by half of 2^-53 of itself, moves it by ln(theta) times
that, and the power's result is off by at most one unit, so f is off by at most
(2 + ln theta) 2^-53 of itself, and the angle by |p| times that."""
import math

import numpy as np
import pytest
import torch

from generate_ref import rope_freqs, rope_table_wide
from test_gpu_rope_table import BOUND


def rows_at_once(half):
    """Rows that the grid takes in one pass: six blocks of 256 threads an SM, 4 pairs a thread or 1."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    return sms * 6 * (256 // (half // 4 if half % 4 == 0 else half))


def check(cos, sin, positions, freqs, rows):
    assert bool(cos.isfinite().all()) and bool(sin.isfinite().all())      # every row was written
    want = rope_table_wide(positions, freqs)
    for got, ref in ((cos, want[0]), (sin, want[1])):
        assert np.abs(got[rows].cpu().double().numpy() - ref).max() <= BOUND


@pytest.mark.gpu
@pytest.mark.parametrize("rot", [2, 46, 96, 128, 250, 256])
@pytest.mark.parametrize("given", [False, True])
def test_several_passes_over_the_rows(h3, rot, given):
    """Two whole passes and a part of one; the rows around their ends and others between."""
    once = rows_at_once(rot // 2)
    N = 2 * once + once // 3 + 1
    rows = np.unique(np.concatenate([np.arange(5), np.arange(once - 5, once + 5), np.arange(2 * once - 5, 2 * once + 5),
                                     np.linspace(0, N - 1, 700).astype(int), np.arange(N - 5, N)]))
    cos, sin = (torch.full((N, rot // 2), float("nan"), device="cuda") for _ in range(2))
    pos, at = None, np.arange(N, dtype=np.int64) + 12345
    if given:
        at = np.random.RandomState(rot).randint(-2 ** 31, 2 ** 31, N)
        pos = torch.from_numpy(at.astype(np.int32)).cuda()
    h3.h3attn_rope_table(cos, sin, rot, pos=pos, first=0 if given else 12345)
    check(cos, sin, at[rows], rope_freqs(rot), torch.from_numpy(rows).cuda())


@pytest.mark.gpu
def test_another_stream_and_rows_around(h3):
    N, rot = 77, 46
    s = torch.cuda.Stream()
    flat = [torch.full((N * (rot // 2) + 12,), 7.0, device="cuda") for _ in range(2)]
    cos, sin = (f[4:4 + N * (rot // 2)].view(N, rot // 2) for f in flat)
    pos = torch.arange(N, dtype=torch.int32, device="cuda") * 1000
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        pos += 1                                                          # the table is of what the stream has then
        h3.h3attn_rope_table(cos, sin, rot, pos=pos)
    h3.h3attn_rope_table(*(t.clone() for t in (cos, sin)), rot)           # nothing of the other stream's is touched
    s.synchronize()
    check(cos, sin, np.arange(N) * 1000 + 1, rope_freqs(rot), torch.arange(N, device="cuda"))
    assert all(bool((f[:4] == 7).all()) and bool((f[4 + N * (rot // 2):] == 7).all()) for f in flat)


@pytest.mark.gpu
@pytest.mark.parametrize("rot,theta", [(96, 10000.0), (128, 500000.0), (256, 10000.0), (46, 1e6)])
@pytest.mark.parametrize("first", [0, 1 << 20, (1 << 31) - 64])
def test_against_exact_frequencies(h3, rot, theta, first):
    wide = np.longdouble
    freqs = np.power(wide(theta), wide(-2) * np.arange(rot // 2, dtype=wide) / wide(rot))
    at = np.arange(first, first + 64)
    cos, sin = (torch.empty(64, rot // 2, device="cuda") for _ in range(2))
    h3.h3attn_rope_table(cos, sin, rot, theta, first=first)
    want = rope_table_wide(at, freqs)
    bound = BOUND + at[:, None] * freqs.astype(np.float64)[None] * (2 + math.log(theta)) * 2.0 ** -53
    for got, ref in ((cos, want[0]), (sin, want[1])):
        assert bool((np.abs(got.cpu().double().numpy() - ref) <= bound).all())
