"""The references of the 4-bit cache pinned on the CPU: scales against binary16,
hand-worked rows, error bounds, ties, and which tokens an eviction keeps."""
import pytest
import torch

from cache4_ref import evict, scale_values, store, values
from generate_ref import randn


def test_scales_are_the_upper_byte_of_a_binary16():
    bits = (torch.arange(0xD8, dtype=torch.int16) << 7).view(torch.float16).double()
    assert torch.equal(bits, scale_values()[:0xD8])
    assert scale_values()[0xD7] == 3840 and bool(scale_values()[0xD8:].isnan().all())


def test_hand_worked_row():
    """max 7: s = 1, so 2.5 and -2.5 are away from zero, -7 is code 1, and 0.49 is code 8."""
    x = torch.zeros(16)
    x[:7] = torch.tensor([7.0, -7.0, 2.5, -2.5, 0.490234375, 1.0, -1.0])
    codes, scales = store(x.to(torch.bfloat16))
    assert scales.tolist() == [(15 << 3)]
    assert codes.tolist()[:4] == [15 | 1 << 4, 11 | 5 << 4, 8 | 9 << 4, 7 | 8 << 4]
    assert values(codes, scales)[:7].tolist() == [7, -7, 3, -3, 0, 1, -1]


@pytest.mark.parametrize("size", [1e-30, 2.0 ** -18, 1e-5, 1e-3, 1.0, 300.0, 2e4, 2e5, 1e30])
def test_errors_are_within_half_a_scale(size):
    x = randn(400, 64, seed=3, scale=size)
    codes, scales = store(x)
    got, s = values(codes, scales), scale_values()[scales.long()].repeat_interleave(16, -1)
    assert bool(got.isfinite().all()) and torch.equal(got, got.to(torch.bfloat16).double())
    err, cut = (got - x.double()).abs(), (x.double().abs() > 7.5 * s)
    assert bool((err <= torch.where(cut, x.double().abs() - 7 * s, s / 2)).all())
    normal = (s >= 2.0 ** -14) & (s < 3840)
    assert not bool((cut & normal).any())


def test_not_finite():
    x = randn(3, 32, seed=1)
    x[0, 3], x[1, 20] = float("inf"), float("nan")
    v = values(*store(x))
    assert bool(v[0, :16].isnan().all()) and bool(v[1, 16:].isnan().all())
    assert bool(v[0, 16:].isfinite().all()) and bool(v[1, :16].isfinite().all()) and bool(v[2].isfinite().all())


def test_evict_by_hand():
    """6 tokens to 4 with 1 recent: of 0..4 the three heaviest are 1, 3 and 4 (2 ties with 4, and 4 weighs more here)."""
    held = [torch.arange(8).view(4, 2, 1, 1)]
    table = torch.tensor([[2, 0, 3]])                       # tokens 0..5 are rows 4 5 0 1 6 7
    w = torch.tensor([[0.0, 9.0, 1.0, 5.0, 1.5, 0.25]])
    got, weights, lens = evict(held, table, [6], 2, w, 4, 1)
    assert lens.tolist() == [4] and weights.tolist() == [[5.0, 9.0, 1.5, 0.25, 0.0, 0.0]]
    # 3 -> place 0, 4 -> place 2 (the gaps in order), the recent one -> place 3
    assert got[0].view(-1)[[4, 5, 0, 1]].tolist() == [1, 5, 6, 7]
