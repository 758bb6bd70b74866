"""GPU parity of the rotated append to a paged cache.  The arithmetic is fixed
operation by operation, so every written element is compared bit for bit:
normed values with the oracle's emulation, the rotation with float32 operations
taken out in float64 (products of a bf16 and a float32 value are exact there).
Everything that is not written has to stay as it was."""
import numpy as np
import pytest
import torch

import oracle
from generate_ref import paged, randn


def bits(t):
    return t.contiguous().cpu().view(torch.int16).numpy().view(np.uint16)


def from_bits(b):
    return torch.from_numpy(np.ascontiguousarray(b).view(np.int16)).view(torch.bfloat16)


def f32(x):
    return np.float64(np.float32(x))


def reference(x, w, cos, sin, at, rot, interleaved, eps):
    """x [n, H, D] bf16 of tokens at table rows `at` -> bf16 bits [n, H, D]."""
    n_tok, H, D = x.shape
    if w is not None:
        # Normed values before the rotation: a rotation by nothing.  The order of the sum of squares goes by the number of
        # whole 16-channel steps that rotate, and the interleaved layout's is that of a row that rotates whole.
        r = D if interleaved else rot
        ones, zeros = np.ones((n_tok, r // 2), np.float32), np.zeros((n_tok, r // 2), np.float32)
        x = from_bits(oracle.qk_norm_rope_emulate(bits(x)[None], w.numpy(), ones, zeros, r, eps)[0])
    v = x.double().numpy()
    h = rot // 2
    c, s = cos.double().numpy()[at][:, None], sin.double().numpy()[at][:, None]
    a, b = (v[..., 0:rot:2], v[..., 1:rot:2]) if interleaved else (v[..., :h], v[..., h:rot])
    lo, hi = f32(a * c - f32(b * s)), f32(b * c + f32(a * s))
    out = v.copy()
    if interleaved:
        out[..., 0:rot:2], out[..., 1:rot:2] = lo, hi
    else:
        out[..., :h], out[..., h:rot] = lo, hi
    return bits(torch.from_numpy(out.astype(np.float32)).to(torch.bfloat16))


class Case:
    """One append call on CPU copies of everything, run on the GPU and checked."""

    def __init__(self, B, S, Hq, Hkv, D, rot, page=16, norm=True, interleaved=False, start=None, new_len=None, pos=None,
                 rows=None, seed=0, eps=1e-6, spare=3, fused=True):
        self.__dict__.update(B=B, S=S, Hq=Hq, Hkv=Hkv, D=D, rot=rot, page=page, interleaved=interleaved, eps=eps)
        self.kv_len = torch.tensor([7 * b % 40 for b in range(B)] if start is None else start, dtype=torch.int32)
        capacity = int(self.kv_len.clamp(min=0).max()) + S
        self.k_pages, self.v_pages, self.table = paged(B, capacity, page, Hkv, D, seed, spare, poison=False)
        rows = capacity if rows is None else rows
        angle = torch.arange(rows)[:, None].double() * 10000.0 ** (torch.arange(rot // 2) * (-2.0 / max(rot, 1)))
        self.cos, self.sin = angle.cos().float(), angle.sin().float()
        self.wq = self.wk = None
        if norm:
            g = torch.Generator().manual_seed(seed + 9)
            self.wq, self.wk = torch.rand(D, generator=g) + 0.5, torch.rand(D, generator=g) + 0.5
        self.new_len = None if new_len is None else torch.tensor(new_len, dtype=torch.int32)
        self.pos = None if pos is None else torch.tensor(pos, dtype=torch.int32).view(B, S)
        qkv = randn(B, S, (Hq + 2 * Hkv) * D, seed=seed + 5)
        if fused:  # slices of one projection's output
            self.src = tuple(t.unflatten(-1, (-1, D)) for t in qkv.split([Hq * D, Hkv * D, Hkv * D], dim=-1))
            self.dev = tuple(t.unflatten(-1, (-1, D)) for t in qkv.cuda().split([Hq * D, Hkv * D, Hkv * D], dim=-1))
        else:
            self.src = tuple(t.unflatten(-1, (-1, D)).contiguous() for t in qkv.split([Hq * D, Hkv * D, Hkv * D], dim=-1))
            self.dev = tuple(t.cuda() for t in self.src)

    def run(self, h3, in_place=False, stream=None):
        def cuda(t):
            return None if t is None else t.cuda()
        self.dk, self.dv, dl = self.k_pages.cuda(), self.v_pages.cuda(), self.kv_len.cuda()
        cache = h3.PagedKV(self.dk, self.dv, self.table.cuda(), dl)
        q, k, v = self.dev
        self.q_out = q if in_place else torch.full((self.B, self.S, self.Hq, self.D), 3.0, dtype=torch.bfloat16,
                                                   device="cuda")
        self.len_out = torch.full((self.B,), -5, dtype=torch.int32, device="cuda")
        no_q = self.Hq == 0
        h3.h3attn_qk_norm_rope_append(None if no_q else q, k, v, None if no_q else self.q_out, cache,
                                      None if no_q else cuda(self.wq), cuda(self.wk), cuda(self.cos), cuda(self.sin),
                                      self.rot, self.eps, self.interleaved, cuda(self.pos), cuda(self.new_len),
                                      self.len_out, stream)
        torch.cuda.synchronize()
        assert torch.equal(dl.cpu(), self.kv_len), "kv_len was changed"
        return self

    def expected(self, q_before):
        q_out, k, v = bits(q_before), bits(self.k_pages), bits(self.v_pages)
        lens, bad = [], False
        capacity = self.table.shape[1] * self.page
        for b in range(self.B):
            n0 = max(int(self.kv_len[b]), 0)
            n = self.S if self.new_len is None else min(max(int(self.new_len[b]), 0), self.S)
            lens.append(min(n0 + n, capacity))
            if n == 0:
                continue
            place = np.arange(n0, n0 + n)
            p = place if self.pos is None else self.pos[b, :n].numpy()
            lost = (p < 0) | (p >= self.cos.shape[0]) if self.rot else np.zeros(n, bool)
            bad |= bool(lost.any())
            at = np.where(lost, 0, p) if self.rot else np.zeros(n, int)
            rq = reference(self.src[0][b, :n], self.wq, self.cos, self.sin, at, self.rot, self.interleaved, self.eps)
            rk = reference(self.src[1][b, :n], self.wk, self.cos, self.sin, at, self.rot, self.interleaved, self.eps)
            rq[lost], rk[lost] = 0, 0
            q_out[b, :n] = rq
            rv = bits(self.src[2][b, :n])
            for i, t in enumerate(place):
                pg = int(self.table[b, t // self.page]) if t < capacity else -1
                if not 0 <= pg < self.k_pages.shape[0]:
                    bad = True
                    continue
                k[pg, t % self.page], v[pg, t % self.page] = rk[i], rv[i]
        return q_out, k, v, lens, bad

    def check(self, h3, in_place=False):
        before = self.src[0] if in_place else torch.full((self.B, self.S, self.Hq, self.D), 3.0, dtype=torch.bfloat16)
        q_out, k, v, lens, bad = self.expected(before)
        status = h3.h3attn_check_device_status()
        assert status == (h3.H3ATTN_ERR_INVALID_ARG if bad else 0)
        for name, got, ref in (("q_out", self.q_out, q_out), ("k_pages", self.dk, k), ("v_pages", self.dv, v)):
            wrong = np.flatnonzero(bits(got).reshape(-1) != ref.reshape(-1))
            assert wrong.size == 0, f"{name}: {wrong.size} elements differ, first at {wrong[:4]}"
        assert self.len_out.tolist() == lens


@pytest.mark.gpu
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("norm", [True, False])
@pytest.mark.parametrize("D,rot", [(64, 64), (64, 48), (64, 34), (64, 2), (128, 96), (128, 128), (128, 66), (128, 0),
                                   (256, 256), (256, 130), (256, 16), (256, 190)])
def test_layouts(h3, D, rot, norm, interleaved):
    Case(2, 5, 6, 2, D, rot, norm=norm, interleaved=interleaved, seed=D + rot).run(h3).check(h3)


@pytest.mark.gpu
@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (24, 24), (20, 4), (8, 1), (0, 3), (7, 7)])
@pytest.mark.parametrize("B,S,page", [(1, 1, 16), (9, 1, 24), (3, 33, 1), (2, 130, 64), (1, 257, 5)])
def test_shapes_and_pages(h3, Hq, Hkv, B, S, page):
    Case(B, S, Hq, Hkv, 128, 96, page=page, seed=B + S).run(h3).check(h3)


@pytest.mark.gpu
def test_ragged_rows_empty_ones_and_wild_lengths(h3):
    """Lengths below zero count as none, new_len is clamped to [0, S], padding is left as it was."""
    Case(6, 9, 4, 2, 128, 96, start=[0, -3, 15, 16, 17, 40], new_len=[9, 4, 0, 1, -2, 100], seed=3).run(h3).check(h3)


@pytest.mark.gpu
@pytest.mark.parametrize("interleaved", [False, True])
def test_given_positions(h3, interleaved):
    pos = [0, 99, 5, 5, 40, 41, 42, 3]
    Case(2, 4, 4, 4, 128, 96, pos=pos, rows=100, interleaved=interleaved, seed=6).run(h3).check(h3)


@pytest.mark.gpu
@pytest.mark.parametrize("D,rot", [(128, 96), (64, 34)])
def test_positions_outside_the_table_give_zeros_and_a_status(h3, D, rot):
    Case(2, 4, 4, 2, D, rot, pos=[0, -1, 5, 10, 2 ** 31 - 1, 9, -2 ** 31, 1], rows=10, seed=7).run(h3).check(h3)


@pytest.mark.gpu
def test_bad_pages_and_places_past_the_capacity(h3):
    """A token without a row in the cache is not stored; its query row is written, the others are stored."""

    c = Case(3, 6, 4, 2, 128, 96, page=4, start=[0, 3, 9], rows=64, seed=8)
    c.table[0, 1] = -1
    c.table[1, 0] = c.k_pages.shape[0]
    c.table = c.table[:, :3].contiguous()  # capacity 12: the last sequence's tokens from 12 on have no place
    c.run(h3).check(h3)


@pytest.mark.gpu
def test_length_next_to_the_largest_int(h3):
    c = Case(1, 3, 2, 1, 64, 64, start=[5], rows=32, seed=9)
    c.kv_len[0] = 2 ** 31 - 2
    c.pos = torch.tensor([[0, 1, 2]], dtype=torch.int32)
    c.run(h3).check(h3)


@pytest.mark.gpu
def test_contiguous_tensors_and_in_place_queries(h3):
    Case(2, 7, 4, 2, 128, 96, fused=False, seed=10).run(h3).check(h3)
    c = Case(2, 7, 4, 2, 128, 66, fused=False, new_len=[7, 3], seed=11)
    c.run(h3, in_place=True).check(h3, in_place=True)


@pytest.mark.gpu
@pytest.mark.parametrize("D,rot", [(64, 48), (128, 96), (256, 130)])
def test_bit_equal_to_the_contiguous_call(h3, D, rot):
    B, S, Hq, Hkv = 1, 300, 6, 2
    c = Case(B, S, Hq, Hkv, D, rot, start=[0], fused=False, page=32, seed=12).run(h3)
    q, k = torch.empty_like(c.dev[0]), torch.empty_like(c.dev[1])
    h3.h3attn_qk_norm_rope_out(c.dev[0], c.dev[1], q, k, c.wq.cuda(), c.wk.cuda(), c.cos.cuda(), c.sin.cuda(), rot, c.eps)
    assert torch.equal(q.view(torch.int16), c.q_out.view(torch.int16))
    rows = c.dk[c.table[0].long().cuda()].flatten(0, 1)[:S]
    assert torch.equal(rows.view(torch.int16), k[0].view(torch.int16))


@pytest.mark.gpu
def test_pages_past_32_bits(h3):
    """A cache of more than 2^31 elements: the row of the last page is the one that is written."""
    page, Hkv, D = 64, 8, 128
    pages = (1 << 31) // (page * Hkv * D) + 3
    k = torch.zeros(pages, page, Hkv, D, dtype=torch.bfloat16, device="cuda")
    v = torch.zeros_like(k)
    table = torch.tensor([[pages - 1]], dtype=torch.int32, device="cuda")
    cache = h3.PagedKV(k, v, table, torch.tensor([63], dtype=torch.int32, device="cuda"))
    new = randn(1, 1, 2 * Hkv, D, seed=1).cuda()
    h3.h3attn_qk_norm_rope_append(None, new[:, :, :Hkv], new[:, :, Hkv:], None, cache, None, None, None, None, 0)
    assert torch.equal(k[-1, 63], new[0, 0, :Hkv]) and torch.equal(v[-1, 63], new[0, 0, Hkv:])
    assert int(k[:, :, 0, 0].count_nonzero()) == 1 and int(v[:, :, 0, 0].count_nonzero()) == 1


@pytest.mark.gpu
def test_stream_and_graph(h3):
    """On another stream, and captured: a replay appends what the buffers hold then."""
    c = Case(3, 2, 4, 2, 128, 96, fused=False, seed=13)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    c.run(h3, stream=s)
    c.check(h3)
    dk, dv, dl = c.k_pages.cuda(), c.v_pages.cuda(), c.kv_len.cuda()
    cache = h3.PagedKV(dk, dv, c.table.cuda(), dl)
    q, k, v = c.dev
    wq, wk, cos, sin = c.wq.cuda(), c.wk.cuda(), c.cos.cuda(), c.sin.cuda()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        h3.h3attn_qk_norm_rope_append(q, k, v, c.q_out, cache, wq, wk, cos, sin, 96, len_out=c.len_out)
    assert torch.equal(dk.cpu(), c.k_pages)  # nothing ran while capturing
    dl.sub_(5).clamp_(min=0)
    c.kv_len = dl.cpu()
    graph.replay()
    torch.cuda.synchronize()
    c.dk, c.dv = dk, dv
    c.check(h3)
