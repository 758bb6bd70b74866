"""Host-side refusals of the operators that keep a cache small: answered before
any CUDA call, from C and from the Python binding."""
import ctypes

import pytest
import torch

import video_dit_dense_gb300 as h3

M = 0x1000000  # 16 MiB apart: fake device addresses, never used
BAD, ALIGN, HEAD = h3.H3ATTN_ERR_INVALID_ARG, h3.H3ATTN_ERR_MISALIGNED, h3.H3ATTN_ERR_UNSUPPORTED_HEAD_DIM
INF, NAN = float("inf"), float("nan")


@pytest.fixture(scope="module")
def lib():
    h3.build()
    return h3.load()


GEOMETRY = [(dict(B=-1), BAD), (dict(B=65536), BAD), (dict(num_pages=0), BAD), (dict(page_size=0), BAD), (dict(max_pages=0), BAD),
            (dict(Hkv=0), BAD), (dict(D=96), HEAD), (dict(num_pages=2 ** 20, page_size=2 ** 11), BAD),
            (dict(max_pages=2 ** 30, page_size=2), BAD)]
POINTERS = [(dict(k=None), BAD), (dict(v=None), BAD), (dict(t=None), BAD), (dict(n=None), BAD), (dict(k=100 * M + 8), ALIGN),
            (dict(v=120 * M + 4), ALIGN), (dict(t=140 * M + 2), ALIGN), (dict(n=141 * M + 1), ALIGN)]
SCALES = [(dict(ks=None), BAD), (dict(vs=None), BAD), (dict(ks=130 * M + 8), ALIGN), (dict(vs=131 * M + 1), ALIGN)]
FIELDS = ("k", "v", "ks", "vs", "t", "n", "B", "num_pages", "page_size", "max_pages", "Hkv", "D")


def cache(kind, k=100 * M, v=120 * M, ks=130 * M, vs=131 * M, t=140 * M, n=141 * M, B=2, num_pages=9, page_size=16, max_pages=4,
          Hkv=2, D=128):
    if kind == 4:
        return ctypes.byref(h3.h3attn_paged_kv4_t(k, v, ks, vs, t, n, B, num_pages, page_size, max_pages, Hkv, D))
    return ctypes.byref(h3.h3attn_paged_kv_t(k, v, t, n, B, num_pages, page_size, max_pages, Hkv, D))


def split(args, kind=4):
    """The cache of these arguments, and the others."""
    of_cache = {n: args[n] for n in FIELDS if n in args}
    return cache(kind, **of_cache), {n: a for n, a in args.items() if n not in of_cache}


def append(lib, c, q=M, kk=2 * M, vv=3 * M, o=4 * M, wq=5 * M, wk=6 * M, cos=7 * M, sin=8 * M, pos=None, new=None, out=None, S=3, Hq=4,
           qst=4 * 128, kst=2 * 128, vst=2 * 128, rows=100, rot=96, inter=0, eps=1e-6, null=False):
    return lib.h3attn_qk_norm_rope_append_q4(q, kk, vv, o, None if null else c, wq, wk, cos, sin, pos, new, out, S, Hq, qst, kst, vst, rows,
                                             rot, inter, eps, None)


@pytest.mark.parametrize("args,want", GEOMETRY + POINTERS + SCALES + [
    (dict(null=True), BAD), (dict(S=-1), BAD), (dict(rot=95), BAD), (dict(rot=130), BAD), (dict(eps=NAN), BAD), (dict(q=None), BAD),
    (dict(o=None), BAD), (dict(kk=None), BAD), (dict(cos=None), BAD), (dict(qst=511), BAD), (dict(kst=260), ALIGN), (dict(vv=3 * M + 2), ALIGN),
    (dict(o=2 * M), BAD), (dict(o=100 * M), BAD), (dict(o=130 * M + 64), BAD), (dict(v=100 * M + 16), BAD), (dict(ks=100 * M + 64), BAD),
    (dict(vs=130 * M + 16), BAD), (dict(vs=120 * M), BAD), (dict(kk=130 * M), BAD), (dict(out=141 * M), BAD), (dict(out=131 * M), BAD),
    (dict(wk=131 * M), BAD), (dict(S=0), 0), (dict(B=0), 0)])
def test_append_q4(lib, args, want):
    c, rest = split(args)
    assert append(lib, c, **rest) == want


@pytest.mark.parametrize("kind", [4, 16])
@pytest.mark.parametrize("args,want", GEOMETRY + POINTERS + [
    (dict(null=True), BAD), (dict(S=-1), BAD), (dict(ko=None, vo=None), BAD), (dict(ko=2 * M), BAD), (dict(ko=M + 8), ALIGN),
    (dict(vo=2 * M + 2), ALIGN), (dict(first=3 * M + 2), ALIGN), (dict(first=M), BAD), (dict(ko=100 * M), BAD), (dict(vo=120 * M + 64), BAD),
    (dict(vo=140 * M), BAD), (dict(S=2 ** 30), BAD), (dict(S=0), 0), (dict(S=0, ko=None, vo=None), 0), (dict(B=0), 0)])
def test_read(lib, kind, args, want):
    c, rest = split(args, kind)

    def call(ko=M, vo=2 * M, first=None, S=5, null=False):
        f = lib.h3attn_paged_read_q4 if kind == 4 else lib.h3attn_paged_read
        return f(None if null else c, ko, vo, first, S, None)
    assert call(**rest) == want


def test_read_q4_scales(lib):
    for args, want in SCALES + [(dict(ks=M), BAD), (dict(vs=2 * M + 16), BAD)]:
        c, _ = split(args)
        assert lib.h3attn_paged_read_q4(c, M, 2 * M, None, 5, None) == want


DECODE = [(dict(null=True), BAD), (dict(Hq=0), BAD), (dict(Hq=5), BAD), (dict(Hq=65536), BAD), (dict(scale=0.0), BAD),
          (dict(scale=NAN), BAD), (dict(scale=INF), BAD), (dict(scale=3e38), BAD), (dict(q=None), BAD), (dict(o=None), BAD),
          (dict(q=M + 8), ALIGN), (dict(o=2 * M + 2), ALIGN), (dict(o=M), BAD), (dict(o=100 * M + 256), BAD), (dict(o=141 * M), BAD),
          (dict(B=65535, Hkv=65535, Hq=65535), BAD), (dict(B=0), 0)]


@pytest.mark.parametrize("args,want", GEOMETRY + POINTERS + SCALES + DECODE + [
    (dict(ws=3 * M + 8, nbytes=1 << 20), ALIGN), (dict(o=130 * M), BAD), (dict(o=131 * M), BAD)])
def test_decode_q4(lib, args, want):
    c, rest = split(args)

    def call(q=M, o=2 * M, Hq=4, scale=0.1, ws=None, nbytes=0, null=False):
        return lib.h3attn_paged_decode_q4(q, o, None if null else c, Hq, scale, ws, nbytes, None)
    assert call(**rest) == want


@pytest.mark.parametrize("kind", [4, 16])
@pytest.mark.parametrize("args,want", GEOMETRY + POINTERS + DECODE + [
    (dict(w=None), BAD), (dict(ws=None), BAD), (dict(w=4 * M + 2), ALIGN), (dict(ws=3 * M + 8), ALIGN), (dict(w=2 * M), BAD),
    (dict(w=M), BAD), (dict(w=100 * M), BAD), (dict(w=120 * M + 64), BAD), (dict(w=141 * M), BAD), (dict(w=140 * M), BAD)])
def test_decode_weights(lib, kind, args, want):
    c, rest = split(args, kind)

    def call(q=M, o=2 * M, Hq=4, scale=0.1, w=4 * M, ws=3 * M, nbytes=1 << 24, null=False):
        f = lib.h3attn_paged_decode_weights_q4 if kind == 4 else lib.h3attn_paged_decode_weights
        return f(q, o, None if null else c, Hq, scale, w, ws, nbytes, None)
    assert call(**rest) == want


@pytest.mark.parametrize("args,want", GEOMETRY + [(dict(Hq=5), BAD), (dict(B=0), 0)])
def test_decode_workspace_sizes(lib, args, want):
    args = dict(args)
    Hq = args.pop("Hq", 4)
    for name, kind in (("decode_q4", 4), ("decode_weights", 16), ("decode_weights_q4", 4)):
        f, n = getattr(lib, f"h3attn_paged_{name}_workspace_size"), ctypes.c_size_t(123)
        assert f(cache(kind, **args), Hq, ctypes.byref(n)) == want and n.value == 0
        assert f(cache(kind), 4, None) == BAD


@pytest.mark.parametrize("kind", [4, 16])
@pytest.mark.parametrize("args,want", GEOMETRY + POINTERS + [
    (dict(null=True), BAD), (dict(keep=0), BAD), (dict(keep=-1), BAD), (dict(recent=-1), BAD), (dict(recent=11), BAD), (dict(w=None), BAD),
    (dict(out=None), BAD), (dict(ws=None), BAD), (dict(nbytes=16), BAD), (dict(w=M + 2), ALIGN), (dict(out=2 * M + 2), ALIGN),
    (dict(ws=3 * M + 8), ALIGN), (dict(out=141 * M), BAD), (dict(out=M + 4), BAD), (dict(ws=M), BAD), (dict(ws=2 * M), BAD),
    (dict(w=100 * M), BAD), (dict(ws=120 * M), BAD), (dict(out=140 * M), BAD), (dict(v=100 * M), BAD), (dict(t=100 * M), BAD),
    (dict(n=120 * M + 64), BAD), (dict(w=140 * M), BAD), (dict(B=0), 0), (dict(B=0, ws=None), 0)])
def test_evict(lib, kind, args, want):
    c, rest = split(args, kind)

    def call(w=M, keep=10, recent=3, out=2 * M, ws=3 * M, nbytes=1 << 20, null=False):
        f = lib.h3attn_paged_evict_q4 if kind == 4 else lib.h3attn_paged_evict
        return f(None if null else c, w, keep, recent, out, ws, nbytes, None)
    assert call(**rest) == want


def test_evict_workspace_size(lib):
    n = ctypes.c_size_t(123)

    def size(B=2, page=16, pages=4, keep=10, recent=3):
        return lib.h3attn_paged_evict_workspace_size(B, page, pages, keep, recent, ctypes.byref(n))
    # header of 4, both lists of min(keep - recent, 64 - keep), a chain for each of min(recent, 64 - keep), 4 bytes each
    assert size() == 0 and n.value == 2 * 4 * (4 + 2 * 7 + 3)
    assert size(keep=60) == 0 and n.value == 2 * 4 * (4 + 2 * 4 + 3)
    assert size(keep=64) == 0 and n.value == 2 * 4 * 4
    assert size(keep=2 ** 31 - 1, recent=2 ** 31 - 1) == 0 and n.value == 2 * 4 * 4
    assert size(B=0) == 0 and n.value == 0
    for bad in (dict(B=-1), dict(page=0), dict(pages=0), dict(keep=0), dict(recent=11), dict(page=2 ** 16, pages=2 ** 15)):
        assert size(**bad) == BAD and n.value == 0
    assert lib.h3attn_paged_evict_workspace_size(2, 16, 4, 10, 3, None) == BAD


def test_the_binding_refuses_before_any_call(lib):
    """CPU tensors are never taken for device buffers; the wrong kind of cache is said."""
    x = torch.zeros(2, 1, 4, 64, dtype=torch.bfloat16)
    codes, scales = torch.zeros(3, 16, 2, 32, dtype=torch.uint8), torch.zeros(3, 16, 2, 4, dtype=torch.uint8)
    table, lens = torch.zeros(2, 2, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    with pytest.raises(h3.H3AttnError, match="CUDA tensor"):
        h3.PagedKV4(codes, codes, scales, scales, table, lens)
    with pytest.raises(h3.H3AttnError, match="num_pages"):
        h3.PagedKV4(codes[0], codes[0], scales, scales, table, lens)
    with pytest.raises(h3.H3AttnError, match="32 bits"):
        many = torch.zeros(2 ** 32 + 3, 0, 2, 32, dtype=torch.uint8)
        h3.PagedKV4(many, many, many, many, table, lens)
    for call in (lambda: h3.h3attn_paged_decode_q4(x, x, object()),
                 lambda: h3.h3attn_qk_norm_rope_append_q4(x, x, x, x, object(), None, None, None, None),
                 lambda: h3.h3attn_paged_decode_weights(x, x, object(), x, x), lambda: h3.h3attn_paged_read(object(), x, None),
                 lambda: h3.h3attn_paged_evict(object(), lens.float(), 1, 0, lens, lens)):
        with pytest.raises(h3.H3AttnError, match="CUDA tensor"):
            call()
    with pytest.raises(h3.H3AttnError, match="at least one"):
        h3.h3attn_paged_read(object(), None, None)
    with pytest.raises(h3.H3AttnError, match="must be a tensor"):
        h3.h3attn_paged_evict(object(), None, 1, 0, None, None)
