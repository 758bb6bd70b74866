"""Host-side refusals of the generation operators: answered before any CUDA call,
from C and from the Python binding."""
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


def norm(lib, x=M, residual=2 * M, h=3 * M, y=4 * M, w=5 * M, s=None, T=4, C=256, fmt=0, eps=1e-6):
    return lib.h3attn_add_rmsnorm(x, residual, h, y, w, s, T, C, fmt, eps, None)


@pytest.mark.parametrize("args,want", [
    (dict(C=0), BAD), (dict(C=12), BAD), (dict(C=16392), BAD), (dict(T=-1), BAD), (dict(eps=-1.0), BAD), (dict(eps=NAN), BAD),
    (dict(fmt=3), BAD), (dict(fmt=-1), BAD), (dict(fmt=2, s=6 * M, C=40), BAD), (dict(fmt=1), BAD), (dict(s=6 * M), BAD),
    (dict(x=None), BAD), (dict(y=None), BAD), (dict(h=None), BAD), (dict(residual=None), BAD),
    (dict(x=M + 8), ALIGN), (dict(y=4 * M + 2), ALIGN), (dict(h=3 * M + 4), ALIGN), (dict(w=5 * M + 4), ALIGN),
    (dict(fmt=1, s=6 * M + 2), ALIGN),
    (dict(h=4 * M), BAD),                       # h over y
    (dict(h=M + 64), BAD), (dict(y=2 * M + 64), BAD), (dict(y=5 * M), BAD), (dict(h=5 * M), BAD),
    (dict(h=M, y=M), BAD),                      # both outputs over x
    (dict(fmt=1, s=6 * M, y=M), BAD),           # 8 bits over 16
    (dict(fmt=1, s=M), BAD), (dict(fmt=1, s=4 * M), BAD), (dict(fmt=2, s=3 * M), BAD),
    (dict(T=0), 0), (dict(T=0, x=None, y=None), 0)])
def test_add_rmsnorm(lib, args, want):
    assert norm(lib, **args) == want


def table(lib, cos=M, sin=2 * M, pos=None, first=0, N=16, rot=96, theta=10000.0, scaling=None):
    s = None if scaling is None else ctypes.byref(h3.h3attn_rope_scaling_t(*scaling))
    return lib.h3attn_rope_table(cos, sin, pos, first, N, rot, theta, s, None)


@pytest.mark.parametrize("args,want", [
    (dict(N=-1), BAD), (dict(rot=0), BAD), (dict(rot=95), BAD), (dict(rot=258), BAD), (dict(rot=-2), BAD),
    (dict(theta=0.5), BAD), (dict(theta=INF), BAD), (dict(theta=NAN), BAD), (dict(first=-1), BAD),
    (dict(first=2 ** 31 - 15), BAD), (dict(first=2 ** 62), BAD), (dict(first=2 ** 63 - 1), BAD), (dict(first=1, pos=3 * M), BAD),
    (dict(cos=None), BAD), (dict(sin=None), BAD), (dict(cos=M + 4), ALIGN), (dict(pos=3 * M + 2), ALIGN),
    (dict(sin=M), BAD), (dict(pos=M), BAD), (dict(pos=2 * M + 64), BAD),
    # kind, original_len, factor, low, high, amplitude
    (dict(scaling=(4, 1, 2.0, 1.0, 32.0, 1.0)), BAD), (dict(scaling=(-1, 1, 2.0, 1.0, 32.0, 1.0)), BAD),
    (dict(scaling=(1, 1, 0.5, 1.0, 32.0, 1.0)), BAD), (dict(scaling=(1, 1, NAN, 1.0, 32.0, 1.0)), BAD),
    (dict(scaling=(1, 1, 2.0, 1.0, 32.0, 0.0)), BAD), (dict(scaling=(1, 1, 2.0, 1.0, 32.0, INF)), BAD),
    (dict(scaling=(1, 1, 2.0, 1.0, 32.0, 1e300)), BAD), (dict(scaling=(2, 1, 2.0, 1.0, 32.0, 1.0), rot=2), BAD),
    (dict(scaling=(2, 1, 1e300, 1.0, 32.0, 1.0), theta=1e300), BAD),
    (dict(scaling=(3, 0, 2.0, 1.0, 32.0, 1.0)), BAD), (dict(scaling=(3, 9, 2.0, -1.0, 32.0, 1.0)), BAD),
    (dict(scaling=(3, 9, 2.0, 5.0, 5.0, 1.0)), BAD), (dict(scaling=(3, 9, 2.0, 5.0, INF, 1.0)), BAD),
    (dict(scaling=(3, 9, 2.0, NAN, 5.0, 1.0)), BAD), (dict(N=0), 0)])
def test_rope_table(lib, args, want):
    assert table(lib, **args) == want


GEOMETRY = [(dict(B=-1), BAD), (dict(B=65536), BAD), (dict(num_pages=0), BAD), (dict(page_size=0), BAD), (dict(max_pages=0), BAD),
            (dict(Hkv=0), BAD), (dict(D=96), HEAD), (dict(num_pages=2 ** 20, page_size=2 ** 11), BAD),
            (dict(max_pages=2 ** 30, page_size=2), BAD)]


def kv(k=100 * M, v=120 * M, t=140 * M, n=141 * M, B=2, num_pages=9, page_size=16, max_pages=4, Hkv=2, D=128):
    return h3.h3attn_paged_kv_t(k, v, t, n, B, num_pages, page_size, max_pages, Hkv, D)


def append(lib, q=M, k=2 * M, v=3 * M, o=4 * M, wq=5 * M, wk=6 * M, cos=7 * M, sin=8 * M, pos=None, new=None, out=None, S=3,
           Hq=4, qs=4 * 128, ks=2 * 128, vs=2 * 128, rows=100, rot=96, inter=0, eps=1e-6, null=False, **cache):
    c = None if null else ctypes.byref(kv(**cache))
    return lib.h3attn_qk_norm_rope_append(q, k, v, o, c, wq, wk, cos, sin, pos, new, out, S, Hq, qs, ks, vs, rows, rot, inter,
                                          eps, None)


@pytest.mark.parametrize("args,want", GEOMETRY + [
    (dict(null=True), BAD), (dict(S=-1), BAD), (dict(Hq=-1), BAD), (dict(rot=95), BAD), (dict(rot=130), BAD), (dict(rot=-2), BAD),
    (dict(eps=NAN), BAD), (dict(rows=-1), BAD), (dict(q=None), BAD), (dict(o=None), BAD), (dict(Hq=0), BAD),
    (dict(q=None, o=None, Hq=0), BAD),          # a query weight without queries
    (dict(k=None), BAD), (dict(v=None), BAD), (dict(cos=None), BAD), (dict(qs=511), BAD), (dict(ks=255), BAD), (dict(vs=-256), BAD),
    (dict(vs=2 ** 62), BAD), (dict(S=2 ** 30), BAD),
    (dict(qs=516), ALIGN), (dict(ks=260), ALIGN), (dict(q=M + 8), ALIGN), (dict(v=3 * M + 2), ALIGN), (dict(wk=6 * M + 4), ALIGN),
    (dict(pos=9 * M + 2), ALIGN), (dict(new=9 * M + 1), ALIGN), (dict(out=9 * M + 3), ALIGN), (dict(k=2 * M + 8), ALIGN),
    (dict(t=140 * M + 2), ALIGN), (dict(n=141 * M + 1), ALIGN), (dict(t=None), BAD), (dict(n=None), BAD),
    (dict(o=2 * M), BAD), (dict(o=M, qs=1024), BAD), (dict(o=M + 512), BAD), (dict(o=7 * M), BAD),
    (dict(v=120 * M), BAD), (dict(q=100 * M + 4096), BAD), (dict(o=120 * M), BAD),
    (dict(out=141 * M), BAD), (dict(out=10 * M, new=10 * M), BAD), (dict(out=4 * M), BAD), (dict(pos=100 * M), BAD),
    (dict(S=0), 0), (dict(B=0), 0)])
def test_append(lib, args, want):
    cache = {n: args[n] for n in ("B", "num_pages", "page_size", "max_pages", "Hkv", "D", "t", "n") if n in args}
    rest = {n: a for n, a in args.items() if n not in cache}
    assert append(lib, **rest, **cache) == want


def decode(lib, q=M, o=2 * M, Hq=4, scale=0.1, ws=None, nbytes=0, null=False, **cache):
    return lib.h3attn_paged_decode(q, o, None if null else ctypes.byref(kv(**cache)), Hq, scale, ws, nbytes, None)


@pytest.mark.parametrize("args,want", GEOMETRY + [
    (dict(null=True), BAD), (dict(Hq=0), BAD), (dict(Hq=5), BAD), (dict(Hq=65536), BAD), (dict(scale=0.0), BAD), (dict(scale=-1.0), BAD),
    (dict(scale=NAN), BAD), (dict(scale=INF), BAD), (dict(scale=3e38), BAD), (dict(q=None), BAD), (dict(o=None), BAD), (dict(k=None), BAD), (dict(v=None), BAD),
    (dict(t=None), BAD), (dict(n=None), BAD), (dict(q=M + 8), ALIGN), (dict(o=2 * M + 2), ALIGN), (dict(k=100 * M + 8), ALIGN),
    (dict(t=140 * M + 2), ALIGN), (dict(ws=3 * M + 8, nbytes=1 << 20), ALIGN), (dict(o=M), BAD), (dict(o=100 * M + 256), BAD),
    (dict(o=141 * M), BAD), (dict(B=65535, Hkv=65535, Hq=65535), BAD), (dict(B=0), 0)])
def test_decode(lib, args, want):
    assert decode(lib, **args) == want


@pytest.mark.parametrize("args,want", GEOMETRY + [(dict(Hq=5), BAD), (dict(B=0), 0)])
def test_decode_workspace_size(lib, args, want):
    args = dict(args)
    Hq, n = args.pop("Hq", 4), ctypes.c_size_t(123)
    assert lib.h3attn_paged_decode_workspace_size(ctypes.byref(kv(**args)), Hq, ctypes.byref(n)) == want
    assert n.value == 0
    assert lib.h3attn_paged_decode_workspace_size(ctypes.byref(kv()), 4, None) == BAD


def test_the_binding_refuses_before_any_call(lib):
    """CPU tensors are never taken for device buffers."""
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    with pytest.raises(h3.H3AttnError, match="CUDA tensor"):
        h3.h3attn_add_rmsnorm(x, None, None, x)
    with pytest.raises(h3.H3AttnError, match="CUDA tensor"):
        h3.h3attn_rope_table(torch.zeros(4, 48), torch.zeros(4, 48), 96)
    pages = torch.zeros(3, 16, 2, 128, dtype=torch.bfloat16)
    with pytest.raises(h3.H3AttnError, match="CUDA tensor"):
        h3.PagedKV(pages, pages, torch.zeros(1, 2, dtype=torch.int32), torch.zeros(1, dtype=torch.int32))
    with pytest.raises(h3.H3AttnError, match="num_pages"):
        h3.PagedKV(pages[0], pages[0], torch.zeros(1, 2, dtype=torch.int32), torch.zeros(1, dtype=torch.int32))


def test_the_compiled_host_path_is_bound_to_the_library(lib):
    """Wrong counts and kinds of arguments are Python errors, nothing else."""
    step = h3._get_step()
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    with pytest.raises(TypeError):
        step.add_rmsnorm(x)
    with pytest.raises(h3.H3AttnError, match="x must be a tensor"):
        h3.h3attn_add_rmsnorm(None, None, None, x)
    with pytest.raises(h3.H3AttnError, match="CUDA tensor"):
        h3.h3attn_paged_decode(x, x, object())
    with pytest.raises(h3.H3AttnError, match="CUDA tensor"):
        h3.h3attn_qk_norm_rope_append(x, x, x, x, object(), None, None, None, None)
    with pytest.raises(h3.H3AttnError, match="unknown scaling"):
        h3.RopeScaling("cubic")
    for n in (2 ** 31, 2 ** 32 + 1, -2 ** 40):  # ctypes would keep the low 32 bits
        with pytest.raises(h3.H3AttnError, match="original_len"):
            h3.RopeScaling("by_parts", 2.0, n)
    pages = torch.zeros(2 ** 32 + 3, 0, 2, 128, dtype=torch.bfloat16)
    with pytest.raises(h3.H3AttnError, match="32 bits"):
        h3.PagedKV(pages, pages, torch.zeros(1, 2, dtype=torch.int32), torch.zeros(1, dtype=torch.int32))
