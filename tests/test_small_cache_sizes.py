"""Workspace sizes from the binding: numbers that do not fit the C interface's 32
bits are refused, not taken modulo 2^32."""
import types

import pytest

import video_dit_dense_gb300 as h3


@pytest.fixture(scope="module")
def built():
    h3.build()


def cache(bits, B=2):
    """A descriptor without a device: 4 pages of 16 tokens a sequence."""
    if bits == 4:
        return types.SimpleNamespace(_struct=h3.h3attn_paged_kv4_t(*[None] * 6, B, 9, 16, 4, 2, 128))
    return types.SimpleNamespace(_struct=h3.h3attn_paged_kv_t(*[None] * 4, B, 9, 16, 4, 2, 128))


@pytest.mark.parametrize("keep,recent", [(2 ** 32 + 10, 3), (10, 2 ** 32 + 3), (10, 3 - 2 ** 32), (10 - 2 ** 32, 3), (2 ** 31, 0),
                                         (2 ** 64 + 10, 3)])
def test_evict(built, keep, recent):
    with pytest.raises(h3.H3AttnError, match="32 bits") as e:
        h3.h3attn_paged_evict_workspace_size(cache(4), keep, recent)
    assert e.value.status == h3.H3ATTN_ERR_INVALID_ARG
    # header of 4, both lists of min(10 - 3, 64 - 10), a chain for each of min(3, 64 - 10), 4 bytes each
    assert h3.h3attn_paged_evict_workspace_size(cache(4), 10, 3) == 2 * 4 * (4 + 2 * 7 + 3)


@pytest.mark.parametrize("Hq", [2 ** 32 + 4, 2 ** 31, 4 - 2 ** 32, -2 ** 31 - 1])
def test_decode(built, Hq):
    for size, bits in ((h3.h3attn_paged_decode_workspace_size, 16), (h3.h3attn_paged_decode_q4_workspace_size, 4),
                       (h3.h3attn_paged_decode_weights_workspace_size, 16)):
        with pytest.raises(h3.H3AttnError, match="32 bits") as e:
            size(cache(bits, B=0), Hq)
        assert e.value.status == h3.H3ATTN_ERR_INVALID_ARG
        assert size(cache(bits, B=0), 4) == 0
