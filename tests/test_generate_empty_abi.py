"""Empty batches and steps of the generation operators, answered before any CUDA
call: an empty tensor has no address, so its null pointer is no fault."""
import pytest

from test_generate_abi import ALIGN, BAD, M, append, decode, lib, norm, table  # noqa: F401  (lib is the fixture)

NO_ROWS = dict(q=None, k=None, v=None, o=None)


@pytest.mark.parametrize("args", [dict(S=0, **NO_ROWS), dict(B=0, **NO_ROWS), dict(S=0, B=0, **NO_ROWS),
                                  dict(B=0, t=None, n=None, **NO_ROWS), dict(S=0, wq=None, wk=None, **NO_ROWS)])
def test_append_of_no_tokens(lib, args):  # noqa: F811
    assert append(lib, **args) == 0


def test_the_others_of_no_rows(lib):  # noqa: F811
    assert norm(lib, T=0, x=None, residual=None, h=None, y=None) == 0
    assert table(lib, N=0, cos=None, sin=None) == 0
    assert decode(lib, B=0, q=None, o=None, t=None, n=None) == 0


@pytest.mark.parametrize("args,want", [
    (dict(out=9 * M + 3), ALIGN), (dict(out=141 * M), BAD), (dict(out=141 * M + 4), BAD), (dict(out=140 * M), BAD),
    (dict(out=100 * M), BAD), (dict(out=120 * M + 64), BAD), (dict(out=9 * M, new=9 * M), BAD), (dict(out=9 * M, n=None), BAD),
    (dict(out=9 * M, n=141 * M + 2), ALIGN), (dict(out=9 * M, B=0), 0), (dict(out=9 * M + 3, B=0), 0)])
def test_lengths_of_a_step_without_tokens(lib, args, want):  # noqa: F811
    """len_out is written by a step without tokens too, so its place is looked at."""
    assert append(lib, S=0, **NO_ROWS, **args) == want
