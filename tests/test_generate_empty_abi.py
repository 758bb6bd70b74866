"""Empty batches and steps of the generation operators, answered before any CUDA
call: an empty tensor has no address, so its null pointer is no fault."""
import pytest

from test_generate_abi import append, decode, lib, norm, table  # noqa: F401  (lib is the fixture)

NO_ROWS = dict(q=None, k=None, v=None, o=None)


@pytest.mark.parametrize("args", [dict(S=0, **NO_ROWS), dict(B=0, **NO_ROWS), dict(S=0, B=0, **NO_ROWS),
                                  dict(B=0, t=None, n=None, **NO_ROWS), dict(S=0, wq=None, wk=None, **NO_ROWS)])
def test_append_of_no_tokens(lib, args):  # noqa: F811
    assert append(lib, **args) == 0


def test_the_others_of_no_rows(lib):  # noqa: F811
    assert norm(lib, T=0, x=None, residual=None, h=None, y=None) == 0
    assert table(lib, N=0, cos=None, sin=None) == 0
    assert decode(lib, B=0, q=None, o=None, t=None, n=None) == 0
