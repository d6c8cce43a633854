"""Sizes at the ends of their types, refused on a host without a GPU."""
from __future__ import annotations

import pytest

from causal_depthwise_conv1d_fwd_gb300 import _lib, build
from test_layer_abi import NULLP, OK, SIZE, STRIDE, verify

MAX = (1 << 31) - 1


@pytest.fixture(scope="module")
def lib():
    build.build()
    return _lib.load()


@pytest.mark.parametrize("sizes", [dict(drafts=MAX), dict(drafts=MAX - 1), dict(drafts=MAX, batch=MAX), dict(batch=MAX, drafts=0, vocab=9000),
                                   dict(batch=MAX, drafts=1), dict(batch=1 << 16, drafts=(1 << 15) - 1), dict(vocab=MAX),
                                   dict(batch=MAX, drafts=MAX, vocab=MAX), dict(batch=1 << 14, drafts=0, vocab=1 << 30)])
def test_verify_refuses_more_rows_than_a_grid_has(lib, sizes):
    assert verify(lib, wsb=(1 << 63) - 1, **sizes) == SIZE
    d = dict(batch=2, drafts=3, vocab=1000)
    d.update(sizes)
    assert lib.spec_verify_workspace(d["batch"], d["drafts"], d["vocab"]) == 0


def test_verify_checks_come_in_order(lib):
    """Strides before sizes that depend on the vocabulary, those before pointers; nothing to do is no error."""
    assert verify(lib, drafts=MAX, tb=-1) == STRIDE
    assert verify(lib, drafts=MAX, t=None) == SIZE
    assert verify(lib, t=None) == NULLP
    assert verify(lib, batch=0, drafts=MAX) == OK


def test_verify_workspace_grows_with_the_sizes(lib):
    sizes = [lib.spec_verify_workspace(b, s, v) for b, s, v in ((1, 0, 1), (1, 1, 1), (4, 3, 32003), (64, 4, 131072), (64, 4, 1 << 20))]
    assert sizes == sorted(sizes) and sizes[0] > 0
    assert lib.spec_verify_workspace(0, 3, 100) == lib.spec_verify_workspace(2, 3, 0) == 0
