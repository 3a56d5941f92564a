"""Sizes past which the step calls' kernels would count beyond 32 bits are
refused on the host (no GPU is needed; the pointers are never followed)."""

import pytest

from tests.test_step_refusals import UNSUPPORTED, ops, prefix, rope, step, verify  # noqa: F401


@pytest.mark.parametrize("S,refused", [(2**30 + 1, True), (2**31 - 1, True), (2**30, False)])
def test_step_requests(ops, S, refused):  # noqa: F811
    assert (step(ops, S=S, width=1, K=1, ring_size=0 if not refused else 8) == UNSUPPORTED) is refused


@pytest.mark.parametrize("rows,refused", [(2**30 + 1, True), (2**31 - 1, True), (2**30, False)])
def test_verification_rows(ops, rows, refused):  # noqa: F811
    assert (verify(ops, mq=rows, cu=None) == UNSUPPORTED) is refused


@pytest.mark.parametrize("H,J,refused", [(2**30 - 2, 2**30 - 2, True), (2, 2**29, True), (2**29, 2**28, True),
                                         (2**29, 2**28 - 1, False)])
def test_heads_of_a_token(ops, H, J, refused):  # noqa: F811
    got = rope(ops, T=1, H=H, J=J, D=2, rot=0, qs=2 * H, ks=2 * J, vs=2 * J, os=2 * H, q=None)
    assert (got == UNSUPPORTED) is refused
