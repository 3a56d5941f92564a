"""Sizes that attention behind a shared prefix cannot count are refused before
anything is launched (no GPU is needed; the pointers are never followed)."""

import pytest

from tests.test_step_refusals import UNSUPPORTED, ops, prefix  # noqa: F401


@pytest.mark.parametrize("S,most,refused", [(2048, 2**24, True), (2048, 2**24 - 16, False),
                                            (512, 2**26, True), (1, 2**31 - 1, False)])
def test_tokens_of_all_sequences(ops, S, most, refused):  # noqa: F811
    """Chunks of 16 tokens of all sequences together stay below 2^31."""
    got = prefix(ops, S=S, T=S, ml=most, width=2**26, wb=0)
    assert (got == UNSUPPORTED) is refused
