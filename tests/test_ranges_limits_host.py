"""Attention over ranges of keys at the limits of what it takes, without a GPU."""
import pytest

from test_ranges_host import NO, P, WS, made


@pytest.mark.parametrize("change, status", [
    (dict(documents=None, docs=-1, mask=None), WS), (dict(documents=None, docs=1 << 30, mask=None), WS),  # docs is ignored
    (dict(docs=(1 << 31) - 1), NO), (dict(docs=(1 << 29) + 1), NO), (dict(docs=1 << 29, n=100), WS),
])
def test_documents_of_a_mask(fa_lib, change, status):
    assert made(fa_lib, **change) == status
