"""PagedKVCache without a GPU: what it holds cannot be exchanged under its packed descriptor."""
from __future__ import annotations

import pytest

import packed_varlen_rope_gb300 as pr


@pytest.mark.parametrize("name", ["k_pages", "v_pages"])
def test_pages_cannot_be_reassigned(name):
    """The descriptor holds the pages' addresses: a cache whose pages were exchanged would go on
    writing to the old ones, which nothing keeps alive any more."""
    cache = object.__new__(pr.PagedKVCache)
    with pytest.raises(AttributeError):
        setattr(cache, name, None)
