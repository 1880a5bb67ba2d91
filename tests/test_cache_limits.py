"""CPU tests of the paged cache's limits: sizes that its arithmetic cannot hold
are refused before anything touches the device."""
import pytest

import test_cache_host as H
from hadamard_rotation_preprocessing_amd import _lib as L


@pytest.mark.parametrize("kw", [
    dict(new_rows=65536, max_pages=32768, bytes_=1 << 40),
    dict(rows=65536, max_pages=32768, bytes_=1 << 40),
    dict(new_rows=1 << 28, max_pages=8, bytes_=1 << 40),
])
def test_update_of_tables_that_are_not_counted_in_31_bits(kw):
    """As many pages as 2^31 could be asked for, and wrap to a negative place
    in the list of free pages."""
    H.refused(H.update(**kw), L.HR_EUNSUPPORTED, "below 2^31")


def test_compact_of_tables_that_are_not_counted_in_31_bits():
    H.refused(H.compact(rows=1 << 20, max_pages=2048, bytes_=1 << 40), L.HR_EUNSUPPORTED, "below 2^31")
