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


@pytest.mark.parametrize("call", [
    lambda: H.append(k=H.POOL - (1 << 30), kst=1 << 36, tokens=1 << 30),          # 2^67 bytes of k
    lambda: H.append(v=H.POOL - (1 << 30), vst=1 << 40, tokens=1 << 30),
    lambda: H.append(pool=H.P - (1 << 40), n_pages=1 << 30, spec=H.cspec(heads=1 << 16, d=256, page=256, g=32, sd=L.HR_F32),
                     kst=1 << 24, ksh=256, vst=1 << 24, vsh=256),                     # 2^63 bytes of pages, through k
    lambda: H.attention(out=H.Q - (1 << 20), ost=1 << 36, osh=128, tokens=1 << 24),
    lambda: H.update(layers=1 << 20, n_pages=1 << 30, bytes_=1 << 40),            # 2^66 bytes of pages
    lambda: H.compact(layers=1 << 20, n_pages=1 << 30, bytes_=1 << 40),
    lambda: H.compact(layers=1 << 20, into=H.X1, into_pages=1 << 30, pool=H.X1 - (1 << 30), bytes_=1 << 40),
])
def test_sizes_beyond_63_bits_still_overlap(call):
    """Sizes whose product does not fit 63 bits are held at the largest, not
    wrapped: the overlap that they make is found."""
    H.refused(call(), L.HR_EINVAL, "overlaps")

