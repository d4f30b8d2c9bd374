"""Views of E4M3 rows, without a GPU."""
import pytest

import chunk_causal_wavefront_b200 as wfb


def test_first_rows_are_counted():
    q = wfb.E4M3Rows.empty(130, 96, "cpu")
    for n in (0, 1, 128, 130):
        assert q.first(n).shape == (n, 96)
    for n in (-1, 131):                       # not "all but the last", nor fewer rows than asked for
        with pytest.raises(ValueError, match="130 rows"):
            q.first(n)
