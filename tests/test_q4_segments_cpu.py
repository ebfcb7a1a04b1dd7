"""The automatic number of key segments of paged_attention_q4, read from its workspace's size."""
import pytest

from paged_attention_int8_gb300 import _lib, build as pkg_build


@pytest.fixture(scope="module", autouse=True)
def lib():
    pkg_build.build()
    return _lib.load()


def _segments(seqs, hq, hk, d, max_query_len, max_seq_len):
    size = _lib.paged_attention_q4_workspace_size(seqs, seqs, hq, hk, d, max_query_len, max_seq_len)
    return 1 if size == 256 else (size - 256) // (seqs * hq * (d + 2) * 4)


# thread blocks an SM: each has four rings of 16-key blocks (20 D bytes) beside 1 KB of the 228 KB
@pytest.mark.parametrize("d,stages,by_registers", [(128, 6, 3), (256, 4, 2)])
@pytest.mark.parametrize("hq,hk", [(32, 8), (4, 1), (48, 6)])
def test_one_long_sequence_is_one_round(d, stages, by_registers, hq, hk):
    places = 152 * min(by_registers, 228 * 1024 // (4 * stages * 20 * d + 1024))
    assert places == {128: 456, 256: 304}[d]
    # (64 segments at most)
    assert _segments(1, hq, hk, d, 1, 131072) == min(64, places // hk)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("seqs", [1, 3, 20, 500])
def test_short_sequences_stay_whole(d, seqs):
    assert _segments(seqs, 32, 8, d, 1, 256) == 1
    assert _segments(seqs, 32, 8, d, 1, 1) == 1
