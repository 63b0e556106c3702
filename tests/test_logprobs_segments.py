"""Segments that rows of logits are cut into, by the workspace that a call
asks for: none of them is empty, however a row lies in memory."""
import pytest

CELL = 12           # a segment's maximum and two sums
UNIT = 8192         # values of a step of a workgroup
MOST = 64           # segments of a row


def _segments(L, tokens, vocab, top):
    need = L.fp8w_logprobs_workspace_bytes(tokens, vocab, top)
    cell = CELL + 8 * top
    assert need % (tokens * cell) == 0
    return max(need // (tokens * cell), 1)


@pytest.fixture(scope="module")
def L():
    import fp8_block_scaled_02_amd as F
    return F.lib()


@pytest.mark.parametrize("tokens", [1, 3, 4, 30, 100, 511, 512, 1023, 1024, 5000])
@pytest.mark.parametrize("top", [0, 5, 64])
def test_no_segment_is_empty(L, tokens, top):
    """The last segment starts before the row's last value."""
    for vocab in [UNIT * u + d for u in (1, 2, 4, 8, 16, 17, 64, 65, 128, 129, 1000) for d in (-8, -7, -1, 0, 1, 7, 8)]:
        segs = _segments(L, tokens, vocab, top)
        units = -(-vocab // UNIT)
        assert 1 <= segs <= min(units, MOST), (vocab, segs)
        per = -(-units // segs)
        assert (segs - 1) * per * UNIT < vocab, (vocab, segs)


def test_segments_of_few_rows(L):
    assert _segments(L, 3, 65536, 5) == 8 and _segments(L, 3, 65537, 5) == 9
    assert _segments(L, 4, 131072, 20) == 16 and _segments(L, 4, 8192, 20) == 1
