"""Limits of the 4-bit window cache's arguments, on the CPU: calls that the library refuses beside the
nearest ones that it takes (of no sequences, so that nothing is launched)."""
import pytest

from test_kv4_oracle import cache, call_attention, hq  # noqa: F401  (hq: a fixture)

FLT_MAX = 3.4028234663852886e38


@pytest.mark.parametrize("cap,taken", [
    (0.0, True), (2.0 ** -20, True), (30.0, True), (2.0 ** 100, True), (2.0 ** 120, True),
    (2.0 ** 120 * 1.001, False), (2.0 ** 127, False), (FLT_MAX, False), (2.0 ** -20 * 0.999, False),
    (-0.0, True), (-1.0, False)])
def test_caps(hq, cap, taken):
    """cap log2(e) and 1 / cap have to be normal fp32 numbers: above 2.36e38 the first was infinite."""
    got = call_attention(hq, cache(hq, n_seqs=0), cap=cap)
    assert got == (hq.HQ_OK if taken else hq.HQ_ERR_INVALID)


@pytest.mark.parametrize("scale,taken", [
    (0.0, True), (0.1, True), (-2.0 ** 120, True), (2.0 ** 120, True), (2.0 ** 120 * 1.001, False),
    (2.0 ** 127, False), (-FLT_MAX, False), (FLT_MAX, False), (float("nan"), False)])
def test_scales(hq, scale, taken):
    """scale log2(e) has to be finite: above 2.36e38 every score was infinite or NaN."""
    got = call_attention(hq, cache(hq, n_seqs=0), scale=scale)
    assert got == (hq.HQ_OK if taken else hq.HQ_ERR_INVALID)
