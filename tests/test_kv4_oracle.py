"""The 4-bit window cache without a GPU: pins of its numpy reference
(oracle/kv4.py) against the definition in 64 bits, and the calls that the
library refuses before it launches anything (their pointers are never read)."""
import ctypes

import numpy as np
import pytest

from oracle import kv4 as R

MASK = [0x12345678, 0xDEADBEEF, 0x00FF00FF, 0x80000001]


def hadamard():
    i = np.arange(128)
    par = np.array([[bin(a & b).count("1") & 1 for b in i] for a in i])
    return (1.0 - 2.0 * par) / np.sqrt(128.0)


def test_transform_is_the_orthonormal_hadamard():
    H = hadamard()
    assert np.allclose(H @ H.T, np.eye(128), atol=1e-12)
    x = np.random.default_rng(0).standard_normal((5, 128))
    assert np.allclose(R.fwht(x) / np.sqrt(128.0), x @ H, atol=1e-12)


def test_codes_are_those_of_the_definition():
    """Codes by the fp32 steps and by the definition in 64 bits differ only where y / s is
    within the fp32 error of a border: 7 rounded stages, the scale's products and the
    quotient, below 16 u of |y| / s <= 7.6 of a step, u = 2^-24."""
    x = np.random.default_rng(1).standard_t(4, (400, 128)).astype(np.float32)
    c, s, bad = R.quantize(x, MASK)
    assert not bad.any()
    y = (x.astype(np.float64) * R.signs_of(MASK)) @ hadamard()
    t = y / s[:, None].astype(np.float64) + 8.0
    assert np.abs(np.abs(y).max(-1) / 7.5 / s - 1).max() <= 2.0 ** -8    # bf16: half a step
    want = np.clip(np.floor(t), 0, 15)
    far = np.abs(t - np.round(t)) > 64 * 8 * 2.0 ** -24
    assert (c == want)[far].all() and far.mean() > 0.999
    # an element is off by at most half a step, and by one bf16 rounding of the scale at the rim
    assert np.abs((c - 7.5) * s[:, None] - y).max(-1).max() <= (0.5 + 8 * 2.0 ** -8) * s.max()


def test_pages_hold_what_was_put_and_attention_is_softmax():
    rng = np.random.default_rng(2)
    nh, P = 2, 32
    pages = R.new_pages(4, nh, P, fill=0xA5)
    table = np.array([[2, 0]])
    n = 45
    k, v = (rng.standard_normal((n, nh, 128)).astype(np.float32) for _ in range(2))
    assert R.append(pages, table, k, v, [0] * n, range(n), MASK) == (False, False)
    assert (pages[1] == 0xA5).all() and (pages[3] == 0xA5).all()
    vals = [R.back(R.rotated(pages, table, 0, n, w), MASK) for w in (0, 1)]
    for x, got in zip((k, v), vals):
        c, s, _ = R.quantize(x, MASK)
        want = ((c - 7.5) * s[..., None].astype(np.float64)) @ hadamard() * R.signs_of(MASK)
        assert np.allclose(got, want.transpose(1, 0, 2), atol=1e-12)
        # 16 levels over +-max: the rows come back to about 1/10 of their size
        assert np.linalg.norm(got - x.transpose(1, 0, 2)) < 0.15 * np.linalg.norm(x)
        r = R.read32(pages, 2, 1, 7, 0 if x is k else 1, MASK)
        assert np.abs(r - want[7, 1]).max() <= 16 * 2.0 ** -24 * np.linalg.norm(want[7, 1])
    q = rng.standard_normal((1, 2, 4, 128))
    a = R.attention(pages, table, [n], q, MASK, 0.1, cap=5.0)
    for j in range(2):
        m = n - 1 + j
        for hq in range(4):
            z = 5.0 * np.tanh(vals[0][hq // 2, :m] @ q[0, j, hq] * 0.1 / 5.0)
            p = np.exp(z) / np.exp(z).sum()
            assert np.allclose(a["out"][0, j, hq], p @ vals[1][hq // 2, :m], atol=1e-10)
            assert np.isclose(a["lse"][0, j, hq], np.log(np.exp(z).sum()))
    assert np.isclose(a["added"].sum(), 8.0)
    assert R.append(pages, table, k[:1], v[:1], [0], [64], MASK) == (False, True)
    k[0, 0, 3] = np.inf
    assert R.append(pages, table, k[:1], v[:1], [0], [5], MASK) == (True, False)


def test_keep():
    m = np.array([3.0, 1.0, 2.0, 2.0, np.nan, 2.0, 9.0, 0.0])
    assert R.keep(m, 8, 8, 2).tolist() == list(range(8))
    assert R.keep(m, 8, 4, 1).tolist() == [0, 2, 6, 7]
    assert R.keep(m, 8, 4, 4).tolist() == [4, 5, 6, 7]
    assert R.keep(m, 7, 6, 0).tolist() == [0, 1, 2, 3, 5, 6]


# ------------------------------------------------------------------ refusals
@pytest.fixture(scope="module")
def hq():
    from weights_hq_encode_gb300 import build
    build.build()
    from weights_hq_encode_gb300 import hq as H
    return H


FAKE = 1 << 20                                   # an address that is never read


def cache(hq, **kw):
    c = dict(d_pages=FAKE, n_pages=8, page_tokens=32, n_kv_heads=2, d_table=FAKE, n_seqs=3,
             table_width=4, d_signs=FAKE)
    c.update(kw)
    return hq.hq_kv4_cache(*[c[n] for n, _ in hq.hq_kv4_cache._fields_])


BAD_CACHES = [dict(page_tokens=24), dict(page_tokens=0), dict(page_tokens=-16), dict(n_kv_heads=0),
              dict(n_pages=-1), dict(n_pages=0), dict(n_pages=1 << 28), dict(n_seqs=-1), dict(n_seqs=70000), dict(table_width=-1),
              dict(table_width=1 << 26), dict(d_pages=None), dict(d_pages=FAKE + 8),
              dict(d_table=None), dict(d_signs=None), dict(d_table=FAKE + 2)]


def call_rows(hq, name, c, **kw):
    a = dict(k=FAKE, v=FAKE, kind=0, st=(256, 128, 256, 128), seq=FAKE, pos=FAKE, n=3, status=FAKE)
    a.update(kw)
    L = hq.lib()
    c = None if c is None else ctypes.byref(c)
    if name == "append":
        return L.hq_kv4_append(c, a["k"], a["v"], a["kind"], *a["st"], a["seq"], a["pos"], a["n"],
                               a["status"], None)
    return L.hq_kv4_read(c, a["seq"], a["pos"], a["n"], a["k"], a["v"], a["kind"], *a["st"],
                         a["status"], None)


@pytest.mark.parametrize("name", ["append", "read"])
def test_rows_refusals(hq, name):
    for bad in BAD_CACHES:
        assert call_rows(hq, name, cache(hq, **bad)) == hq.HQ_ERR_INVALID, bad
    assert call_rows(hq, name, None) == hq.HQ_ERR_INVALID
    for bad in (dict(k=None), dict(v=None), dict(seq=None), dict(pos=None), dict(status=None),
                dict(kind=3), dict(kind=-1), dict(n=-1), dict(n=1 << 40), dict(k=FAKE + 1),
                dict(kind=1, v=FAKE + 2)):
        assert call_rows(hq, name, cache(hq), **bad) == hq.HQ_ERR_INVALID, bad
    assert call_rows(hq, name, cache(hq), n=0) == hq.HQ_OK


def call_attention(hq, c, **kw):
    a = dict(lengths=FAKE, q=FAKE, q_kind=0, st=(512, 512, 128), q_len=1, Hq=4, scale=0.1, cap=0.0,
             out=FAKE, out_kind=0, lse=None, mass_in=None, mass_out=None, ws=FAKE, ws_bytes=1 << 30,
             status=FAKE)
    a.update(kw)
    return hq.lib().hq_kv4_attention(
        None if c is None else ctypes.byref(c), a["lengths"], a["q"], a["q_kind"], *a["st"],
        a["q_len"], a["Hq"], a["scale"], a["cap"], a["out"], a["out_kind"], a["lse"], a["mass_in"],
        a["mass_out"], a["ws"], a["ws_bytes"], a["status"], None)


def test_attention_refusals(hq):
    for bad in BAD_CACHES:
        assert call_attention(hq, cache(hq, **bad)) == hq.HQ_ERR_INVALID, bad
    for bad in (dict(lengths=None), dict(q=None), dict(out=None), dict(ws=None), dict(status=None),
                dict(q_kind=7), dict(out_kind=7), dict(q_len=0), dict(q_len=1 << 17), dict(Hq=0),
                dict(Hq=3), dict(scale=float("nan")), dict(scale=float("inf")), dict(cap=-1.0), dict(cap=1e-7),
                dict(cap=float("inf")), dict(mass_in=FAKE), dict(ws_bytes=0), dict(ws=FAKE + 16),
                dict(out=FAKE + 4), dict(q=FAKE + 1), dict(lse=FAKE + 2), dict(mass_out=FAKE + 1)):
        assert call_attention(hq, cache(hq), **bad) == hq.HQ_ERR_INVALID, bad
    assert call_attention(hq, cache(hq, n_seqs=0)) == hq.HQ_OK
    need = hq.lib().hq_kv4_attention_workspace_bytes
    plain, mass = (need(ctypes.byref(cache(hq)), 2, 4, m) for m in (0, 1))
    # the scores of every row and position are kept when the mass is wanted
    assert mass >= plain + 3 * 2 * 4 * 128 * 4
    assert call_attention(hq, cache(hq), mass_out=FAKE, ws_bytes=plain) == hq.HQ_ERR_INVALID
    assert need(ctypes.byref(cache(hq)), 2, 3, 0) == 0 and need(ctypes.byref(cache(hq)), 0, 4, 0) == 0


def call_evict(hq, src, dst, **kw):
    a = dict(lengths=FAKE, mass=FAKE, budget=64, recent=8, kept=FAKE + 4096,
             new_lengths=FAKE + 8192, new_mass=FAKE + 12288, status=FAKE)
    a.update(kw)
    return hq.lib().hq_kv4_evict(ctypes.byref(src), a["lengths"], a["mass"], ctypes.byref(dst),
                                 a["budget"], a["recent"], a["kept"], a["new_lengths"],
                                 a["new_mass"], a["status"], None)


def test_evict_refusals(hq):
    other = dict(d_table=FAKE + 4096)
    for bad in BAD_CACHES:
        assert call_evict(hq, cache(hq, **bad), cache(hq, **other)) == hq.HQ_ERR_INVALID, bad
        assert call_evict(hq, cache(hq), cache(hq, **{**other, **bad})) == hq.HQ_ERR_INVALID, bad
    for bad in (dict(lengths=None), dict(mass=None), dict(kept=None), dict(new_lengths=None),
                dict(new_mass=None), dict(status=None), dict(budget=0), dict(budget=-1),
                dict(recent=-1), dict(recent=65), dict(mass=FAKE + 2), dict(kept=FAKE + 1),
                dict(budget=(1 << 30) + 1), dict(budget=0x7FFFFFFF), dict(new_lengths=FAKE),
                dict(new_mass=FAKE)):                     # in place of an input
        assert call_evict(hq, cache(hq), cache(hq, **other), **bad) == hq.HQ_ERR_INVALID, bad
    for dst in (dict(n_seqs=2), dict(n_kv_heads=1), dict(table_width=1)):
        assert call_evict(hq, cache(hq), cache(hq, **{**other, **dst})) == hq.HQ_ERR_INVALID, dst
    assert call_evict(hq, cache(hq), cache(hq)) == hq.HQ_ERR_INVALID      # its own pages
    assert call_evict(hq, cache(hq, n_seqs=0), cache(hq, n_seqs=0)) == hq.HQ_OK


def test_header_symbols_layout_and_sizes(hq):
    import os
    import re
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    src = re.sub(r"/\*.*?\*/", "", open(os.path.join(root, "include", "hq_kv4.h")).read(), flags=re.S)
    names = set(re.findall(r"\b(hq_kv4_[a-z0-9_]+)\s*\(", src))
    assert names == {n for n in hq.EXPORTED if n.startswith("hq_kv4_")}
    for n in names:
        assert hasattr(hq.lib(), n)
    assert ctypes.sizeof(hq.hq_kv4_cache) == 48 and hq.hq_kv4_cache.d_table.offset == 24
    assert hq.hq_kv4_page_bytes(8, 16) == 8 * 2112 and hq.hq_kv4_page_bytes(1, 24) == 0
    assert hq.hq_kv4_page_bytes(0, 16) == 0 and hq.hq_kv4_page_bytes(3, 64) == 12 * 2112
    assert hq.hq_status_string(hq.HQ_ERR_PAGE) != hq.hq_status_string(3)


def test_binding_refuses_what_does_not_fit(hq):
    import torch
    with pytest.raises(ValueError):                      # not on a CUDA device
        hq.make_kv4_cache(torch.zeros(2112, dtype=torch.uint8), torch.zeros((1, 1), dtype=torch.int32),
                          16, 1, torch.zeros(4, dtype=torch.int32))
    with pytest.raises(ValueError):
        hq.make_kv4_cache(torch.zeros(2112, dtype=torch.uint8), torch.zeros((1, 1), dtype=torch.int32),
                          24, 1, torch.zeros(4, dtype=torch.int32))
    with pytest.raises(ValueError):                      # 16 once cut to 32 bits
        hq.make_kv4_cache(torch.zeros(2112, dtype=torch.uint8), torch.zeros((1, 1), dtype=torch.int32),
                          (1 << 32) + 16, 1, torch.zeros(4, dtype=torch.int32))
    with pytest.raises(ValueError):
        hq.hq_kv4_page_bytes(1 << 32 | 1, 16)
    with pytest.raises(TypeError):
        hq.make_kv4_cache(torch.zeros(2112), torch.zeros((1, 1), dtype=torch.int32), 16, 1,
                          torch.zeros(4, dtype=torch.int32))
