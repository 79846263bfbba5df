"""A serving step's calls around the 4-bit window cache on the GPU at sizes, scores and values where
they reach their limits, against their reference (oracle/serving.py).  Bounds are those that
test_serving_gpu.py derives."""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

from oracle import kv4 as R
from oracle import serving as S
from test_kv4_gpu import DT, HALF_STEP, MASK, U, Cache, queries
from test_kv4_gpu import hq  # noqa: F401  (the fixture)
from test_kv4_scores_gpu import LN2, SCORES, fill, raw_score, unit_query
from test_serving_gpu import Pool, room, tree, trees

pytestmark = pytest.mark.gpu
HERE = os.path.dirname(os.path.abspath(__file__))


# ------------------------------------------------------------------ resize
def resize_there_and_back(hq, B):
    rng = np.random.default_rng(B)
    lens = [int(x) for x in rng.integers(0, 30, B)]
    have = sum(-(-n // 16) for n in lens)
    pool = Pool(hq, rng, B, 16, 5, have + B // 2, lens)
    granted = pool.step(hq, lens, [int(x) for x in rng.integers(0, 80, B)], 50 * B)
    pool.step(hq, granted, lens, 50 * B)


@pytest.mark.parametrize("B", [4010, 4011, 4096, 4097, 16384])
def test_resize_of_many_sequences_first(hq, B):
    """In a process of its own, whose first large resize it is: no call may need another before it."""
    code = ("import test_serving_range_gpu as t\nfrom weights_hq_encode_gb300 import hq\n"
            f"t.resize_there_and_back(hq, {B})\nt.resize_there_and_back(hq, 600)\n"
            f"t.resize_there_and_back(hq, {B})\n")
    path = os.pathsep.join([os.path.dirname(HERE), HERE, os.environ.get("PYTHONPATH", "")])
    got = subprocess.run([sys.executable, "-c", code], env=dict(os.environ, PYTHONPATH=path), cwd=HERE,
                         capture_output=True, text=True, timeout=300)
    assert got.returncode == 0, got.stderr[-2000:]


# ------------------------------------------------------------------ tree attention
def check(C, lens, parents, q, scale, cap, got, kind="f32", wide=False, least=0.0):
    """`wide`: the kernel of 128-row tiles ran, which rounds a weight once to fp16 for outputs of 16
    bits, by 2^-11 of it (and 2^-31 of the row's largest, which is not counted here).  `least`: what fp32 has no room for."""
    ref = S.tree(C.pages, C.table, lens, parents, q.double().cpu().numpy(), MASK, scale, cap)
    out, lse = (t.double().cpu().numpy() for t in got)
    steps = ((np.array(lens) + q.shape[1]) / 16)[:, None, None]
    score = 30 * U * ref["zeta"] + 566 * U * ref["zeta_codes"] + 8 * U * np.minimum(cap, 4 * ref["zeta"])
    tol = ((2 * score + (68 * steps + 100) * U) * np.linalg.norm(ref["size"], axis=-1) +
           1200 * U * np.sqrt(128.0) * ref["scales"]) + least
    if kind != "f32" and wide:
        tol += 2.0 ** -11 * np.linalg.norm(ref["size"], axis=-1)
    rounding = HALF_STEP[kind] * np.linalg.norm(ref["out"], axis=-1) * 1.01
    err = np.linalg.norm(out - ref["out"], axis=-1)
    assert (err <= tol + rounding).all(), (err / (tol + rounding + 1e-300)).max()
    empty = np.isneginf(ref["lse"])
    assert not out[empty].any() and np.array_equal(np.isneginf(lse), empty)
    d = np.abs(lse[~empty] - ref["lse"][~empty])
    assert (d <= (score + (2 * steps + 24) * U)[~empty] + 4 * U * np.abs(ref["lse"][~empty])).all()


def rows_for(C, k, v):
    """The same rows k, v [tokens][nh][128] for every sequence."""
    for b in range(len(C.lens)):
        R.append(C.pages, C.table, k.astype(np.float32), v.astype(np.float32), [b] * len(k), range(len(k)), MASK)
    C.upload()


@pytest.mark.parametrize("n,G", [(4, 4), (48, 4)])
@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("value,up", [(0.0, 200), (2.0 ** -60, 100)])
def test_tree_scores_of_rows_without_value(hq, n, G, out, value, up):
    """Values of zero, or of 2^-160 of those before, under scores far above all before them; values under scores
    a little below those.  (Weights below 2^-126 of the largest are none in fp32.)"""
    rng = np.random.default_rng(81)
    m, nh = 1500, 2
    C = Cache(hq, rng, [m + n] * 2, nh, 16, width=room(2, nh, n * G, 16, 98), empty=True)
    k, v = (rng.standard_normal((m + n, nh, 128)) for _ in range(2))
    d = rng.standard_normal(128)
    d /= np.linalg.norm(d)
    k[128:900] += up * d                         # from a block of 128 tokens on
    k[900:] += (up - 3) * d
    v[128:900] *= value
    v[:128] *= 2.0 ** 100 if value else 1.0
    rows_for(C, k, v)
    parents = trees(rng, 2, n, "random")
    q = torch.from_numpy((d + 0.02 * rng.standard_normal((2, n, nh * G, 128))).astype(np.float32)).cuda()
    for lens in ([m, m], [600, 700], [m, 850]):  # the last with no other value near the largest score
        got = tree(hq, C, lens, parents, q, 1.0, 0.0, DT[out])
        assert torch.isfinite(got[0]).all() and torch.isfinite(got[1]).all() and int(C.status) == 0
        check(C, lens, parents, q, 1.0, 0.0, got, out, wide=n * G > 32,
              least=1e-36 if value == 0 else 2.0 ** -126 * 2.0 ** 100 * 128 * 24)       # 128 rows of norm 24 at most


@pytest.mark.parametrize("n,G", [(4, 4), (48, 4)])
@pytest.mark.parametrize("value", [1.0, 2.0 ** 119, 2.0 ** -100])
def test_tree_keys_and_values_of_any_size(hq, n, G, value):
    """Keys up to 2^119 under small queries or scales, tiny ones under large ones: scores of a few units."""
    rng = np.random.default_rng(82)
    m, nh = 700, 2
    parents = trees(rng, 2, n, "random")
    for key, query, scale in ((118, -80, 2.0 ** -40), (119, -10, 2.0 ** -111), (114, -84, 2.0 ** -32), (-104, 90, 2.0 ** 12),
                              (-100, 40, 2.0 ** 58), (-100, 0, 2.0 ** 98)):
        C = Cache(hq, rng, [m + n] * 2, nh, 16, width=room(2, nh, n * G, 16, 47), empty=True)
        k, v = (rng.standard_normal((m + n, nh, 128)) for _ in range(2))
        rows_for(C, k * 2.0 ** key, v * value)
        q = queries(rng, 2, n, nh * G, "f32", size=1.0)
        q = (q.double() * 2.0 ** query).float()
        for cap in (0.0, 8.0):
            got = tree(hq, C, [m, 300], parents, q, scale, cap, torch.float32)
            check(C, [m, 300], parents, q, scale, cap, got)
            assert int(C.status) == 0


@pytest.mark.parametrize("n,G", [(4, 4), (48, 4)])
def test_tree_no_scale_over_large_keys(hq, n, G):
    """A scale of 0, or next to it, over keys of any size: equal weights."""
    rng = np.random.default_rng(84)
    m, nh = 500, 2
    parents = trees(rng, 2, n, "random")
    C = Cache(hq, rng, [m + n] * 2, nh, 16, width=room(2, nh, n * G, 16, 47), empty=True)
    k, v = (rng.standard_normal((m + n, nh, 128)) for _ in range(2))
    rows_for(C, k * 2.0 ** 119, v)
    q = queries(rng, 2, n, nh * G, "f32", size=1.0)
    for scale in (0.0, -0.0, 1e-45):
        check(C, [m, 300], parents, q, scale, 0.0, tree(hq, C, [m, 300], parents, q, scale, 0.0, torch.float32))
    assert int(C.status) == 0


@pytest.mark.parametrize("n,G", [(4, 4), (48, 4)])
@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("bits", [0x7FFF, 0xFFFF, 0x7F80, 0xFF80, 0xBF80, 0x7F7F, 0x0001, 0x0000])
def test_tree_behind_padding_holds_no_scales(hq, n, G, out, bits):
    """Drafts whose path leads to padding get no weight and give none, whatever lies in their places: NaN,
    infinities, negative, huge and tiny values for scales."""
    rng = np.random.default_rng(80)
    lens, nh = [300, 77], 2
    C = Cache(hq, rng, [m + n for m in lens], nh, 16, width=room(2, nh, n * G, 16, 22))
    parents = [[-1, -2, 1] + [0] * (n - 3), [-1] * (n - 2) + [-2, n - 2]]
    for b, j in ((0, 1), (0, 2), (1, n - 2), (1, n - 1)):
        t = lens[b] + j
        unit = C.pages[C.table[b, t // 16], :, 0]
        for at in (2048, 2080):
            unit[:, at + 2 * (t % 16):at + 2 * (t % 16) + 2] = (bits & 255, bits >> 8)
    C.upload()
    q = queries(rng, 2, n, nh * G, "f32")
    got = tree(hq, C, lens, parents, q, 0.1, 0.0, DT[out])
    assert int(C.status) == hq.HQ_ERR_PAGE
    check(C, lens, parents, q, 0.1, 0.0, got, out, wide=n * G > 32)


@pytest.mark.parametrize("n,G", [(4, 4), (48, 4)])
def test_tree_equal_and_lone_scores(hq, n, G):
    """Scores beyond 2^24, all equal or one far above the others: outputs are the means of V that they
    stand for, V's scales rising 2^20-fold along one sequence and falling along the other."""
    rng = np.random.default_rng(83)
    lens, nh = [1500, 300], 2
    full = [m + n for m in lens]
    C = Cache(hq, rng, full, nh, 16, width=room(2, nh, n * G, 16, 98), empty=True)
    q = unit_query()
    k = rng.standard_normal(128)
    k[5] = 3.0
    rise = [0.03 * 2.0 ** (20.0 * np.arange(m) / m) for m in full]
    rise[1] = rise[1][::-1]
    v = [rng.standard_normal((m, 128)) * r[:, None] for m, r in zip(full, rise)]
    dq = torch.from_numpy(np.broadcast_to(q, (2, n, nh * G, 128)).copy()).cuda()
    for lone in (None, 0, 700, 1100):
        rows = [np.broadcast_to(k, (m, 128)).copy() for m in full]
        if lone is not None:
            for b in range(2):
                rows[b][min(lone, lens[b] - 1)] *= 2.0
        fill(C, rows, v)
        raw = raw_score(C, 0, 1, q)
        for z in [3.0] + SCORES:
            if lone is not None and z < 1e4:
                continue
            got = tree(hq, C, lens, [[-1] * n] * 2, dq, z * LN2 / raw, 0.0, torch.float32)
            out = got[0].double().cpu().numpy()
            for b in range(2):
                V = R.back(R.rotated(C.pages, C.table, b, full[b], 1), MASK)
                size = np.abs(R.rotated(C.pages, C.table, b, full[b], 1))
                s = np.concatenate([R.raw_rows(C.pages, p, 1)[1] for p in C.table[b, :-(-full[b] // 16)]], 1)
                for j in range(n):
                    p = np.zeros(full[b])
                    if lone is None:
                        p[:lens[b]] = p[lens[b] + j] = 1.0 / (lens[b] + 1)
                    else:
                        p[min(lone, lens[b] - 1)] = 1.0
                    for h in range(nh):
                        tol = ((68 * full[b] / 16 + 100) * U * np.linalg.norm(p @ size[h]) +
                               1200 * U * np.sqrt(128.0) * (p @ s[h, :full[b]].astype(np.float64)))
                        err = np.linalg.norm(out[b, j, h * G:(h + 1) * G] - p @ V[h], axis=-1)
                        assert (err <= tol).all(), (lone, z, b, j, err.max() / tol)
    assert int(C.status) == 0


SIZES = [  # committed lengths, nh, G, drafts, page, cap, q type, out type
    ([300, 1, 64], 2, 8, 3, 48, 30.0, "bf16", "bf16"),                    # 24 rows a head
    ([130, 2, 77], 3, 4, 8, 32, 0.0, "f16", "f16"),                       # 32
    ([257, 31], 2, 5, 13, 64, 0.0, "f32", "f16"),                         # 65
    ([1100, 40, 0], 1, 4, 64, 64, 0.0, "f16", "bf16"),                    # 256
]


@pytest.mark.parametrize("case,wide", [(i, w) for i, c in enumerate(SIZES) for w in (False, True)
                                       if not w or c[2] * c[3] > 32])
def test_tree_weights_in_two_parts(hq, case, wide):
    """Outputs of 16 bits: the kernel of 16-row tiles rounds nothing but them."""
    lens, nh, G, n, page, cap, dq, do = SIZES[case]
    rng = np.random.default_rng(90 + case)
    parents = trees(rng, len(lens), n, "random")
    width = -(-(max(lens) + n) // page)
    C = Cache(hq, rng, [a + n for a in lens], nh, page,
              width=room(len(lens), nh, n * G, page, width) if wide else width)
    q = queries(rng, len(lens), n, nh * G, dq)
    got = tree(hq, C, lens, parents, q, 128 ** -0.5, cap, DT[do])
    assert int(C.status) == 0
    check(C, lens, parents, q, 128 ** -0.5, cap, got, do, wide=wide)
