"""The 4-bit window cache's attention at scores, queries, keys and caps of any size
against its reference (oracle/kv4.py).

A score beyond 2^24 (in log2 units) has no fraction left in fp32, and its own
error is large.  What must not depend on it: an output is a weighted mean of
rows of V.  Where all weights are known - one token, equal scores, equal rows of
V, one score far above the others - only the value side's error is left, as
tests/test_kv4_gpu.py derives it, in the norm of an output row (u = 2^-24, A =
sum p |V'| in the transformed domain, s V's scales, T tokens):
  |d out| <= (34 T / 16 + 100) u |A| + 600 u sqrt(128) sum p s.
Equal scores have to come out equal for that.  They do for a query whose
transform is +-1 in every coordinate: its fp16 parts are exact, so that every
token's score is one and the same chain of roundings."""
import numpy as np
import pytest
import torch

from oracle import kv4 as R
from test_kv4_gpu import MASK, U, Cache, attend, check, hq, queries  # noqa: F401  (hq: a fixture)

pytestmark = pytest.mark.gpu

LN2 = float(np.log(2.0))
SCORES = [1.7e7, -1.7e7, 5e7, 5e8, -5e8, 2.0 ** 60, 2.0 ** 100]     # in log2 units
ROWS = [3, 4, 8, 16]                             # query rows a head: blocks of 4, 8 and 16


def unit_query():
    """A query of one coordinate whose transform is exactly +-1 in fp32."""
    a = np.float32(np.sqrt(128.0))
    near = np.array([a, np.nextafter(a, np.float32(0)), np.nextafter(a, np.float32(99))], np.float32)
    exact = near[near * np.float32(0.08838834764831845) == 1]
    assert len(exact)
    q = np.zeros(128, np.float32)
    q[5] = exact[0]
    return q


def fill(C, k, v):
    """Sequence b of the cache gets K and V rows k[b], v[b] [tokens, 128] for every head."""
    for b in range(len(C.lens)):
        wide = [np.repeat(np.asarray(x[b], np.float32)[:, None], C.nh, 1) for x in (k, v)]
        R.append(C.pages, C.table, *wide, [b] * C.lens[b], range(C.lens[b]), MASK)
    C.upload()


def raw_score(C, b, t, q):
    """q . Khat of head 0 in 64 bits."""
    return float(R.back(R.rotated(C.pages, C.table, b, t + 1, 0), MASK)[0, t] @ q.astype(np.float64))


def value_bound(size, scales, T):
    return (34 * T / 16 + 100) * U * np.linalg.norm(size, axis=-1) + 600 * U * np.sqrt(128.0) * scales


def check_mean(C, got, weights):
    """Every output row of sequence b is the mean of the head's rows of V by weights[b]."""
    out = got[0].double().cpu().numpy()
    G = out.shape[2] // C.nh
    for b, n in enumerate(C.lens):
        V = R.rotated(C.pages, C.table, b, n, 1)
        s = np.concatenate([R.raw_rows(C.pages, p, 1)[1] for p in C.table[b, :-(-n // C.page)]], 1)[:, :n]
        p = weights[b]
        for h in range(C.nh):
            want = R.back(p @ V[h], MASK)
            tol = value_bound(p @ np.abs(V[h]), float(p @ s[h].astype(np.float64)), n)
            err = np.linalg.norm(out[b, :, h * G:(h + 1) * G] - want, axis=-1)
            assert (err <= tol).all(), (b, h, err.max() / tol)


def check_lse(got, want, zeta):
    """Scores' own errors, below 330 u of zeta = |scale| |q| max s (max(|c|, 7.5 sqrt(128)))."""
    d = np.abs(got[1].double().cpu().numpy() - want)
    assert (d <= 340 * U * (zeta + abs(want)) + 1e-5).all()


@pytest.mark.parametrize("G", ROWS)
@pytest.mark.parametrize("width", [1, 64])
def test_one_token_is_its_value(hq, G, width):
    """Blocks that end a row themselves, for a narrow table and for a wide one."""
    rng = np.random.default_rng(100 + G)
    sizes = [0.03, 0.5, 1.0, 2.0 ** 15]          # V's scales
    C = Cache(hq, rng, [1] * 4, 2, 16, width=width, empty=True)
    q = unit_query()
    k = rng.standard_normal((1, 128))
    k[0, 5] = 3.0                                # a score that is no small rest of its addends
    fill(C, [k] * 4, [2.6 * a * rng.standard_normal((1, 128)) for a in sizes])
    raw = raw_score(C, 0, 0, q)
    dq = torch.from_numpy(np.broadcast_to(q, (4, 1, 2 * G, 128)).copy()).cuda()
    for z in SCORES:
        for cap in (0.0, 4e8):
            got = attend(hq, C, dq, z * LN2 / raw, cap, torch.float32)
            check_mean(C, got, [np.ones(1)] * 4)
            want = z * LN2 if cap == 0 else cap * np.tanh(z * LN2 / cap)
            check_lse(got, want, 100.0 * abs(z))
    assert int(C.status) == 0


@pytest.mark.parametrize("G", ROWS)
@pytest.mark.parametrize("lens,width", [([600, 37], 38), ([700, 37], 44), ([700, 37], 200), ([3000, 1], 188)])
def test_equal_scores_give_the_mean(hq, G, lens, width):
    """All weights equal, beside V's scales that rise 2^20-fold along one sequence and fall along the
    other: in one block, and in several whose sums are joined."""
    rng = np.random.default_rng(200 + G)
    C = Cache(hq, rng, lens, 2, 16, width=width, empty=True)
    q = unit_query()
    k = rng.standard_normal(128)
    k[5] = 3.0
    rise = [0.03 * 2.0 ** (20.0 * np.arange(n) / n) for n in lens]
    rise[1] = rise[1][::-1]
    fill(C, [np.broadcast_to(k, (n, 128)) for n in lens],
         [rng.standard_normal((n, 128)) * r[:, None] for n, r in zip(lens, rise)])
    raw = raw_score(C, 0, 0, q)
    dq = torch.from_numpy(np.broadcast_to(q, (2, 1, 2 * G, 128)).copy()).cuda()
    for z in [3.0] + SCORES:
        got = attend(hq, C, dq, z * LN2 / raw, 0.0, torch.float32)
        check_mean(C, got, [np.full(n, 1.0 / n) for n in lens])


@pytest.mark.parametrize("G", ROWS)
def test_equal_values_are_the_output(hq, G):
    """Any weights at all: rows of V that are all the same are the output."""
    rng = np.random.default_rng(300 + G)
    lens = [700, 90]
    C = Cache(hq, rng, lens, 2, 16, width=50, empty=True)
    v = rng.standard_normal((2, 128))
    fill(C, [rng.standard_normal((n, 128)) for n in lens],
         [np.broadcast_to(v[b], (n, 128)) for b, n in enumerate(lens)])
    q = queries(rng, 2, 1, 2 * G, "f32")
    for scale in (1.0, 1e6, -1e7, 1e8):
        got = attend(hq, C, q, scale, 0.0, torch.float32)
        check_mean(C, got, [np.full(n, 1.0 / n) for n in lens])


@pytest.mark.parametrize("G", ROWS)
def test_one_score_far_above_the_others(hq, G):
    """Keys of one direction whose sizes fall by 5% a step: the first by far takes all the weight,
    wherever it lies, whatever the scales of V beside it."""
    rng = np.random.default_rng(400 + G)
    lens = [700, 333, 45]
    C = Cache(hq, rng, lens, 2, 16, width=60, empty=True)
    k = rng.standard_normal(128)
    k[5] = 3.0
    q = unit_query()
    rank = [np.minimum(rng.permutation(n), 100) for n in lens]
    v = [rng.standard_normal((n, 128)) * 2.0 ** rng.uniform(-15, 15, (n, 1)) for n in lens]
    fill(C, [k[None] * 1.05 ** -r[:, None] for r in rank], v)
    tops = [int(np.argmin(r)) for r in rank]
    sign = np.sign(raw_score(C, 0, tops[0], q))
    dq = torch.from_numpy(np.broadcast_to(q, (3, 1, 2 * G, 128)).copy()).cuda()
    raw = abs(raw_score(C, 0, tops[0], q))
    for z in (1.7e7, 5e7, 5e8, 2.0 ** 60, 2.0 ** 100):
        got = attend(hq, C, dq, sign * z * LN2 / raw, 0.0, torch.float32)
        check_mean(C, got, [np.eye(n)[t] for n, t in zip(lens, tops)])


@pytest.mark.parametrize("G", ROWS)
@pytest.mark.parametrize("lens,width", [([600, 90], 38), ([2000, 90], 130)])
def test_scores_that_climb(hq, G, lens, width):
    """Scores that go from far below to far above zero along the tokens, by steps below and above
    what starts a row anew: three equal ones at the end share the weight."""
    rng = np.random.default_rng(450 + G)
    C = Cache(hq, rng, lens, 2, 16, width=width, empty=True)
    k = rng.standard_normal(128)
    k[5] = 3.0
    q = unit_query()
    steps = np.array([-1.0, -2.0 ** -4, -2.0 ** -9, 2.0 ** -12, 2.0 ** -6, 2.0 ** -2, 2.0 ** -1])
    size = [steps[np.arange(n) * len(steps) // n] for n in lens]
    shares = []
    for a in size:
        a[[-1, -2, -40]] = 1.0
        shares.append((a == 1.0) / 3.0)
    fill(C, [k[None] * a[:, None] for a in size],
         [rng.standard_normal((n, 128)) * 2.0 ** rng.uniform(-15, 15, (n, 1)) for n in lens])
    raw = raw_score(C, 0, lens[0] - 1, q)
    dq = torch.from_numpy(np.broadcast_to(q, (2, 1, 2 * G, 128)).copy()).cuda()
    mass = torch.zeros((2, 2, C.width * 16), device="cuda")
    for z in (1e4, 1e6, 3e6, 1.7e7, 5e8, 2.0 ** 60, 2.0 ** 100):
        got = attend(hq, C, dq, z * LN2 / raw, 0.0, torch.float32, mass)
        check_mean(C, got, shares)
        M = got[2].double().cpu().numpy()
        for b, n in enumerate(lens):
            assert (np.abs(M[b, :, :n] - G * shares[b]) <= mass_bound(n, G) * G * shares[b]).all()


# ------------------------------------------------------------------ accumulated weights
# A weight is 2^((z - m) - log2 l) from the row's own m and l: 4 u for the power, 17 u for log2 l (below
# 16: a step of 16 u, and half of one for the difference, times ln 2), l's sum with its terms' powers
# (T / 16 + 24) u, and one rounded addition for each of a head's G rows.
def mass_bound(T, G):
    return (T / 16 + 50 + G) * U


@pytest.mark.parametrize("G", ROWS)
@pytest.mark.parametrize("lens,width", [([600, 37], 38), ([1, 16], 64), ([3000, 1], 188)])
def test_mass_of_equal_scores(hq, G, lens, width):
    """Every token of a row gets the same weight, whatever the scores; mass that was there stays."""
    rng = np.random.default_rng(500 + G)
    C = Cache(hq, rng, lens, 2, 16, width=width, empty=True)
    q = unit_query()
    k = rng.standard_normal(128)
    k[5] = 3.0
    fill(C, [np.broadcast_to(k, (n, 128)) for n in lens], [rng.standard_normal((n, 128)) for n in lens])
    raw = raw_score(C, 0, 0, q)
    dq = torch.from_numpy(np.broadcast_to(q, (2, 1, 2 * G, 128)).copy()).cuda()
    for mass in (torch.zeros((2, 2, C.width * 16), device="cuda"),
                 torch.rand((2, 2, C.width * 16), device="cuda")):
        for z in [3.0, 1e5, 3e6] + SCORES:
            M = attend(hq, C, dq, z * LN2 / raw, 0.0, torch.float32, mass)[2].double().cpu().numpy()
            before = mass.double().cpu().numpy()
            for b, n in enumerate(lens):
                want = before[b, :, :n] + G / n
                assert (np.abs(M[b, :, :n] - want) <= mass_bound(n, G) * G / n + U * want).all(), (z, b)


@pytest.mark.parametrize("G", ROWS)
def test_mass_of_any_scores_adds_up(hq, G):
    """A row's weights add up to 1: random scores up to some 10^8, and one far above the others."""
    rng = np.random.default_rng(600 + G)
    lens = [700, 90]
    C = Cache(hq, rng, lens, 2, 16, width=50)
    q = queries(rng, 2, 1, 2 * G, "f32")
    mass = torch.zeros((2, 2, C.width * 16), device="cuda")
    for scale in (0.1, 1.0, 1e3, 1e5, -1e6, 1e7):
        M = attend(hq, C, q, scale, 0.0, torch.float32, mass)[2].double().cpu().numpy()
        for b, n in enumerate(lens):
            assert (np.abs(M[b, :, :n].sum(-1) / G - 1) <= mass_bound(n, G)).all(), (scale, b)


# ------------------------------------------------------------------ sizes of operands and caps
@pytest.mark.parametrize("power", [-90, -40, 0, 40, 90])
def test_queries_and_keys_of_any_size(hq, power):
    """Queries 2^power large over keys 2^-power large, so that the scores are of ordinary size, under
    caps from 2^-20 to 2^120 and without one; the bound is that of tests/test_kv4_gpu.py."""
    rng = np.random.default_rng(700 + power)
    lens = [333, 20]
    C = Cache(hq, rng, lens, 2, 16, empty=True)
    fill(C, [rng.standard_normal((n, 128)) * 2.0 ** -power for n in lens],
         [rng.standard_normal((n, 128)) for n in lens])
    for G in (4, 6):
        q = queries(rng, 2, 1, 2 * G, "f32") * 2.0 ** power
        for cap in (0.0, 2.0 ** -20, 1.0, 30.0, 2.0 ** 20, 2.0 ** 60, 2.0 ** 100, 2.0 ** 120):
            check(C, q, 0.1, cap, attend(hq, C, q, 0.1, cap, torch.float32))


@pytest.mark.parametrize("G", ROWS)
def test_the_largest_scale(hq, G):
    """Large scales beside small queries: scores of ordinary size, and of some 10^10."""
    rng = np.random.default_rng(800 + G)
    C = Cache(hq, rng, [100, 7], 2, 16)
    q = queries(rng, 2, 1, 2 * G, "f32") * 2.0 ** -90
    for scale in (2.0 ** 86, 2.0 ** 120):
        got = attend(hq, C, q, scale, 0.0, torch.float32)
        if scale < 2.0 ** 100:
            check(C, q, scale, 0.0, got)
        for b, n in enumerate(C.lens):           # inside the hull of V's rows
            V = R.rotated(C.pages, C.table, b, n, 1)
            s = np.concatenate([R.raw_rows(C.pages, p, 1)[1] for p in C.table[b, :-(-n // 16)]], 1)[:, :n]
            hull = np.abs(R.back(V, MASK)).max()
            tol = value_bound(V, s, n).max()
            assert (got[0][b].double().abs() <= hull + tol).all()     # NaN fails as well


# ------------------------------------------------------------------ size of the error
# A score is 8 steps of the tensor cores over centred codes: 16 products, each of at most 17/16 |q'| |c - 7.5|,
# and the sum so far.  A step may cut each of the 17 addends by 2 u of the largest, and no partial sum is
# beyond |q'| |c - 7.5|: with 30 u for the query's transform and parts, the multipliers and the scale,
#   |dz| <= (30 + 8 x 34 x 17/16) u zeta <= 320 u zeta,   zeta = |scale| |q| max |Khat|,
# where tests/test_kv4_gpu.py still counts uncentred codes (30 u zeta + 294 u zeta_codes, some 3 times as much).
# These are worst cases; a loss of precision shows earlier in all rows together.  With scores of rms 1 the
# largest addend is about the partial sum, below the score itself, so a step's 17 cuts are
# sqrt(17) 2 u / sqrt(3) = 4.8 u and 8 steps 14 u; they are independent from token to token, so that an
# output's norm is off by 14 u.  The value side adds T / 64 steps of 4.8 u a warp to a sum
# that grows to the output's size, below 14 u for T = 500.
# sqrt(14^2 + 14^2) u = 20 u is the limit; as every largest addend is counted at the full score, a kernel of
# centred codes stays below it (5 to 10 u), one of uncentred codes, whose partial sums are 7.5 |sum q'| and
# more, does not (33 to 43 u).
@pytest.mark.parametrize("G", ROWS)
def test_errors_of_all_rows_together(hq, G):
    rng = np.random.default_rng(900 + G)
    lens = [500, 467]
    C = Cache(hq, rng, lens, 2, 16, empty=True)
    fill(C, *[[rng.standard_normal((n, 128)) for n in lens] for _ in range(2)])
    q = queries(rng, 2, 1, 2 * G, "f32", size=1.0)
    scale = 128 ** -0.5
    out, lse, _ = attend(hq, C, q, scale, 0.0, torch.float32)
    ref = R.attention(C.pages, C.table, lens, q.double().cpu().numpy(), MASK, scale)
    err = np.linalg.norm(out.double().cpu().numpy() - ref["out"], axis=-1)
    score = 320 * U * ref["zeta"]
    bound = ((2 * score + (34 * max(lens) / 16 + 100) * U) * np.linalg.norm(ref["size"], axis=-1) +
             600 * U * np.sqrt(128.0) * ref["scales"])
    assert (err <= bound).all()
    assert (np.abs(lse.double().cpu().numpy() - ref["lse"]) <= score + (max(lens) / 16 + 50) * U).all()
    assert np.linalg.norm(err) <= 20 * U * np.linalg.norm(ref["out"])
