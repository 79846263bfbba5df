"""The 4-bit window cache on the GPU against its reference (oracle/kv4.py).

Pages, codes, scales and kept positions are compared exactly; rows read as
fp32 are bit-identical to the reference's fp32 steps, and as bf16 or fp16 to
their rounding.

Tolerance of the attention, to first order in u = 2^-24.  The rotated query
q' = H D q / sqrt(128) takes 9 roundings (9 u of |q|); its two fp16 parts miss
it by 2^-22 |q'_i| + 2^-36 of the row's largest value (4 u), the codes c are
exact.  A score is summed in 8 steps of the tensor cores from the start -7.5
sum q'.  A step adds 16 products and the sum so far; its adder may align the 17
addends to the largest and cut what falls below, 2 u of the largest for each:
34 u a step.  No product and no partial sum exceeds |q'| s_t |c_t| in norm,
|c_t| = max(norm of a row's codes, 7.5 sqrt(128)), so 8 x 34 u of that, 18 u for
the start and the pairing of dimensions, and 4 u for the products with the
scales: |dz| <= 30 u zeta + 294 u zeta_c, zeta = |scale| |q| max |Khat_t|,
zeta_c = |scale| |q| max s_t |c_t|, plus 8 u min(cap, 4 zeta) for the capped form:
tanh(y) is off by at most 8 u (e^2|y| by 4 u and 2 |y| u, of which less than half
arrives, a quotient by 4 u, a sum and a difference by u each), and below |y| = 1/4,
where a series takes over, by 6 u for its rest and u for each of 4 roundings of y.  exp2 is off
by 4 u, so the softmax's weights are off by 2 |dz| + 12 u and their sum by u
for each of at most T / 16 + 20 additions on a thread and across threads.  The value
side splits the weights into two fp16 parts (4 u) and adds centred codes: an
even dimension's c - 7.5, and c_e - 7.5 + 16 (c_o - 7.5) for an odd one, which
is a sixteenth of the difference of the two.  A step adds 16 products and the
sum so far, 34 u of the largest; over the at most T / 16 steps of a warp that
is 34 u sum_t p_t s_t x 7.5 for every dimension if each step's largest addend is
a product of its own tokens, and 34 u T / 16 of the row's sum if it is the sum so
far, at most A = sum_t p_t |y_t| (V in the transformed domain).  With more than 4
rows a head the low parts are steps of their own into the same sum, with products
2^-11 of the others: a warp has n <= 2 ceil(T / 128) units, so 2 n - 1 <= T / 32 + 3 steps
that meet a sum, no more than the T / 16 counted from T = 96 on.  Below, 3 steps
are 102 u: with the 31 u that the 100 below leave, at most 35 u |A| more than
counted (T = 17; up to 16 tokens it is one step), and as |A| <= 7.5 sqrt(128)
sum p s, 263 u sqrt(128) sum p s of the 345 u that the 600 below leave beside the 255
of the products.  With 60 u for the
joining of the parts and the transform back (9 u), in the norm of an output row:
  |d out| <= (2 |dz| + (34 T / 16 + 100) u) |A| + 600 u sqrt(128) sum_t p_t s_t
plus half a step of the output's type, element by element.

These are worst cases.  The roundings are independent, so the error is of the
order of their root: of the 8 x 17 cuts of a score sqrt(136) x 2 u / sqrt(3), of
addends that are 16 of a row's codes times |q'| / sqrt(128) and less.  With |q| of
17, scales s_t near 1/2 and scale 0.1, as in most cases here, that is below 10^-5
for a score, and so for a weight and an output row in fp32; `check` holds all
rows together to twice that where its caller says that the case is such a one."""
import numpy as np
import pytest
import torch

from oracle import kv4 as R

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
MASK = [0x12345678, 0xDEADBEEF, 0x00FF00FF, 0x80000001]
DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
HALF_STEP = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11, "f32": U}


@pytest.fixture(scope="module")
def hq():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from weights_hq_encode_gb300 import build
    build.build()
    from weights_hq_encode_gb300 import hq as H
    return H


class Cache:
    """Pages in use on both sides, with every sequence's table in a random order."""

    def __init__(self, hq, rng, lens, nh, page, width=None, fill=0xFF, empty=False):
        self.hq, self.nh, self.page, self.lens = hq, nh, page, list(lens)
        self.width = max(1, -(-max(lens) // page)) if width is None else width
        n = len(lens) * self.width
        self.pages = R.new_pages(n + 3, nh, page, fill)      # 0xFF: NaN scales where nothing is
        self.table = rng.permutation(n + 3)[:n].reshape(len(lens), self.width).astype(np.int32)
        if not empty:
            for b, m in enumerate(lens):
                k, v = (rng.standard_normal((m, nh, 128)) * np.exp(0.5 * rng.standard_normal((m, nh, 1)))
                        for _ in range(2))
                R.append(self.pages, self.table, k.astype(np.float32), v.astype(np.float32),
                         [b] * m, range(m), MASK)
        self.upload()

    def upload(self):
        hq = self.hq
        self.d_pages = torch.from_numpy(self.pages.copy()).cuda()
        self.d_table = torch.from_numpy(self.table.copy()).cuda()
        self.d_lens = torch.tensor(self.lens, dtype=torch.int32).cuda()
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.c = hq.make_kv4_cache(self.d_pages, self.d_table, self.page, self.nh,
                                   hq.signs_tensor([MASK]).flatten())

    def same_pages(self):
        torch.cuda.synchronize()
        return np.array_equal(self.d_pages.cpu().numpy(), self.pages)


def ints(x):
    return torch.tensor(list(x), dtype=torch.int32).cuda()


def rows(rng, n, nh, dtype, layout):
    """K and V rows [n, nh, 128] of a layout, and their fp32 values."""
    x = rng.standard_normal((2, n, nh, 128)) * np.exp(rng.standard_normal((2, 1, nh, 128)))
    t = torch.from_numpy(x.astype(np.float32)).to(DT[dtype]).cuda()
    if layout == "fused":                        # slices of a projection's rows
        buf = torch.zeros((n, 3 * nh + 1, 128), dtype=DT[dtype], device="cuda")
        k, v = buf[:, nh:2 * nh], buf[:, 2 * nh + 1:]
    elif layout == "heads":                      # head-major slabs
        k, v = (torch.zeros((nh, n, 128), dtype=DT[dtype], device="cuda").transpose(0, 1)
                for _ in range(2))
    elif layout == "odd":                        # rows that start off 16-byte boundaries
        buf = torch.zeros(2 * n * nh * 131 + 3, dtype=DT[dtype], device="cuda")
        k, v = (buf[1 + i * n * nh * 131:].as_strided((n, nh, 128), (nh * 131, 131, 1))
                for i in range(2))
    else:
        k, v = (torch.zeros((n, nh, 128), dtype=DT[dtype], device="cuda") for _ in range(2))
    k.copy_(t[0])
    v.copy_(t[1])
    return k, v, t[0].float().cpu().numpy(), t[1].float().cpu().numpy()


# ------------------------------------------------------------------ append and read
@pytest.mark.parametrize("dtype,layout,nh,page,n", [
    ("bf16", "plain", 8, 16, 1), ("bf16", "fused", 3, 48, 100), ("f16", "heads", 2, 64, 77),
    ("f32", "odd", 1, 32, 65), ("bf16", "odd", 2, 16, 33), ("f32", "fused", 5, 128, 50)])
def test_append_bytes(hq, dtype, layout, nh, page, n):
    rng = np.random.default_rng(n)
    C = Cache(hq, rng, [n + 9, 40], nh, page, fill=0x5A, empty=True)
    k, v, kx, vx = rows(rng, n, nh, dtype, layout)
    seq = np.where(np.arange(n) % 7 == 3, -1, np.arange(n) % 2 * (np.arange(n) // 2 < 40))
    pos = np.where(seq == 1, np.arange(n) // 2, np.arange(n) + 9)
    assert R.append(C.pages, C.table, kx, vx, seq, pos, MASK) == (False, False)
    assert hq.hq_kv4_append(C.c, k, v, ints(seq), ints(pos), C.status) == hq.HQ_OK
    assert C.same_pages() and int(C.status) == 0


def test_append_special_rows_and_places(hq):
    """Zeros, tiny, huge and non-finite rows; sequences, positions and pages outside their range
    are left out and reported."""
    rng = np.random.default_rng(3)
    nh, page, n = 2, 16, 24
    C = Cache(hq, rng, [40, 20], nh, page, fill=0x11, empty=True)
    k, v, kx, vx = rows(rng, n, nh, "f32", "plain")
    for i, val in ((0, 0.0), (1, 1e-38), (2, 1e-36), (3, np.inf), (4, np.nan), (5, 3e38), (6, 2e36),
                   (7, 1e-45)):
        kx[i] = val
    kx[8, 0, 5] = np.nan
    k.copy_(torch.from_numpy(kx))
    seq, pos = np.array([0] * n), np.arange(n)
    C.table[0, 1] = C.pages.shape[0]             # positions 16 .. 31 of sequence 0 have no page
    seq[12], pos[13], pos[14], seq[15] = 2, -1, 48, -5
    C.upload()
    assert R.append(C.pages, C.table, kx, vx, seq, pos, MASK) == (True, True)
    assert hq.hq_kv4_append(C.c, k, v, ints(seq), ints(pos), C.status) == hq.HQ_OK
    assert C.same_pages() and int(C.status) == hq.HQ_ERR_RANGE | hq.HQ_ERR_PAGE
    assert hq.hq_kv4_append(C.c, k[:0], v[:0], ints([]), ints([]), C.status) == hq.HQ_OK


@pytest.mark.parametrize("dtype,layout,nh,page,n", [
    ("f32", "plain", 2, 16, 60), ("bf16", "heads", 3, 48, 50), ("f16", "fused", 1, 32, 1),
    ("bf16", "odd", 2, 64, 33), ("f32", "odd", 1, 16, 17)])
def test_read_bits(hq, dtype, layout, nh, page, n):
    rng = np.random.default_rng(n + 1)
    C = Cache(hq, rng, [n, 30], nh, page)
    seq = np.where(np.arange(n) % 5 == 1, 1, 0)
    pos = np.where(seq == 1, np.arange(n) % 30, rng.permutation(n))
    seq[n // 2] = -1                             # a padding token
    k, v, _, _ = rows(rng, n, nh, dtype, layout)
    before = k.clone(), v.clone()
    assert hq.hq_kv4_read(C.c, ints(seq), ints(pos), k, v, C.status) == hq.HQ_OK
    assert int(C.status) == 0
    for which, got, old in ((0, k, before[0]), (1, v, before[1])):
        for i in range(n):
            if seq[i] < 0:
                assert torch.equal(got[i], old[i])
                continue
            want = np.stack([R.read32(C.pages, C.table[seq[i], pos[i] // page], h, pos[i] % page,
                                      which, MASK) for h in range(nh)])
            assert torch.equal(got[i].cpu(), torch.from_numpy(want).to(DT[dtype]))
    seq[0], pos[n - 1] = 2, 30 + page * C.width
    assert hq.hq_kv4_read(C.c, ints(seq), ints(pos), k, v, C.status) == hq.HQ_OK
    assert int(C.status) == hq.HQ_ERR_PAGE and not k[0].any() and not v[n - 1].any()


def test_read_window_into_the_lattice_codec(hq):
    """A window's rows as head-major slabs go straight to the encoder."""
    rng = np.random.default_rng(5)
    n, nh = 64, 2
    C = Cache(hq, rng, [n], nh, 16)
    k, v, _, _ = rows(rng, n, nh, "bf16", "heads")
    assert hq.hq_kv4_read(C.c, ints([0] * n), ints(range(n)), k, v, C.status) == hq.HQ_OK
    signs = hq.signs_tensor([MASK])
    p = hq.make_params(hq.HQ_E8, 3, 6.0, 1, 22, signs, 1 << 40)
    got = hq.decode(hq.encode(k.transpose(0, 1), p), torch.float32).view(nh, n, 128)
    x = k.transpose(0, 1).float()
    assert (got - x).norm() < 0.1 * x.norm()


# ------------------------------------------------------------------ attention
def attend(hq, C, q, scale, cap, out_dtype, mass=None, ws=None, lse=True):
    B, q_len, Hq, _ = q.shape
    out = torch.full((B, q_len, Hq, 128), 7.0, dtype=out_dtype, device="cuda")
    L = torch.full((B, q_len, Hq), 7.0, device="cuda") if lse else None
    M = None
    if mass is not None:
        M = torch.full((B, C.nh, C.width * C.page), -3.0, device="cuda")
    if ws is None:
        ws = torch.full((hq.hq_kv4_attention_workspace_bytes(C.c, q_len, Hq, mass is not None),), 0xFF,
                        dtype=torch.uint8, device="cuda")
    assert hq.hq_kv4_attention(C.c, C.d_lens, q, scale, cap, out, L, mass, M, ws, C.status) == hq.HQ_OK
    return out, L, M


def check(C, q, scale, cap, got, kind="f32", mass=None, lens=None, plain=False):
    """Outputs against the reference within the bound derived above; returns the worst share."""
    lens = C.lens if lens is None else lens
    m = None if mass is None else mass.cpu().numpy().astype(np.float64)
    ref = R.attention(C.pages, C.table, lens,
                      q.double().cpu().numpy(), MASK, scale, cap, m)
    out, lse, mass_out = (None if t is None else t.double().cpu().numpy() for t in got)
    steps = max(lens) / 16 if len(lens) else 0
    min_cap = np.minimum(cap, 4 * ref["zeta"])
    score = 30 * U * ref["zeta"] + 294 * U * ref["zeta_codes"] + 8 * U * min_cap
    tol = ((2 * score + (34 * steps + 100) * U) * np.linalg.norm(ref["size"], axis=-1) +
           600 * U * np.sqrt(128.0) * ref["scales"])
    rounding = HALF_STEP[kind] * np.linalg.norm(ref["out"], axis=-1) * 1.01
    err = np.linalg.norm(out - ref["out"], axis=-1)
    assert (err <= tol + rounding).all(), (err / (tol + rounding + 1e-300)).max()
    rel = np.linalg.norm(err) / (np.linalg.norm(ref["out"]) + 1e-300)
    assert not plain or rel <= 2e-5, rel
    if lse is not None:
        empty = np.isneginf(ref["lse"])
        assert np.array_equal(np.isneginf(lse), empty)
        assert not out[empty].any()
        d = np.abs(lse[~empty] - ref["lse"][~empty])
        assert (d <= (score + (steps + 24) * U)[~empty] + 4 * U * np.abs(ref["lse"][~empty])).all()
    if mass_out is not None:
        for b, n in enumerate(lens):
            d = np.abs(mass_out[b, :, :n] - ref["mass"][b, :, :n])
            assert (d <= (2 * score[b].max() + (steps + 40) * U) * ref["added"][b, :, :n] +
                    2 * U * np.abs(ref["mass"][b, :, :n]) + 1e-37).all()
            assert (mass_out[b, :, n:] == -3.0).all()
    return (err / (tol + rounding + 1e-300)).max()


def queries(rng, B, q_len, Hq, dtype, layout="plain", size=1.5):
    x = torch.from_numpy(rng.standard_normal((B, q_len, Hq, 128)) * size).to(DT[dtype]).cuda()
    if layout == "plain":
        return x
    if layout == "fused":
        buf = torch.zeros((B, q_len, Hq + 2, 128), dtype=DT[dtype], device="cuda")
        buf[:, :, :Hq] = x
        return buf[:, :, :Hq]
    buf = torch.zeros(B * q_len * Hq * 129 + 1, dtype=DT[dtype], device="cuda")     # "odd"
    y = buf[1:].as_strided((B, q_len, Hq, 128), (q_len * Hq * 129, 129, q_len * 129, 1))
    y.copy_(x)
    return y


CASES = [
    # lens, nh, G, q_len, page, cap, q type, out type, layout, mass
    ([1], 1, 1, 1, 16, 0.0, "bf16", "f32", "plain", False),
    ([15, 16, 17, 0, 33], 2, 4, 1, 16, 0.0, "f32", "f32", "plain", True),
    ([300, 1, 64], 2, 8, 1, 48, 30.0, "bf16", "bf16", "fused", False),
    ([130, 2, 77], 3, 1, 4, 32, 0.0, "f16", "f32", "odd", True),          # rows that see nothing
    ([257, 31], 2, 5, 3, 64, 50.0, "f32", "f16", "odd", False),           # 15 rows a head
    ([500], 1, 16, 1, 128, 0.0, "bf16", "f32", "plain", True),            # 16 rows a head
    ([200, 19], 1, 6, 7, 16, 5.0, "bf16", "f32", "fused", True),          # 42 rows a head
    ([5000, 129], 1, 4, 1, 32, 0.0, "f32", "f32", "plain", True),
    ([1100, 40], 1, 4, 40, 64, 0.0, "f16", "bf16", "plain", False),       # 160 rows a head
    ([0, 0], 2, 4, 2, 16, 0.0, "f32", "f32", "plain", True),
]


@pytest.mark.parametrize("case", range(len(CASES)))
def test_attention_against_reference(hq, case):
    lens, nh, G, q_len, page, cap, dq, do, layout, mass = CASES[case]
    rng = np.random.default_rng(case)
    C = Cache(hq, rng, lens, nh, page, width=max(1, -(-max(lens) // page)) + case % 2)
    for b, n in enumerate(lens):                 # entries past the length are not read
        C.table[b, -(-n // page):] = -1 if case % 3 == 0 else 1 << 30
    C.upload()
    q = queries(rng, len(lens), q_len, nh * G, dq, layout)
    m = torch.rand((len(lens), nh, C.width * page), device="cuda") if mass else None
    got = attend(hq, C, q, 128 ** -0.5, cap, DT[do], m)
    assert int(C.status) == 0 and C.same_pages()
    check(C, q, 128 ** -0.5, cap, got, do, m, plain=do == "f32")
    again = attend(hq, C, q, 128 ** -0.5, cap, DT[do], m, lse=False)
    assert torch.equal(got[0], again[0])         # the order of the sums is fixed
    assert got[2] is None or torch.equal(got[2], again[2])


@pytest.mark.parametrize("cap", [2.0 ** 10, 2.0 ** 20, 2.0 ** 100])
def test_attention_caps_far_above_the_scores(hq, cap):
    """Scores that the cap hardly bends keep their own precision, not the cap's."""
    rng = np.random.default_rng(19)
    C = Cache(hq, rng, [300, 33], 2, 32)
    for G in (4, 6):
        q = queries(rng, 2, 1, 2 * G, "f32")
        check(C, q, 0.1, cap, attend(hq, C, q, 0.1, cap, torch.float32), plain=True)


def test_attention_many_ragged_sequences(hq):
    """More (sequence, head) pairs than resident blocks, lengths 0 .. 400."""
    rng = np.random.default_rng(20)
    lens = [int(x) for x in rng.integers(0, 400, 130)]
    C = Cache(hq, rng, lens, 4, 16)
    q = queries(rng, len(lens), 1, 8, "bf16")
    check(C, q, 0.1, 0.0, attend(hq, C, q, 0.1, 0.0, torch.float32), plain=True)


@pytest.mark.parametrize("case", range(4))
def test_attention_rows_that_many_blocks_share(hq, case):
    """Joins by one and by eight warps, of more blocks than are read ahead, listed by (sequence,
    head) and by block, beside sequences without tokens."""
    rng = np.random.default_rng(40 + case)
    lens, nh, G = (([2900] * 6 + [0] + [2900] * 6, 3, 16), ([22000, 0], 1, 4), ([0, 7000], 1, 16),
                   ([int(x) for x in rng.integers(0, 200, 160)] + [4000], 2, 8))[case]
    C = Cache(hq, rng, lens, nh, 16 * (1 + case))
    q = queries(rng, len(lens), 1, nh * G, "bf16")
    got = attend(hq, C, q, 0.1, 0.0, torch.float32)
    check(C, q, 0.1, 0.0, got, plain=True)
    assert torch.equal(got[0], attend(hq, C, q, 0.1, 0.0, torch.float32)[0])


def test_attention_sharp_flat_and_uneven(hq):
    """Scores far apart (zeta about 10^3), all equal, negative scale, and V scales of very
    different size, the largest on a token of no weight."""
    rng = np.random.default_rng(21)
    n, nh, page = 700, 2, 16
    C = Cache(hq, rng, [n, n], nh, page)
    for size, scale in ((60.0, 1.0), (0.0, 0.1), (1.5, -0.3)):
        q = queries(rng, 2, 1, 8, "f32", size=size)
        check(C, q, scale, 0.0, attend(hq, C, q, scale, 0.0, torch.float32))
    k, v = (rng.standard_normal((n, nh, 128)).astype(np.float32) for _ in range(2))
    d = rng.standard_normal(128).astype(np.float32)
    k[100] = -40 * d
    v[100] *= 1e30                               # no weight, a huge value
    v[300:] *= 1e-3
    v[500:] *= 1e-30
    R.append(C.pages, C.table, k, v, [0] * n, range(n), MASK)
    C.upload()
    q = torch.from_numpy(np.broadcast_to(d, (2, 1, 8, 128)).copy()).cuda()
    check(C, q, 1.0, 0.0, attend(hq, C, q, 1.0, 0.0, torch.float32))


def test_attention_sink_and_equal_rest(hq):
    """One token of weight near 1 and thousands of equal tokens of weight 2^-18 each: the
    small weights' roundings do not add up."""
    rng = np.random.default_rng(22)
    n, nh, page = 4000, 1, 32
    C = Cache(hq, rng, [n], nh, page, empty=True)
    d = rng.standard_normal(128).astype(np.float32)
    k = np.broadcast_to(d * 0.1, (n, nh, 128)).copy()
    v = np.broadcast_to(rng.standard_normal(128), (n, nh, 128)).astype(np.float32).copy()
    k[0], v[0] = d * 0.1 + d * (18 * np.log(2.0) / float(d @ d)), 0.0
    R.append(C.pages, C.table, k, v, [0] * n, range(n), MASK)
    C.upload()
    q = torch.from_numpy(np.broadcast_to(d, (1, 1, 4, 128)).copy()).cuda()
    m = torch.zeros((1, 1, C.width * page), device="cuda")
    check(C, q, 1.0, 0.0, attend(hq, C, q, 1.0, 0.0, torch.float32, m), mass=m)


def test_attention_nan_query_stays_in_its_row(hq):
    rng = np.random.default_rng(23)
    C = Cache(hq, rng, [90], 2, 16)
    q = queries(rng, 1, 1, 8, "f32")
    want = attend(hq, C, q, 0.1, 0.0, torch.float32)[0]
    q2 = q.clone()
    q2[0, 0, 3, 5] = float("nan")
    got = attend(hq, C, q2, 0.1, 0.0, torch.float32)[0]
    assert torch.isnan(got[0, 0, 3]).all()
    keep = [0, 1, 2, 4, 5, 6, 7]
    assert torch.equal(got[:, :, keep], want[:, :, keep])


def test_attention_bad_pages_and_lengths(hq):
    """A page outside the pool weighs nothing and is reported, as are lengths outside
    [0, capacity]."""
    rng = np.random.default_rng(24)
    page, n = 16, 100
    C = Cache(hq, rng, [n, n, n], 2, page)
    good = C.table.copy()
    C.table[0, 2], C.table[2, 0] = -1, C.pages.shape[0]
    C.upload()
    C.d_lens = ints([n, -4, n])
    q = queries(rng, 3, 1, 4, "f32")
    m = torch.zeros((3, 2, C.width * page), device="cuda")
    out, lse, M = attend(hq, C, q, 0.1, 0.0, torch.float32, m)
    assert int(C.status) == hq.HQ_ERR_PAGE
    assert not out[1].any() and torch.isneginf(lse[1]).all()
    # the same as a cache without those tokens
    C.table = good
    for b, drop in ((0, 2), (2, 0)):
        D = Cache(hq, rng, [n - page], 2, page, empty=True)
        left = [j for j in range(C.width) if j != drop]
        D.table = np.arange(len(left), dtype=np.int32)[None]
        D.pages[:len(left)] = C.pages[good[b, left]]
        D.upload()
        D.lens = [n - page]
        check(D, q[b:b + 1], 0.1, 0.0, (out[b:b + 1], lse[b:b + 1], None), plain=True)
        assert not M[b, :, drop * page:(drop + 1) * page].any()
    C.upload()
    C.d_lens = ints([n, C.width * page + 1, n])
    attend(hq, C, q, 0.1, 0.0, torch.float32)
    assert int(C.status) == hq.HQ_ERR_PAGE


def test_attention_on_streams_in_graphs_and_in_place_mass(hq):
    """Two calls at once with workspaces of their own; one call captured and replayed over
    changed lengths, queries and mass; mass accumulated in place."""
    rng = np.random.default_rng(25)
    C = Cache(hq, rng, [900, 333], 2, 16)
    qs = [queries(rng, 2, 1, 8, "bf16") for _ in range(2)]
    alone = [attend(hq, C, q, 0.1, 0.0, torch.float32) for q in qs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [None, None]
    for _ in range(3):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i] = attend(hq, C, qs[i], 0.1, 0.0, torch.float32)
    torch.cuda.synchronize()
    for a, g in zip(alone, got):
        assert torch.equal(a[0], g[0]) and torch.equal(a[1], g[1])
    # an explicit stream argument
    ws = torch.empty(hq.hq_kv4_attention_workspace_bytes(C.c, 1, 8, True), dtype=torch.uint8,
                     device="cuda")
    q, mass = qs[0].clone(), torch.zeros((2, 2, C.width * 16), device="cuda")
    out, lse = torch.zeros((2, 1, 8, 128), device="cuda"), torch.zeros((2, 1, 8), device="cuda")
    torch.cuda.synchronize()
    assert hq.hq_kv4_attention(C.c, C.d_lens, q, 0.1, 0.0, out, lse, mass, mass, ws, C.status,
                               stream=streams[0]) == hq.HQ_OK
    streams[0].synchronize()
    assert torch.equal(out, alone[0][0])
    first = mass.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):                # behind copies and a fill, as in a serving step
        q.copy_(qs[1])
        out.zero_()
        hq.hq_kv4_attention(C.c, C.d_lens, q, 0.1, 0.0, out, lse, mass, mass, ws, C.status)
    for lens in ([900, 333], [17, 0], [400, 333]):
        C.d_lens.copy_(ints(lens))
        q.zero_()
        before = mass.clone()
        graph.replay()
        torch.cuda.synchronize()
        check(C, q, 0.1, 0.0, (out, lse, None), lens=lens, plain=True)
        add = (mass - before).double().sum().item()
        assert abs(add - 8 * sum(n > 0 for n in lens)) < 1e-2
    assert abs(first.double().sum().item() - 16) < 1e-3 and int(C.status) == 0


def test_attention_shared_pages(hq):
    """Sequences that share a prefix's pages read the same rows."""
    rng = np.random.default_rng(26)
    C = Cache(hq, rng, [96, 96], 2, 32)
    C.table[1, :2] = C.table[0, :2]
    C.upload()
    q = queries(rng, 1, 1, 4, "f32").expand(2, 1, 4, 128)
    got = attend(hq, C, q, 0.1, 0.0, torch.float32)
    check(C, q, 0.1, 0.0, got)


def test_pool_past_four_gigabytes(hq):
    """Pages behind byte 2^32 and token index 2^31 / 128 of the pool."""
    nh, page = 8, 128
    per = hq.hq_kv4_page_bytes(nh, page)
    n_pages = (1 << 32) // per + 40
    rng = np.random.default_rng(27)
    C = Cache(hq, rng, [300, 140], nh, page)
    big = torch.zeros(n_pages * per, dtype=torch.uint8, device="cuda")
    ids = n_pages - 1 - C.table.astype(np.int64)
    for old, new in zip(C.table.flatten(), ids.flatten()):
        big[new * per:(new + 1) * per] = C.d_pages[int(old)].flatten()
    table = torch.from_numpy(ids.astype(np.int32)).cuda()
    c = hq.make_kv4_cache(big, table, page, nh, hq.signs_tensor([MASK]).flatten())
    C2 = C
    q = queries(rng, 2, 1, 16, "bf16")
    want = attend(hq, C, q, 0.1, 0.0, torch.float32)
    small = C.c
    C2.c = c
    got = attend(hq, C2, q, 0.1, 0.0, torch.float32)
    assert torch.equal(got[0], want[0])
    k, v = (torch.empty((300, nh, 128), device="cuda") for _ in range(2))
    k2, v2 = torch.empty_like(k), torch.empty_like(v)
    where = ints([0] * 300), ints(range(300))
    hq.hq_kv4_read(small, *where, k, v, C.status)
    hq.hq_kv4_append(c, v, k, *where, C.status)            # swapped, back in place
    hq.hq_kv4_read(c, *where, k2, v2, C.status)
    assert (k2 - v).norm() < 0.2 * v.norm() and (v2 - k).norm() < 0.2 * k.norm()


# ------------------------------------------------------------------ eviction
def evict(hq, C, mass, budget, recent, page=None):
    B, page = len(C.lens), C.page if page is None else page
    width = max(1, -(-min(budget, C.width * C.page) // page))
    pages = torch.full((B * width + 2, C.nh, page // 16, 2112), 0x77, dtype=torch.uint8, device="cuda")
    table = torch.randperm(B * width + 2)[:B * width].to(torch.int32).view(B, width).cuda()
    dst = hq.make_kv4_cache(pages, table, page, C.nh, hq.signs_tensor([MASK]).flatten())
    kept = torch.full((B, C.nh, budget), -9, dtype=torch.int32, device="cuda")
    n = torch.full((B,), -9, dtype=torch.int32, device="cuda")
    m = torch.full((B, C.nh, width * page), -5.0, device="cuda")
    assert hq.hq_kv4_evict(C.c, C.d_lens, mass, dst, recent, kept, n, m, C.status) == hq.HQ_OK
    torch.cuda.synchronize()
    return dst, pages, table, kept, n, m


@pytest.mark.parametrize("lens,nh,page,budget,recent,new_page", [
    ([40], 1, 16, 16, 4, None), ([300, 5, 0, 64, 65], 2, 16, 64, 16, 32),
    ([5000, 4097, 63], 2, 48, 1000, 0, None), ([200, 90], 3, 32, 77, 77, 16),
    ([33, 32], 1, 16, 1, 0, None), ([70], 2, 16, 500, 20, 64),
    ([60001, 49155, 49151], 1, 128, 2500, 50, None)])            # more keys than shared memory has
def test_evict_against_reference(hq, lens, nh, page, budget, recent, new_page):
    rng = np.random.default_rng(budget)
    C = Cache(hq, rng, lens, nh, page)
    mass = np.floor(rng.random((len(lens), nh, C.width * page)) * 40).astype(np.float32) / 8
    mass[:, :, 3::50] = np.nan
    mass[:, :, 4::60] = np.inf
    mass[:, :, 5::40] = -0.0
    mass[:, :, 6::90] = -1.0
    dst, pages, table, kept, n, m = evict(hq, C, torch.from_numpy(mass).cuda(), budget, recent, new_page)
    assert int(C.status) == 0 and C.same_pages()
    pages, table, P = pages.cpu().numpy(), table.cpu().numpy(), dst.page_tokens
    for b, length in enumerate(lens):
        assert int(n[b]) == min(length, budget)
        for h in range(nh):
            want = R.keep(mass[b, h], length, budget, recent)
            got = kept[b, h].cpu().numpy()
            assert np.array_equal(got[:len(want)], want) and (got[len(want):] == -1).all()
            gm = m[b, h].cpu().numpy()
            assert np.array_equal(gm[:len(want)].view(np.int32), mass[b, h, want].view(np.int32))
            assert (gm[len(want):] == -5.0).all()
            for which in range(2):
                for i, t in list(enumerate(want))[:40]:
                    c0, s0 = R.raw_rows(C.pages, C.table[b, t // page], which)
                    c1, s1 = R.raw_rows(pages, table[b, i // P], which)
                    assert np.array_equal(c0[h, t % page], c1[h, i % P])
                    assert s0[h, t % page] == s1[h, i % P]


@pytest.mark.parametrize("n,budget,recent", [(5, 3, 0), (1030, 700, 6), (1031, 700, 6), (8300, 100, 99),
                                             (50000, 3, 1), (50000, 49990, 7)])
def test_evict_positions_of_distinct_and_equal_masses(hq, n, budget, recent):
    """Sequences on both sides of every limit of the selection (1024 and 8192 tokens that compete,
    49152 keys in shared memory), masses all distinct, in steps and negative, on 16-byte boundaries and off."""
    rng = np.random.default_rng(n)
    C = Cache(hq, rng, [n], 1, 16, empty=True)
    draws = rng.random(C.width * 16)
    for mass in (draws, np.floor(draws * 50) / 50, -draws, np.exp(-40 * draws)):
        for off in (0, 1):
            buf = torch.zeros(mass.size + off, device="cuda")
            d = buf[off:].view(1, 1, -1)
            d.copy_(torch.from_numpy(mass))
            kept = evict(hq, C, d, budget, recent)[3]
            want = R.keep(mass.astype(np.float32), n, budget, recent)
            assert np.array_equal(kept[0, 0].cpu().numpy(), want)


def test_evict_equal_masses_and_bad_pages(hq):
    """All masses equal: the lowest positions win; rows whose page is outside the pool are left
    out and reported."""
    rng = np.random.default_rng(31)
    C = Cache(hq, rng, [9000], 1, 64)
    mass = torch.zeros((1, 1, C.width * 64), device="cuda")
    _, _, _, kept, _, _ = evict(hq, C, mass, 4500, 100)
    assert torch.equal(kept[0, 0], torch.cat([torch.arange(4400), torch.arange(8900, 9000)]).int().cuda())
    C.table[0, 1] = -7
    C.upload()
    _, pages, table, kept, n, _ = evict(hq, C, mass, 4500, 100)
    assert int(C.status) == hq.HQ_ERR_PAGE and int(n) == 4500
    assert (pages[int(table[0, 1])] == 0x77).all()


# ------------------------------------------------------------------ together
def test_a_serving_loop(hq):
    """Prompts appended, tokens decoded with their weights accumulated, the cache cut to its
    budget whenever it is over it: page bytes equal the reference's, outputs within the bound."""
    rng = np.random.default_rng(40)
    B, nh, G, page, width, budget, recent = 3, 2, 4, 16, 8, 64, 16
    lens = [70, 20, 1]
    C = Cache(hq, rng, lens, nh, page, width=width, empty=True)
    k, v, kx, vx = rows(rng, sum(lens), nh, "bf16", "fused")
    seq = np.repeat(np.arange(B), lens)
    pos = np.concatenate([np.arange(n) for n in lens])
    R.append(C.pages, C.table, kx, vx, seq, pos, MASK)
    hq.hq_kv4_append(C.c, k, v, ints(seq), ints(pos), C.status)
    mass = torch.zeros((B, nh, width * page), device="cuda")
    spare = None
    for step in range(20):
        k, v, kx, vx = rows(rng, B, nh, "bf16", "plain")
        R.append(C.pages, C.table, kx, vx, range(B), C.lens, MASK)
        hq.hq_kv4_append(C.c, k, v, ints(range(B)), C.d_lens, C.status)
        C.d_lens += 1
        C.lens = [n + 1 for n in C.lens]
        assert C.same_pages()
        q = queries(rng, B, 1, nh * G, "bf16")
        out, lse, new = attend(hq, C, q, 0.1, 0.0, torch.float32, mass)
        check(C, q, 0.1, 0.0, (out, lse, new), mass=mass)
        new[new == -3.0] = 0.0
        mass = new
        if max(C.lens) > budget + 10:
            if spare is None:
                spare = torch.zeros_like(C.d_pages), torch.arange(B * width, dtype=torch.int32).view(B, width).cuda()
            dst = hq.make_kv4_cache(spare[0], spare[1], page, nh, hq.signs_tensor([MASK]).flatten())
            kept = torch.empty((B, nh, budget), dtype=torch.int32, device="cuda")
            n, m = torch.empty(B, dtype=torch.int32, device="cuda"), torch.zeros_like(mass)
            hq.hq_kv4_evict(C.c, C.d_lens, mass, dst, recent, kept, n, m, C.status)
            torch.cuda.synchronize()
            for b in range(B):
                for h in range(nh):
                    want = R.keep(mass[b, h].cpu().numpy(), C.lens[b], budget, recent)
                    assert np.array_equal(kept[b, h, :len(want)].cpu().numpy(), want)
            spare, C.c, mass = (C.d_pages, C.d_table), dst, m
            C.d_pages, C.d_table, C.d_lens = dst._pages, dst._table, n
            C.pages, C.table = C.d_pages.cpu().numpy(), C.d_table.cpu().numpy()
            C.lens = n.tolist()
    assert int(C.status) == 0 and max(C.lens) <= budget + 10


def test_a_chain_without_waits(hq):
    """Torch kernels that write the next call's inputs, appends, attentions and reads behind one
    another in a stream, each launched while the one before it runs: the same bits as with a
    wait after every call."""
    def run(wait):
        rng = np.random.default_rng(41)
        B, nh, page, width = 4, 2, 16, 40
        C = Cache(hq, rng, [600, 33, 15, 1], nh, page, width=width)
        g = torch.Generator(device="cuda")
        g.manual_seed(7)
        ws = torch.zeros(hq.hq_kv4_attention_workspace_bytes(C.c, 1, 8, True), dtype=torch.uint8,
                         device="cuda")
        mass = torch.zeros((B, nh, width * page), device="cuda")
        k, v = (torch.empty((B, nh, 128), device="cuda") for _ in range(2))
        q, out = torch.empty((B, 1, 8, 128), device="cuda"), torch.empty((B, 1, 8, 128), device="cuda")
        seq, rows_k, rows_v = ints(range(B)), torch.empty_like(k), torch.empty_like(k)
        seen = []
        for _ in range(25):
            for t in (k, v, q):
                t.normal_(generator=g)
            hq.hq_kv4_append(C.c, k, v, seq, C.d_lens, C.status)
            if wait:
                torch.cuda.synchronize()
            hq.hq_kv4_read(C.c, seq, C.d_lens, rows_k, rows_v, C.status)
            C.d_lens += 1
            if wait:
                torch.cuda.synchronize()
            hq.hq_kv4_attention(C.c, C.d_lens, q, 0.1, 0.0, out, None, mass, mass, ws, C.status)
            if wait:
                torch.cuda.synchronize()
            seen += [out.clone(), rows_k.clone(), rows_v.clone()]
        torch.cuda.synchronize()
        assert int(C.status) == 0
        return seen + [mass, C.d_pages]

    for a, b in zip(run(True), run(False)):
        assert torch.equal(a, b)


def test_binding_checks(hq):
    rng = np.random.default_rng(50)
    C = Cache(hq, rng, [20, 30], 2, 16)
    k, v, _, _ = rows(rng, 2, 2, "bf16", "plain")
    one = ints([0, 1])
    with pytest.raises(ValueError):
        hq.hq_kv4_append(C.c, k[:1], v, one, one, C.status)
    with pytest.raises(ValueError):
        hq.hq_kv4_append(C.c, k, v, one, one[:1], C.status)
    with pytest.raises(ValueError):
        hq.hq_kv4_append(C.c, k.cpu(), v, one, one, C.status)
    with pytest.raises(TypeError):
        hq.hq_kv4_append(C.c, k, v.float(), one, one, C.status)
    with pytest.raises(TypeError):
        hq.hq_kv4_append(C.c, k.double(), v.double(), one, one, C.status)
    with pytest.raises(TypeError):
        hq.hq_kv4_read(C.c, one.long(), one, k, v, C.status)
    with pytest.raises(ValueError):
        hq.hq_kv4_read(C.c, one, one, k.expand(2, 2, 128)[..., ::2], v, C.status)
    q = queries(rng, 2, 1, 4, "bf16")
    out = torch.empty((2, 1, 4, 128), device="cuda")
    ws = torch.empty(1 << 20, dtype=torch.uint8, device="cuda")
    with pytest.raises(ValueError):
        hq.hq_kv4_attention(C.c, C.d_lens[:1], q, 0.1, 0.0, out, None, None, None, ws, C.status)
    with pytest.raises(ValueError):
        hq.hq_kv4_attention(C.c, C.d_lens, q, 0.1, 0.0, out[:1], None, None, None, ws, C.status)
    assert hq.hq_kv4_attention(C.c, C.d_lens, q, 0.1, 0.0, out, None, None, None, ws[:16],
                               C.status) == hq.HQ_ERR_INVALID
    with pytest.raises(ValueError):
        hq.hq_kv4_attention(C.c, C.d_lens, q, 0.1, 0.0, out, None, None,
                            torch.zeros((2, 2, 16), device="cuda"), ws, C.status)
