"""Attention over packed prompts on the GPU where weights, values and the cut of a batch reach
their limits, against its reference (oracle/serving.py).

The bound is test_prompt_gpu.py's with a term of its own for small weights in fp16: a weight
enters its product as 2^(z - m) with the reference m chosen so that a row's largest weight is
2^10 to 2^15; below fp16's normal range it is off by at most 2^-25, that is 2^-35 of the
largest weight, which is at most 1:  2^-35 sum |v|, where that file allows 2^-19."""
import numpy as np
import pytest
import torch

from oracle import serving as S
from test_kv4_gpu import HALF_STEP, U
from test_kv4_gpu import hq  # noqa: F401  (the fixture)
from test_prompt_gpu import call, offsets, tensors

pytestmark = pytest.mark.gpu


def check(q, k, v, starts, k_starts, scale, cap, got, rows=None):
    kind = "bf16" if q.dtype == torch.bfloat16 else "f16"
    h = HALF_STEP[kind]
    ref = S.prompt(*(t.double().cpu().numpy() for t in (q, k, v)), starts,
                   starts if k_starts is None else k_starts, scale, cap, rows)
    out, lse = (t.double().cpu().numpy() for t in got)
    live = ~np.isnan(ref["lse"][:, 0])
    dz = (280 * U * ref["zeta"] + 8 * U * np.minimum(cap, 4 * ref["zeta"]))[live]
    T = ref["keys"][live]
    tol = 1.01 * ((h + 2 * dz + (34 * T / 16 + 100) * U)[..., None] * ref["size"][live] +
                  h * np.abs(ref["out"][live]))
    if kind == "f16":
        tol += 2.0 ** -35 * ref["every"][live] + 2.0 ** -25        # and outputs below fp16's normal range
    err = np.abs(out[live] - ref["out"][live])
    assert (err <= tol).all(), (err / (tol + 1e-300)).max()
    want = ref["lse"][live]
    d = np.abs(lse[live] - want)
    assert (d <= dz + (T / 2 + 40) * U + 8 * U * (np.abs(want) + ref["zeta"][live])).all()


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("spread", [0.7, 0.01])
@pytest.mark.parametrize("new,old,at,cap", [
    (3, 4093, 0, 0.0), (3, 16381, 0, 0.0), (2, 65500, 40, 0.0), (3, 16381, 20, 60.0), (3, 16381, 9000, 0.0),
    (8192, 0, 0, 0.0), (5000, 0, 33, 60.0)])
def test_one_heavy_key_of_small_value(hq, dtype, spread, new, old, at, cap):
    """One key 14 above all others, which share a part of the weight between them, and whose values are
    20 times larger: small weights count as much as large ones."""
    rng = np.random.default_rng(70)
    m, dt = new + old, torch.float16 if dtype == "f16" else torch.bfloat16
    d = rng.standard_normal(128)
    d /= np.linalg.norm(d)
    k = spread / 4 * rng.standard_normal((m, 1, 128))
    k[at] += 3.5 * d
    v = 0.5 + 0.5 * rng.standard_normal((m, 1, 128))
    v[at] *= 0.05
    q = np.broadcast_to(4 * d, (new, 1, 128)) + 0.01 * rng.standard_normal((new, 1, 128))
    q, k, v = (torch.from_numpy(x).to(dt).cuda() for x in (q, k, v))
    starts, k_starts = [0, new], None if old == 0 else [0, m]
    rows = None if new < 10 else {0, 127, 1000, new - 129, new - 1}
    check(q, k, v, starts, k_starts, 1.0, cap, call(hq, q, k, v, starts, k_starts, 1.0, cap), rows)


@pytest.mark.parametrize("case", range(4))
def test_equal_sequences_cut_into_pieces(hq, case):
    """Batches that are cut, with several sequences of one length, or more keys than the sort by length tells
    apart: the same bits in every call."""
    new, old, nh, G, cap, dtype = (
        ([128] * 2, [20000] * 2, 8, 2, 0.0, "bf16"), ([1] * 5, [19000] * 5, 2, 4, 0.0, "f16"),
        ([1] * 9, [5000] * 9, 1, 3, 20.0, "bf16"), ([1, 3, 2], [131300, 140000, 135000], 1, 1, 0.0, "bf16"))[case]
    rng = np.random.default_rng(71 + case)
    starts, k_starts = offsets(new), offsets([a + b for a, b in zip(new, old)])
    q, k, v = tensors(rng, starts[-1], k_starts[-1], nh, G, dtype, "plain")
    first = call(hq, q, k, v, starts, k_starts, 128 ** -0.5, cap)
    for _ in range(30):
        again = call(hq, q, k, v, starts, k_starts, 128 ** -0.5, cap)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])
    if case > 0:
        check(q, k, v, starts, k_starts, 128 ** -0.5, cap, first)


@pytest.mark.parametrize("value", [2.0 ** 80, 2.0 ** 68, 1.0, 2.0 ** -80])
def test_values_of_any_size(hq, value):
    """Values far from 1 under scores that climb and fall by up to 85 in steps of any size, many of
    them equal, whole prompts and pieces."""
    rng = np.random.default_rng(75)
    d = rng.standard_normal(128)
    d /= np.linalg.norm(d)
    for n, m, up in ((900, 900, 19.0), (900, 900, -19.0), (900, 900, 42.0), (900, 900, 0.0), (5, 9000, 42.0), (5, 9000, 0.0)):
        q = np.broadcast_to(d, (n, 4, 128)) + 0.03 * rng.standard_normal((n, 4, 128))
        k = up * np.linspace(-1, 1, m)[:, None, None] * d + 0.5 * rng.standard_normal((m, 2, 128))
        v = value * rng.standard_normal((m, 2, 128))
        q, k, v = (torch.from_numpy(x).to(torch.bfloat16).cuda() for x in (q, k, v))
        for cap in (0.0, 64.0):
            starts, k_starts = [0, n], None if n == m else [0, m]
            got = call(hq, q, k, v, starts, k_starts, 1.0, cap)
            assert torch.isfinite(got[0]).all() and torch.isfinite(got[1]).all()
            check(q, k, v, starts, k_starts, 1.0, cap, got, {0, 1, 4, 130, 513, n - 1})


def test_no_scale_over_large_products(hq):
    """A scale of 0, or next to it, over products up to fp32's limit: equal weights."""
    rng = np.random.default_rng(76)
    q, k = (torch.from_numpy(rng.standard_normal((300, h, 128)) * s).to(torch.bfloat16).cuda()
            for h, s in ((4, 2.0 ** 61), (2, 2.0 ** 60)))
    v = torch.from_numpy(rng.standard_normal((300, 2, 128))).to(torch.bfloat16).cuda()
    for scale, cap in ((0.0, 0.0), (-0.0, 0.0), (1e-45, 0.0), (0.0, 5.0)):
        check(q, k, v, [0, 300], None, scale, cap, call(hq, q, k, v, [0, 300], None, scale, cap))
