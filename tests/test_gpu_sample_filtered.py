"""qg_sample_filtered against the oracle, row by row.

Tokens and kept counts are equal: both sides weigh in float64, the library
rounds each weight to 2^-44 (or finer than V^-1 2^-62 of the total), so a
border that a random u or top_p meets within that is not expected in any of
these cases (about 1e-8 a row). The log-probability is log(w / S): S is off
by at most V 2^-45, the rest is float64, then one rounding to fp32."""
import math

import numpy as np
import pytest
import torch

from oracle import qg_oracle as O
from tests.gpu_util import dev

pytestmark = pytest.mark.gpu

qg = pytest.importorskip("weight_only_quantized_03_b200")


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def check(logits, u, temperature=None, top_k=None, top_p=None, min_p=None, ld=None):
    B, V = logits.shape
    f32 = lambda a: None if a is None else dev(np.asarray(a, np.float32))
    wide = torch.full((B, ld or V), 1e30, device="cuda")
    wide[:, :V] = dev(np.asarray(logits, np.float32))
    ld_ = wide[:, :V]
    out, kept = (torch.full((B,), -9, dtype=torch.int32, device="cuda") for _ in range(2))
    lp = torch.full((B,), 7.0, device="cuda")
    qg.qg_sample_filtered(ld_, f32(u), out, f32(temperature),
                          None if top_k is None else dev(np.asarray(top_k, np.int32)), f32(top_p),
                          f32(min_p), kept, lp)
    out, kept, lp = out.cpu().numpy(), kept.cpu().numpy(), lp.cpu().numpy().astype(np.float64)
    at = lambda a, b, d: d if a is None else np.float32(np.asarray(a)[b])
    for b in range(B):
        want = O.sample_filtered(np.asarray(logits[b], np.float32), np.float32(u[b]),
                                 at(temperature, b, 1.0),
                                 0 if top_k is None else int(top_k[b]), at(top_p, b, 1.0),
                                 at(min_p, b, 0.0))
        assert (int(out[b]), int(kept[b])) == want[:2], (b, out[b], kept[b], want)
        if math.isnan(want[2]):
            assert math.isnan(lp[b])
        else:
            tol = V * 2.0 ** -44 + 1e-12 + O.U32 * 1.01 * abs(want[2])
            assert abs(lp[b] - want[2]) <= tol, (b, lp[b], want)
    return out, kept


def params(rng, B, V):
    pick = lambda *v: rng.choice(v, size=B)
    return dict(u=rng.random(B).astype(np.float32),
                temperature=pick(0.0, 0.2, 0.7, 1.0, 1.5, 5.0),
                top_k=pick(0, 0, 1, 2, 50, V // 2, V, V + 5),
                top_p=pick(0.0, 0.1, 0.5, 0.9, 0.99, 1.0, 1.0),
                min_p=pick(0.0, 0.0, 0.01, 0.2, 1.0, 3.0))


@pytest.mark.parametrize("B,V,ld", [(7, 1, None), (9, 2, None), (16, 31, 37), (33, 1000, None),
                                    (160, 2048, None), (20, 4097, 4099), (5, 9001, None),
                                    (3, 40000, None), (12, 70001, 70003), (1, 151936, None),
                                    (32, 151936, None)])
def test_random_rows(B, V, ld):
    rng = np.random.default_rng(V + B)
    for spread in ((2.5,) if V > 50000 else (0.3, 2.5, 12.0)):
        l = (rng.standard_normal((B, V)) * spread).astype(np.float32)
        check(l, ld=ld, **params(rng, B, V))
        check(l, rng.random(B).astype(np.float32), ld=ld)   # no filters at all


@pytest.mark.parametrize("name", ["u", "temperature", "top_k", "top_p", "min_p"])
def test_each_filter_alone(name):
    rng = np.random.default_rng(5)
    B, V = 64, 5000
    p = params(rng, B, V)
    l = (rng.standard_normal((B, V)) * 2).astype(np.float32)
    check(l, p["u"], **({} if name == "u" else {name: p[name]}))


@pytest.mark.parametrize("V", [9, 3000, 50000])
def test_ties_go_by_index(V):
    rng = np.random.default_rng(V)
    B = 12
    l = np.round(rng.standard_normal((B, V)) * 1.5).astype(np.float32)   # a few values
    l[0] = 4.0                                                           # one value
    l[1] = np.where(np.arange(V) % 3 == 0, -0.0, 0.0)
    l[2] = np.where(np.arange(V) < V // 2, 1.0, 2.0)
    check(l, **params(rng, B, V))
    check(l, rng.random(B).astype(np.float32), top_k=rng.integers(1, V + 1, B))
    check(l, rng.random(B).astype(np.float32), top_p=rng.random(B).astype(np.float32))


@pytest.mark.parametrize("V", [700, 30000, 151936])
def test_outliers_and_masked_values(V):
    """Values that crowd into one bin of the first histogram: an outlier far
    above or below, masks of -1e9 and of the lowest float, and -inf."""
    rng = np.random.default_rng(V + 1)
    B = 10
    l = (rng.standard_normal((B, V)) * 2).astype(np.float32)
    l[0, 3] = 1e30
    l[1, 5] = -1e30
    l[2, rng.random(V) < 0.9] = -1e9
    l[3, rng.random(V) < 0.9] = np.finfo(np.float32).min
    l[4, rng.random(V) < 0.99] = -np.inf
    l[5, 7], l[5, 8] = np.finfo(np.float32).max, np.finfo(np.float32).min
    l[6] = (1000.0 + rng.integers(0, 3, V) * 2.0 ** -13).astype(np.float32)
    l[7] *= 1e-30
    l[8] = np.where(rng.random(V) < 0.5, l[8] * 1e-38, l[8] * 1e30)
    l[9] = -np.abs(l[9]) * 1e-42
    for top_k in (0, 40, V // 3, V - 1):
        p = params(rng, B, V)
        p["top_k"] = np.full(B, top_k)
        p["temperature"] = np.full(B, 0.9)
        check(l, **p)
    check(l, rng.random(B).astype(np.float32), temperature=np.full(B, 1e-3),
          top_k=np.full(B, V // 2))
    check(l, rng.random(B).astype(np.float32), temperature=np.full(B, np.inf))
    check(l, rng.random(B).astype(np.float32), temperature=np.full(B, 1e-45))


def test_rows_that_are_not_numbers():
    nan, inf = np.nan, np.inf
    V = 6000
    rng = np.random.default_rng(0)
    l = rng.standard_normal((8, V)).astype(np.float32)
    l[0] = nan
    l[1] = -inf
    l[2, :] = nan
    l[2, 4321] = -5.0
    l[3, rng.random(V) < 0.5] = nan
    l[4, [17, 400, 5999]] = inf
    l[5] = inf
    l[6, 9] = inf
    l[6, rng.random(V) < 0.3] = -inf
    u = np.array([0.3, 0.3, 0.3, 0.7, 0.5, 0.99, 0.2, 0.6], np.float32)
    check(l, u)
    check(l, u, top_p=np.full(8, 0.7), min_p=np.full(8, 0.5), top_k=np.full(8, 2))
    check(l, u, temperature=np.zeros(8))


def test_ends_of_u_and_parameters_that_are_not_numbers():
    rng = np.random.default_rng(1)
    l = rng.standard_normal((4, 3000)).astype(np.float32)
    out, _ = check(l, np.array([0.0, 1.0, 0.0, 1.0], np.float32), top_k=[0, 0, 5, 5])
    assert out[0] == l[0].argmax() and out[2] == l[2].argmax()
    # u beyond its range and NaN are clamped; NaN filters are off, a NaN
    # temperature is greedy
    nan = np.nan
    got = [torch.empty(4, dtype=torch.int32, device="cuda") for _ in range(2)]
    ld = dev(l)
    f = lambda *a: torch.tensor(a, dtype=torch.float32, device="cuda")
    qg.qg_sample_filtered(ld, f(-3.0, 2.0, nan, 0.4), got[0], top_p=f(nan, nan, nan, nan),
                          min_p=f(nan, nan, nan, nan))
    qg.qg_sample_filtered(ld, f(0.0, 1.0, 0.0, 0.4), got[1])
    assert torch.equal(*got)
    qg.qg_sample_filtered(ld, f(0.9, 0.9, 0.9, 0.9), got[0], temperature=f(nan, -1.0, 0.0, nan))
    assert got[0].tolist() == l.argmax(1).tolist()


def test_a_vocabulary_beyond_the_resident_slices():
    rng = np.random.default_rng(2)
    V = 700001                      # slices larger than shared memory holds
    l = (rng.standard_normal((3, V)) * 3).astype(np.float32)
    check(l, np.array([0.2, 0.9, 0.5], np.float32), top_p=np.array([1.0, 0.95, 0.5]),
          top_k=[0, 1000, 300000])


def test_batches_beyond_one_wave_and_same_bits_in_a_graph():
    rng = np.random.default_rng(3)
    B, V = 400, 20000
    l = (rng.standard_normal((B, V)) * 2).astype(np.float32)
    p = params(rng, B, V)
    want, _ = check(l, **p)
    ld = dev(l)
    out = torch.zeros(B, dtype=torch.int32, device="cuda")
    args = {k: dev(np.asarray(v, np.int32 if k == "top_k" else np.float32)) for k, v in p.items()}
    u = args.pop("u")
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        qg.qg_sample_filtered(ld, u, out, **args)
    for _ in range(3):
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert np.array_equal(out.cpu().numpy(), want)


@pytest.mark.parametrize("B,V", [(170, 6000), (149, 8192), (8, 151936), (2, 8190), (300, 4095)])
def test_batches_and_slices_at_the_ends_of_the_rules(B, V):
    """Two blocks an SM, clusters of 8 in place of 16, slices of 2047 values;
    random rows, and rows of a few distinct values."""
    rng = np.random.default_rng(V + 7 * B)
    l = (rng.standard_normal((B, V)) * 2).astype(np.float32)
    if V < 50000:
        l[::3] = np.round(l[::3] * 2) / 2
    check(l, **params(rng, B, V))


@pytest.mark.parametrize("B,V", [(3, 151936), (148, 5000), (300, 3000)])
def test_collections_of_many_calls_side_by_side(B, V):
    """Rows whose members come from every CTA of a cluster and every warp of a
    CTA, on two streams at once, many times: the same tokens each time. (A
    CTA's count of members and their place in the list are words of their own:
    threads read the first while the other is set.)"""
    rng = np.random.default_rng(B + V)
    l = (rng.standard_normal((B, V)) * 2).astype(np.float32)
    p = dict(u=rng.random(B).astype(np.float32), top_k=rng.integers(20, 200, B),
             top_p=np.full(B, 0.95), temperature=np.full(B, 1.1))
    want, kept = check(l, **p)
    ld = dev(l)
    args = {k: dev(np.asarray(v, np.int32 if k == "top_k" else np.float32)) for k, v in p.items()}
    u = args.pop("u")
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    outs = torch.full((2, 40, 2, B), -1, dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    for i in range(40):
        for s, stream in enumerate(streams):
            with torch.cuda.stream(stream):
                qg.qg_sample_filtered(ld, u, outs[s, i, 0], kept=outs[s, i, 1], **args)
    torch.cuda.synchronize()
    got = outs.cpu().numpy()
    assert np.all(got[:, :, 0] == want) and np.all(got[:, :, 1] == kept)


@pytest.mark.parametrize("V", [1 << 22, (1 << 21) + 12345, (1 << 20) + 17])
def test_crowded_rows_of_the_largest_vocabularies(V):
    """A slice of more than 65536 values in one bin, whose weights' lower
    pieces add up past 32 bits: one larger logit and the rest equal (a floor,
    or a finite mask within reach), and a few crowded values. The weights are
    no round numbers; each is rounded to 2^-40 of the largest, 2^-41 / 1e-4 of
    the smallest one here, which moves a border by at most 0.02 candidates."""
    B = 4
    l = np.zeros((B, V), np.float32)
    l[0, 17] = 6.5
    l[1, V // 2:] = -0.375
    l[1, V - 3] = 9.25
    l[2] = -3.0 + np.random.default_rng(V).integers(0, 3, V) * 2.0 ** -12
    l[2, 5] = 4.5
    l[3, V // 3] = 6.5
    u = np.array([0.9, 0.7, 0.4, 0.9], np.float32)
    check(l, u)
    check(l, u, top_p=[0.9, 0.65, 0.97, 1.0], top_k=[0, 0, 0, V - 5], min_p=[0, 0, 0, 1e-3])


@pytest.mark.parametrize("V", [300, 5000, 151936])
def test_a_min_p_below_the_weights_resolution(V):
    """min-p keeps every weight of at least min_p, also those that the sums
    round to 0: from 2^-40 down to the least positive float, with the other
    filters off and on, over values whose weights reach far below it."""
    rng = np.random.default_rng(V + 3)
    B = 10
    l = (rng.standard_normal((B, V)) * 30).astype(np.float32)
    l[8, 3] = np.inf
    l[9, rng.random(V) < 0.3] = -np.inf
    min_p = np.array([1e-12, 3e-14, 1e-15, 1e-20, 1e-30, 1e-37, 1e-40, 1.5e-45, 1e-20, 1e-20],
                     np.float32)
    assert 0 < min_p.min() < 2.0 ** -148
    u = rng.random(B).astype(np.float32)
    for k in (0, 60, V - 7):
        for p in (1.0, 0.97):
            check(l, u, top_k=np.full(B, k), top_p=np.full(B, p), min_p=min_p)
    check(l, u, temperature=np.full(B, 0.05), min_p=min_p)
    check(l, u, temperature=np.full(B, np.inf), min_p=min_p)
