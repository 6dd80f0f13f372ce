"""qg_paged_attention against the oracle (``rows_attention`` in float64 over
the exact cached values).

Tolerance of an output o = sum_t p_t v_t (u = 2^-24), from the kernels'
arithmetic (csrc/paged_attention.cu):
- a score: products are exact, their sum over D terms in the tensor core's
  fp32 (a truncating add: 2u each, gamma(2D)), three factors (scale, K scale,
  q's unit: 4u), and the terms an fp32 q is carried in (2^-21); times
  scale * sum |q k|.
- a log-weight: that, the rounding of the score and of its difference to the
  reference (2u (|s| + |m|)), its exp2 (2^-22), and one rescaling exp2
  (2^-22 and u |m| each) per move of the reference, at most range / 4 log2
  units, and two merges. It moves the output by sum p |e| |v - o|, times
  e^(2 max e) for the second order.
- the weights' rounding in the numerator alone: w_round * sum p |v|, with
  w_round 2^-11 (fp16) or 2^-8 (bf16) for one term, 2^-21 / 2^-22 for the terms
  of an fp32 output, and fp16's floor, 2^-35 max|v| a token.
- fp32 sums over L tokens: gamma(2L + 64) (sum p |v| + |o|), one division.
- the store: 2^-8 |o| for bf16."""
import math

import numpy as np
import pytest
import torch

import qg_synth
from oracle import qg_oracle as O
from tests.gpu_util import dev, host64
from tests.paged_util import Cache, bf16_bits, starts

pytestmark = pytest.mark.gpu

qg = pytest.importorskip("weight_only_quantized_03_b200")

U = O.U32


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def reference(q, k, v, H, Hkv, D, scale, kind, exact, out_bf16):
    """(value, bound) for rows q [n, H*D] over k, v [Hkv, L, D]."""
    n, L = q.shape[0], k.shape[1]
    out, tol = np.zeros((n, H, D)), np.zeros((n, H, D))
    seen = np.arange(L)[None] <= np.arange(L - n, L)[:, None]
    w_round = (2.0 ** -21 if kind == "int8" else 2.0 ** -22) if exact else (
        2.0 ** -11 if kind == "int8" else 2.0 ** -8)
    for h in range(H):
        K, V = k[h // (H // Hkv)], v[h // (H // Hkv)]
        x = q.reshape(n, H, D)[:, h]
        s = np.where(seen, x @ K.T * scale, -np.inf)
        m = s.max(1, keepdims=True)
        p = np.exp(s - m)
        p /= p.sum(1, keepdims=True)
        o = p @ V
        fin = np.where(seen, s, m)
        ds = (O.gamma(2 * D) + 4 * U + 2.0 ** -21) * scale * (np.abs(x) @ np.abs(K).T)
        rng = (m - fin.min(1, keepdims=True)) / math.log(2)
        moves = rng / 4 + 4
        e = ds + 2 * U * (np.abs(fin) + np.abs(m)) + 2.0 ** -22 + moves * (2.0 ** -22 + U * np.abs(m))
        e = np.where(seen, e, 0.0)
        pv = p @ np.abs(V)
        # sum_t p_t e_t |v_t - o| <= (p e) |V| + |o| sum p e
        move = (p * e) @ np.abs(V) + np.abs(o) * (p * e).sum(1, keepdims=True)
        tol[:, h] = (np.exp(2 * e.max(1, keepdims=True)) * move + w_round * pv
                     + L * 2.0 ** -35 * np.abs(V).max(initial=0.0)
                     + O.gamma(2 * L + 64) * (pv + np.abs(o)) + U * np.abs(o))
        out[:, h] = o
    if out_bf16:
        tol = tol + 2.0 ** -8 * np.abs(out)
    return out.reshape(n, H * D), 1.01 * tol.reshape(n, H * D)


def run(cache, n, lens, H, xt, ot, seed, scale=None, q_scale=1.0, row_start=True, pad=0):
    """(got, q, D-scaled q, kv, table): one call with junk in out and after
    the last row."""
    T, D = sum(n), cache.D
    q = qg_synth.gaussian((T, H * D), q_scale, seed)
    qv = q if xt == torch.float32 else O.bf16_bits_to_f64(bf16_bits(q))
    kv, table = cache.upload(qg)
    qd = torch.zeros((T + pad, H * D), dtype=xt, device="cuda")
    qd[:T] = torch.from_numpy(np.asarray(qv, np.float64)).to(xt).cuda()
    out = torch.full((T + pad, H * D), 55.0, dtype=ot, device="cuda")
    ws = torch.full((qg.qg_paged_attention_workspace_size(D),), 255, dtype=torch.uint8,
                    device="cuda")
    qg.qg_paged_attention(kv, table, dev(np.array(lens, np.int32)), qd, out, H,
                          1 / math.sqrt(D) if scale is None else scale, ws,
                          row_start=dev(starts(n)) if row_start else None)
    return host64(out), np.asarray(qv, np.float64)


def check(kind, D, page, H, Hkv, n, lens, xt, ot, seed, scale=None, q_scale=1.0, row_start=True,
          cap=None, pad=0):
    cache = Cache(kind, len(n), Hkv, D, page, cap or max(lens), lens, seed)
    got, q = run(cache, n, lens, H, xt, ot, seed + 1, scale, q_scale, row_start, pad)
    exact = torch.float32 in (xt, ot)
    r0 = starts(n)
    worst = 0.0
    for b in range(len(n)):
        if not n[b]:
            continue
        g = got[r0[b]:r0[b + 1]]
        k, v = cache.values(b, lens[b])
        want, tol = reference(q[r0[b]:r0[b + 1]], k, v, H, Hkv, D,
                              1 / math.sqrt(D) if scale is None else scale, kind, exact,
                              ot == torch.bfloat16)
        err = np.abs(g - want)
        assert np.all(err <= tol), (b, float((err - tol).max()), float(err.max()))
        worst = max(worst, float((err / tol).max()))
    assert np.all(got[sum(n):] == 55.0)
    return worst


BF, F32 = torch.bfloat16, torch.float32

# kind, D, page, H, Hkv, rows per sequence, lengths, q type, out type
CASES = [
    ("int8", 128, 64, 16, 8, [1], [1], BF, BF),
    ("int8", 128, 64, 16, 8, [1], [512], BF, BF),
    ("int8", 128, 64, 16, 8, [1, 1, 1], [513, 17, 16], BF, BF),
    ("int8", 128, 16, 5, 1, [1, 1], [2049, 100], BF, BF),
    ("int8", 128, 48, 8, 1, [1], [4093], F32, F32),
    ("int8", 64, 32, 16, 16, [1, 1], [1500, 3], BF, BF),
    ("int8", 64, 16, 6, 2, [1] * 5, [1, 15, 16, 17, 333], F32, BF),
    ("int8", 256, 32, 8, 2, [1, 1], [700, 31], BF, BF),
    ("int8", 256, 16, 2, 2, [3], [100], BF, F32),
    ("int8", 128, 64, 16, 1, [1, 1], [300, 5], BF, BF),       # 16 query heads a KV head
    ("int8", 128, 64, 16, 8, [4, 4, 0, 1], [200, 4, 9, 77], BF, BF),
    ("int8", 128, 64, 4, 2, [5, 30], [64, 31], BF, BF),       # 16 columns a tile
    ("int8", 128, 32, 4, 2, [5, 30], [64, 31], F32, F32),
    ("bf16", 128, 64, 16, 8, [1], [1], BF, BF),
    ("bf16", 128, 16, 16, 8, [1, 1, 1], [513, 17, 16], BF, BF),
    ("bf16", 128, 64, 8, 1, [1], [4093], F32, F32),
    ("bf16", 64, 48, 16, 16, [1, 1], [1500, 3], BF, BF),
    ("bf16", 64, 32, 6, 2, [1] * 5, [1, 15, 16, 17, 333], BF, F32),
    ("bf16", 256, 32, 8, 2, [1, 1], [700, 31], F32, BF),
    ("bf16", 256, 16, 2, 2, [3], [100], BF, BF),
    ("bf16", 128, 64, 4, 2, [5, 30], [64, 31], BF, BF),
    ("bf16", 64, 16, 3, 1, [33], [33], BF, BF),
]


@pytest.mark.parametrize("case", CASES,
                         ids=lambda c: f"{c[0]}-d{c[1]}-p{c[2]}-h{c[3]}.{c[4]}-n{c[5]}-l{c[6]}")
def test_attention(case):
    kind, D, page, H, Hkv, n, lens, xt, ot = case
    check(kind, D, page, H, Hkv, n, lens, xt, ot, 500, cap=max(lens) + 100, pad=3)


@pytest.mark.parametrize("kind,D,H,Hkv,n,lens", [
    ("int8", 128, 16, 8, [700, 1, 600], [700, 300, 900]),
    ("bf16", 128, 16, 8, [900, 0, 333], [1000, 7, 333]),
    ("int8", 64, 24, 8, [401, 402], [401, 1000]),
    ("bf16", 64, 40, 8, [250, 3], [257, 3]),
])
def test_prompt_rows(kind, D, H, Hkv, n, lens):
    """Enough columns for the kernel that gives a warp 32 of them."""
    check(kind, D, 64, H, Hkv, n, lens, BF, BF, 600, pad=5)


@pytest.mark.parametrize("kind", ["int8", "bf16"])
@pytest.mark.parametrize("q_scale", [1e-3, 30.0])
def test_flat_and_peaked_scores(kind, q_scale):
    """Nearly equal weights over a long cache, and a softmax that moves its
    maximum often and ends on one token."""
    for xt, ot in ((BF, BF), (F32, F32)):
        check(kind, 128, 64, 4, 2, [1, 2], [3000, 777], xt, ot, 700, q_scale=q_scale)


def test_one_row_each_without_row_start_many_sequences():
    lens = [1 + (37 * i) % 600 for i in range(70)]
    check("int8", 128, 64, 4, 2, [1] * 70, lens, BF, BF, 800, row_start=False)
    check("bf16", 64, 32, 2, 2, [1] * 70, lens, BF, F32, 801, row_start=False)


@pytest.mark.parametrize("kind", ["int8", "bf16"])
def test_blocks_of_very_different_scales(kind):
    """K and V scales over 40 binades: the weights' unit follows them."""
    D, Hkv, L = 128, 1, 640
    cache = Cache(kind, 1, Hkv, D, 64, L, [L], 900)
    if kind == "int8":
        rng = np.random.default_rng(1)
        cache.vs *= (2.0 ** rng.integers(-30, 10, cache.vs.shape)).astype(np.float32)
        cache.vs[cache.table[0, 3], 0, 1] = 0.0
        cache.ks *= (2.0 ** rng.integers(-6, 2, cache.ks.shape)).astype(np.float32)
    for xt, ot in ((BF, BF), (F32, F32)):
        got, q = run(cache, [1, 1][:1], [L], 2, xt, ot, 901)
        k, v = cache.values(0, L)
        want, tol = reference(q, k, v, 2, Hkv, D, 1 / math.sqrt(D), kind, F32 in (xt, ot), ot == BF)
        assert np.all(np.abs(got - want) <= tol)


def test_rows_without_keys_and_lengths_out_of_range():
    """Zero rows for a length that is 0, shorter than the rows or longer
    than the table; the others are untouched by them."""
    for kind in ("int8", "bf16"):
        cache = Cache(kind, 4, 2, 128, 64, 128, [100, 100, 100, 100], 910)
        got, q = run(cache, [1, 2, 3, 1], [0, 1, 129, 100], 4, BF, BF, 911)
        assert np.all(got[:6] == 0.0)
        k, v = cache.values(3, 100)
        want, tol = reference(q[6:], k, v, 4, 2, 128, 1 / math.sqrt(128), kind, False, True)
        assert np.all(np.abs(got[6:] - want) <= tol)


def test_bad_pages_give_nan_to_the_rows_that_see_them():
    for kind in ("int8", "bf16"):
        n, lens = [4, 1, 40], [66, 130, 90]
        cache = Cache(kind, 3, 2, 128, 64, 192, lens, 920)
        good = cache.table.copy()
        cache.table[0, 1] = cache.k.shape[0]    # tokens 64 and 65: rows 2 and 3 see them
        cache.table[1, 2] = -7                  # tokens 128, 129
        cache.table[2, 2] = -1                  # past its length: never read
        got, q = run(cache, n, lens, 4, BF, BF, 921)
        cache.table = good
        assert np.isnan(got[2:5]).all()
        for b, rows in ((0, slice(0, 2)), (2, slice(5, 45))):
            k, v = cache.values(b, lens[b])
            r0 = starts(n)
            want, tol = reference(q[r0[b]:r0[b + 1]], k, v, 4, 2, 128, 1 / math.sqrt(128), kind,
                                  False, True)
            m = rows.stop - rows.start
            assert np.all(np.abs(got[rows] - want[:m]) <= tol[:m])


@pytest.mark.parametrize("kind", ["int8", "bf16"])
@pytest.mark.parametrize("rows", [20, 1300])
def test_values_that_are_not_finite_stay_with_the_rows_that_see_them(kind, rows):
    """K and V of a later row are NaN or infinite: earlier rows are exact,
    as if they were finite."""
    D, H, Hkv = 128, 16, 8
    L = rows + 40
    cache = Cache(kind, 1, Hkv, D, 64, L, [L], 930)
    bad = L - 3 if kind == "bf16" else (L - 3) // 16 * 16  # an int8 block is NaN as a whole
    k, v = cache.values(0, L)
    p, r = cache.place(0, bad)
    if kind == "bf16":
        cache.k[p, 2, r, 5] = 0x7FC0
        cache.v[p, 4, r, 7] = 0x7F80
    else:
        cache.ks[p, 2, r // 16] = np.nan
        cache.vs[p, 4, r // 16] = np.nan
    got, q = run(cache, [rows], [L], H, BF, BF, 931)
    want, tol = reference(q, k, v, H, Hkv, D, 1 / math.sqrt(D), kind, False, True)
    first = bad - (L - rows)  # the first row that sees it
    assert 0 < first < rows
    assert np.all(np.abs(got[:first] - want[:first]) <= tol[:first])
    g = got[first:].reshape(-1, H, D)
    assert np.isnan(g[:, 4:6]).all()            # K NaN: all of KV head 2's heads
    if kind == "bf16":
        assert not np.isfinite(g[:, 8:10, 7]).any()
        ok = np.ones((H, D), bool)
        ok[4:6] = False
        ok[8:10, 7] = False
        w, t = (a[first:].reshape(-1, H, D)[:, ok] for a in (want, tol))
        assert np.all(np.abs(g[:, ok] - w) <= t)
    else:
        assert np.isnan(g[:, 8:10]).all()
        ok = [h for h in range(H) if h not in (4, 5, 8, 9)]
        w, t = (a[first:].reshape(-1, H, D)[:, ok] for a in (want, tol))
        assert np.all(np.abs(g[:, ok] - w) <= t)


def test_same_bits_each_time_on_streams_and_from_two_graphs():
    """Two captured graphs with workspaces of their own, replayed at once;
    the pages' and lengths' contents may change between replays."""
    n, lens = [1, 1, 4, 1], [700, 33, 500, 1999]
    cache = Cache("int8", 4, 2, 128, 64, 2048, lens, 940)
    kv, table = cache.upload(qg)
    T = sum(n)
    q = torch.randn((T, 4 * 128), device="cuda").bfloat16()
    ld, rs = dev(np.array(lens, np.int32)), dev(starts(n))
    outs = [torch.zeros_like(q) for _ in range(4)]
    wss = [torch.empty(qg.qg_paged_attention_workspace_size(128), dtype=torch.uint8,
                       device="cuda") for _ in range(3)]
    call = lambda i, w: qg.qg_paged_attention(kv, table, ld, q, outs[i], 4, 0.1, wss[w],
                                              row_start=rs)
    call(0, 0)
    side = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    with torch.cuda.stream(side[0]):
        call(1, 0)
    torch.cuda.synchronize()
    graphs = []
    for i in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side[i]):
            call(2 + i, 1 + i)
        graphs.append(g)
    for _ in range(3):
        for i in range(2):
            with torch.cuda.stream(side[i]):
                graphs[i].replay()
    torch.cuda.synchronize()
    for o in outs[1:]:
        assert torch.equal(o, outs[0])
    ld.copy_(dev(np.array([650, 30, 490, 1], np.int32)))
    call(0, 0)
    torch.cuda.synchronize()
    graphs[0].replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[2], outs[0]) and not torch.equal(outs[3], outs[0])


def test_a_pool_beyond_32_bit_offsets():
    """Pages whose byte offsets pass 2^32: append, gather and attend there."""
    Hkv, D, page = 8, 128, 64
    P = 70000                       # 4.6 GB of codes, K and V each
    assert P * Hkv * page * D > 1 << 32
    kv = qg.PagedKV.empty(P, page, Hkv, D)
    L = 130
    table = dev(np.array([[P - 1, 65536, P - 3]], np.int32))
    x = torch.randn((L, 2 * Hkv * D), device="cuda")
    qg.qg_paged_kv_append(kv, table, dev(np.array([L], np.int32)), x[:, :1024], x[:, 1024:],
                          row_start=dev(starts([L])), rotary_dim=0)
    k, v = (torch.empty((L, Hkv * D), device="cuda") for _ in range(2))
    qg.qg_paged_kv_gather(kv, table, None, dev(starts([L])), k, v)
    for got, want in ((k, x[:, :1024]), (v, x[:, 1024:])):
        step = torch.empty((L, Hkv), device="cuda")
        for t in range(0, L, 16):
            step[t:t + 16] = want[t:t + 16].view(-1, Hkv, D).abs().amax((0, 2)) / 127
        err = (got - want).view(L, Hkv, D).abs().amax(-1)
        assert bool((err <= step * 0.5001 + 1e-6).all())
    q = torch.randn((1, 16 * D), device="cuda").bfloat16()
    out = torch.empty_like(q)
    ws = torch.empty(qg.qg_paged_attention_workspace_size(D), dtype=torch.uint8, device="cuda")
    qg.qg_paged_attention(kv, table, dev(np.array([L], np.int32)), q, out, 16, D ** -0.5, ws)
    kh = host64(k).reshape(L, Hkv, D).transpose(1, 0, 2)
    vh = host64(v).reshape(L, Hkv, D).transpose(1, 0, 2)
    want, tol = reference(host64(q), kh, vh, 16, Hkv, D, D ** -0.5, "int8", False, True)
    # (the gathered values are rounded to fp32: u each)
    assert np.all(np.abs(host64(out) - want) <= tol + 4 * U * np.abs(vh).max())


def test_rows_of_values_that_are_not_finite():
    """Whole rows of V past the first prompt rows are infinite or NaN in more
    than half of their dims; the other dims are as if nothing had happened."""
    D, H, Hkv, rows = 128, 4, 2, 300
    L = rows + 40
    cache = Cache("bf16", 1, Hkv, D, 64, L, [L], 950)
    k, v = cache.values(0, L)
    bad = {L - 1: (0x7F80, slice(0, 100)), L - 20: (0xFF80, slice(20, 90)),
           L - 3: (0x7FC0, slice(64, 80)), 17: (0x7F80, slice(0, 1))}
    for t, (bits, dims) in bad.items():
        p, r = cache.place(0, t)
        cache.v[p, 1, r, dims] = bits
    got, q = run(cache, [rows], [L], H, BF, BF, 951)
    want, tol = reference(q, k, v, H, Hkv, D, 1 / math.sqrt(D), "bf16", False, True)
    g, w, t = (a.reshape(rows, H, D) for a in (got, want, tol))
    hit = np.zeros((rows, H, D), bool)
    for at, (_, dims) in bad.items():
        hit[max(0, at - (L - rows)):, 2:, dims] = True
    assert not np.isfinite(g[hit]).any()
    assert np.all(np.abs(g[~hit] - w[~hit]) <= t[~hit])
    # which kind: the last row sees +inf at dims 0..99, -inf at 20..89, NaN at 64..79
    last = g[-1, 2:]
    assert np.isposinf(last[:, 1:20]).all() and np.isnan(last[:, 20:90]).all()
    assert np.isposinf(last[:, 90:100]).all()
    before = g[-2, 2:]
    assert np.isneginf(before[:, 20:64]).all() and np.isnan(before[:, 64:80]).all()


@pytest.mark.parametrize("case", [
    ("int8", 128, 64, 4, 2, [40, 0, 33], [2100, 0, 35]),
    ("int8", 64, 16, 16, 1, [9, 200], [2053, 200]),
    ("bf16", 128, 32, 16, 16, [65], [1100]),
    ("bf16", 64, 16, 6, 2, [50, 1], [2113, 700]),
    ("bf16", 128, 128, 16, 1, [70, 5, 2], [1000, 5, 900]),
], ids=lambda c: f"{c[0]}-d{c[1]}-h{c[3]}.{c[4]}-n{c[5]}-l{c[6]}")
def test_few_prompt_rows_over_many_tokens(case):
    """A tile's keys shared by up to eight blocks, some of them without any."""
    kind, D, page, H, Hkv, n, lens = case
    check(kind, D, page, H, Hkv, n, lens, BF, BF, 970, cap=max(lens) + 50, pad=5)


def test_prompt_rows_of_a_wrong_length_beside_a_long_cache():
    """kv_len below the sequence's rows: zero rows, the others as they are."""
    D, H, Hkv, n = 128, 4, 2, [33, 64, 20]
    lens = [2100, 64, 2090]
    cache = Cache("int8", 3, Hkv, D, 64, 2200, lens, 980)
    got, q = run(cache, n, [2100, 10, 2090], H, BF, BF, 981)
    r0 = starts(n)
    assert np.all(got[r0[1]:r0[2]] == 0.0)
    for b in (0, 2):
        k, v = cache.values(b, lens[b])
        rows = slice(r0[b], r0[b + 1])
        want, tol = reference(q[rows], k, v, H, Hkv, D, 1 / math.sqrt(D), "int8", False, True)
        assert np.all(np.abs(got[rows] - want) <= tol)


LONG = [
    ("int8", 128, 64, 16, 8, [1, 1, 1], [513, 17, 1], BF, BF),
    ("int8", 64, 32, 6, 2, [1, 3, 0, 1], [1000, 15, 0, 129], F32, BF),
    ("int8", 256, 16, 8, 2, [1, 1], [700, 31], BF, BF),
    ("int8", 128, 64, 16, 1, [1, 1], [300, 5], BF, BF),
    ("bf16", 128, 16, 8, 1, [1], [2093], F32, F32),
    ("bf16", 64, 48, 16, 16, [1, 1], [900, 3], BF, BF),
    ("bf16", 256, 32, 8, 2, [2, 1], [700, 31], F32, BF),
    ("bf16", 128, 64, 16, 8, [1] * 40, [1 + 29 * i for i in range(40)], BF, BF),
]


@pytest.mark.parametrize("case", LONG,
                         ids=lambda c: f"{c[0]}-d{c[1]}-h{c[3]}.{c[4]}-n{len(c[5])}-l{c[6][0]}")
def test_page_tables_far_longer_than_the_sequences(case):
    """Room for 20000 tokens a sequence: the work is cut into pieces whose
    parts a second launch merges, most of them of a chunk or two."""
    kind, D, page, H, Hkv, n, lens, xt, ot = case
    cap = 20000 if len(n) < 10 else 5000
    check(kind, D, page, H, Hkv, n, lens, xt, ot, 990, cap=cap, pad=2)


@pytest.mark.parametrize("kind", ["int8", "bf16"])
def test_a_cluster_with_idle_blocks_and_empty_sequences(kind):
    """Eight blocks an item and keys for one, several and all of them; a
    sequence without rows and one of a wrong length."""
    D, H, Hkv = 128, 4, 2
    n, lens = [1, 0, 1, 1, 1], [1, 300, 130, 1000, 40]
    cache = Cache(kind, 5, Hkv, D, 64, 1000, lens, 995)
    got, q = run(cache, n, [1, 300, 130, 1000, 5000], H, BF, BF, 996)
    r0 = starts(n)
    assert np.all(got[3] == 0.0)
    for b in (0, 2, 3):
        k, v = cache.values(b, lens[b])
        rows = slice(r0[b], r0[b + 1])
        want, tol = reference(q[rows], k, v, H, Hkv, D, 1 / math.sqrt(D), kind, False, True)
        assert np.all(np.abs(got[rows] - want) <= tol)


# Room for far more tokens than there are: the tcgen05 kernel, eight blocks a
# tile, whatever the number of rows.
ROOM = 20000


@pytest.mark.parametrize("case", [
    ("int8", 128, 64, 4, 2, [40, 0, 33], [2100, 0, 35]),
    ("int8", 64, 16, 16, 1, [9, 200], [2053, 200]),
    ("int8", 128, 16, 12, 4, [1, 14, 30], [1, 300, 64]),
    ("bf16", 128, 32, 16, 16, [65], [1100]),
    ("bf16", 64, 16, 6, 2, [50, 1], [2113, 700]),
    ("bf16", 128, 128, 16, 1, [70, 5, 2], [1000, 5, 900]),
    ("int8", 128, 64, 16, 8, [5] * 40, [5 + 31 * i for i in range(40)]),
], ids=lambda c: f"{c[0]}-d{c[1]}-h{c[3]}.{c[4]}-n{c[5][:3]}-l{c[6][:3]}")
def test_prompt_rows_with_room_for_many_tokens(case):
    kind, D, page, H, Hkv, n, lens = case
    check(kind, D, page, H, Hkv, n, lens, BF, BF, 1010,
          cap=ROOM if len(n) < 10 else 6000, pad=5)


@pytest.mark.parametrize("kind", ["int8", "bf16"])
@pytest.mark.parametrize("q_scale", [1e-3, 30.0])
@pytest.mark.parametrize("room", [0, ROOM])
def test_flat_and_peaked_scores_of_prompt_rows(kind, q_scale, room):
    check(kind, 128, 64, 16, 4, [150], [1200], BF, BF, 1020, q_scale=q_scale, cap=room or 1200)


@pytest.mark.parametrize("kind", ["int8", "bf16"])
@pytest.mark.parametrize("room", [0, ROOM])
def test_prompt_rows_over_blocks_of_very_different_scales(kind, room):
    D, Hkv, L, n = 128, 2, 640, 300
    cache = Cache(kind, 1, Hkv, D, 64, room or L, [L], 1030)
    if kind == "int8":
        rng = np.random.default_rng(2)
        cache.vs *= (2.0 ** rng.integers(-30, 10, cache.vs.shape)).astype(np.float32)
        cache.vs[cache.table[0, 3], 0, 1] = 0.0
        cache.ks *= (2.0 ** rng.integers(-6, 2, cache.ks.shape)).astype(np.float32)
        cache.ks[cache.table[0, 5], 1, 2] *= -1.0
    got, q = run(cache, [n], [L], 8, BF, BF, 1031)
    k, v = cache.values(0, L)
    want, tol = reference(q, k, v, 8, Hkv, D, 1 / math.sqrt(D), kind, False, True)
    assert np.all(np.abs(got - want) <= tol)


@pytest.mark.parametrize("kind", ["int8", "bf16"])
def test_bad_pages_and_lengths_among_prompt_rows(kind):
    """Rows that see a page outside the pool are NaN, a wrong length gives
    zero rows, the others are untouched."""
    n, lens = [33, 20, 70, 9], [130, 20, 90, 40]
    cache = Cache(kind, 4, 2, 128, 64, ROOM, lens, 1040)
    good = cache.table.copy()
    cache.table[0, 2] = cache.k.shape[0]        # tokens 128 and 129: the last two rows
    cache.table[2, 2] = -1                      # past its length: never read
    got, q = run(cache, n, [130, 20, 90, 5], 8, BF, BF, 1041)
    cache.table = good
    r0 = starts(n)
    assert np.isnan(got[31:33]).all() and np.all(got[r0[3]:] == 0.0)
    for b, rows in ((0, slice(0, 31)), (1, slice(33, 53)), (2, slice(53, 123))):
        k, v = cache.values(b, lens[b])
        want, tol = reference(q[r0[b]:r0[b + 1]], k, v, 8, 2, 128, 1 / math.sqrt(128), kind, False,
                              True)
        m = rows.stop - rows.start
        assert np.all(np.abs(got[rows] - want[:m]) <= tol[:m])


@pytest.mark.parametrize("room", [0, 20000])
@pytest.mark.parametrize("xt,ot", [(BF, BF), (F32, F32), (F32, BF), (BF, F32)])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_infinite_keys_and_values_that_a_row_sees(D, xt, ot, room):
    """bf16 pages, one row: an infinite V value makes that dim infinite (NaN
    where both signs meet), whatever terms the weights are carried in; a K row
    with a score of -inf is as if it were not there, one with +inf gives NaN."""
    H, Hkv, L = 4, 2, 300
    cache = Cache("bf16", 2, Hkv, D, 64, room or L, [L, L], 1200)
    v_bad = {5: (0x7F80, [0, 3]), 130: (0xFF80, [1, 3]), 299: (0x7F80, [D - 1])}
    for t, (bits, dims) in v_bad.items():
        p, r = cache.place(0, t)
        cache.v[p, 0, r, dims] = bits
    q = qg_synth.gaussian((2, H * D), 1.0, 1201)
    qv = q if xt == F32 else O.bf16_bits_to_f64(bf16_bits(q))
    # sequence 1: token 77's score is -inf for KV head 0's first query head (and
    # the second one, by the sign it gets), token 200's NaN for KV head 1's
    sign = qv[1].reshape(H, D)
    qv = np.asarray(qv, np.float64).copy()
    qv[1].reshape(H, D)[1, 9] = abs(sign[1, 9]) * np.sign(sign[0, 9])
    p, r = cache.place(1, 77)
    cache.k[p, 0, r, 9] = 0xFF80 if sign[0, 9] > 0 else 0x7F80
    p, r = cache.place(1, 200)
    cache.k[p, 1, r, 9] = 0x7F80 if sign[2, 9] > 0 else 0xFF80
    kv, table = cache.upload(qg)
    qd = torch.from_numpy(qv).to(xt).cuda()
    out = torch.full((2, H * D), 55.0, dtype=ot, device="cuda")
    ws = torch.empty(qg.qg_paged_attention_workspace_size(D), dtype=torch.uint8, device="cuda")
    qg.qg_paged_attention(kv, table, dev(np.array([L, L], np.int32)), qd, out, H, 1 / math.sqrt(D),
                          ws)
    got, exact = host64(out).reshape(2, H, D), F32 in (xt, ot)
    args = (H, Hkv, D, 1 / math.sqrt(D), "bf16", exact, ot == BF)
    with np.errstate(invalid="ignore"):
        k, v = cache.values(0, L)
    hit = sorted({d for _, dims in v_bad.values() for d in dims})
    want, tol = reference(qv[:1], k, np.where(np.isfinite(v), v, 0.0), *args)
    keep = np.ones((H, D), bool)
    keep[:2, hit] = False
    assert np.all(np.abs(got[0] - want.reshape(H, D))[keep] <= tol.reshape(H, D)[keep])
    assert np.isposinf(got[0, :2, [0, D - 1]]).all() and np.isneginf(got[0, :2, 1]).all()
    assert np.isnan(got[0, :2, 3]).all()
    k, v = (np.delete(a, 77, 1) for a in cache.values(1, L))
    k[1] = np.where(np.isfinite(k[1]), k[1], 0.0)
    want, tol = reference(qv[1:], k, v, *args)
    assert np.all(np.abs(got[1] - want.reshape(H, D))[:2] <= tol.reshape(H, D)[:2])
    assert np.isnan(got[1, 2]).all()


@pytest.mark.parametrize("D,H,Hkv,n,lens,cap", [
    (64, 16, 16, [1, 1, 1], [1500, 300, 7], 0), (128, 16, 8, [1, 1], [700, 33], 0),
    (128, 8, 2, [1, 1], [700, 33], 20000), (256, 4, 2, [1, 2], [300, 40], 0),
    (64, 6, 2, [1, 2, 0, 1], [1000, 15, 0, 129], 20000),
])
def test_weights_of_bf16_pages_keep_16_bits(D, H, Hkv, n, lens, cap):
    """Single tokens and a few rows with bf16 q and out: a weight is cut to
    bf16 (2^-7) and its rest rounded to bf16 (2^-8 of that, at most): within
    2^-15 of it. The tolerance is that of exact weights, with sum p |v| taken from
    its difference to the one with 8 bits."""
    cache = Cache("bf16", len(n), Hkv, D, 64, cap or max(lens), lens, 1210)
    got, q = run(cache, n, lens, H, BF, BF, 1211)
    r0 = starts(n)
    for b in range(len(n)):
        if not n[b]:
            continue
        rows = slice(r0[b], r0[b + 1])
        k, v = cache.values(b, lens[b])
        args = (q[rows], k, v, H, Hkv, D, 1 / math.sqrt(D), "bf16")
        want, tol = reference(*args, True, True)
        pv = (reference(*args, False, True)[1] - tol) / (1.01 * (2.0 ** -8 - 2.0 ** -22))
        err = np.abs(got[rows] - want)
        assert np.all(err <= tol + 2.0 ** -15 * pv), (b, float((err - tol).max()))


@pytest.mark.parametrize("case", [
    ("int8", 128, 64, 16, 8, [100, 37, 1, 0, 250], [400, 37, 290, 5, 250], F32, F32, 0),
    ("bf16", 128, 64, 16, 8, [100, 37, 1, 0, 250], [400, 37, 290, 5, 250], F32, F32, 0),
    ("int8", 64, 32, 12, 4, [130, 7, 300], [500, 900, 300], F32, BF, 0),
    ("bf16", 64, 16, 6, 2, [200, 150], [200, 620], BF, F32, 0),
    ("int8", 256, 32, 8, 2, [90, 3, 110], [200, 333, 110], BF, BF, 0),
    ("bf16", 256, 64, 4, 2, [70, 140], [300, 140], F32, F32, 0),
    ("int8", 128, 64, 4, 1, [60] * 5, [60 + 75 * i for i in range(5)], F32, F32, 20000),
    ("bf16", 128, 128, 4, 2, [45, 0, 210], [700, 3, 210], F32, BF, 20000),
], ids=lambda c: f"{c[0]}-d{c[1]}-h{c[3]}.{c[4]}-n{c[5][:3]}-room{c[9]}")
def test_hundreds_of_rows_in_fp32_or_with_wide_heads(case):
    """What the prompt kernel does not take, in hundreds of rows: many items a
    piece of the line, cuts inside items and before their first chunk."""
    kind, D, page, H, Hkv, n, lens, xt, ot, room = case
    check(kind, D, page, H, Hkv, n, lens, xt, ot, 1220, cap=room or max(lens), pad=3)


@pytest.mark.parametrize("xt,ot", [(BF, BF), (F32, F32)])
@pytest.mark.parametrize("lens", [[1], [16], [128], [129], [1, 128, 1, 129, 2, 127],
                                  [46 + i for i in range(25)], [257] * 40, [3000, 1, 1, 1]],
                         ids=lambda l: f"{len(l)}x{l[0]}")
def test_cuts_of_the_line(lens, xt, ot):
    """Room for 20000 tokens, so that the line is cut: items of one chunk and
    of the least and the most tokens of one, pieces of a single unit, pieces
    that begin or end in an item's part that stands for no chunk."""
    for n in (1, 2):
        rows = [min(n, x) for x in lens]
        check("int8", 64, 64, 4, 2, rows, lens, xt, ot, 1230, cap=20000)
