"""qg_paged_kv_append and qg_paged_kv_gather against the oracle.

Tolerances, per value, with u = 2^-24 (include/qg.h states the arithmetic):
the normed and rotated row x is a float32 chain; its error e is the norm's
relative bound (``rmsnorm_rel_bound``) and three roundings on |a cos| + |b
sin|, and 2^-22 (|a| + |b|) for the sine and cosine (the reduced angle is
rounded to float32: at most pi 2^-25, sincospi: 2 ulp). A bf16 store is the
rounding of a value within e. An int8 block's scale is max|x| / 127 within
max(e) / 127 and one rounding; x / s is then within
e / s + |x / s| (max(e) / max|x| + 3 u), and its code within half a step
more. A requantised code is within half a step and 127 times the scales'
relative error."""
import numpy as np
import pytest
import torch

import qg_synth
from oracle import qg_oracle as O
from tests.gpu_util import bf16_dev, dev, host64
from tests.paged_util import BLOCK, Cache, bf16_bits, starts

pytestmark = pytest.mark.gpu

qg = pytest.importorskip("weight_only_quantized_03_b200")

U = O.U32
EPS, THETA = 1e-6, 1e6


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def turned(x, w_bits, pos, D, rd):
    """(value, bound) of the norm (w_bits or None) and rotation of x [heads*D]."""
    n = x if w_bits is None else O.rmsnorm_perhead(x, w_bits, EPS, D)
    rho = 0.0 if w_bits is None else O.rmsnorm_rel_bound(D)
    v = O.rope_neox(n, pos, THETA, D, rd) if rd else n
    h = np.abs(n).reshape(-1, D)
    e = rho * h
    if rd:
        half = rd // 2
        a = pos * O.rope_inv_freq(THETA, rd)
        c, s = np.abs(np.cos(a)), np.abs(np.sin(a))
        lo, hi = h[:, :half], h[:, half:rd]
        sc = 2.0 ** -22 * (lo + hi)
        e[:, :half] = (rho + O.gamma(4)) * (lo * c + hi * s) + sc
        e[:, half:rd] = (rho + O.gamma(4)) * (hi * c + lo * s) + sc
    return v, 1.01 * e.reshape(v.shape)


def check_append(cache, kv, n, lens, k, v, k_norm, rd, dropped=()):
    """The device pool against the host pool with the rows appended."""
    got = cache.download(kv)
    D, Hkv = cache.D, cache.Hkv
    r0 = starts(n)
    for which, (rows, w, pages, scales) in enumerate(
            ((k, k_norm, cache.k, cache.ks), (v, None, cache.v, cache.vs))):
        g_pages, g_scales = got[2 * which], got[2 * which + 1]
        same = np.ones(pages.shape[:3], bool)  # rows that must be as they were
        if scales is not None:
            same_s = np.ones(scales.shape, bool)
        for b in range(cache.B):
            if b in dropped or not n[b]:
                continue
            x = np.zeros((n[b], Hkv, D))
            e = np.zeros((n[b], Hkv, D))
            p0 = lens[b] - n[b]
            for i in range(n[b]):
                a = rows[r0[b] + i]
                val, err = turned(a, w, p0 + i, D, rd) if which == 0 else (a, np.zeros_like(a))
                x[i], e[i] = val.reshape(Hkv, D), err.reshape(Hkv, D)
            for t0 in range(p0 // BLOCK * BLOCK, lens[b], BLOCK):
                lo, hi = max(t0, p0), min(t0 + BLOCK, lens[b])
                p, r = cache.place(b, t0)
                o = lo - t0
                xs, es = x[lo - p0:hi - p0], e[lo - p0:hi - p0]
                if scales is None:
                    same[p, :, r + o:r + hi - t0] = False
                    g = O.bf16_bits_to_f64(g_pages[p, :, r + o:r + hi - t0]).transpose(1, 0, 2)
                    assert np.all(O.bf16_rounding_ok(xs, g, 0.0, es)), (which, b, t0)
                    continue
                same[p, :, r:r + hi - t0] = False
                same_s[p, :, r // BLOCK] = False
                for h in range(Hkv):
                    s_old = float(scales[p, h, r // BLOCK])
                    codes, s = O.kv_block_append(pages[p, h, r:r + BLOCK], s_old, o, xs[:, h])
                    g, gs = g_pages[p, h, r:r + BLOCK].astype(float), float(g_scales[p, h, r // BLOCK])
                    if np.isnan(s):
                        assert np.isnan(gs)
                        continue
                    top, etop = np.abs(xs[:, h]).max(), es[:, h].max()
                    assert abs(gs - s) <= etop / 127 + 2 * U * s + 2.0 ** -149, (which, b, t0, h)
                    if s == 0:
                        assert not g[:hi - t0].any()
                        continue
                    rel = etop / (127 * s) + 3 * U  # of the scale, and the quotient's rounding
                    want = np.clip(xs[:, h] / s, -127, 127)
                    tol = 0.5 + es[:, h] / s + np.abs(want) * rel
                    assert np.all(np.abs(g[o:hi - t0] - want) <= tol), (which, b, t0, h)
                    if o and gs != s_old:
                        want = pages[p, h, r:r + o] * (s_old / s)
                        assert np.all(np.abs(g[:o] - want) <= 0.5 + 127 * 2 * rel), (which, b, t0)
                    elif o:
                        assert np.array_equal(g[:o], pages[p, h, r:r + o])
        assert np.array_equal(g_pages[same_of(same, g_pages)], pages[same_of(same, pages)])
        if scales is not None:
            np.testing.assert_array_equal(g_scales[same_s], scales[same_s])


def same_of(mask, a):
    return np.broadcast_to(mask[..., None], a.shape)


# kind, x type, D, page, H, Hkv, norm, rotary_dim, rows per sequence, lengths
CASES = [
    ("int8", "f32", 128, 64, 16, 8, True, 128, [1], [1]),
    ("int8", "f32", 128, 64, 16, 8, True, 128, [1, 1, 1], [512, 33, 16]),
    ("int8", "bf16", 128, 16, 4, 2, False, 128, [17, 0, 31, 1, 5], [17, 0, 100, 1, 20]),
    ("int8", "f32", 64, 48, 3, 3, True, 32, [2, 16, 33], [47, 31, 50]),
    ("int8", "bf16", 256, 32, 2, 1, True, 64, [19, 3], [40, 3]),
    ("int8", "f32", 64, 16, 5, 1, False, 0, [40], [41]),
    ("bf16", "f32", 128, 64, 16, 8, True, 128, [1, 1], [200, 64]),
    ("bf16", "bf16", 64, 32, 2, 2, False, 64, [20, 1, 0, 70], [51, 33, 9, 70]),
    ("bf16", "f32", 256, 16, 3, 1, True, 256, [18], [30]),
    ("bf16", "bf16", 128, 128, 0, 4, True, 8, [5, 6], [5, 140]),
]


def _inputs(case, seed):
    kind, xt, D, page, H, Hkv, norm, rd, n, lens = case
    B, T = len(n), sum(n)
    cache = Cache(kind, B, Hkv, D, page, max(lens) + page, np.array(lens) - n, seed)
    x = qg_synth.gaussian((T + 3, (H + 2 * Hkv) * D), 1.5, seed + 1)
    xb = x if xt == "f32" else O.bf16_bits_to_f64(bf16_bits(x))
    w = [bf16_bits(1 + 0.2 * qg_synth.gaussian((D,), 1.0, seed + 2 + i)) if norm else None
         for i in range(2)]
    return cache, np.asarray(xb, np.float64), w


@pytest.mark.parametrize("case", CASES, ids=lambda c: f"{c[0]}-{c[1]}-d{c[2]}-p{c[3]}-{c[8]}")
def test_append(case):
    kind, xt, D, page, H, Hkv, norm, rd, n, lens = case
    cache, x, w = _inputs(case, 100)
    T, W = sum(n), Hkv * D
    xd = torch.from_numpy(x).to(torch.float32 if xt == "f32" else torch.bfloat16).cuda()
    # q, k, v are slices of one projection's rows; three padding rows follow
    q, k, v = xd.split((H * D, W, W), 1)
    kv, table = cache.upload(qg)
    wd = [None if a is None else bf16_dev(a) for a in w]
    for qt in (torch.bfloat16, torch.float32):
        kv, table = cache.upload(qg)
        q_out = torch.full((T + 3, H * D), 77.0, dtype=qt, device="cuda")
        qg.qg_paged_kv_append(kv, table, dev(np.array(lens, np.int32)), k, v,
                              row_start=dev(starts(n)), q=q if H else None,
                              q_out=q_out if H else None, q_norm=wd[0], k_norm=wd[1], eps=EPS,
                              theta=THETA, rotary_dim=rd)
        check_append(cache, kv, n, lens, x[:, H * D:H * D + W], x[:, H * D + W:], w[1], rd)
        got, r0 = host64(q_out), starts(n)
        for b in range(len(n)):
            for i in range(n[b]):
                val, err = turned(x[r0[b] + i, :H * D], w[0], lens[b] - n[b] + i, D, rd)
                g = got[r0[b] + i]
                if qt == torch.float32:
                    assert np.all(np.abs(g - val) <= err + U * np.abs(val))
                else:
                    assert np.all(O.bf16_rounding_ok(val, g, 0.0, err))
        assert np.all(got[T:] == 77.0)


@pytest.mark.parametrize("kind", ["int8", "bf16"])
def test_append_one_row_each_without_row_start_and_in_place(kind):
    case = (kind, "f32", 128, 32, 4, 2, True, 128, [1] * 40, [1 + 7 * i for i in range(40)])
    cache, x, w = _inputs(case, 200)
    kv, table = cache.upload(qg)
    x = x[:40]
    q, k, v = (torch.from_numpy(a.copy()).float().cuda()
               for a in np.split(x, (4 * 128, 6 * 128), 1))
    lens = np.array(case[9], np.int32)
    want = torch.empty_like(q)
    wd = [bf16_dev(a) for a in w]
    kv2, _ = cache.upload(qg)
    qg.qg_paged_kv_append(kv2, table, dev(lens), k, v, q=q, q_out=want, q_norm=wd[0], k_norm=wd[1])
    qg.qg_paged_kv_append(kv, table, dev(lens), k, v, q=q, q_out=q, q_norm=wd[0], k_norm=wd[1])
    check_append(cache, kv, [1] * 40, case[9], x[:, 512:768], x[:, 768:], w[1], 128)
    assert torch.equal(q, want)
    # again on the same state: the rows are what they were
    qg.qg_paged_kv_append(kv2, table, dev(lens), k, v, q=want.clone(), q_out=want, q_norm=wd[0],
                          k_norm=wd[1])
    for a, b in zip(cache.download(kv), cache.download(kv2)):
        np.testing.assert_array_equal(a, b)


def test_append_far_positions_keep_their_angle():
    """Position 2^20 - 1: the reduction of the angle keeps fp32 accuracy."""
    D, page, L = 64, 65536, 1 << 20
    cache = Cache("bf16", 1, 1, D, page, page, [0], 7)
    cache.max_pages = L // page
    cache.table = np.zeros((1, cache.max_pages), np.int32) + 1
    kv, table = cache.upload(qg)
    x = qg_synth.gaussian((1, 2 * D), 1.0, 8).astype(np.float64)
    xd = torch.from_numpy(x).float().cuda()
    qg.qg_paged_kv_append(kv, table, dev(np.array([L], np.int32)), xd[:, :D], xd[:, D:])
    val, err = turned(x[0, :D], None, L - 1, D, D)
    got = O.bf16_bits_to_f64(cache.download(kv)[0][1, 0, page - 1])
    assert np.all(O.bf16_rounding_ok(val, got, 0.0, err))


def test_append_values_that_are_not_finite():
    """They poison their block's scale and no other block."""
    D, Hkv = 64, 2
    cache = Cache("int8", 1, Hkv, D, 64, 64, [3], 9)
    x = np.array(qg_synth.gaussian((37, 2 * Hkv * D), 1.0, 10), np.float64)
    x[20, 5] = np.inf          # k, head 0, token 23: block 1
    x[36, Hkv * D + 70] = np.nan  # v, head 1, token 39: block 2
    kv, table = cache.upload(qg)
    xd = torch.from_numpy(x).float().cuda()
    qg.qg_paged_kv_append(kv, table, dev(np.array([40], np.int32)), xd[:, :128], xd[:, 128:],
                          row_start=dev(starts([37])), rotary_dim=0)
    check_append(cache, kv, [37], [40], x[:, :128], x[:, 128:], None, 0)
    k, v = (torch.empty((48, 128), device="cuda") for _ in range(2))
    qg.qg_paged_kv_gather(kv, table, None, dev(starts([48])), k, v)
    k, v = host64(k), host64(v)
    assert np.isnan(k[16:32, :64]).all() and not np.isnan(k[:16]).any()
    assert not np.isnan(k[16:40, 64:]).any()
    assert np.isnan(v[32:, 64:]).all() and not np.isnan(v[:32]).any()


def test_append_drops_bad_pages_and_bad_lengths():
    case = ("int8", "f32", 64, 16, 2, 1, False, 64, [4, 4, 4, 4], [20, 40, 20, 20])
    cache, x, _ = _inputs(case, 300)
    P = cache.k.shape[0]
    cache.table[0, 1] = P        # tokens 16..19 of sequence 0
    cache.table[2, 1] = -1
    kv, table = cache.upload(qg)
    xd = torch.from_numpy(x).float().cuda()
    q_out = torch.full((19, 128), 77.0, device="cuda")
    over = cache.max_pages * cache.page + 1
    lens = [20, over, 20, 3]     # sequence 1 beyond its table, sequence 3 shorter than its rows
    qg.qg_paged_kv_append(kv, table, dev(np.array(lens, np.int32)), xd[:, 128:192], xd[:, 192:],
                          row_start=dev(starts(case[8])), q=xd[:, :128], q_out=q_out)
    check_append(cache, kv, case[8], case[9], x[:, 128:192], x[:, 192:], None, 64,
                 dropped=(0, 1, 2, 3))
    got = host64(q_out)
    assert np.all(got[4:8] == 77) and np.all(got[12:] == 77)
    assert not np.any(got[:4] == 77) and not np.any(got[8:12] == 77)


@pytest.mark.parametrize("kind,D,page,dt", [("int8", 128, 64, "bf16"), ("int8", 64, 16, "f32"),
                                            ("bf16", 256, 32, "bf16"), ("bf16", 64, 48, "f32")])
def test_gather(kind, D, page, dt):
    lens = [70, 1, 0, 33]
    cache = Cache(kind, 4, 3, D, page, 96, lens, 11)
    kv, table = cache.upload(qg)
    first, n = [5, 0, 0, 32], [65, 1, 0, 1]
    tt = torch.float32 if dt == "f32" else torch.bfloat16
    k, v = (torch.full((70, 3 * D), 55.0, dtype=tt, device="cuda") for _ in range(2))
    qg.qg_paged_kv_gather(kv, table, dev(np.array(first, np.int32)), dev(starts(n)), k, v)
    r0 = starts(n)
    for got, which in ((host64(k), 0), (host64(v), 1)):
        for b in range(4):
            want = cache.values(b, lens[b])[which][:, first[b]:first[b] + n[b]]
            want = want.transpose(1, 0, 2).reshape(n[b], 3 * D)
            g = got[r0[b]:r0[b + 1]]
            if dt == "bf16":
                assert np.all(O.bf16_rounding_ok(want, g, 2 * U))
            else:
                assert np.all(np.abs(g - want) <= U * np.abs(want))
        assert np.all(got[67:] == 55.0)
    # one row each, K alone; a token beyond the table and a bad page give NaN
    cache.table[1, 0] = -5
    kv, table = cache.upload(qg)
    k = torch.zeros((4, 3 * D), dtype=tt, device="cuda")
    qg.qg_paged_kv_gather(kv, table, dev(np.array([0, 0, 1 << 30, -1], np.int32)), None, k)
    got = host64(k)
    assert not np.isnan(got[0]).any() and np.isnan(got[1:]).all()


def test_append_on_a_side_stream_and_captured():
    """Same bits eagerly, on another stream and from a replayed graph."""
    case = ("int8", "bf16", 128, 64, 4, 2, True, 128, [3, 1, 30], [50, 1, 64])
    cache, x, w = _inputs(case, 400)
    lens, rs = dev(np.array(case[9], np.int32)), dev(starts(case[8]))
    xd = torch.from_numpy(x).bfloat16().cuda()
    q, k, v = xd.split((512, 256, 256), 1)
    wd = [bf16_dev(a) for a in w]

    def call(kv, table, out):
        qg.qg_paged_kv_append(kv, table, lens, k, v, row_start=rs, q=q, q_out=out, q_norm=wd[0],
                              k_norm=wd[1])

    outs, pools = [], []
    for how in range(3):
        kv, table = cache.upload(qg)
        out = torch.zeros((37, 512), dtype=torch.bfloat16, device="cuda")
        side = torch.cuda.Stream()
        torch.cuda.synchronize()
        if how == 0:
            call(kv, table, out)
        elif how == 1:
            with torch.cuda.stream(side):
                call(kv, table, out)
        else:
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=side):
                call(kv, table, out)
            g.replay()
        torch.cuda.synchronize()
        outs.append(out)
        pools.append(cache.download(kv))
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])
    for a, b, c in zip(*pools):
        np.testing.assert_array_equal(a, b)
        np.testing.assert_array_equal(a, c)


@pytest.mark.parametrize("kind", ["int8", "bf16"])
def test_append_of_prompts_in_place_and_apart_are_the_same(kind):
    """q rotated onto itself, K and V slices of one projection: the same bits
    as from tensors of their own, whole blocks and their ends."""
    D, H, Hkv, page = 128, 6, 2, 32
    n, before = [37, 0, 3, 16], [5, 9, 30, 0]
    T, B = sum(n), len(n)
    g = torch.Generator(device="cuda").manual_seed(77)
    dt = torch.int8 if kind == "int8" else torch.bfloat16
    x = torch.randn((T, (H + 2 * Hkv) * D), generator=g, device="cuda").bfloat16()
    w = [(1 + 0.1 * torch.randn(D, generator=g, device="cuda")).bfloat16() for _ in range(2)]
    table = torch.randperm(B * 4, generator=g, device="cuda").view(B, 4).int()
    lens = dev(np.array([a + b for a, b in zip(n, before)], np.int32))
    rs = dev(starts(n))
    got = []
    for apart in (False, True):
        kv = qg.PagedKV.empty(B * 4, page, Hkv, D, dt)
        for t in (kv.k_pages, kv.v_pages, kv.k_scales, kv.v_scales):
            if t is not None:
                t.zero_()
        q, k, v = x.split((H * D, Hkv * D, Hkv * D), 1)
        q = q.contiguous()
        out = torch.zeros_like(q) if apart else q
        if apart:
            k, v = k.contiguous(), v.contiguous()
        qg.qg_paged_kv_append(kv, table, lens, k, v, row_start=rs, q=q, q_out=out, q_norm=w[0],
                              k_norm=w[1], theta=1e4, rotary_dim=96)
        torch.cuda.synchronize()
        got.append([out] + [t for t in (kv.k_pages, kv.v_pages, kv.k_scales, kv.v_scales)
                            if t is not None])
    assert all(torch.equal(a, b) for a, b in zip(*got))
    assert got[0][0].abs().max() > 0 and got[0][1].float().abs().max() > 0


def _matching_sequences(rs, T):
    """Sequences whose range of block slots holds a slot, by the rule of
    csrc/paged_kv.cu: {slot: [(first row, rows), ...]} where it is several."""
    c = [min(max(r, 0), T) for r in rs]
    out = {}
    for u in range(T // BLOCK + 2 * (len(rs) - 1)):
        m = [(c[i], c[i + 1] - c[i]) for i in range(len(rs) - 1)
             if c[i] // BLOCK + 2 * i <= u < c[i + 1] // BLOCK + 2 * (i + 1)]
        if len(m) > 1:
            out[u] = m
    return out


@pytest.mark.parametrize("kind", ["int8", "bf16"])
def test_append_with_row_starts_that_decrease_stays_within_its_rows(kind):
    """Slots that two sequences claim: a mix of one's first row and the
    other's rows would reach past the call's rows."""
    T, rs = 200, [0, 200, 50, 60, 190, 200]
    claims = _matching_sequences(rs, T)
    assert max(r + n for m in claims.values() for r, _ in m for _, n in m) > T
    D, Hkv, H, page, B = 64, 2, 2, 32, 5
    cache = Cache(kind, B, Hkv, D, page, 256, [0] * B, 500)
    kv, table = cache.upload(qg)
    x = torch.randn((2 * T, (H + 2 * Hkv) * D), device="cuda")
    q, k, v = (a[:T] for a in x.split((H * D, Hkv * D, Hkv * D), 1))
    out = torch.full((2 * T, H * D), 77.0, device="cuda")
    lens = dev(np.array([200, 10, 10, 130, 10], np.int32))
    qg.qg_paged_kv_append(kv, table, lens, k, v, row_start=dev(np.array(rs, np.int32)), q=q,
                          q_out=out[:T])
    torch.cuda.synchronize()
    assert bool((out[T:] == 77.0).all())
    assert not bool(torch.isnan(out).any())
    # the pages of nobody (two spare ones) are as they were
    spare = np.setdiff1d(np.arange(cache.k.shape[0]), cache.table)
    got = cache.download(kv)
    np.testing.assert_array_equal(got[0][spare], cache.k[spare])
    np.testing.assert_array_equal(got[2][spare], cache.v[spare])


def _codes32(codes, s_old, o, x):
    """kv_block_append as include/qg.h states it in fp32: (codes, scale) of a
    block [16, D] after rows x (fp32 values) at place o."""
    f = np.float32
    codes, s_old = codes.copy(), f(s_old) if o else f(0)
    s = max(s_old, np.abs(x).max() / f(127))
    s = s if s >= f(2.0 ** -126) else f(0)
    n = len(x)
    if s == 0:
        codes[:o + n] = 0
        return codes, s
    if s != s_old:
        codes[:o] = np.rint(codes[:o].astype(f) * (s_old / s))
    codes[o:o + n] = np.clip(np.rint(x / s), -127, 127)
    return codes, s


@pytest.mark.parametrize("xt", ["f32", "bf16"])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_append_codes_are_the_fp32_quotients(xt, D):
    """Without norm and rotation every step is one fp32 operation, so codes
    and scales are equal, also where x / s lies at a tie between two codes or
    next to one: half the largest value and other odd multiples of s / 2."""
    Hkv, page, n = 3, 32, [40, 1, 16, 9, 8, 5, 3]
    lens = [45, 1, 16, 25, 31, 37, 8]
    dt = torch.float32 if xt == "f32" else torch.bfloat16
    f32 = lambda a: torch.from_numpy(a).to(dt).float().numpy()
    rng = np.random.default_rng(D)
    cache = Cache("int8", len(n), Hkv, D, page, 64, np.array(lens) - n, 600)
    cache.ks *= np.float32(0.3)
    x = f32(rng.standard_normal((sum(n), 2 * Hkv, D)).astype(np.float32) * 1.5)
    # near ties: (k + 1/2) s for the scale of a row's own largest value
    s = np.abs(x).max(-1, keepdims=True) / np.float32(127)
    k = rng.integers(-127, 127, x.shape).astype(np.float32) + np.float32(0.5)
    near = f32(k * s) if xt == "f32" else f32(np.sign(k) * np.abs(x).max(-1, keepdims=True) / 2)
    near = np.nextafter(near, np.float32(9) * rng.integers(-1, 2, x.shape).astype(np.float32)) \
        if xt == "f32" else near
    x = np.where((rng.random(x.shape) < 0.5) & (np.abs(near) < np.abs(x).max(-1, keepdims=True)),
                 near, x).astype(np.float32)
    kv, table = cache.upload(qg)
    xd = torch.from_numpy(x.reshape(sum(n), -1)).to(dt).cuda()
    qg.qg_paged_kv_append(kv, table, dev(np.array(lens, np.int32)), xd[:, :Hkv * D],
                          xd[:, Hkv * D:], row_start=dev(starts(n)), rotary_dim=0)
    got, r0 = cache.download(kv), starts(n)
    ties = 0
    for which, (pages, scales) in enumerate(((cache.k, cache.ks), (cache.v, cache.vs))):
        for b in range(len(n)):
            p0 = lens[b] - n[b]
            rows = x[r0[b]:r0[b + 1], which * Hkv:(which + 1) * Hkv]
            for t0 in range(p0 // BLOCK * BLOCK, lens[b], BLOCK):
                lo, hi = max(t0, p0), min(t0 + BLOCK, lens[b])
                p, r = cache.place(b, t0)
                for h in range(Hkv):
                    want, s = _codes32(pages[p, h, r:r + BLOCK], scales[p, h, r // BLOCK],
                                       lo - t0, rows[lo - p0:hi - p0, h])
                    q = rows[lo - p0:hi - p0, h] / s
                    ties += int((np.abs(np.abs(q - np.rint(q)) - 0.5) < 1e-4).sum())
                    assert got[2 * which + 1][p, h, r // BLOCK] == s, (which, b, t0, h)
                    np.testing.assert_array_equal(got[2 * which][p, h, r:hi - t0 + r],
                                                  want[:hi - t0], err_msg=str((which, b, t0, h)))
    assert ties > 20


@pytest.mark.parametrize("which", ["q_norm", "k_norm"])
def test_append_refuses_norm_weights_of_another_type(which):
    """A refused call leaves the cache as it was; bf16 bits as int16 are the
    same weights."""
    D = 64
    cache = Cache("int8", 1, 1, D, 16, 16, [3], 700)
    kv, table = cache.upload(qg)
    x = torch.randn((1, 3 * D), device="cuda")
    w = (1 + 0.1 * torch.randn(D, device="cuda"))
    lens, out = dev(np.array([4], np.int32)), torch.zeros((1, D), device="cuda")
    call = lambda w: qg.qg_paged_kv_append(kv, table, lens, x[:, D:2 * D], x[:, 2 * D:],
                                           q=x[:, :D], q_out=out, **{which: w})
    for bad in (w.half(), w, w[:32].bfloat16()):
        with pytest.raises(ValueError, match="64 bf16 values"):
            call(bad)
    for a, b in zip(cache.download(kv), (cache.k, cache.ks, cache.v, cache.vs)):
        np.testing.assert_array_equal(a, b)
    call(w.bfloat16())
    first = [out.clone()] + [torch.from_numpy(a) for a in cache.download(kv)]
    kv, _ = cache.upload(qg)
    call(w.bfloat16().view(torch.int16))
    again = [out] + [torch.from_numpy(a) for a in cache.download(kv)]
    assert all(torch.equal(a.cpu().nan_to_num(7.5), b.cpu().nan_to_num(7.5))
               if a.is_floating_point() else torch.equal(a, b) for a, b in zip(first, again))
