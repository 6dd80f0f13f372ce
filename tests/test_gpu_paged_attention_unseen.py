"""qg_paged_attention on int8 pages: what a row does not see (later blocks,
their scales, the padding behind the last token) must not reach it, and scales
of 0 and very small ones keep their bits. Rows go to the prompt kernel with one
CTA a tile (many KV heads) and with clusters (room for many tokens), and few
rows to the other kernels.

Tolerance: ``test_gpu_paged_attention.reference`` over the tokens that the rows
of a check see, so that its terms in max|V| are theirs; and 2^-134, half of bf16's
step below 2^-126 (its least numbers are multiples of 2^-133), which rounding by
2^-8 |o| does not count."""
import math

import numpy as np
import pytest
import torch

import qg_synth
from oracle import qg_oracle as O
from tests.gpu_util import dev, host64
from tests.paged_util import Cache, bf16_bits, starts
from tests.test_gpu_paged_attention import ROOM, reference

pytestmark = pytest.mark.gpu

qg = pytest.importorskip("weight_only_quantized_03_b200")

BF = torch.bfloat16
# query and KV heads, room for tokens: tiles of 128 rows, of 64 rows, clusters
FORMS = [(8, 8, 0), (16, 8, 0), (2, 2, ROOM), (4, 2, ROOM)]


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def attend(cache, q, n, lens, H, scale):
    """(out, q as bf16) of the rows q."""
    D = cache.D
    q = O.bf16_bits_to_f64(bf16_bits(q))
    kv, table = cache.upload(qg)
    qd = torch.from_numpy(q).to(BF).cuda()
    out = torch.full_like(qd, 55.0)
    ws = torch.empty(qg.qg_paged_attention_workspace_size(D), dtype=torch.uint8, device="cuda")
    qg.qg_paged_attention(kv, table, dev(np.array(lens, np.int32)), qd, out, H, scale, ws,
                          row_start=dev(starts(n)))
    return host64(out), q


def check(cache, got, q, n, lens, H, scale, splits=()):
    """Rows of each sequence against the oracle; `splits`: tokens at which a
    sequence's rows are checked apart, by what they see."""
    r0 = starts(n)
    for b in range(len(n)):
        k, v = cache.values(b, lens[b])
        first = lens[b] - n[b]  # the first row's token
        ends = [t for t in splits if first < t < lens[b]] + [lens[b]]
        at = first
        for end in ends:
            rows = slice(r0[b] + at - first, r0[b] + end - first)
            want, tol = reference(q[rows], k[:, :end], v[:, :end], H, cache.Hkv, cache.D, scale,
                                  "int8", False, True)
            err, tol = np.abs(got[rows] - want), tol + 2.0 ** -134
            assert np.all(err <= tol), (b, at, end, float((err / tol).max()))
            at = end


def _rows(H, D, T, seed):
    return qg_synth.gaussian((T, H * D), 1.0, seed)


@pytest.mark.parametrize("small", [0.0, 2.0 ** -126, 1e-30])
@pytest.mark.parametrize("H,Hkv,room", FORMS)
def test_a_block_of_small_keys_that_rows_do_not_see(H, Hkv, room, small):
    """Blocks of K with scale 0 (what an append of zeros stores) or a very
    small one, behind rows whose own scores lie far below 0: their softmax
    goes by the scores that they see."""
    D, L = 128, 300
    cache = Cache("int8", 1, Hkv, D, 64, room or L, [L], 1100)
    cache.k = np.where(cache.k < 0, cache.k, -1 - np.maximum(cache.k, 0).clip(0, 126)).astype(np.int8)
    blocks = [2, 6, 11, 13, 17]
    for j in blocks:
        p, r = cache.place(0, 16 * j)
        if small == 0.0:
            cache.k[p, :, r:r + 16] = 0
        cache.ks[p, :, r // 16] = small
    q = np.abs(_rows(H, D, L, 1101)) * 3.0
    got, q = attend(cache, q, [L], [L], H, 0.5)
    check(cache, got, q, [L], [L], H, 0.5, splits=[16 * j for j in blocks])


@pytest.mark.parametrize("v_scale", [1e-6, 1e-9, 1e-13])
@pytest.mark.parametrize("H,Hkv,room", FORMS)
def test_small_values_with_lengths_that_end_inside_a_step(H, Hkv, room, v_scale):
    """What lies behind the last token does not set the unit of V."""
    D = 128
    lens = [17, 1, 65, 70, 33, 130, 48, 200] * (3 if not room else 1)
    n = [x if i % 3 else min(x, 20) for i, x in enumerate(lens)]
    cache = Cache("int8", len(n), Hkv, D, 64, room or 200, lens, 1110)
    cache.vs *= np.float32(v_scale)
    q = _rows(H, D, sum(n), 1111)
    got, q = attend(cache, q, n, lens, H, 1 / math.sqrt(D))
    assert np.abs(got).max() > 0
    check(cache, got, q, n, lens, H, 1 / math.sqrt(D))


@pytest.mark.parametrize("H,Hkv,room", FORMS)
@pytest.mark.parametrize("v_scale", [1.0, 2.0 ** -116])
def test_values_of_zero(H, Hkv, room, v_scale):
    """Blocks of V with scale 0: the first ones (a whole step, and more than
    one), every block of a head, and the last ones; the others with ordinary and
    with the smallest scales."""
    D, L = 128, 300
    cache = Cache("int8", 1, Hkv, D, 64, room or L, [L], 1120)
    cache.vs *= np.float32(v_scale)
    for h, (lo, hi) in ((0, (0, 80)), (1, (0, 304))):
        for t in range(lo, min(hi, L), 16):
            p, r = cache.place(0, t)
            cache.v[p, h, r:r + 16] = 0
            cache.vs[p, h, r // 16] = 0.0
    q = _rows(H, D, L, 1121)
    got, q = attend(cache, q, [L], [L], H, 1 / math.sqrt(D))
    G = H // Hkv
    assert np.all(got.reshape(L, H, D)[:, G:2 * G] == 0.0)
    check(cache, got, q, [L], [L], H, 1 / math.sqrt(D), splits=[80])


@pytest.mark.parametrize("H,Hkv,room", FORMS)
def test_a_block_of_large_values_that_rows_do_not_see(H, Hkv, room):
    """V of a later block is 2^30 times as large: rows before it keep the
    bits that they would have without it."""
    D, L = 128, 300
    cache = Cache("int8", 1, Hkv, D, 64, room or L, [L], 1130)
    blocks = [3, 7, 10, 15]
    for i, j in enumerate(blocks):
        p, r = cache.place(0, 16 * j)
        cache.vs[p, :, r // 16] *= np.float32(2.0 ** (20 + 10 * i))
    q = _rows(H, D, L, 1131)
    got, q = attend(cache, q, [L], [L], H, 1 / math.sqrt(D))
    check(cache, got, q, [L], [L], H, 1 / math.sqrt(D), splits=[16 * j for j in blocks])


@pytest.mark.parametrize("n", [1, 3, 20])
def test_few_rows_over_such_blocks(n):
    """The kernels for few rows: the same contents."""
    D, L, H, Hkv = 128, 300, 4, 2
    cache = Cache("int8", 2, Hkv, D, 64, L, [L, 17], 1140)
    for j, (ks, vs) in {1: (0.0, 2.0 ** 30), 17: (2.0 ** -126, 0.0), 18: (0.0, 2.0 ** 20)}.items():
        p, r = cache.place(0, 16 * j)
        cache.ks[p, :, r // 16] = ks
        if ks == 0.0:
            cache.k[p, :, r:r + 16] = 0
        cache.vs[p, :, r // 16] *= np.float32(vs)
        if vs == 0.0:
            cache.v[p, :, r:r + 16] = 0
    cache.vs[cache.table[1, 0], :, :2] *= np.float32(1e-9)
    m = [n, min(n, 17)]
    q = _rows(H, D, sum(m), 1141)
    got, q = attend(cache, q, m, [L, 17], H, 1 / math.sqrt(D))
    check(cache, got, q, m, [L, 17], H, 1 / math.sqrt(D), splits=[16 * 17, 16 * 18])
