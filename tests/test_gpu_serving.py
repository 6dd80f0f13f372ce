"""The serving operators together, as a decode loop uses them: prompts of a
ragged batch are appended and attended, then every step appends one token a
sequence, attends and samples, eagerly and from a replayed CUDA graph.

Each step is checked from the device's own cache (teacher-forced): attention
against the oracle over the gathered values (tolerance of
``test_gpu_paged_attention.reference``, and u |v| for the values' rounding to
fp32), the token against the oracle on the device's logits. At the end every
cached value is within half a step of its block's scale for its own rounding,
and half for each later growth of the scale."""
import math

import numpy as np
import pytest
import torch

from oracle import qg_oracle as O
from tests.gpu_util import dev, host64
from tests.paged_util import BLOCK, starts
from tests.test_gpu_paged_attention import reference

pytestmark = pytest.mark.gpu

qg = pytest.importorskip("weight_only_quantized_03_b200")

H, HKV, D, PAGE, V = 4, 2, 64, 16, 500
PROMPTS, STEPS = [37, 1, 20], 21
SCALE = 1 / math.sqrt(D)


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


class Loop:
    def __init__(self, dtype, seed):
        g = torch.Generator().manual_seed(seed)
        n = lambda *s: torch.randn(s, generator=g).cuda()
        B = len(PROMPTS)
        self.B, most = B, (max(PROMPTS) + STEPS + PAGE - 1) // PAGE
        self.kv = qg.PagedKV.empty(B * most + 1, PAGE, HKV, D, dtype)
        self.table = torch.randperm(B * most + 1, generator=g)[:B * most].view(B, most).int().cuda()
        self.embed = n(V, (H + 2 * HKV) * D)
        self.head = n(H * D, V) * 0.7
        self.w = [(1 + 0.1 * n(D)).bfloat16() for _ in range(2)]
        self.len = torch.zeros(B, dtype=torch.int32, device="cuda")
        self.tok = torch.zeros(B, dtype=torch.int32, device="cuda")
        self.u = torch.rand((STEPS, B), generator=g).cuda()
        self.at = torch.zeros(1, dtype=torch.int64, device="cuda")
        self.q = torch.empty((B, H * D), dtype=torch.bfloat16, device="cuda")
        self.out = torch.empty_like(self.q)
        self.logits = torch.empty((B, V), device="cuda")
        self.ws = torch.empty(qg.qg_paged_attention_workspace_size(D), dtype=torch.uint8,
                              device="cuda")
        self.temp = torch.tensor([0.8, 1.0, 0.0], device="cuda")
        self.top_k = torch.tensor([0, 40, 0], dtype=torch.int32, device="cuda")
        self.top_p = torch.tensor([0.9, 1.0, 1.0], device="cuda")
        self.x = None

    def append(self, x, q, row_start=None):
        a, k, v = x.split((H * D, HKV * D, HKV * D), 1)
        qg.qg_paged_kv_append(self.kv, self.table, self.len, k, v, row_start=row_start, q=a,
                              q_out=q, q_norm=self.w[0], k_norm=self.w[1], theta=1e4)

    def prompt(self, tokens):
        rs = dev(starts(PROMPTS))
        self.len += dev(np.array(PROMPTS, np.int32))
        x = self.embed[tokens.long()]
        q = torch.empty((x.shape[0], H * D), dtype=torch.bfloat16, device="cuda")
        out = torch.empty_like(q)
        self.append(x, q, rs)
        qg.qg_paged_attention(self.kv, self.table, self.len, q, out, H, SCALE, self.ws,
                              row_start=rs)
        return q, out

    def step(self):
        self.len += 1
        self.x = self.embed[self.tok.long()]
        self.append(self.x, self.q)
        qg.qg_paged_attention(self.kv, self.table, self.len, self.q, self.out, H, SCALE, self.ws)
        torch.matmul(self.out.float(), self.head, out=self.logits)
        qg.qg_sample_filtered(self.logits, self.u.index_select(0, self.at)[0], self.tok, self.temp, self.top_k,
                              self.top_p)
        self.at += 1

    def cached(self, lens):
        k, v = (torch.empty((sum(lens), HKV * D), device="cuda") for _ in range(2))
        qg.qg_paged_kv_gather(self.kv, self.table, None, dev(starts(lens)), k, v)
        f = lambda t: [a.reshape(-1, HKV, D).transpose(1, 0, 2)
                       for a in np.split(host64(t), np.cumsum(lens)[:-1])]
        return f(k), f(v)


def _check_attention(loop, q, out, n, lens, kind):
    k, v = loop.cached(lens)
    q, out, r0 = host64(q), host64(out), starts(n)
    for b in range(loop.B):
        rows = slice(r0[b], r0[b + 1])
        want, tol = reference(q[rows], k[b], v[b], H, HKV, D, SCALE, kind, False, True)
        assert np.all(np.abs(out[rows] - want) <= tol + 4 * O.U32 * np.abs(v[b]).max())


@pytest.mark.parametrize("kind", ["int8", "bf16"])
def test_a_decode_loop(kind):
    dtype = torch.int8 if kind == "int8" else torch.bfloat16
    loop = Loop(dtype, 5)
    tokens = torch.randint(0, V, (sum(PROMPTS),), generator=torch.Generator().manual_seed(6)).int()
    seqs = [list(t) for t in np.split(tokens.numpy(), np.cumsum(PROMPTS)[:-1])]
    q, out = loop.prompt(tokens.cuda())
    _check_attention(loop, q, out, PROMPTS, PROMPTS, kind)
    lens = list(PROMPTS)
    for i in range(STEPS):
        fed = loop.tok.cpu().numpy()
        loop.step()
        torch.cuda.synchronize()
        lens = [x + 1 for x in lens]
        for b in range(loop.B):
            seqs[b].append(int(fed[b]))
        _check_attention(loop, loop.q, loop.out, [1] * loop.B, lens, kind)
        logits, u = loop.logits.cpu().numpy(), loop.u[i].cpu().numpy()
        for b in range(loop.B):
            want = O.sample_filtered(logits[b], u[b], float(loop.temp[b]), int(loop.top_k[b]),
                                     np.float32(float(loop.top_p[b])))[0]
            assert int(loop.tok[b]) == want, (i, b)
    # the cache against the exact rows
    k, v = loop.cached(lens)
    embed = host64(loop.embed)
    wk = loop.w[1].view(torch.int16).cpu().numpy().view(np.uint16)
    for b in range(loop.B):
        for which, got in ((0, k[b]), (1, v[b])):
            exact = np.zeros((HKV, lens[b], D))
            for t in range(lens[b]):
                row = embed[seqs[b][t], (H + which * HKV) * D:(H + (which + 1) * HKV) * D]
                if which == 0:
                    row = O.rope_neox(O.rmsnorm_perhead(row, wk, 1e-6, D), t, 1e4, D)
                exact[:, t] = row.reshape(HKV, D)
            err = np.abs(got - exact)
            if kind == "bf16":
                assert np.all(err <= 2.0 ** -8 * np.abs(exact) + 1e-5)
                continue
            for t0 in range(0, lens[b], BLOCK):
                part = exact[:, t0:t0 + BLOCK]
                top = np.maximum.accumulate(np.abs(part).max(2), 1)          # [HKV, rows]
                s = top[:, -1] / 127
                for h in range(HKV):
                    for r in range(part.shape[1]):
                        # scales after this row's: each growth rounds once more
                        later = np.unique(top[h, r:]).size
                        bound = 0.5 * s[h] * later * (1 + 1e-4) + 1e-5
                        assert err[h, t0 + r].max() <= bound, (b, which, t0, h, r)


@pytest.mark.parametrize("kind", ["int8", "bf16"])
def test_the_loop_from_a_graph_gives_the_same_bits(kind):
    dtype = torch.int8 if kind == "int8" else torch.bfloat16
    tokens = torch.randint(0, V, (sum(PROMPTS),), generator=torch.Generator().manual_seed(6)).int()
    runs = []
    for graphed in (False, True):
        loop = Loop(dtype, 5)
        loop.prompt(tokens.cuda())
        toks = []
        if not graphed:
            for _ in range(STEPS):
                loop.step()
                toks.append(loop.tok.clone())
        else:
            state = [t.clone() for t in (loop.len, loop.tok, loop.at, loop.kv.k_pages,
                                         loop.kv.v_pages)]
            scales = [None if t is None else t.clone()
                      for t in (loop.kv.k_scales, loop.kv.v_scales)]
            side = torch.cuda.Stream()
            side.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(side):
                loop.step()     # (the libraries under the loop warm up outside the capture)
            torch.cuda.synchronize()
            for t, s in zip((loop.len, loop.tok, loop.at, loop.kv.k_pages, loop.kv.v_pages), state):
                t.copy_(s)
            for t, s in zip((loop.kv.k_scales, loop.kv.v_scales), scales):
                if t is not None:
                    t.copy_(s)
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=side):
                loop.step()
            for _ in range(STEPS):
                g.replay()
                torch.cuda.synchronize()
                toks.append(loop.tok.clone())
        torch.cuda.synchronize()
        lens = [p + STEPS for p in PROMPTS]
        runs.append((torch.stack(toks), loop.out.clone(), loop.cached(lens)))
    assert torch.equal(runs[0][0], runs[1][0]) and torch.equal(runs[0][1], runs[1][1])
    for a, b in zip(runs[0][2], runs[1][2]):
        for x, y in zip(a, b):
            np.testing.assert_array_equal(x, y)


@pytest.mark.parametrize("kind", ["int8", "bf16"])
@pytest.mark.parametrize("n", [[1, 1, 2], [40, 1, 70]])
def test_rows_before_the_first_and_behind_the_last_sequence_stay(kind, n):
    """row_start begins past 0 and ends before T: append, attention and
    gather leave the rows outside alone (and do not read them: they are NaN),
    the rows inside are those of the same call without them."""
    dtype = torch.int8 if kind == "int8" else torch.bfloat16
    lens = [x + 13 * i for i, x in enumerate(n)]
    g = torch.Generator(device="cuda").manual_seed(31)
    B, T, lead, tail = len(n), sum(n), 21, 5
    most = max(lens) // PAGE + 1
    table = torch.randperm(B * most, generator=g, device="cuda").view(B, most).int()
    x = torch.randn((T, (H + 2 * HKV) * D), generator=g, device="cuda").bfloat16()
    ws = torch.empty(qg.qg_paged_attention_workspace_size(D), dtype=torch.uint8, device="cuda")
    ld, runs = dev(np.array(lens, np.int32)), []
    for before, behind in ((0, 0), (lead, tail)):
        kv = qg.PagedKV.empty(B * most, PAGE, HKV, D, dtype)
        for t in (kv.k_pages, kv.v_pages, kv.k_scales, kv.v_scales):
            if t is not None:
                t.zero_()
        all_rows = before + T + behind
        rows = slice(before, before + T)
        wide = torch.full((all_rows, x.shape[1]), math.nan, dtype=torch.bfloat16, device="cuda")
        wide[rows] = x
        rs = dev(starts(n) + before)
        full = lambda w, dt=torch.bfloat16: torch.full((all_rows, w), 55.0, dtype=dt, device="cuda")
        q, out, k, v = full(H * D), full(H * D), full(HKV * D), full(HKV * D)
        a, b, c = wide.split((H * D, HKV * D, HKV * D), 1)
        qg.qg_paged_kv_append(kv, table, ld, b, c, row_start=rs, q=a, q_out=q)
        qg.qg_paged_attention(kv, table, ld, q, out, H, SCALE, ws, row_start=rs)
        qg.qg_paged_kv_gather(kv, table, ld - torch.tensor(n, device="cuda").int(), rs, k, v)
        torch.cuda.synchronize()
        for t in (q, out, k, v):
            assert bool((t[:before] == 55.0).all()) and bool((t[before + T:] == 55.0).all())
            assert bool(torch.isfinite(t).all())
        runs.append([t[rows].clone() for t in (q, out, k, v)] +
                    [t for t in (kv.k_pages, kv.v_pages) if t is not None])
    assert all(torch.equal(s, t) for s, t in zip(*runs))


@pytest.mark.parametrize("kind", ["int8", "bf16"])
@pytest.mark.parametrize("heads,rows", [(256, 1), (16, 70), (4, 2), (3, 33)])
def test_a_row_of_q_that_is_not_finite_stays_alone(kind, heads, rows):
    """One query head's values NaN or infinite: that head's row is NaN, its
    neighbours in a tile are as they were."""
    dtype = torch.int8 if kind == "int8" else torch.bfloat16
    g = torch.Generator(device="cuda").manual_seed(32)
    L, hkv = 130, 1
    kv = qg.PagedKV.empty(9, PAGE, hkv, D, dtype)
    table = torch.arange(9, device="cuda", dtype=torch.int32).view(1, 9)
    x = torch.randn((L, 2 * hkv * D), generator=g, device="cuda")
    qg.qg_paged_kv_append(kv, table, dev(np.array([L], np.int32)), x[:, :D], x[:, D:],
                          row_start=dev(starts([L])))
    q = torch.randn((rows, heads * D), generator=g, device="cuda").bfloat16()
    ws = torch.empty(qg.qg_paged_attention_workspace_size(D), dtype=torch.uint8, device="cuda")
    outs = []
    for bad in (False, True):
        if bad:
            q.view(rows, heads, D)[rows // 2, heads // 2, 3] = math.inf
            q.view(rows, heads, D)[rows - 1, 0, :] = math.nan
        out = torch.empty_like(q)
        qg.qg_paged_attention(kv, table, dev(np.array([L], np.int32)), q, out, heads, SCALE, ws,
                              row_start=dev(starts([rows])))
        outs.append(out.view(rows, heads, D))
    same = torch.ones((rows, heads), dtype=torch.bool, device="cuda")
    same[rows // 2, heads // 2] = same[rows - 1, 0] = False
    assert torch.equal(outs[0][same], outs[1][same])
    assert bool(torch.isnan(outs[1][~same]).all())
