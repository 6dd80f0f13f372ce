"""Kernels that start before the one ahead of them on the stream has ended:
what reads attention's rows, right behind it, must see all of them."""
import math

import numpy as np
import pytest
import torch

import qg_synth
from tests.gpu_util import dev
from tests.paged_util import starts

pytestmark = pytest.mark.gpu

qg = pytest.importorskip("weight_only_quantized_03_b200")


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def _pool(Hkv, D, tokens, page=64, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    kv = qg.PagedKV.empty(tokens // page, page, Hkv, D, torch.int8)
    for t in (kv.k_pages, kv.v_pages):
        t.copy_(torch.randint(-127, 128, t.shape, generator=g, device="cuda", dtype=torch.int8))
    for t in (kv.k_scales, kv.v_scales):
        t.copy_(0.01 + 0.01 * torch.rand(t.shape, generator=g, device="cuda"))
    return kv, g


@pytest.mark.parametrize("B,Hkv,tokens", [
    (74, 8, 8192),    # twice as many (sequence, head) items as pieces: none is cut
    (37, 8, 16384),   # an item is a block
    (37, 8, 16320),
    (5, 8, 100),      # an item is one chunk
    (40, 1, 16384),   # some items cut
])
def test_the_next_kernel_sees_all_rows(B, Hkv, tokens):
    """The sequences share their pages. q_out of an append without norm and
    rotation is its q: attention's rows as that kernel read them."""
    D, H, page = 128, 2 * Hkv, 64
    kv, g = _pool(Hkv, D, (tokens + page - 1) // page * page, page)
    most = kv.k_pages.shape[0]
    table = torch.arange(most, dtype=torch.int32, device="cuda").repeat(B, 1)
    lens = torch.full((B,), tokens, dtype=torch.int32, device="cuda")
    q = torch.randn((B, H * D), generator=g, device="cuda").bfloat16()
    ws = torch.empty(qg.qg_paged_attention_workspace_size(D), dtype=torch.uint8, device="cuda")
    want = torch.empty_like(q)
    attend = lambda out: qg.qg_paged_attention(kv, table, lens, q, out, H, 1 / math.sqrt(D), ws)
    attend(want)
    torch.cuda.synchronize()
    assert torch.isfinite(want).all()
    other = qg.PagedKV.empty(B, 16, 1, D, torch.bfloat16)
    one = torch.arange(B, dtype=torch.int32, device="cuda").view(B, 1)
    first = torch.ones(B, dtype=torch.int32, device="cuda")
    k = torch.zeros((B, D), dtype=torch.bfloat16, device="cuda")
    for _ in range(5):
        out, seen = torch.full_like(q, math.nan), torch.full_like(q, math.nan)
        torch.cuda.synchronize()
        attend(out)
        qg.qg_paged_kv_append(other, one, first, k, k, q=out, q_out=seen, rotary_dim=0)
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(seen, want)


@pytest.mark.parametrize("T,N", [(256, 512), (24, 4096)])
def test_a_prompt_before_products_on_tensor_memory(T, N):
    """The kernel behind takes tensor memory before it waits: prompt rows,
    their output projection, prompt rows again."""
    D, H, Hkv, B = 128, 16, 8, 2
    K = H * D
    kv, g = _pool(Hkv, D, 4096, seed=1)
    # (room for many more tokens, so that the few rows take that kernel too)
    table = torch.arange(64, dtype=torch.int32, device="cuda").view(2, 32).repeat(1, 13)
    n = [T - 7, 7]
    rs, lens = dev(starts(n)), dev(np.array([2000, 900], np.int32))
    w, s, b = (dev(a) for a in qg_synth.affine8_packed(N, K, 7))
    q = torch.randn((T, K), generator=g, device="cuda").bfloat16()
    ws = torch.empty(qg.qg_paged_attention_workspace_size(D), dtype=torch.uint8, device="cuda")
    err = torch.zeros(64, dtype=torch.int32, device="cuda")

    def chain(sync):
        x = q
        for _ in range(3):
            out, y = torch.full_like(q, math.nan), torch.empty((T, N), device="cuda")
            qg.qg_paged_attention(kv, table, lens, x, out, H, 1 / math.sqrt(D), ws, row_start=rs)
            if sync:
                torch.cuda.synchronize()
            qg.qg_gemm_affine8_g64(w, s, b, out, y, ws=err)
            if sync:
                torch.cuda.synchronize()
            x = out
        return out, y

    want = chain(True)
    assert all(torch.isfinite(t).all() for t in want)
    for _ in range(3):
        got = chain(False)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
