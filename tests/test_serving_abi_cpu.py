"""Refusals of the serving entry points before any launch (no GPU needed):
each names the argument at fault."""
import ctypes

import pytest
import torch

import weight_only_quantized_03_b200 as qg

FAKE = 0x7F0000000000  # aligned, never dereferenced


def _status(name, *args):
    st = getattr(qg.lib, name)(*args)
    return st, qg.last_error()


def _kv(**kw):
    f = dict(k_pages=FAKE, v_pages=FAKE, k_scales=FAKE, v_scales=FAKE, num_pages=10, page_size=64,
             kv_heads=2, head_dim=128, dtype=qg.QG_KV_INT8)
    f.update(kw)
    return qg.qg_paged_kv(**f)


def _append(kv=None, **kw):
    a = dict(table=FAKE, max_pages=4, kv_len=FAKE, row_start=None, q=FAKE, q_ld=512, k=FAKE,
             k_ld=256, v=FAKE, v_ld=256, xdt=qg.QG_F32, qn=None, kn=None, eps=1e-6, theta=1e6,
             rd=128, qo=FAKE, qdt=qg.QG_BF16, B=2, T=2, H=4)
    a.update(kw)
    ref = ctypes.byref(kv if kv is not None else _kv())
    return _status("qg_paged_kv_append", ref, *a.values(), None)


def test_pool_refusals_name_the_field():
    U, I, M = qg.QG_ERR_UNSUPPORTED_SHAPE, qg.QG_ERR_INVALID_ARGUMENT, qg.QG_ERR_MISALIGNED
    for kv, code, word in ((_kv(head_dim=96), U, "head_dim=96"), (_kv(page_size=24), U, "page_size=24"),
                           (_kv(page_size=0), U, "page_size=0"), (_kv(kv_heads=0), U, "kv_heads=0"),
                           (_kv(dtype=3), I, "dtype=3"), (_kv(num_pages=-1), U, "num_pages=-1"),
                           (_kv(k_pages=None), I, "k_pages"), (_kv(v_pages=FAKE + 8), M, "v_pages"),
                           (_kv(k_scales=None), I, "k_scales"), (_kv(v_scales=FAKE + 2), M, "scales")):
        st, msg = _append(kv)
        assert st == code and word in msg, (st, msg)
        st, msg = _status("qg_paged_kv_gather", ctypes.byref(kv), FAKE, 4, FAKE, None, FAKE, FAKE,
                          qg.QG_F32, 2, 2, None)
        assert st == code and word in msg, (st, msg)
    assert _status("qg_paged_kv_append", None, *([0] * 0), FAKE, 4, FAKE, None, None, 0, FAKE, 256,
                   FAKE, 256, 0, None, None, 1e-6, 1e6, 0, None, 0, 1, 1, 0, None)[0] == I
    st, msg = _append(max_pages=1 << 28)
    assert st == U and "max_pages" in msg


def test_append_refusals():
    U, I, M = qg.QG_ERR_UNSUPPORTED_SHAPE, qg.QG_ERR_INVALID_ARGUMENT, qg.QG_ERR_MISALIGNED
    for kw, code, word in ((dict(T=3), U, "row_start"), (dict(B=-1), U, "B=-1"),
                           (dict(xdt=5), I, "x_dtype=5"), (dict(qdt=5), I, "q_out_dtype=5"),
                           (dict(rd=130), U, "rotary_dim=130"), (dict(rd=12), U, "rotary_dim=12"),
                           (dict(theta=0.0), I, "theta"), (dict(table=None), I, "page_table"),
                           (dict(kv_len=None), I, "kv_len"), (dict(k=None), I, "k or v"),
                           (dict(q=None), I, "q"), (dict(qo=None), I, "q_out"),
                           (dict(k_ld=128), U, "k_ld=128"), (dict(v_ld=258), M, "k or v"),
                           (dict(k=FAKE + 8), M, "k or v"), (dict(q_ld=514), M, "q or q_out"),
                           (dict(qo=FAKE + 4), M, "q_out"), (dict(row_start=FAKE + 2), M, "row_start")):
        st, msg = _append(**kw)
        assert st == code and word in msg, (kw, st, msg)
    # empty work launches nothing
    assert _append(B=0, T=0, k=None)[0] == qg.QG_OK
    assert _append(row_start=FAKE, T=0)[0] == qg.QG_OK


def test_more_sequences_than_a_call_takes():
    """Every block looks through the sequences: past 65536 that would take
    the GPU for minutes."""
    B = (1 << 16) + 1
    st, msg = _append(B=B, T=B)
    assert st == qg.QG_ERR_UNSUPPORTED_SHAPE and "too large" in msg
    st, _ = _status("qg_paged_kv_gather", ctypes.byref(_kv()), FAKE, 4, FAKE, None, FAKE, FAKE,
                    qg.QG_F32, B, B, None)
    assert st == qg.QG_ERR_UNSUPPORTED_SHAPE


def test_gather_refusals():
    ref = ctypes.byref(_kv())
    g = lambda *a: _status("qg_paged_kv_gather", ref, *a, None)
    assert g(FAKE, 4, FAKE, None, FAKE, FAKE, qg.QG_F32, 2, 3)[0] == qg.QG_ERR_UNSUPPORTED_SHAPE
    assert g(FAKE, 4, FAKE, None, FAKE, FAKE, 9, 2, 2)[0] == qg.QG_ERR_INVALID_ARGUMENT
    assert g(None, 4, FAKE, None, FAKE, FAKE, 0, 2, 2)[0] == qg.QG_ERR_INVALID_ARGUMENT
    assert g(FAKE, 4, FAKE, None, FAKE + 8, None, 0, 2, 2)[0] == qg.QG_ERR_MISALIGNED
    assert g(FAKE, 4, FAKE, None, None, None, 0, 2, 2)[0] == qg.QG_OK


def test_python_refusals():
    """The binding refuses host tensors, layouts and types that the C side
    could not see."""
    pages = lambda dt: torch.zeros((2, 1, 16, 64), dtype=dt)
    with pytest.raises(TypeError):
        qg.PagedKV(pages(torch.float16), pages(torch.float16))
    with pytest.raises(ValueError, match="k_scales"):
        qg.PagedKV(pages(torch.int8), pages(torch.int8))
    with pytest.raises(ValueError, match="v_scales"):
        qg.PagedKV(pages(torch.int8), pages(torch.int8), torch.zeros(2, 1, 1), torch.zeros(2, 1, 2))
    with pytest.raises(ValueError, match="contiguous"):
        t = torch.zeros((2, 16, 1, 64), dtype=torch.bfloat16).transpose(1, 2).expand(2, 3, 16, 64)
        qg.PagedKV(t, t)
    with pytest.raises(ValueError, match="one type"):
        qg.PagedKV(pages(torch.bfloat16), pages(torch.int8))
    with pytest.raises(ValueError, match="unit stride"):
        qg._rows_of("k", torch.zeros(64, 4).t(), 64)
    assert qg._rows_of("k", torch.zeros(4, 96)[:, 32:], 64) == 96
    with pytest.raises(ValueError, match="int32"):
        qg._check_index(-1, "kv_len", torch.zeros(3), 3)
    with pytest.raises(ValueError, match="of 4 values"):
        qg._check_index(-1, "kv_len", torch.zeros(3, dtype=torch.int32), 4)
    with pytest.raises(ValueError, match="cpu"):
        qg._check_index(0, "kv_len", torch.zeros(3, dtype=torch.int32), 3)
    with pytest.raises(ValueError, match="cpu"):
        qg._check_device(0, ("k", torch.zeros(3)))


def _attend(kv=None, **kw):
    need = qg.lib.qg_paged_attention_workspace_size(128)
    a = dict(table=FAKE, max_pages=4, kv_len=FAKE, row_start=None, q=FAKE, qdt=qg.QG_BF16, out=FAKE,
             odt=qg.QG_BF16, B=2, T=2, H=4, scale=0.1, ws=FAKE, ws_bytes=need)
    a.update(kw)
    return _status("qg_paged_attention", ctypes.byref(kv if kv is not None else _kv()),
                   *a.values(), None)


def test_attention_refusals():
    U, I, M = qg.QG_ERR_UNSUPPORTED_SHAPE, qg.QG_ERR_INVALID_ARGUMENT, qg.QG_ERR_MISALIGNED
    need = qg.lib.qg_paged_attention_workspace_size(128)
    assert need > 0 and qg.lib.qg_paged_attention_workspace_size(0) == 0
    for kw, code, word in ((dict(T=3), U, "row_start"), (dict(H=5), U, "H=5"), (dict(H=0), U, "H=0"),
                           (dict(B=1 << 17, T=1 << 17), U, "too large"),
                           (dict(row_start=FAKE, T=1 << 29), U, "too large"),
                           (dict(qdt=4), I, "q_dtype=4"), (dict(odt=4), I, "out_dtype=4"),
                           (dict(scale=0.0), I, "scale"), (dict(scale=float("nan")), I, "scale"),
                           (dict(scale=float("inf")), I, "scale"), (dict(q=None), I, "q or out"),
                           (dict(out=FAKE + 8), M, "out"), (dict(kv_len=FAKE + 1), M, "kv_len"),
                           (dict(ws_bytes=need - 1), qg.QG_ERR_WORKSPACE_TOO_SMALL, str(need)),
                           (dict(ws=None), qg.QG_ERR_WORKSPACE_TOO_SMALL, str(need)),
                           (dict(ws=FAKE + 16), M, "ws")):
        st, msg = _attend(**kw)
        assert st == code and word in msg, (kw, st, msg)
    st, msg = _attend(_kv(num_pages=1 << 29))
    assert st == U and "too large" in msg
    assert _attend(B=0, T=0, q=None)[0] == qg.QG_OK


def test_sample_filtered_refusals():
    U, I, M = qg.QG_ERR_UNSUPPORTED_SHAPE, qg.QG_ERR_INVALID_ARGUMENT, qg.QG_ERR_MISALIGNED

    def call(**kw):
        a = dict(logits=FAKE, ld=1000, B=2, V=1000, t=None, k=None, p=None, m=None, u=FAKE, out=FAKE,
                 kept=None, lp=None)
        a.update(kw)
        return _status("qg_sample_filtered", *a.values(), None)

    for kw, code, word in ((dict(V=0), U, "V=0"), (dict(V=1 << 23, ld=1 << 23), U, "V="),
                           (dict(ld=999), U, "ld=999"), (dict(B=-1), U, "B=-1"),
                           (dict(B=70000), U, "B=70000"), (dict(logits=None), I, "logits"),
                           (dict(u=None), I, "u"), (dict(out=None), I, "out"),
                           (dict(t=FAKE + 2), M, "aligned"), (dict(logits=FAKE + 1), M, "aligned")):
        st, msg = call(**kw)
        assert st == code and word in msg, (kw, st, msg)
    assert call(B=0, logits=None)[0] == qg.QG_OK


def test_norm_weights_are_bf16():
    """fp16 weights have two bytes as well, but other bits: refused."""
    for good in (torch.ones(64).bfloat16(), torch.ones(64).bfloat16().view(torch.int16),
                 torch.ones(64).bfloat16().view(torch.uint16)):
        qg._check_norm(good, 64)
    for bad in (torch.ones(64).half(), torch.ones(64), torch.ones(32).bfloat16(),
                torch.ones(128).bfloat16()[::2]):
        with pytest.raises(ValueError, match="64 bf16 values"):
            qg._check_norm(bad, 64)


@pytest.mark.parametrize("B,T,H,Hkv,pages", [(54606, 16777284, 8, 2, 84), (40555, 33554509, 8, 2, 41),
                                             (1, 1 << 27, 8, 8, 6), (1, 1000, 16, 8, 1 << 18),
                                             (65536, 65536, 64, 64, 340), (3, 70, 2, 2, 1 << 19)])
def test_attention_takes_what_the_header_allows(B, T, H, Hkv, pages):
    """The rule on rows, heads and pages, at fp32 (where no call goes to the
    kernel that it does not bound), with q missing: a call within the rule is
    refused for that, one beyond for its sizes."""
    kv = _kv(kv_heads=Hkv, page_size=192)
    room = lambda pages: (T * H // 8 + B * Hkv) * (pages * 192 // 128 + 3)
    most = next(p for p in range(pages, -1, -1) if room(p) < 1 << 31)
    call = lambda pages: _attend(kv, row_start=FAKE, B=B, T=T, H=H, max_pages=pages, q=None,
                                 qdt=qg.QG_F32)
    st, msg = call(most)
    assert st == qg.QG_ERR_INVALID_ARGUMENT and "q or out" in msg, (st, msg)
    if 2 * room(most) > 1 << 31 and 192 * (2 * most + 8) < 0x7FFFFFFF - 65536:
        st, msg = call(2 * most + 8)
        assert st == qg.QG_ERR_UNSUPPORTED_SHAPE and "too many" in msg, (st, msg)
