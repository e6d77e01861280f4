"""Refusals of the paged and rotary entry points, before any device work (no GPU): the C ABI with fake
aligned pointers, and the Python binding's own checks."""
import ctypes

import pytest
import torch

import decode_attention_11_b200 as tq

FAKE = 0x10000
BAD, UNSUPPORTED, WORKSPACE = tq.TQ_ERR_INVALID_ARG, tq.TQ_ERR_UNSUPPORTED, tq.TQ_ERR_WORKSPACE


def pool(**kw):
    c = dict(B=8, Hkv=2, T_cap=64, head_dim=128, k_bits=3, v_bits=3, qjl_m=128, k_codes=FAKE, k_signs=FAKE,
             k_norm=FAKE, k_rnorm=FAKE, v_codes=FAKE, v_norm=FAKE)
    c.update(kw)
    return tq._Cache(**c)


def params(**kw):
    p = dict(Pi=FAKE, S=FAKE, k_centroids=FAKE, k_thresholds=FAKE, v_centroids=FAKE, v_thresholds=FAKE)
    p.update(kw)
    return tq._Params(**p)


def table(**kw):
    t = dict(n_seq=4, max_pages=8, num_pages=8, page_size=64, table=FAKE, seq_lens=FAKE, refs=FAKE, status=FAKE)
    t.update(kw)
    return tq._PageTable(**t)


R = ctypes.byref

# a cache that is no pool: wrong layout, page size, too many slots, too large a page
NO_POOL = [(dict(layout=tq.TQ_LAYOUT_MIXED, k_bits=4, v_bits=4), UNSUPPORTED), (dict(T_cap=24), BAD),
           (dict(B=1 << 25, T_cap=64), BAD), (dict(Hkv=1 << 20, T_cap=64, B=1), BAD), (dict(head_dim=64), UNSUPPORTED),
           (dict(k_bits=5), UNSUPPORTED), (dict(qjl_m=64), UNSUPPORTED), (dict(k_norm=FAKE + 8), BAD), (dict(k_codes=None), BAD)]


def rope(q=FAKE, qs=(1024, 128), Hq=8, k=FAKE, ks=(256, 128), Hkv=2, dtype=tq.TQ_BF16, N=4, pos=FAKE, pos_stride=4, axes=1,
         axis=bytes(64), base=1e4, style=tq.TQ_ROPE_HALF, q_out=FAKE * 2, k_out=FAKE * 2):
    return tq.lib().tq_rope(q, *qs, Hq, k, *ks, Hkv, dtype, N, pos, pos_stride, axes, axis, base, style, 0, q_out, k_out, None)


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=2), UNSUPPORTED), (dict(style=2), UNSUPPORTED), (dict(N=-1), BAD), (dict(Hq=-1), BAD), (dict(q=None), BAD),
    (dict(k_out=None), BAD), (dict(q=FAKE + 8), BAD), (dict(q_out=FAKE + 4), BAD), (dict(qs=(1024, 4)), BAD),
    (dict(qs=(-1024, 128)), BAD), (dict(pos=None), BAD), (dict(pos=FAKE + 2), BAD), (dict(axes=0), BAD),
    (dict(axis=bytes([1] * 64)), BAD), (dict(axes=2, pos_stride=-1), BAD), (dict(base=0.0), BAD), (dict(base=float("inf")), BAD),
    (dict(base=float("nan")), BAD), (dict(q_out=FAKE, qs=(2048, 128)), BAD)])
def test_rope_refuses(kw, status):
    assert rope(**kw) == status and tq.last_error()


def test_rope_with_nothing_to_do():
    assert rope(N=0, q=None, k=None, q_out=None, k_out=None, pos=None) == tq.TQ_OK
    assert rope(Hq=0, Hkv=0) == tq.TQ_OK


@pytest.mark.parametrize("kw", [dict(n_seq=0), dict(max_pages=0), dict(num_pages=0), dict(page_size=8), dict(page_size=40),
                                dict(table=None), dict(seq_lens=None), dict(refs=None), dict(status=None), dict(refs=FAKE + 4),
                                dict(table=FAKE + 2), dict(max_pages=1 << 26), dict(num_pages=1 << 26)])
def test_page_table_refused(kw):
    L, t = tq.lib(), table(**kw)
    ws = 1 << 20
    assert L.tq_pages_reserve(R(t), FAKE, FAKE, 1, FAKE, 4, FAKE, ws, None) == BAD
    assert L.tq_pages_fork(R(t), FAKE, FAKE, 1, R(pool()), 1, FAKE, ws, None) == BAD
    assert L.tq_pages_free(R(t), FAKE, 1, None) == BAD
    assert L.tq_pages_compact(R(t), R(pool()), 1, FAKE, ws, None) == BAD


def test_page_calls_refuse():
    L, t, p, ws = tq.lib(), table(), pool(), 1 << 20
    assert L.tq_pages_workspace_size(None, 1) == 0 and L.tq_pages_workspace_size(R(t), -1) == 0
    need = L.tq_pages_workspace_size(R(t), 3)
    assert need > 0
    # lists
    assert L.tq_pages_reserve(R(t), None, FAKE, 1, FAKE, 4, FAKE, ws, None) == BAD
    assert L.tq_pages_reserve(R(t), FAKE, FAKE + 2, 1, FAKE, 4, FAKE, ws, None) == BAD
    assert L.tq_pages_reserve(R(t), FAKE, FAKE, -1, FAKE, 4, FAKE, ws, None) == BAD
    assert L.tq_pages_reserve(R(t), FAKE, FAKE, 1, None, 4, FAKE, ws, None) == BAD
    assert L.tq_pages_reserve(R(t), FAKE, FAKE, 1, FAKE, -4, FAKE, ws, None) == BAD
    assert L.tq_pages_free(R(t), None, 1, None) == BAD
    assert L.tq_pages_copy(R(p), 1, FAKE, None, 1, None, None) == BAD
    assert L.tq_pages_copy(R(p), 1, FAKE, FAKE, 1, FAKE + 1, None) == BAD
    # workspaces
    assert L.tq_pages_reserve(R(t), FAKE, FAKE, 3, FAKE, 4, FAKE, need - 1, None) == WORKSPACE
    assert L.tq_pages_fork(R(t), FAKE, FAKE, 3, R(p), 1, None, ws, None) == BAD
    assert L.tq_pages_compact(R(t), R(p), 1, FAKE, 8, None) == WORKSPACE
    # pools: not of this table, unequal, none where some are said to be, no pools at all
    assert L.tq_pages_fork(R(t), FAKE, FAKE, 1, R(pool(B=9)), 1, FAKE, ws, None) == BAD
    assert L.tq_pages_compact(R(t), R(pool(T_cap=32)), 1, FAKE, ws, None) == BAD
    two = (tq._Cache * 2)(p, pool(k_bits=4))
    assert L.tq_pages_fork(R(t), FAKE, FAKE, 1, two, 2, FAKE, ws, None) == BAD
    assert "differs" in tq.last_error()
    assert L.tq_pages_copy(None, 1, FAKE, FAKE, 1, None, None) == BAD
    assert L.tq_pages_copy(R(p), -1, FAKE, FAKE, 1, None, None) == BAD
    for kw, status in NO_POOL:
        assert L.tq_pages_copy(R(pool(**kw)), 1, FAKE, FAKE, 1, None, None) == status, kw
    # empty lists do nothing
    assert L.tq_pages_free(R(t), None, 0, None) == tq.TQ_OK
    assert L.tq_pages_fork(R(t), None, None, 0, R(p), 1, FAKE, ws, None) == tq.TQ_OK
    assert L.tq_pages_copy(R(p), 1, None, None, 0, None, None) == tq.TQ_OK
    assert L.tq_pages_reserve(R(t), None, None, 0, None, 0, FAKE, ws, None) == tq.TQ_OK


def quantize(p=None, c=None, k=FAKE, v=FAKE, dtype=tq.TQ_BF16, sn=256, sh=128, N=4, slots=FAKE):
    return tq.lib().tq_paged_quantize(R(p or params()), k, v, dtype, sn, sh, N, slots, R(c or pool()), None)


def read(p=None, c=None, slots=FAKE, N=4, dtype=tq.TQ_BF16, k=FAKE, v=FAKE, s=FAKE, r=FAKE):
    return tq.lib().tq_paged_read(R(p or params()), R(c or pool()), slots, N, dtype, k, v, s, r, None)


def test_row_calls_refuse():
    for kw, status in NO_POOL:
        assert quantize(c=pool(**kw)) == status, kw
        assert read(c=pool(**kw)) == status, kw
    for f in (quantize, read):
        assert f(p=params(Pi=None)) == BAD and f(p=params(S=None)) == BAD
        assert f(slots=None) == BAD and f(slots=FAKE + 2) == BAD and f(N=-1) == BAD and f(N=1 << 30) == BAD
        assert f(dtype=7) == UNSUPPORTED
        assert f(k=None) == BAD and f(v=FAKE + 8) == BAD
    assert read(k=FAKE + 16) == BAD and read(v=FAKE + 16) == BAD
    assert quantize(sn=-256) == BAD and quantize(sh=4) == BAD and quantize(sn=257) == BAD
    assert quantize(N=0, k=None, v=None, slots=None) == tq.TQ_OK
    bare = pool(qjl_m=0, k_signs=None, k_rnorm=None)
    assert read(c=bare) == BAD and read(c=bare, s=None) == BAD and read(s=FAKE + 4) == BAD and read(r=FAKE + 2) == BAD
    assert read(N=0, k=None, v=None, slots=None) == tq.TQ_OK


def decode(p=None, q=FAKE, q_dtype=tq.TQ_F32, B=2, Hq=8, c=None, t=FAKE, stride=8, max_pages=8, lens=FAKE, window=0, out=FAKE,
           out_dtype=tq.TQ_F32, lse=FAKE, ws=FAKE, ws_bytes=1 << 30):
    return tq.lib().tq_paged_decode_attn(R(p or params()), q, q_dtype, B, Hq, R(c or pool()), t, stride, max_pages, lens,
                                         window, 0.0, out, out_dtype, lse, ws, ws_bytes, None)


@pytest.mark.parametrize("kw,status", [
    (dict(q_dtype=3), UNSUPPORTED), (dict(out_dtype=3), UNSUPPORTED), (dict(B=0), BAD), (dict(B=70000), BAD), (dict(Hq=7), BAD),
    (dict(Hq=0), BAD), (dict(max_pages=0), BAD), (dict(stride=7), BAD), (dict(max_pages=1 << 25, stride=1 << 25), BAD),
    (dict(window=-1), BAD), (dict(q=None), BAD), (dict(q=FAKE + 8), BAD), (dict(out=None), BAD), (dict(t=None), BAD),
    (dict(t=FAKE + 2), BAD), (dict(lens=None), BAD), (dict(lse=FAKE + 2), BAD), (dict(ws=None), BAD), (dict(ws_bytes=1024), WORKSPACE),
    (dict(p=params(k_centroids=None)), BAD)])
def test_decode_refuses(kw, status):
    assert decode(**kw) == status and tq.last_error()


def test_decode_refuses_what_is_no_pool():
    for kw, status in NO_POOL:
        assert decode(c=pool(**kw)) == status, kw
    assert tq.lib().tq_paged_decode_workspace_size(2, 7, R(pool())) == 0
    assert tq.lib().tq_paged_decode_workspace_size(0, 8, R(pool())) == 0
    assert tq.lib().tq_paged_decode_workspace_size(2, 8, None) == 0


def test_binding_refuses():
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32)
    q = torch.zeros(4, 8, 128)
    with pytest.raises(ValueError, match="CUDA device"):
        tq.rope(q, None, i32(4))
    with pytest.raises(ValueError, match="both None"):
        tq.rope(None, None, i32(4))
    with pytest.raises(ValueError, match="pos"):
        tq.rope(q, None, torch.zeros(4))
    with pytest.raises(ValueError, match="pos"):
        tq.rope(q, None, i32(3))
    with pytest.raises(ValueError, match="sections"):
        tq.rope(q, None, i32(4), sections=(32, 16))
    with pytest.raises(ValueError, match="dtype"):
        tq.rope(q, q.to(torch.bfloat16), i32(4))
    with pytest.raises(ValueError, match="64 entries"):
        tq.rope(q, None, i32(4), axis_of_pair=[0] * 63)
    cache = tq.Cache.allocate(8, 2, 64, 3, 3, device="cpu")
    pt = tq.PageTable.allocate(4, 8, 8, 64, device="cpu")
    pr = tq.Params.create(torch.eye(128).numpy(), torch.ones(128, 128).numpy(), 3, 3, device="cpu")
    with pytest.raises(ValueError, match="int32"):
        tq.pages_free(pt, torch.zeros(2, dtype=torch.int64))
    with pytest.raises(ValueError, match="CUDA device"):
        tq.pages_free(pt, i32(2))
    with pytest.raises(ValueError, match="same length"):
        tq.pages_fork(pt, i32(2), i32(3), [cache])
    with pytest.raises(ValueError, match="same length"):
        tq.pages_reserve(pt, i32(2), i32(3), 4)
    with pytest.raises(ValueError, match="contiguous"):
        tq.pages_copy([cache], i32(4)[::2], i32(2))
    with pytest.raises(ValueError, match="entry per token"):
        tq.paged_quantize(pr, q[:, :2], q[:, :2], cache, i32(3))
    with pytest.raises(ValueError, match=r"\[N, 2, 128\]"):
        tq.paged_quantize(pr, q, q, cache, i32(4))
    with pytest.raises(ValueError, match="strides"):
        tq.paged_quantize(pr, q[:, :2], torch.zeros(4, 2, 128), cache, i32(4))
    with pytest.raises(TypeError):
        tq.paged_read(pr, cache, i32(4), dtype=torch.float16)
    with pytest.raises(ValueError, match="table"):
        tq.paged_decode_attn(pr, q, cache, i32(3, 8), i32(4))
    with pytest.raises(ValueError, match="seq_lens"):
        tq.paged_decode_attn(pr, q, cache, i32(4, 8), i32(3))
    with pytest.raises(ValueError, match="CUDA device"):
        tq.paged_decode_attn(pr, q, cache, i32(4, 8), i32(4))
    pt.status[0] = tq.TQ_PAGES_NO_ROOM
    with pytest.raises(ValueError, match="free pages"):
        pt.check()
    pt.check()
