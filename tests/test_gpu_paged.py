"""Paged quantize, read and decode attention on the GPU against the float64 oracle.

Attention tolerance (fp32 output).  q', S q' and the weights enter the products as fp16 hi + lo (2^-22
relative), products accumulate in fp32 over at most 24 steps (24 * 2^-23).  With |q| <= 15 and key
norms below 30, a score is off by at most |q| |k| / sqrt(128) * (2 * 2^-22 + 24 * 2^-23) = 40 * 3.3e-6 =
1.4e-4, which scales a weight by as much, in the numerator and in the sum: 3e-4 relative to the output's
norm.  A bf16 output adds eps / 2 = 2^-8 of each value.  lse: the score's 1.4e-4, and 2^-23 of its value."""
import math

import numpy as np
import pytest
import torch

import decode_attention_11_b200 as tq
import workloads as W
from oracle import tq_oracle as O

from _parity import NORM_ULP, ulp_distance_f32

pytestmark = pytest.mark.gpu

PI, S = W.make_rotation(1234), W.make_qjl_matrix(2345)
ARRAYS = ("k_codes", "k_signs", "k_norm", "k_rnorm", "v_codes", "v_norm")


def params(kb, vb, qjl=True):
    return tq.Params.create(PI, S if qjl else None, kb, vb)


def filled_pool(pages, Hkv, ps, kb, vb, qjl=True, seed=0):
    """A pool of random codes and signs with key norms below 30."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    pool = tq.Cache.allocate(pages, Hkv, ps, kb, vb, 128 if qjl else 0)
    for n in ("k_codes", "k_signs", "v_codes"):
        if getattr(pool, n) is not None:
            getattr(pool, n).random_(0, 256, generator=g)
    pool.k_norm.uniform_(1.0, 29.0, generator=g)
    pool.v_norm.uniform_(1.0, 29.0, generator=g)
    if qjl:
        pool.k_rnorm.copy_(0.15 * pool.k_norm)
    return pool


def table_for(lens, ps, pages, seed=0, extra=1):
    """Shuffled distinct pages for each sequence; entries past its last page are -1 or nonsense."""
    g = torch.Generator().manual_seed(seed)
    order = torch.randperm(pages, generator=g).tolist()
    per = max(1, max(-(-n // ps) for n in lens)) + extra
    rows = []
    for b, n in enumerate(lens):
        need = -(-n // ps)
        rows.append([order.pop() for _ in range(need)] + [-1 if b % 2 else 10**9] * (per - need))
    return torch.tensor(rows, dtype=torch.int32, device="cuda")


def rows_of(pool, table, b, t):
    """The pool's rows of tokens t of sequence b, as [1, Hkv, len(t), ...] host arrays."""
    page = table[b, torch.as_tensor(t // pool.T_cap, device="cuda")].long()
    off = torch.as_tensor(t % pool.T_cap, device="cuda")
    out = {}
    for n in ARRAYS:
        a = getattr(pool, n)
        if a is not None:
            out[n] = a.transpose(1, 2)[page, off].transpose(0, 1)[None].cpu().numpy()
    return out


def reference(q, pool, table, lens, window=0, scale=None, qjl=True):
    q = q.double().cpu().numpy()
    B, Hq, _ = q.shape
    out, lse = np.zeros((B, Hq, 128)), np.full((B, Hq), -np.inf)
    sc = scale or 1.0 / math.sqrt(128)
    for b, n in enumerate(lens):
        t = np.arange(max(0, n - window) if window else 0, n)
        if not len(t):
            continue
        c = rows_of(pool, table, b, t)
        out[b] = O.decode_attention(q[b:b + 1], PI, S if qjl else None, c, pool.k_bits, pool.v_bits, len(t), scale=sc)[0]
        for h in range(Hq):
            kv = h // (Hq // pool.Hkv)
            est = sc * O.score_estimates(q[b, h], PI, S if qjl else None, c["k_codes"][0, kv], c["k_norm"][0, kv],
                                         pool.k_bits, c["k_signs"][0, kv] if qjl else None, c["k_rnorm"][0, kv] if qjl else None)
            lse[b, h] = est.max() + math.log(np.exp(est - est.max()).sum())
    return out, lse


def assert_close(out, lse, ref, ref_lse):
    got = out.double().cpu().numpy()
    assert np.isfinite(got).all()
    err = np.abs(got - ref)
    # half a step of bf16, below its smallest normal value nothing
    half = torch.finfo(torch.bfloat16).eps / 2 if out.dtype == torch.bfloat16 else 0.0
    rest = np.maximum(err - half * np.abs(ref), 0.0)
    norm = np.linalg.norm(ref, axis=-1, keepdims=True)
    assert (np.linalg.norm(rest, axis=-1, keepdims=True) <= 3e-4 * (1 + half) * norm).all(), \
        (np.linalg.norm(rest, axis=-1) / np.maximum(norm[..., 0], 1e-30)).max()
    if lse is not None:
        l = lse.double().cpu().numpy()
        assert np.array_equal(np.isinf(l), np.isinf(ref_lse)) and (l[np.isinf(l)] < 0).all()
        f = np.isfinite(ref_lse)
        assert (np.abs(l[f] - ref_lse[f]) <= 1.4e-4 + 2.0**-22 * np.abs(ref_lse[f])).all()


def queries(B, Hq, dtype=torch.float32, seed=5):
    g = torch.Generator(device="cuda").manual_seed(seed)
    q = torch.randn(B, Hq, 128, generator=g, device="cuda")
    return (q * (q.norm(dim=-1, keepdim=True).clamp_max(15.0) / q.norm(dim=-1, keepdim=True))).to(dtype)


# ------------------------------------------------------------------------------------------ decode

@pytest.mark.parametrize("kb,vb,qjl,Hq,Hkv,ps", [
    (4, 4, True, 8, 2, 64), (4, 4, True, 16, 2, 16), (3, 3, True, 8, 8, 32), (3, 2, True, 16, 2, 48),
    (2, 2, True, 5, 1, 16), (2, 4, False, 6, 2, 64), (4, 3, False, 40, 2, 128), (3, 4, True, 24, 2, 256),
    (2, 3, True, 9, 3, 16), (4, 2, True, 7, 1, 32), (3, 2, False, 17, 1, 64), (4, 4, False, 3, 1, 16)])
def test_decode_ragged(kb, vb, qjl, Hq, Hkv, ps):
    lens = [1, 0, 17, ps, ps + 1, 3 * ps - 1, 700, 0, 2, 16, 333]
    pages = sum(-(-n // ps) for n in lens) + 3
    pool = filled_pool(pages, Hkv, ps, kb, vb, qjl)
    table = table_for(lens, ps, pages)
    p = params(kb, vb, qjl)
    for dtype in (torch.float32, torch.bfloat16):
        q = queries(len(lens), Hq, dtype)
        out, lse = tq.paged_decode_attn(p, q, pool, table, torch.tensor(lens, dtype=torch.int32, device="cuda"),
                                        out_dtype=dtype, return_lse=True)
        ref, rl = reference(q, pool, table, lens, qjl=qjl)
        assert_close(out, lse, ref, rl)
        assert (out[1] == 0).all() and (out[7] == 0).all()
    assert tq.decode_device_errors() == 0


@pytest.mark.parametrize("window", [1, 15, 16, 17, 64, 100, 5000])
@pytest.mark.parametrize("Hq,Hkv", [(4, 1), (16, 2)])
def test_decode_window(window, Hq, Hkv):
    ps, lens = 32, [1000, 16, 1, 0, 129, 64]
    pages = sum(-(-n // ps) for n in lens)
    pool = filled_pool(pages, Hkv, ps, 4, 4, seed=window)
    table = table_for(lens, ps, pages, extra=0)
    q = queries(len(lens), Hq)
    out, lse = tq.paged_decode_attn(params(4, 4), q, pool, table, torch.tensor(lens, dtype=torch.int32, device="cuda"),
                                    window=window, scale=0.07, return_lse=True)
    assert_close(out, lse, *reference(q, pool, table, lens, window, scale=0.07))


@pytest.mark.parametrize("B,Hkv,Hq,lens", [(1, 1, 1, [20011]), (2, 2, 16, [9000, 31]), (300, 1, 4, None), (40, 8, 32, None)])
def test_decode_long_and_many(B, Hkv, Hq, lens):
    """One unit over many CTAs, and many units per CTA (lengths that end inside CTA ranges)."""
    ps = 64
    if lens is None:
        r = np.random.RandomState(B)
        lens = r.randint(0, 220, B).tolist()
    pages = sum(-(-n // ps) for n in lens) + 1
    pool = filled_pool(pages, Hkv, ps, 4, 4, seed=B)
    table = table_for(lens, ps, pages)
    q = queries(B, Hq)
    out, lse = tq.paged_decode_attn(params(4, 4), q, pool, table, torch.tensor(lens, dtype=torch.int32, device="cuda"),
                                    return_lse=True)
    assert_close(out, lse, *reference(q, pool, table, lens))


@pytest.mark.parametrize("B,Hkv,Hq,window", [(600, 2, 8, 0), (520, 2, 10, 9)])
def test_decode_large_batches(B, Hkv, Hq, window):
    """More sequences than a CTA keeps lengths of (512), and more heads than the merge kernel takes in one round;
    one sequence in three is empty."""
    ps = 16
    r = np.random.RandomState(B)
    lens = (r.randint(1, 70, B) * (r.randint(0, 3, B) > 0)).tolist()
    lens[0] = lens[-1] = 0
    pages = sum(-(-n // ps) for n in lens) + 1
    pool = filled_pool(pages, Hkv, ps, 3, 2, seed=B)
    table = table_for(lens, ps, pages)
    q = queries(B, Hq)
    out, lse = tq.paged_decode_attn(params(3, 2), q, pool, table, torch.tensor(lens, dtype=torch.int32, device="cuda"),
                                    window=window, return_lse=True)
    assert_close(out, lse, *reference(q, pool, table, lens, window))
    assert tq.decode_device_errors() == 0


@pytest.mark.parametrize("kb", [2, 3, 4])
@pytest.mark.parametrize("vb", [2, 3, 4])
@pytest.mark.parametrize("qjl", [True, False])
@pytest.mark.parametrize("Hq", [2, 6])
def test_decode_every_width(kb, vb, qjl, Hq):
    """Every pair of widths, with and without a sketch, up to four and up to eight heads per kv-head."""
    ps, lens = 16, [33, 5]
    pool = filled_pool(5, 1, ps, kb, vb, qjl, seed=kb + vb)
    table = table_for(lens, ps, 5)
    q = queries(2, Hq)
    out, lse = tq.paged_decode_attn(params(kb, vb, qjl), q, pool, table, torch.tensor(lens, dtype=torch.int32, device="cuda"),
                                    return_lse=True)
    assert_close(out, lse, *reference(q, pool, table, lens, qjl=qjl))


@pytest.mark.parametrize("vs,ks", [(1e-20, 1.0), (1e-6, 1e-5), (1e7, 1e6), (1e25, 1e15), ("growing", 1.0), ("falling", 1e-3)])
def test_decode_scales(vs, ks):
    """Values and keys of any magnitude (queries the other way, so that scores stay as they are); value norms
    that grow, or fall, by 2^40 along a sequence; zero values first."""
    ps, lens = 32, [700, 40]
    pages = 24
    pool = filled_pool(pages, 1, ps, 4, 4)
    table = table_for(lens, ps, pages)
    if isinstance(vs, str):
        for b, n in enumerate(lens):
            t = torch.arange(n, device="cuda")
            x = 2.0 ** (40.0 * (t if vs == "growing" else n - t) / n - 20)
            x[:17] = 0
            pool.v_norm[table[b, t // ps].long(), 0, t % ps] = x.float()
    else:
        pool.v_norm *= vs
    pool.k_norm *= ks
    pool.k_rnorm *= ks
    q = queries(2, 6) / ks
    out, lse = tq.paged_decode_attn(params(4, 4), q, pool, table, torch.tensor(lens, dtype=torch.int32, device="cuda"),
                                    return_lse=True)
    assert_close(out, lse, *reference(q, pool, table, lens))


def test_decode_batch_past_shared_memory():
    """More sequences than a CTA keeps the lengths of; empty ones in between and at both ends."""
    B, ps = 700, 16
    r = np.random.RandomState(3)
    lens = r.randint(0, 60, B)
    lens[r.rand(B) < 0.3] = 0
    lens[0] = lens[-1] = lens[300:340] = 0
    lens = lens.tolist()
    pages = sum(-(-n // ps) for n in lens) + 1
    pool = filled_pool(pages, 1, ps, 3, 3)
    table = table_for(lens, ps, pages)
    q = queries(B, 2)
    lt = torch.tensor(lens, dtype=torch.int32, device="cuda")
    for w in (0, 20):
        out, lse = tq.paged_decode_attn(params(3, 3), q, pool, table, lt, window=w, return_lse=True)
        assert_close(out, lse, *reference(q, pool, table, lens, w))


def test_decode_ignores_what_is_not_shown():
    """NaN norms and any codes in rows past the length, before the window, and in pages of no sequence."""
    ps, lens, window = 32, [45, 100, 0, 64], 40
    pages = 12
    pool = filled_pool(pages, 2, ps, 4, 4)
    table = table_for(lens, ps, pages)
    lt = torch.tensor(lens, dtype=torch.int32, device="cuda")
    q = queries(len(lens), 8)
    p = params(4, 4)
    shown = torch.zeros(pages, ps, dtype=torch.bool, device="cuda")
    for b, n in enumerate(lens):
        for t in range(max(0, n - window), n):
            shown[table[b, t // ps].long(), t % ps] = True
    want, wl = tq.paged_decode_attn(p, q, pool, table, lt, window=window, return_lse=True)
    hide = ~shown[:, None].expand(-1, 2, -1)
    for v in (float("nan"), float("inf"), -float("inf"), -3.4e38):
        for n in ("k_norm", "k_rnorm", "v_norm"):
            getattr(pool, n)[hide] = v
        pool.k_codes[hide] = 255
        got, gl = tq.paged_decode_attn(p, q, pool, table, lt, window=window, return_lse=True)
        assert torch.equal(got, want) and torch.equal(gl, wl)


def test_decode_equals_contiguous_decode_within_rounding():
    """Pages laid out in order are the contiguous cache's rows."""
    w = W.CONFIGS["llama3_8b_128k_b4"].scaled(T=512, B=2, Hkv=2, Hq=8)
    K, V = W.make_kv(w, "k").cuda(), W.make_kv(w, "v").cuda()
    p = tq.Params.create(W.rotation_for(w), W.qjl_for(w), 4, 4)
    flat = tq.Cache.allocate(2, 2, 512, 4, 4)
    tq.quantize(p, K, V, flat)
    pool = tq.Cache.allocate(16, 2, 64, 4, 4)
    slots = torch.arange(1024, device="cuda", dtype=torch.int32)
    tok = lambda x: x.permute(0, 2, 1, 3).reshape(1024, 2, 128)
    tq.paged_quantize(p, tok(K), tok(V), pool, slots)
    for n in ARRAYS:
        a, b = getattr(flat, n), getattr(pool, n)
        b = b.view(2, 8, 2, 64, *b.shape[3:]).transpose(1, 2).reshape(a.shape)
        if n in ("k_norm", "v_norm", "k_rnorm"):
            # the contract of the pipeline's side (tests/_parity.py): norms within NORM_ULP of the exact
            # value's rounding, ||r|| within 1e-5; the few-rows route rounds the exact value (2^-24)
            tol = 1e-5 + 2.0**-23 if n == "k_rnorm" else (NORM_ULP + 1) * 2.0**-23
            assert ((a - b).abs() <= tol * a.abs()).all(), n
        else:
            assert torch.equal(a, b), n
    q = W.make_queries(w).cuda()
    table = torch.arange(16, device="cuda", dtype=torch.int32).view(2, 8)
    a = tq.decode_attn(p, q, flat, 500)
    b = tq.paged_decode_attn(p, q, pool, table, torch.full((2,), 500, dtype=torch.int32, device="cuda"))
    assert (a - b).norm() <= 6e-4 * a.norm()


def test_decode_bad_pages_and_lengths_are_recorded():
    ps, lens = 32, [100, 70, 90]
    pool = filled_pool(12, 2, ps, 4, 4)
    table = table_for(lens, ps, 12)
    q, p = queries(3, 8), params(4, 4)
    lt = torch.tensor(lens, dtype=torch.int32, device="cuda")
    want = tq.paged_decode_attn(p, q, pool, table, lt)
    for bad in (12, -1, 2**31 - 1):
        t2 = table.clone()
        t2[1, 1] = bad
        got = tq.paged_decode_attn(p, q, pool, t2, lt)
        assert tq.decode_device_errors() == 16
        tq.reset_device_errors()
        for b in (0, 2):
            assert (got[b] - want[b]).norm() <= 1e-5 * want[b].norm()
    for n in (-1, table.shape[1] * ps + 1):
        l2 = lt.clone()
        l2[1] = n
        got = tq.paged_decode_attn(p, q, pool, table, l2)
        assert tq.decode_device_errors() == 16
        tq.reset_device_errors()
        for b in (0, 2):
            assert (got[b] - want[b]).norm() <= 1e-5 * want[b].norm()
    assert torch.equal(tq.paged_decode_attn(p, q, pool, table, lt), want) and tq.decode_device_errors() == 0


def test_decode_graph_streams_workspace_and_strides():
    ps, lens = 16, [200, 33, 0, 77]
    pool = filled_pool(40, 2, ps, 3, 3)
    table = table_for(lens, ps, 40)
    p, q = params(3, 3), queries(4, 8)
    lt = torch.tensor(lens, dtype=torch.int32, device="cuda")
    want = tq.paged_decode_attn(p, q, pool, table, lt)
    wide = torch.full((4, table.shape[1] + 7), 99, dtype=torch.int32, device="cuda")
    wide[:, 2:2 + table.shape[1]] = table
    assert torch.equal(tq.paged_decode_attn(p, q, pool, wide[:, 2:2 + table.shape[1]], lt), want)
    n = tq.paged_decode_workspace_size(4, 8, pool)
    ws = torch.full((n + 64,), 255, dtype=torch.uint8, device="cuda")
    assert torch.equal(tq.paged_decode_attn(p, q, pool, table, lt, workspace=ws[:n]), want)
    assert (ws[n:] == 255).all()
    with pytest.raises(tq.TqError):
        tq.paged_decode_attn(p, q, pool, table, lt, workspace=ws[:n - 256])
    # two calls at once on two streams, each with a workspace of its own
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    outs = [tq.paged_decode_attn(p, q, pool, table, lt, stream=s) for _ in range(20) for s in (s1, s2)]
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in outs)
    # one captured graph, replayed as lengths and pages change
    out = torch.empty_like(want)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        tq.paged_decode_attn(p, q, pool, table, lt, out=out, workspace=ws[:n])
    for new in ([1, 0, 0, 5], [0, 0, 0, 0], [200, 33, 0, 77]):
        lt.copy_(torch.tensor(new, dtype=torch.int32))
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, tq.paged_decode_attn(p, q, pool, table, lt))


def test_joined_by_lse():
    """Attention over two parts joined by their lse equals attention over the whole."""
    ps, n = 16, 160
    pool = filled_pool(10, 2, ps, 4, 4)
    p, q = params(4, 4), queries(1, 8)
    table = torch.arange(10, dtype=torch.int32, device="cuda")[None]
    L = lambda x: torch.tensor([x], dtype=torch.int32, device="cuda")
    whole, wl = tq.paged_decode_attn(p, q, pool, table, L(n), return_lse=True)
    a, al = tq.paged_decode_attn(p, q, pool, table, L(96), return_lse=True)
    b, bl = tq.paged_decode_attn(p, q, pool, table, L(n), window=64, return_lse=True)
    lse = torch.logaddexp(al, bl)
    both = a * (al - lse).exp()[..., None] + b * (bl - lse).exp()[..., None]
    assert (both - whole).norm() <= 6e-4 * whole.norm() and (lse - wl).abs().max() <= 3e-4


def test_offsets_past_32_bits():
    """A page whose rows lie past 4 GB of the code arrays."""
    ps, Hkv = 256, 8
    pages = (5 << 30) // (ps * Hkv * 64)
    pool = tq.Cache.allocate(pages, Hkv, ps, 4, 4)
    lens = [300]
    src = filled_pool(2, Hkv, ps, 4, 4)
    table = torch.tensor([[pages - 1, pages - 2]], dtype=torch.int32, device="cuda")
    for n in ARRAYS:
        getattr(pool, n)[pages - 1], getattr(pool, n)[pages - 2] = getattr(src, n)[0], getattr(src, n)[1]
    p, q = params(4, 4), queries(1, 32)
    lt = torch.tensor(lens, dtype=torch.int32, device="cuda")
    got = tq.paged_decode_attn(p, q, pool, table, lt)
    assert torch.equal(got, tq.paged_decode_attn(p, q, src, torch.tensor([[0, 1]], dtype=torch.int32, device="cuda"), lt))
    slots = torch.tensor([(pages - 1) * ps + 3, (pages - 2) * ps + 255], dtype=torch.int32, device="cuda")
    for a, b in zip(tq.paged_read(p, pool, slots), tq.paged_read(p, src, torch.tensor([3, 511], dtype=torch.int32, device="cuda"))):
        assert torch.equal(a, b)


# ------------------------------------------------------------------------------------------ rows

def check_rows(pool, slots, K, V, kb, vb, qjl):
    """The pool's rows against the oracle's quantization of K, V [N, Hkv, 128] (any float dtype)."""
    s = slots.cpu().numpy()
    keep = np.flatnonzero((s >= 0) & (s < pool.B * pool.T_cap))
    page, off = s[keep] // pool.T_cap, s[keep] % pool.T_cap
    at = lambda n: getattr(pool, n).transpose(1, 2)[torch.as_tensor(page, device="cuda"), torch.as_tensor(off, device="cuda")].cpu().numpy()
    Hkv = pool.Hkv
    x = lambda t: t.double().cpu().numpy()[keep].reshape(-1, 128)
    for name, X, bits, slot_of in (("k", x(K), kb, O.k_slot_of_coord), ("v", x(V), vb, O.v_slot_of_coord)):
        r = O.quantize_vectors(X, PI, bits, S if qjl and name == "k" else None)
        codes = at(name + "_codes").reshape(-1, 16 * bits)
        ex = O.code_exempt(r["u"], bits)
        got = O.unpack_codes(codes, bits, slot_of)
        assert not ((got != r["idx"]) & ~ex).any(), name
        assert ulp_distance_f32(at(name + "_norm").reshape(-1), r["n"].astype(np.float32)).max() <= NORM_ULP
        if "signs" in r:
            sx = O.sign_exempt(r["sproj"], ex)
            assert not ((O.unpack_signs(at("k_signs").reshape(-1, 16)) != r["signs"]) & ~sx).any()
            rn, clean = at("k_rnorm").reshape(-1), ~ex.any(1)
            assert (np.abs(rn - r["rnorm"])[clean] <= 1e-5 * r["rnorm"][clean] + 1e-30).all()


@pytest.mark.parametrize("kb,vb,qjl,dtype,N,Hkv,ps", [
    (4, 4, True, torch.bfloat16, 1, 8, 64), (4, 4, True, torch.bfloat16, 64, 8, 64), (3, 3, True, torch.float32, 37, 2, 16),
    (2, 2, False, torch.bfloat16, 129, 1, 32), (3, 2, True, torch.bfloat16, 601, 8, 16), (4, 3, True, torch.float32, 700, 8, 64),
    (4, 4, True, torch.bfloat16, 1300, 8, 128), (2, 3, False, torch.float32, 2500, 2, 48), (3, 4, True, torch.bfloat16, 2600, 2, 256)])
def test_quantize_rows(kb, vb, qjl, dtype, N, Hkv, ps):
    """Both routes (few rows, many rows), padding, and rows of other tokens left as they were."""
    torch.manual_seed(N)
    scale = torch.exp(0.5 * torch.randn(Hkv, 128, device="cuda"))
    scale[:, :3] *= 15
    K, V = ((torch.randn(N, Hkv, 128, device="cuda") * scale).to(dtype) for _ in range(2))
    pages = -(-N // ps) + 4
    slots = torch.randperm(pages * ps, device="cuda")[:N].to(torch.int32)
    if N > 1:
        slots[torch.rand(N, device="cuda") < 0.1] = -1
        slots[0] = pages * ps  # outside the pool: not written either
    pool = tq.Cache.allocate(pages, Hkv, ps, kb, vb, 128 if qjl else 0)
    for n in ARRAYS:
        if getattr(pool, n) is not None:
            getattr(pool, n).view(torch.uint8).fill_(0xA5)
    tq.paged_quantize(params(kb, vb, qjl), K, V, pool, slots)
    assert tq.quantize_device_errors() == 0
    check_rows(pool, slots, K, V, kb, vb, qjl)
    used = torch.zeros(pages * ps, dtype=torch.bool, device="cuda")
    used[slots[(slots >= 0) & (slots < pages * ps)].long()] = True
    rest = ~used.view(pages, 1, ps).expand(-1, Hkv, -1)
    for n in ARRAYS:
        if getattr(pool, n) is not None:
            a = getattr(pool, n)
            a = a.view(torch.uint8).view(pages, Hkv, ps, -1)
            assert (a[rest] == 0xA5).all(), n


@pytest.mark.parametrize("N", [24, 1700])
def test_quantize_in_a_graph_and_on_a_stream(N):
    """Both routes captured: a replay quantizes the inputs and slots as they are then; nothing to do for N = 0."""
    K, V = (torch.randn(N, 3, 128, device="cuda").to(torch.bfloat16) for _ in range(2))
    p, pool = params(4, 4), tq.Cache.allocate(-(-N // 16) + 2, 3, 16, 4, 4)
    slots = torch.arange(N, device="cuda", dtype=torch.int32)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        tq.paged_quantize(p, K, V, pool, slots)
    for _ in range(2):
        K.copy_(torch.randn(N, 3, 128, device="cuda"))
        slots.copy_(torch.randperm(pool.B * 16, device="cuda")[:N])
        g.replay()
        check_rows(pool, slots, K, V, 4, 4, True)
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    other = tq.Cache.allocate(pool.B, 3, 16, 4, 4)
    torch.cuda.synchronize()
    for _ in range(10):
        tq.paged_quantize(p, K, V, pool, slots, stream=a)
        tq.paged_quantize(p, V, K, other, slots, stream=b)
    torch.cuda.synchronize()
    check_rows(pool, slots, K, V, 4, 4, True)
    check_rows(other, slots, V, K, 4, 4, True)
    before = [getattr(pool, n).clone() for n in ARRAYS]
    tq.paged_quantize(p, K[:0], V[:0], pool, slots[:0])
    k, v, sg, rn = tq.paged_read(p, pool, slots[:0])
    assert k.shape == v.shape == sg.shape == (0, 3, 128) and rn.shape == (0, 3)
    assert all(torch.equal(a, getattr(pool, n)) for a, n in zip(before, ARRAYS))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("N", [40, 1700])
def test_quantize_special_rows_and_strides(dtype, N):
    """Zero rows, basis vectors, tiny and huge rows; a slice of a wider projection (strided rows)."""
    wide = torch.randn(N, 7, 128, device="cuda").to(dtype)
    wide[0] = 0
    wide[1] = 0
    wide[1, :, 5] = 3
    wide[2] *= 1e-30
    wide[3] *= 1e30
    K, V = wide[:, 1:4], wide[:, 4:7]
    slots = torch.arange(N, device="cuda", dtype=torch.int32)
    pool = tq.Cache.allocate(-(-N // 16), 3, 16, 4, 4)
    tq.paged_quantize(params(4, 4), K, V, pool, slots)
    check_rows(pool, slots, K, V, 4, 4, True)


@pytest.mark.parametrize("kb,vb,qjl,ps", [(4, 4, True, 16), (3, 3, True, 64), (2, 2, True, 32), (3, 2, False, 16), (4, 3, True, 48), (2, 4, True, 16)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_read_rows(kb, vb, qjl, ps, dtype):
    """Values to half a step of the output type plus the fp32 product's two roundings."""
    Hkv, pages, N = 3, 9, 211
    pool = filled_pool(pages, Hkv, ps, kb, vb, qjl)
    slots = torch.randint(-1, pages * ps, (N,), device="cuda", dtype=torch.int32)
    slots[7], slots[8] = pages * ps, slots[9]  # outside; a repeat
    k, v, signs, rn = tq.paged_read(params(kb, vb, qjl), pool, slots, dtype=dtype)
    s = slots.cpu().numpy()
    live = (s >= 0) & (s < pages * ps)
    page, off = torch.as_tensor(np.where(live, s, 0) // ps, device="cuda"), torch.as_tensor(np.where(live, s, 0) % ps, device="cuda")
    at = lambda n: getattr(pool, n).transpose(1, 2)[page, off].cpu().numpy()
    for got, name, bits, slot_of in ((k, "k", kb, O.k_slot_of_coord), (v, "v", vb, O.v_slot_of_coord)):
        idx = O.unpack_codes(at(name + "_codes").reshape(-1, 16 * bits), bits, slot_of).reshape(N, Hkv, 128)
        ref = O.codebook(bits).centroids[idx] * (at(name + "_norm").astype(np.float64) / math.sqrt(128))[..., None]
        ref[~live] = 0
        tol = (torch.finfo(dtype).eps / 2 * 1.001 + 3 * 2.0**-24) * np.abs(ref)
        assert (np.abs(got.double().cpu().numpy() - ref) <= tol).all()
    if not qjl:
        assert signs is None and rn is None
        return
    want = 2 * O.unpack_signs(at("k_signs").reshape(-1, 16)).reshape(N, Hkv, 128) - 1
    want[~live] = 0
    assert np.array_equal(signs.cpu().numpy(), want)
    assert np.array_equal(rn.cpu().numpy(), np.where(live[:, None], at("k_rnorm"), 0))


def test_a_serving_loop():
    """Rotate, reserve, quantize, attend, fork, free, compact: as a server runs them, one check per step
    against attention over the rows read back."""
    torch.manual_seed(0)
    Hq, Hkv, ps, n_seq = 8, 2, 16, 6
    p = params(4, 4)
    pool = tq.Cache.allocate(40, Hkv, ps, 4, 4)
    pt = tq.PageTable.allocate(n_seq, 10, 40, ps)
    ints = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    lens = [0] * n_seq

    def feed(seqs, counts):
        N = sum(counts)
        pos = ints([lens[s] + i for s, c in zip(seqs, counts) for i in range(c)])
        q = torch.randn(N, Hq, 128, device="cuda").to(torch.bfloat16)
        k = torch.randn(N, Hkv, 128, device="cuda").to(torch.bfloat16)
        v = torch.randn(N, Hkv, 128, device="cuda").to(torch.bfloat16)
        q, k = tq.rope(q, k, pos)
        slots = tq.pages_reserve(pt, ints(seqs), ints(counts), N + 3)
        tq.paged_quantize(p, torch.cat([k, k[:3]]), torch.cat([v, v[:3]]), pool, slots)
        for s, c in zip(seqs, counts):
            lens[s] += c
        return q

    def attend():
        q = torch.randn(n_seq, Hq, 128, device="cuda")
        out = tq.paged_decode_attn(p, q, pool, pt.table, pt.seq_lens)
        assert pt.seq_lens.tolist() == lens
        Sd, Pd = torch.tensor(S, device="cuda").double(), torch.tensor(PI, device="cuda").double()
        for b, n in enumerate(lens):
            if n == 0:
                assert (out[b] == 0).all()
                continue
            t = torch.arange(n, device="cuda")
            slots = (pt.table[b, t // ps] * ps + t % ps).to(torch.int32)
            k, v, sg, rn = (x.double() for x in tq.paged_read(p, pool, slots))
            k = k + (rn * math.sqrt(math.pi / 2) / 128)[..., None] * (sg @ Sd)
            qr = (q[b].double() @ Pd.T).view(Hkv, Hq // Hkv, 128)
            w = torch.softmax(torch.einsum("hgd,nhd->hgn", qr, k) / math.sqrt(128), -1)
            ref = torch.einsum("hgn,nhd->hgd", w, v).reshape(Hq, 128) @ Pd
            assert (out[b].double() - ref).norm() <= 3e-4 * ref.norm()
        pt.check()

    feed([0, 1, 2], [37, 16, 80])
    attend()
    for _ in range(3):
        feed([0, 1, 2], [1, 1, 1])
        attend()
    tq.pages_fork(pt, ints([0, 0]), ints([4, 5]), [pool])
    lens[4] = lens[5] = lens[0]
    attend()
    feed([0, 4, 5], [3, 20, 1])
    attend()
    tq.pages_free(pt, ints([0, 2]))
    lens[0] = lens[2] = 0
    tq.pages_compact(pt, [pool])
    attend()
    used = int((pt.refs > 0).sum())
    assert (pt.refs[:used] > 0).all() and (pt.refs[used:] == 0).all()
    feed([3, 2, 5], [50, 5, 1])
    attend()
    assert tq.decode_device_errors() == 0 and tq.quantize_device_errors() == 0
