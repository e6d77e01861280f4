"""Cases that measure the operators around a paged compressed cache: rotary positions with several
axes, page management (reserve, fork, free, compact), quantizing rows into pages, reading rows back,
and single-token attention over pages of 2..4-bit codes.

Every case has a plain form (elementary torch operations) and the framework's own calls, chosen by
the module's `own`.  A pool is six arrays [pages, kv-heads, page_size, ...]: packed key codes, sign
bits, key norms, residual norms, packed value codes, value norms (the row layout of include/tq.h).
"""
import functools
import math
import random

import numpy as np
import torch

own = False

D = 128
HALF_PI_ROOT = math.sqrt(math.pi / 2.0)
ROW_KEYS = ("k_codes", "k_signs", "k_norm", "k_rnorm", "v_codes", "v_norm")


# ------------------------------------------------------------------------------------------ cases

def listed():
    return [
        # one decode step of 64 sequences: rotate the new queries and keys
        dict(name="rope_step_64", op="rope", N=64, Hq=32, Hkv=8, axes=1, style="half", dtype="bf16",
             inverse=False, base=10000.0, far=32768),
        # a prompt with pictures and film frames: three axes, positions of a long context
        dict(name="rope_prompt_3axes", op="rope", N=16384, Hq=32, Hkv=8, axes=3, style="half", dtype="bf16",
             inverse=False, base=1000000.0, far=1048576),
        # the gradient of the same rotation in fp32, neighbouring pairs, two axes, an odd length
        dict(name="rope_grad_2axes", op="rope", N=5003, Hq=16, Hkv=2, axes=2, style="pair", dtype="f32",
             inverse=True, base=10000.0, far=131072),
        # best-of-n: drop the losing branches of 16 prompts and fork the winners again, 8 layers
        dict(name="fork_16_branches", op="fork", n=16, T=2000, page_size=64, Hkv=8, k_bits=4, v_bits=4, layers=8),
        # the older half of a busy pool leaves, the rest moves down, new sequences take the room
        dict(name="compact_pool", op="compact", n=256, T=4096, page_size=64, Hkv=8, k_bits=4, v_bits=4, layers=1),
        # one decode step of 64 sequences: 64 new rows per kv-head into their pages, and back
        dict(name="append_step_64", op="append", N=64, Hkv=8, page_size=64, k_bits=4, v_bits=4, dtype="bf16", pad=0.1),
        # a prefill chunk of 8192 tokens, compressed and read back for the chunk's own attention
        dict(name="append_chunk_8k", op="append", N=8192, Hkv=8, page_size=64, k_bits=4, v_bits=4, dtype="bf16", pad=0.0),
        # a cached prefix read back for a dense attention over it
        dict(name="read_prefix_32k", op="read", N=32768, Hkv=8, page_size=64, k_bits=3, v_bits=3, dtype="bf16"),
        # the smallest decode: one sequence of a few hundred tokens
        dict(name="decode_short_b1", op="decode", B=1, Hq=32, Hkv=8, T=500, ragged=False, page_size=64, k_bits=3,
             v_bits=3, window=0, dtype="bf16"),
        # a serving batch: 64 ragged sequences up to 16K tokens, eight heads per kv-head
        dict(name="decode_ragged_b64", op="decode", B=64, Hq=64, Hkv=8, T=16384, ragged=True, page_size=64, k_bits=3,
             v_bits=2, window=0, dtype="bf16"),
        # long contexts of equal length in 4 bits
        dict(name="decode_128k_b4", op="decode", B=4, Hq=32, Hkv=8, T=131072, ragged=False, page_size=128, k_bits=4,
             v_bits=4, window=0, dtype="bf16"),
        # a sliding window over long sequences, small pages, fp32 queries
        dict(name="decode_window_b32", op="decode", B=32, Hq=16, Hkv=2, T=40000, ragged=True, page_size=16, k_bits=4,
             v_bits=4, window=4096, dtype="f32"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "fork", "compact", "append", "read", "decode", "decode", "decode"])
    Hq, Hkv = rng.choice([(32, 8), (64, 8), (16, 2), (16, 1), (8, 8)])
    ps = rng.choice([16, 32, 64, 128, 256])
    kb, vb = rng.choice([(4, 4), (3, 3), (3, 2), (2, 2), (4, 3)])
    if op == "rope":
        return dict(op=op, N=_log_int(rng, 1, 16384), Hq=Hq if Hq < 64 else 32, Hkv=Hkv, axes=rng.choice([1, 2, 3]),
                    style=rng.choice(["half", "pair"]), dtype=rng.choice(["bf16", "f32"]) if Hq < 32 else "bf16",
                    inverse=rng.random() < 0.3, base=rng.choice([10000.0, 500000.0, 1000000.0]),
                    far=_log_int(rng, 2048, 1048576))
    if op == "fork":
        return dict(op=op, n=_log_int(rng, 1, 16), T=_log_int(rng, 1, 2000), page_size=ps, Hkv=Hkv, k_bits=kb,
                    v_bits=vb, layers=rng.randint(1, 8))
    if op == "compact":
        return dict(op=op, n=2 * _log_int(rng, 1, 64), T=_log_int(rng, 16, 4096), page_size=ps, Hkv=Hkv, k_bits=kb,
                    v_bits=vb, layers=rng.randint(1, 2))
    if op == "append":
        return dict(op=op, N=_log_int(rng, 1, 8192), Hkv=Hkv, page_size=ps, k_bits=kb, v_bits=vb,
                    dtype=rng.choice(["bf16", "bf16", "f32"]), pad=rng.choice([0.0, 0.1]))
    if op == "read":
        return dict(op=op, N=_log_int(rng, 1, 32768), Hkv=Hkv, page_size=ps, k_bits=kb, v_bits=vb,
                    dtype=rng.choice(["bf16", "f32"]))
    T = _log_int(rng, 16, 131072)
    most = max(1, (4 * 131072 * 8) // (T * Hkv))
    B = min(_log_int(rng, 1, 256), most)
    return dict(op=op, B=B, Hq=Hq, Hkv=Hkv, T=T, ragged=B > 1 and rng.random() < 0.7, page_size=ps, k_bits=kb,
                v_bits=vb, window=_log_int(rng, 1, T) if rng.random() < 0.25 else 0,
                dtype=rng.choice(["bf16", "bf16", "f32"]))


def lens_of(case):
    """Tokens of each sequence: a decode batch's lengths, the same for every seed."""
    if not case["ragged"]:
        return [case["T"]] * case["B"]
    r = random.Random(17 * case["B"] + case["T"])
    lens = [_log_int(r, max(1, case["T"] // 64), case["T"]) for _ in range(case["B"])]
    lens[0] = case["T"]
    lens[-1] = 0 if case["B"] > 2 else lens[-1]  # a slot of the batch that holds no sequence
    return lens


def row_bytes(case):
    return 16 * case["k_bits"] + 16 + 4 + 4 + 16 * case["v_bits"] + 4


def work(case):
    op = case["op"]
    if op == "rope":
        es = 2 if case["dtype"] == "bf16" else 4
        n = case["N"] * (case["Hq"] + case["Hkv"]) * D
        return {"bytes": 2 * es * n + 4 * case["axes"] * case["N"], "flops": 3 * n}
    if op == "fork":
        pages = case["n"] if case["T"] % case["page_size"] else 0
        moved = 2 * pages * case["page_size"] * case["Hkv"] * row_bytes(case) * case["layers"]
        return {"bytes": moved + 3 * 4 * case["n"] * pages_of(case["T"], case["page_size"]) + 64, "flops": 0}
    if op == "compact":
        per = pages_of(case["T"], case["page_size"]) * (case["n"] // 2)
        return {"bytes": 2 * per * case["page_size"] * case["Hkv"] * row_bytes(case) * case["layers"] + 32 * per,
                "flops": 0}
    if op in ("append", "read"):
        es = 2 if case["dtype"] == "bf16" else 4
        rows = case["N"] * case["Hkv"]
        back = 2 * D * es + D + 4  # values, signs and the residual norm of a row
        b = rows * (row_bytes(case) + back) + 4 * case["N"]
        if op == "read":
            return {"bytes": b, "flops": 2 * rows * D}
        return {"bytes": b + rows * 2 * D * es, "flops": 3 * 2 * rows * D * D}
    w = case["window"]
    tokens = sum(min(n, w) if w else n for n in lens_of(case))
    es = 2 if case["dtype"] == "bf16" else 4
    rows = case["B"] * case["Hq"]
    return {"bytes": tokens * case["Hkv"] * row_bytes(case) + rows * (2 * D * es + 4),
            "flops": 2 * 3 * tokens * case["Hq"] * D + 3 * 2 * rows * D * D}


def pages_of(tokens, page_size):
    return -(-tokens // page_size)


# ------------------------------------------------------------------------------- shared constants

def _cdf(x):
    return 0.5 * math.erfc(-x / math.sqrt(2.0))


def _pdf(x):
    return 0.0 if math.isinf(x) else math.exp(-0.5 * x * x) / math.sqrt(2.0 * math.pi)


@functools.lru_cache(None)
def codebook(bits):
    """Lloyd-Max grid of N(0,1): centroids rounded to fp16, thresholds their exact midpoints."""
    L = 1 << bits
    c = [3.0 * (k - (L - 1) / 2) / L for k in range(L)]
    move = 1.0
    while move > 1e-13:
        t = [-math.inf] + [0.5 * (c[i] + c[i + 1]) for i in range(L - 1)] + [math.inf]
        n = [(_pdf(t[k]) - _pdf(t[k + 1])) / (_cdf(t[k + 1]) - _cdf(t[k])) for k in range(L)]
        move = max(abs(a - b) for a, b in zip(c, n))
        c = n
    c = np.array(c)
    c = (0.5 * (c - c[::-1])).astype(np.float16).astype(np.float64)
    return c, 0.5 * (c[1:] + c[:-1])


def inv_freq(base):
    return float(base) ** (-torch.arange(0, D, 2, dtype=torch.float64) / D)


def sections_of(axes):
    return {1: (64,), 2: (32, 32), 3: (16, 24, 24)}[axes]


def layout_maps():
    """Where coordinate j (or sketch row j) of a row sits: key slot, value slot, sign bit."""
    j = torch.arange(D)
    a, h, t, e = j // 16, (j // 8) % 2, (j // 2) % 4, j % 2
    return 32 * t + 4 * a + 2 * h + e, 16 * (j % 8) + j // 8, 32 * t + 2 * a + h + 16 * e


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _dtype(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


# ---------------------------------------------------------------------------------------- prepare

def _constants(case, g):
    """The layer's constants: rotation, sketch, codebooks and the product sketch x rotation."""
    q, r = torch.linalg.qr(torch.randn(D, D, generator=g, device="cuda", dtype=torch.float64))
    Pi = (q * torch.sign(torch.diagonal(r))).float().contiguous()
    S = torch.randn(D, D, generator=g, device="cuda").half().float()
    f = lambda x: torch.tensor(x, dtype=torch.float32, device="cuda")
    (kc, kt), (vc, vt) = codebook(case["k_bits"]), codebook(case["v_bits"])
    ks, vs, sb = layout_maps()
    return dict(Pi=Pi, S=S, S_Pi=S.double() @ Pi.double(), kc=f(kc), kt=f(kt), vc=f(vc), vt=f(vt),
                ks=ks.cuda(), vs=vs.cuda(), sb=sb.cuda(), k_bits=case["k_bits"], v_bits=case["v_bits"])


def _empty_pool(case, pages, layers=()):
    u8 = dict(dtype=torch.uint8, device="cuda")
    f32 = dict(dtype=torch.float32, device="cuda")
    s = (*layers, pages, case["Hkv"], case["page_size"])
    return dict(k_codes=torch.zeros(*s, 16 * case["k_bits"], **u8), k_signs=torch.zeros(*s, 16, **u8),
                k_norm=torch.zeros(*s, **f32), k_rnorm=torch.zeros(*s, **f32),
                v_codes=torch.zeros(*s, 16 * case["v_bits"], **u8), v_norm=torch.zeros(*s, **f32))


def _pack(codes, bits):
    """Codes [rows, 128] in slot order to a little-endian bit stream [rows, 16 * bits]."""
    b = (codes.unsqueeze(-1) >> torch.arange(bits, device=codes.device, dtype=torch.uint8)) & 1
    b = b.reshape(codes.shape[0], 16 * bits, 8) << torch.arange(8, device=codes.device, dtype=torch.uint8)
    return b.sum(-1, dtype=torch.uint8)


def _fill_codes(dst, thresholds, slot, g, most=1 << 18):
    """Codes of Gaussian coordinates (what the rotation makes of any vector), packed into rows."""
    rows = dst.view(-1, dst.shape[-1])
    bits = dst.shape[-1] // 16
    for at in range(0, rows.shape[0], most):
        n = min(most, rows.shape[0] - at)
        u = torch.randn(n, D, generator=g, device="cuda")
        codes = torch.bucketize(u, thresholds, right=True).to(torch.uint8)
        rows[at:at + n] = _pack(codes, bits)


def _filled_pool(case, pages, const, g, layers=()):
    pool = _empty_pool(case, pages, layers)
    _fill_codes(pool["k_codes"], const["kt"], const["ks"], g)
    _fill_codes(pool["v_codes"], const["vt"], const["vs"], g)
    pool["k_signs"].random_(0, 256, generator=g)
    f = lambda x: torch.randn(x.shape, generator=g, device="cuda").mul_(0.3).exp_().mul_(math.sqrt(D))
    pool["k_norm"].copy_(f(pool["k_norm"]))
    pool["v_norm"].copy_(f(pool["v_norm"]))
    # the residual's share of the norm: the distortion of the grid, 2.7 x 4^-bits at most
    pool["k_rnorm"].copy_(pool["k_norm"] * math.sqrt(2.4 * 4.0 ** -case["k_bits"]))
    return pool


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    st = dict(case)
    if op == "rope":
        dt = _dtype(case)
        st["q"] = torch.randn(case["N"], case["Hq"], D, generator=g, device="cuda").to(dt)
        st["k"] = torch.randn(case["N"], case["Hkv"], D, generator=g, device="cuda").to(dt)
        st["pos"] = torch.randint(0, case["far"], (case["axes"], case["N"]), generator=g, device="cuda",
                                  dtype=torch.int32)
        st["freq"] = inv_freq(case["base"]).cuda()
        return st
    if op in ("append", "read"):
        const = st["const"] = _constants(case, g)
        pages = pages_of(case["N"], case["page_size"]) + 3
        room = torch.randperm(pages * case["page_size"], generator=g, device="cuda")[:case["N"]]
        if op == "append" and case["N"] > 1024:  # whole pages in a shuffled order, as a prompt fills them
            order = torch.randperm(pages, generator=g, device="cuda")
            t = torch.arange(case["N"], device="cuda")
            room = order[t // case["page_size"]] * case["page_size"] + t % case["page_size"]
        if op == "append" and case["pad"]:  # rows of a padded batch that belong to no sequence
            out = torch.rand(case["N"], generator=g, device="cuda") < case["pad"]
            room = torch.where(out, -1, room)
        st["slots"] = room.to(torch.int32)
        if op == "read":
            st["pool"] = _filled_pool(case, pages, const, g)
            return st
        st["pool"] = _empty_pool(case, pages)
        scale = (0.5 * torch.randn(2, case["Hkv"], D, generator=g, device="cuda")).exp()
        scale[:, :, torch.randperm(D, generator=g, device="cuda")[:3]] *= 15.0  # outlier channels
        x = torch.randn(2, case["N"], case["Hkv"], D, generator=g, device="cuda") * scale[:, None]
        st["k"], st["v"] = x.to(_dtype(case)).unbind(0)
        return st
    if op in ("fork", "compact"):
        n, ps, per = case["n"], case["page_size"], pages_of(case["T"], case["page_size"])
        n_seq = 2 * n if op == "fork" else n
        pages = (n * per + n) if op == "fork" else n * per
        pages += 5
        const = _constants(case, g)
        st["pool"] = _filled_pool(case, pages, const, g, (case["layers"],))
        st["refs"] = torch.zeros(pages, dtype=torch.int32, device="cuda")
        st["lens"] = torch.zeros(n_seq, dtype=torch.int32, device="cuda")
        st["table"] = torch.full((n_seq, per + 2), -1, dtype=torch.int32, device="cuda")
        st["status"] = torch.zeros(1, dtype=torch.int32, device="cuda")
        live = n
        where = torch.randperm(pages, generator=g, device="cuda")[:n * per] if op == "fork" else torch.arange(n * per, device="cuda")
        st["table"][:live, :per] = where.view(live, per).to(torch.int32)
        st["lens"][:live] = case["T"]
        st["refs"][where] = 1
        ids = torch.randperm(n, generator=g, device="cuda").to(torch.int32)
        if op == "fork":
            st["src"], st["dst"] = ids, torch.arange(n, 2 * n, device="cuda", dtype=torch.int32)
        else:
            st["lens"][:live] -= torch.randint(0, ps, (n,), generator=g, device="cuda").clamp_max(case["T"] - (per - 1) * ps - 1).to(torch.int32)
            old = torch.arange(n // 2, device="cuda", dtype=torch.int32)
            st["sets"] = [old, old + n // 2]
            st["grow"] = [st["lens"][s.long()].clone() for s in st["sets"]]
            st["most"] = (n // 2) * case["T"]
        return st
    # decode
    const = st["const"] = _constants(case, g)
    ps = case["page_size"]
    lens = lens_of(case)
    per = max(1, pages_of(max(lens), ps))
    counts = torch.tensor([pages_of(n, ps) for n in lens])
    pages = int(counts.sum()) + 2
    st["pool"] = _filled_pool(case, pages, const, g)
    st["lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
    order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    at = torch.arange(per)[None] + (counts.cumsum(0) - counts)[:, None]
    mine = torch.arange(per)[None] < counts[:, None]
    st["table"] = torch.where(mine.cuda(), order[at.clamp_max(pages - 1).cuda()], -1).to(torch.int32)
    st["q"] = torch.randn(case["B"], case["Hq"], D, generator=g, device="cuda").to(_dtype(case))
    return st


# ------------------------------------------------------------------------------- the framework's calls

def _own_params(tq, c):
    return tq.Params(c["Pi"], c["S"], c["kc"], c["kt"], c["vc"], c["vt"], c["S_Pi"])


def _own_cache(tq, st, pool):
    return tq.Cache(pool["k_norm"].shape[0], st["Hkv"], st["page_size"], st["k_bits"], st["v_bits"], D,
                    *(pool[k] for k in ROW_KEYS))


def _own_table(tq, st):
    return tq.PageTable(st["page_size"], st["table"], st["lens"], st["refs"], st["status"])


def _layers(tq, st):
    return [_own_cache(tq, st, {k: st["pool"][k][i] for k in ROW_KEYS}) for i in range(st["layers"])]


def _run_own(st):
    import decode_attention_11_b200 as tq
    op = st["op"]
    if op == "rope":
        return tq.rope(st["q"], st["k"], st["pos"], sections=sections_of(st["axes"]), base=st["base"],
                       style=tq.TQ_ROPE_HALF if st["style"] == "half" else tq.TQ_ROPE_PAIR, inverse=st["inverse"])
    if op == "append":
        params, cache = _own_params(tq, st["const"]), _own_cache(tq, st, st["pool"])
        tq.paged_quantize(params, st["k"], st["v"], cache, st["slots"])
        return tq.paged_read(params, cache, st["slots"], dtype=st["k"].dtype)
    if op == "read":
        return tq.paged_read(_own_params(tq, st["const"]), _own_cache(tq, st, st["pool"]), st["slots"],
                             dtype=_dtype(st))
    if op == "fork":
        pt, caches = _own_table(tq, st), _layers(tq, st)
        tq.pages_free(pt, st["dst"])
        tq.pages_fork(pt, st["src"], st["dst"], caches)
        return _tables(st)
    if op == "compact":
        pt, caches = _own_table(tq, st), _layers(tq, st)
        tq.pages_free(pt, st["sets"][0])
        tq.pages_compact(pt, caches)
        slots = tq.pages_reserve(pt, st["sets"][0], st["grow"][0], st["most"])
        return _next_half(st, slots)
    return tq.paged_decode_attn(_own_params(tq, st["const"]), st["q"], _own_cache(tq, st, st["pool"]), st["table"],
                                st["lens"], window=st["window"], out_dtype=_dtype(st), return_lse=True)


def _tables(st):
    return dict(table=st["table"], lens=st["lens"], refs=st["refs"], status=st["status"],
                **{k: st["pool"][k] for k in ROW_KEYS})


def _next_half(st, slots):
    st["sets"].reverse()
    st["grow"].reverse()
    return dict(_tables(st), slots=slots)


# ---------------------------------------------------------------------------------- the plain forms

def _unpack(rows, bits, where):
    """Codes of packed rows [..., 16 * bits], as indices [..., 128] in coordinate order."""
    b = (rows.unsqueeze(-1) >> torch.arange(8, device=rows.device, dtype=torch.uint8)) & 1
    b = b.view(*rows.shape[:-1], D, bits)
    codes = (b << torch.arange(bits, device=rows.device, dtype=torch.uint8)).sum(-1, dtype=torch.uint8)
    return codes[..., where].int()


def _sign_bits(rows, where):
    b = (rows.unsqueeze(-1) >> torch.arange(8, device=rows.device, dtype=torch.uint8)) & 1
    return b.view(*rows.shape[:-1], D)[..., where]


def _rope(x, cos, sin, style, dtype):
    x = x.to(cos.dtype)
    if style == "half":
        a, b = x[..., :64], x[..., 64:]
        y = torch.cat([a * cos - b * sin, a * sin + b * cos], -1)
    else:
        a, b = x[..., 0::2], x[..., 1::2]
        y = torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2)
    return y.to(dtype)


def _plain_rope(st, work_dtype=torch.float32):
    axis = torch.repeat_interleave(torch.arange(st["axes"], device="cuda"),
                                   torch.tensor(sections_of(st["axes"]), device="cuda"), output_size=64)
    angle = st["pos"].double()[axis].t() * st["freq"]  # [N, 64], in 64 bits: positions are far
    angle = -angle if st["inverse"] else angle
    cos, sin = angle.cos().to(work_dtype)[:, None], angle.sin().to(work_dtype)[:, None]
    dt = st["q"].dtype if work_dtype == torch.float32 else work_dtype
    return _rope(st["q"], cos, sin, st["style"], dt), _rope(st["k"], cos, sin, st["style"], dt)


def _plain_quantize(x, c, which):
    """(index, norm, u) of rows, in 64 bits: a code next to a threshold depends on every bit."""
    x = x.double()
    n = x.square().sum(-1).sqrt()
    u = math.sqrt(D) * (x @ c["Pi"].double().t()) / torch.where(n > 0, n, torch.ones_like(n))[..., None]
    idx = (u.unsqueeze(-1) >= c[which + "t"].double()).sum(-1)
    return idx, n, u


def _plain_append(st):
    c, dt = st["const"], st["k"].dtype
    ki, kn, ku = _plain_quantize(st["k"], c, "k")
    vi, vn, _ = _plain_quantize(st["v"], c, "v")
    rho = ku - c["kc"].double()[ki]
    rn = (kn * rho.square().sum(-1).sqrt() / math.sqrt(D)).float()
    signs = torch.where(rho @ c["S"].double().t() >= 0, 1, -1).to(torch.int8)
    kept = (st["slots"] >= 0)[:, None]
    k = (kn.float() / math.sqrt(D))[..., None] * c["kc"][ki]
    v = (vn.float() / math.sqrt(D))[..., None] * c["vc"][vi]
    return ((k * kept[..., None]).to(dt), (v * kept[..., None]).to(dt), signs * kept[..., None], rn * kept)


def _rows(st, key):
    """Rows [N, kv-heads, ...] of the slots of a pool array."""
    s = st["slots"].clamp_min(0).long()
    return st["pool"][key][s // st["page_size"], :, s % st["page_size"]]


def _plain_read(st):
    c, dt = st["const"], _dtype(st)
    k = c["kc"][_unpack(_rows(st, "k_codes"), st["k_bits"], c["ks"])] * (_rows(st, "k_norm") / math.sqrt(D))[..., None]
    v = c["vc"][_unpack(_rows(st, "v_codes"), st["v_bits"], c["vs"])] * (_rows(st, "v_norm") / math.sqrt(D))[..., None]
    signs = _sign_bits(_rows(st, "k_signs"), c["sb"]).to(torch.int8) * 2 - 1
    return k.to(dt), v.to(dt), signs, _rows(st, "k_rnorm")


def _plain_free(st, seqs):
    seqs = seqs.long()
    col = torch.arange(st["table"].shape[1], device="cuda")
    held = col < ((st["lens"][seqs] + st["page_size"] - 1) // st["page_size"])[:, None]
    st["refs"].index_add_(0, st["table"][seqs].clamp_min(0).flatten().long(), -held.flatten().int())
    st["table"][seqs] = -1
    st["lens"][seqs] = 0


def _plain_fork(st):
    _plain_free(st, st["dst"])
    ps, src, dst, refs = st["page_size"], st["src"].long(), st["dst"].long(), st["refs"]
    lens, rows = st["lens"][src], st["table"][src]
    full, part = lens // ps, lens % ps > 0
    room = torch.argsort((refs > 0).int(), stable=True)  # the free pages first, lowest first
    new = room[(part.int().cumsum(0) - 1).clamp_min(0)]
    last = rows.gather(1, full.long().clamp_max(rows.shape[1] - 1)[:, None])[:, 0].clamp_min(0).long()
    to = torch.where(part, new, last)
    col = torch.arange(rows.shape[1], device="cuda")
    child = torch.where(col < full[:, None], rows, -1)
    child = torch.where((col == full[:, None]) & part[:, None], to[:, None].int(), child)
    st["table"][dst] = child
    st["lens"][dst] = lens
    refs.index_add_(0, rows.clamp_min(0).flatten().long(), (col < full[:, None]).flatten().int())
    refs.index_add_(0, new, part.int())
    [a.index_copy_(1, to, a.index_select(1, last)) for a in st["pool"].values()]
    return _tables(st)


def _plain_compact(st):
    ps, refs, ids = st["page_size"], st["refs"], torch.arange(st["refs"].shape[0], device="cuda")
    seqs, grow = st["sets"][0].long(), st["grow"][0]
    _plain_free(st, st["sets"][0])
    # live pages above the number of live pages move into the free ones below it, in order
    live = refs > 0
    n_live = live.sum()
    to, frm = torch.nonzero(~live & (ids < n_live))[:, 0], torch.nonzero(live & (ids >= n_live))[:, 0]
    [a.index_copy_(1, to, a.index_select(1, frm)) for a in st["pool"].values()]
    new_id = ids.clone()
    new_id[frm] = to
    st["table"].copy_(torch.where(st["table"] >= 0, new_id[st["table"].clamp_min(0).long()].int(), -1))
    refs[to] = refs[frm]
    refs[frm] = 0
    # the half that left comes back as new sequences: lowest free pages, in the order of the list
    need = (grow + ps - 1) // ps
    room = torch.argsort((refs > 0).int(), stable=True).int()
    col = torch.arange(st["table"].shape[1], device="cuda")
    at = (need.cumsum(0) - need)[:, None] + col
    held = col < need[:, None]
    rows = torch.where(held, room[at.clamp_max(room.shape[0] - 1)], -1)
    st["table"][seqs] = rows
    st["lens"][seqs] = grow
    refs.index_add_(0, rows.clamp_min(0).flatten().long(), held.flatten().int())
    tok = torch.arange(st["most"], device="cuda")
    end = grow.cumsum(0)
    i = (tok[:, None] >= end).sum(-1)
    inside = i < grow.shape[0]
    i = i.clamp_max(grow.shape[0] - 1)
    p = tok - (end - grow)[i]
    slots = rows[i, (p // ps).clamp(0, rows.shape[1] - 1)] * ps + (p % ps).int()
    return _next_half(st, torch.where(inside, slots, -1).int())


def _plain_decode(st):
    c, pool, ps = st["const"], st["pool"], st["page_size"]
    B, Hq, Hkv = st["B"], st["Hq"], st["Hkv"]
    g = Hq // Hkv
    pages = st["table"].clamp_min(0).long()
    T = pages.shape[1] * ps

    def gather(key):  # [B, kv-heads, T, ...]
        x = pool[key][pages]
        return x.transpose(1, 2).reshape(B, Hkv, T, *x.shape[4:])

    q = (st["q"].float() @ c["Pi"].t()).view(B, Hkv, g, D)
    sq = q @ c["S"].t()
    est = (q @ c["kc"][_unpack(gather("k_codes"), st["k_bits"], c["ks"])].transpose(-1, -2)) \
        * (gather("k_norm") / math.sqrt(D))[:, :, None]
    signs = _sign_bits(gather("k_signs"), c["sb"]).float() * 2 - 1
    est += (sq @ signs.transpose(-1, -2)) * (gather("k_rnorm") * (HALF_PI_ROOT / D))[:, :, None]
    del signs
    t = torch.arange(T, device="cuda")
    n = st["lens"][:, None]
    seen = (t < n) & (t >= n - st["window"]) if st["window"] else t < n
    est = torch.where(seen[:, None, None], est / math.sqrt(D), -math.inf)
    top = est.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    p = (est - top).exp()
    total = p.sum(-1, keepdim=True)
    vn = torch.where(seen[:, None], gather("v_norm"), 0.0) / math.sqrt(D)
    o = (p * vn[:, :, None]) @ c["vc"][_unpack(gather("v_codes"), st["v_bits"], c["vs"])]
    o = (o / torch.where(total > 0, total, 1.0)) @ c["Pi"]
    return o.view(B, Hq, D).to(_dtype(st)), (top + total.log()).view(B, Hq)


def run(state):
    if own:
        return _run_own(state)
    return {"rope": _plain_rope, "append": _plain_append, "read": _plain_read, "fork": _plain_fork,
            "compact": _plain_compact, "decode": _plain_decode}[state["op"]](state)


# -------------------------------------------------------------------------- the definitions in 64 bits

def _code_at(row, bits, j_slot):
    """Code at slot j_slot of packed rows, read as a window of two bytes of the bit stream."""
    bit = bits * j_slot
    lo = row[..., bit // 8].long()
    hi = row[..., (bit // 8 + 1).clamp_max(row.shape[-1] - 1)].long()
    return ((lo | (hi << 8)) >> (bit % 8)) & ((1 << bits) - 1)


def _exact_rope(case, st):
    """Each pair as a complex number times e^(i angle)."""
    i = torch.arange(64, device="cuda")
    ends = torch.tensor(sections_of(case["axes"]), device="cuda").cumsum(0)
    axis = (i[:, None] >= ends).sum(-1)
    theta = torch.exp(-math.log(case["base"]) * 2.0 * i.double() / D)
    angle = st["pos"].double().t()[:, axis] * theta * (-1.0 if case["inverse"] else 1.0)
    turn = torch.polar(torch.ones_like(angle), angle)[:, None]
    out = []
    for x in (st["q"].double(), st["k"].double()):
        if case["style"] == "half":
            z = torch.complex(x[..., :64].contiguous(), x[..., 64:].contiguous()) * turn
            out.append(torch.cat([z.real, z.imag], -1))
        else:
            z = torch.view_as_complex(x.unflatten(-1, (64, 2)).contiguous()) * turn
            out.append(torch.view_as_real(z).flatten(-2))
    return tuple(out)


def _exact_append(case, st):
    c = st["const"]
    Pi, S = c["Pi"].double(), c["S"].double()
    res = []
    for x, cc, ct in ((st["k"], c["kc"], c["kt"]), (st["v"], c["vc"], c["vt"])):
        x = x.double()
        n = torch.linalg.vector_norm(x, dim=-1, keepdim=True)
        u = math.sqrt(D) * torch.einsum("ij,nhj->nhi", Pi, x) / n
        val = cc.double()[torch.searchsorted(ct.double(), u, right=True)]
        res.append((n, u, val))
    (kn, ku, kv), (vn, _, vv) = res
    rho = ku - kv
    sign = torch.einsum("lj,nhj->nhl", S, rho) >= 0
    keep = (st["slots"] >= 0).double()[:, None, None]
    return (kn * kv / math.sqrt(D) * keep, vn * vv / math.sqrt(D) * keep, (sign.double() * 2 - 1) * keep,
            (kn * torch.linalg.vector_norm(rho, dim=-1, keepdim=True) / math.sqrt(D) * keep)[..., 0])


def _exact_read(case, st):
    c, s = st["const"], st["slots"].long()
    page, off = s // case["page_size"], s % case["page_size"]
    at = lambda key: st["pool"][key].transpose(1, 2)[page, off]
    k = c["kc"].double()[_code_at(at("k_codes"), case["k_bits"], c["ks"])] * at("k_norm").double()[..., None]
    v = c["vc"].double()[_code_at(at("v_codes"), case["v_bits"], c["vs"])] * at("v_norm").double()[..., None]
    signs = 2.0 * _code_at(at("k_signs"), 1, c["sb"]).double() - 1.0
    return k / math.sqrt(D), v / math.sqrt(D), signs, at("k_rnorm").double()


def _exact_decode(case, st):
    c, ps = st["const"], case["page_size"]
    B, Hq, Hkv = case["B"], case["Hq"], case["Hkv"]
    Pi, S = c["Pi"].double(), c["S"].double()
    out = torch.zeros(B, Hq, D, dtype=torch.float64, device="cuda")
    lse = torch.full((B, Hq), -math.inf, dtype=torch.float64, device="cuda")
    for b, n in enumerate(lens_of(case)):
        first = max(0, n - case["window"]) if case["window"] else 0
        if first >= n:
            continue
        t = torch.arange(first, n, device="cuda")
        page = st["table"][b, t // ps].long()
        for h in range(Hkv):
            at = lambda key: st["pool"][key][page, h, t % ps]
            khat = c["kc"].double()[_code_at(at("k_codes"), case["k_bits"], c["ks"])] * (at("k_norm").double() / math.sqrt(D))[:, None]
            sign = 2.0 * _code_at(at("k_signs"), 1, c["sb"]).double() - 1.0
            # the estimator as one vector per key: khat + ||r|| sqrt(pi/2)/m S^T sign
            khat = khat + (at("k_rnorm").double() * HALF_PI_ROOT / D)[:, None] * (sign @ S)
            hs = slice(h * Hq // Hkv, (h + 1) * Hq // Hkv)
            score = (st["q"][b, hs].double() @ Pi.t()) @ khat.t() / math.sqrt(D)
            lse[b, hs] = torch.logsumexp(score, -1)
            p = (score - lse[b, hs][:, None]).exp()
            vhat = c["vc"].double()[_code_at(at("v_codes"), case["v_bits"], c["vs"])] * (at("v_norm").double() / math.sqrt(D))[:, None]
            out[b, hs] = (p @ vhat) @ Pi
    return out, lse


def exact(case, seed):
    if case["op"] in ("fork", "compact"):  # whole numbers and copied rows: nothing is computed
        return None
    st = prepare(case, seed)
    r = {"rope": _exact_rope, "append": _exact_append, "read": _exact_read, "decode": _exact_decode}[case["op"]](case, st)
    if case["op"] in ("append", "read"):  # the signs are whole numbers
        r = (r[0], r[1], None, r[3])
    return r
