"""Paged decode attention where single tokens are far out of scale, against the float64 oracle.

Output tolerance where one token has all the weight.  Its weight enters as fp16 hi + lo (2^-22) and its
values are exact; sums and normalisation are fewer than 16 fp32 roundings (16 * 2^-24).  The rotation back
drops products of two lo parts and rounds the parts (2^-21 of each product) and sums eight k-steps in fp32
(24 * 2^-24 at most): a coordinate is off by that times sum_j |Pi[j][i]| |o'[j]| <= |o'|, so the vector by
sqrt(128) (2^-21 + 24 * 2^-24) = 2.2e-5 of its norm.  Together below 3e-5.

lse: a score's error is at most |q| |k| / sqrt(128) * (2 * 2^-22 + 24 * 2^-23) (q' and S q' as hi + lo, 24
fp32 sums)."""
import math

import numpy as np
import pytest
import torch

import decode_attention_11_b200 as tq
from oracle import tq_oracle as O

from test_gpu_paged import PI, S, filled_pool, params, reference, rows_of, table_for

pytestmark = pytest.mark.gpu

ALL_WEIGHT = 3e-5
SCORE = 2 * 2.0**-22 + 24 * 2.0**-23


def like_queries(B, Hq, seed=5):
    """Queries of norm 15 whose heads differ little, so that one key stands out for all of them."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    q = torch.randn(B, 1, 128, generator=g, device="cuda") + 0.05 * torch.randn(B, Hq, 128, generator=g, device="cuda")
    return q * (15.0 / q.norm(dim=-1, keepdim=True))


def raise_score(pool, table, q, b, lo, hi, score):
    """The token of [lo, hi) that suits sequence b's queries best gets the key norm that gives head 0 that score."""
    t = np.arange(lo, hi)
    c = rows_of(pool, table, b, t)
    est = O.score_estimates(q[b, 0].double().cpu().numpy(), PI, S, c["k_codes"][0, 0], c["k_norm"][0, 0], pool.k_bits,
                            c["k_signs"][0, 0], c["k_rnorm"][0, 0]) / math.sqrt(128)
    i = int(np.argmax(est / c["k_norm"][0, 0]))
    norm = float(c["k_norm"][0, 0, i] * score / est[i])
    page, off = table[b, t[i] // pool.T_cap].long(), int(t[i]) % pool.T_cap
    pool.k_norm[page, 0, off], pool.k_rnorm[page, 0, off] = norm, 0.15 * norm
    return int(t[i]), norm


@pytest.mark.parametrize("Hq", [3, 6])
@pytest.mark.parametrize("kb,vb", [(4, 4), (3, 2)])
@pytest.mark.parametrize("ratio", [2.0**20, 2.0**30, 2.0**36])
def test_large_value_norm_without_weight(Hq, kb, vb, ratio):
    """A token whose value norm is 2^20 .. 2^36 times the others', at a score about 60 below the maximum (it
    adds less than 1e-14), before and after the token that has the weight, in its group of 16 and in the
    groups beside it (a warp's range is three to five groups here)."""
    away = [1, -1, 3, -3, 7, -7, 16, -16, 20, -20, 33, -33]
    B, ps, T = len(away), 64, 8000
    lens = [T] * B
    pages = B * (-(-T // ps))
    pool = filled_pool(pages, 1, ps, kb, vb, seed=kb)
    pool.k_norm.mul_(0.1)  # scores of a few units
    pool.k_rnorm.mul_(0.1)
    table = table_for(lens, ps, pages)
    q = like_queries(B, Hq)
    norms = []
    for b, d in enumerate(away):
        i, n = raise_score(pool, table, q, b, 4000 + 64 * b, 4064 + 64 * b, 60.0)
        norms.append(n)
        pool.v_norm[table[b, (i + d) // ps].long(), 0, (i + d) % ps] = 10.0 * ratio
    out, lse = tq.paged_decode_attn(params(kb, vb), q, pool, table, torch.tensor(lens, dtype=torch.int32, device="cuda"),
                                    return_lse=True)
    ref, rl = reference(q, pool, table, lens)
    got = out.double().cpu().numpy()
    err = np.linalg.norm(got - ref, axis=-1) / np.linalg.norm(ref, axis=-1)
    assert (err <= ALL_WEIGHT).all(), err.max(axis=1)
    tol = 15.0 * np.array(norms)[:, None] / math.sqrt(128) * SCORE + 2.0**-22 * np.abs(rl)
    assert (np.abs(lse.double().cpu().numpy() - rl) <= tol).all()


@pytest.mark.parametrize("Hq", [4, 8])
@pytest.mark.parametrize("big", [1e28, 1e31, 1e33])
def test_scores_far_below_zero(Hq, big):
    """Scores of +-1e28 .. +-1e33 and more: where all of a head are negative the nearest to zero has the weight,
    and a sequence of one token gives that token whatever its score.  Half the heads are the others' negatives,
    so both signs are there.  (Scores of two tokens that come within their error of each other are left out: the
    fixed inputs have none.)"""
    ps, lens = 16, [1, 1, 5, 40, 1, 0]
    pages = sum(-(-n // ps) for n in lens)
    pool = filled_pool(pages, 1, ps, 4, 4, seed=2)
    table = table_for(lens, ps, pages)
    q = like_queries(len(lens), Hq) * big
    q[:, Hq // 2:] *= -1
    out, lse = tq.paged_decode_attn(params(4, 4), q, pool, table, torch.tensor(lens, dtype=torch.int32, device="cuda"),
                                    return_lse=True)
    ref, rl = reference(q, pool, table, lens)
    f = np.isfinite(rl)
    assert (rl[f] < -1e28).any() and (rl[f] > 1e28).any()
    err = np.linalg.norm(out.double().cpu().numpy() - ref, axis=-1)
    assert (err <= ALL_WEIGHT * np.linalg.norm(ref, axis=-1)).all(), err
    l = lse.double().cpu().numpy()
    assert np.array_equal(np.isfinite(l), f) and (l[~f] == -np.inf).all()
    # a score's error, with key norms below 29; the product with ln 2 adds two roundings of the value
    assert (np.abs(l[f] - rl[f]) <= 15.0 * big * 29.0 / math.sqrt(128) * SCORE + 2.0**-22 * np.abs(rl[f])).all()


# -------------------------------------------------------------------------- fp32 accuracy
#
# At ordinary sizes (|q| = 4, key norms 6 .. 20, so scores of one unit or less) the errors are roundings of
# either sign, which add as a root of squares:
#   weights   a score of s is off by about s * sqrt(24) * 2^-24 + 2^-22: below 6e-7, and alike for a weight; over
#             many tokens the output's part of that keeps its size relative to the output, as both fall alike
#   sums      fp32 over n groups of 16: sqrt(n) 2^-25 of the sum, n <= 148 here: 3.6e-7
#   rotation  products off by 2^-21.7: 3e-7 of the norm; eight k-steps' sums as much again
# together below 1.2e-6; 4e-6 allows three times that.  What it has to catch is larger: a sum over tokens that
# is cut off instead of rounded loses up to 2^-23, on average 2^-24, of the sum so far in each of the 148 groups
# (8.8e-6 at the end, two thirds of it on the growing sum: 6e-6), and a missing lo part 2^-12 (2.4e-4).
# lse: one score's error (one token: |q| |k| / sqrt(128) <= 7 times sqrt(24) 2^-24 and 2^-22 = 3.7e-6), and
# four roundings of a value of at most 14 (3.4e-6): 8e-6.
OUT_FP32, LSE_FP32 = 4e-6, 8e-6


def accurate(out, lse, ref, ref_lse):
    err = np.linalg.norm(out - ref, axis=-1) / np.linalg.norm(ref, axis=-1)
    assert (err <= OUT_FP32).all(), err.max()
    assert (np.abs(lse - ref_lse) <= LSE_FP32).all(), np.abs(lse - ref_lse).max()


def ordinary_pool(pages, Hkv, ps, kb, vb, seed):
    pool = filled_pool(pages, Hkv, ps, kb, vb, seed=seed)
    for n in (pool.k_norm, pool.v_norm):
        n.mul_(0.5).add_(5.5)  # 6 .. 20
    pool.k_rnorm.copy_(0.15 * pool.k_norm)
    return pool


def ordinary_queries(B, Hq, seed=9):
    q = torch.randn(B, Hq, 128, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda")
    return q * (4.0 / q.norm(dim=-1, keepdim=True))


@pytest.mark.parametrize("Hq", [4, 8])
@pytest.mark.parametrize("kb,vb", [(4, 4), (3, 3), (2, 2)])
def test_fp32_accuracy(Hq, kb, vb):
    """One token (the value product and the rotation back alone) to a few thousand."""
    ps, lens = 32, [1, 1, 2, 15, 100, 1000, 5000]
    pages = sum(-(-n // ps) for n in lens)
    pool = ordinary_pool(pages, 1, ps, kb, vb, seed=kb)
    table = table_for(lens, ps, pages)
    q = ordinary_queries(len(lens), Hq)
    out, lse = tq.paged_decode_attn(params(kb, vb), q, pool, table, torch.tensor(lens, dtype=torch.int32, device="cuda"),
                                    return_lse=True)
    accurate(out.double().cpu().numpy(), lse.double().cpu().numpy(), *reference(q, pool, table, lens))


@pytest.mark.parametrize("g", [4, 8])
def test_fp32_accuracy_of_long_sequences(g):
    """Four sequences of 128K tokens, 148 groups of 16 and more to a warp; one kv-head of one is compared."""
    B, Hkv, ps, T, b, kv = 4, 8, 128, 131072, 1, 3
    pages = B * T // ps
    pool = ordinary_pool(pages, Hkv, ps, 4, 4, seed=g)
    table = torch.randperm(pages, generator=torch.Generator().manual_seed(1)).to(torch.int32).view(B, -1).cuda()
    q = ordinary_queries(B, g * Hkv)
    out, lse = tq.paged_decode_attn(params(4, 4), q, pool, table, torch.full((B,), T, dtype=torch.int32, device="cuda"),
                                    return_lse=True)
    one = tq.Cache.allocate(T // ps, 1, ps, 4, 4)  # that kv-head's pages in order
    for n in ("k_codes", "k_signs", "k_norm", "k_rnorm", "v_codes", "v_norm"):
        getattr(one, n)[:, 0] = getattr(pool, n)[table[b].long(), kv]
    heads = slice(kv * g, kv * g + g)
    ref, rl = reference(q[b:b + 1, heads], one, torch.arange(T // ps, dtype=torch.int32, device="cuda")[None], [T])
    accurate(out[b:b + 1, heads].double().cpu().numpy(), lse[b:b + 1, heads].double().cpu().numpy(), ref, rl)


@pytest.mark.parametrize("Hq", [4, 8])
def test_value_norms_over_the_whole_range(Hq):
    """Norms of 1e-8 and of 1e30 in one sequence, the large ones at scores 200 below the maximum (e^-200 1e38
    is below 1e-48 of the output); next to the token that has the weight and in other groups."""
    away = [1, -1, 5, 16, -16, 40]
    B, ps, T = len(away), 16, 500
    lens = [T] * B
    pages = B * (-(-T // ps))
    pool = filled_pool(pages, 1, ps, 4, 4, seed=4)
    pool.k_norm.mul_(0.1)
    pool.k_rnorm.mul_(0.1)
    pool.v_norm.mul_(1e-9)
    table = table_for(lens, ps, pages)
    q = like_queries(B, Hq)
    norms = []
    for b, d in enumerate(away):
        i, n = raise_score(pool, table, q, b, 240 + b, 272 + b, 200.0)
        norms.append(n)
        pool.v_norm[table[b, (i + d) // ps].long(), 0, (i + d) % ps] = 1e30
    out, lse = tq.paged_decode_attn(params(4, 4), q, pool, table, torch.tensor(lens, dtype=torch.int32, device="cuda"),
                                    return_lse=True)
    ref, rl = reference(q, pool, table, lens)
    err = np.linalg.norm(out.double().cpu().numpy() - ref, axis=-1) / np.linalg.norm(ref, axis=-1)
    assert (err <= ALL_WEIGHT).all(), err
    tol = 15.0 * np.array(norms)[:, None] / math.sqrt(128) * SCORE + 2.0**-22 * np.abs(rl)
    assert (np.abs(lse.double().cpu().numpy() - rl) <= tol).all()
