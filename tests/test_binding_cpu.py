"""Structures that the Python binding hands to the library (no GPU)."""
import ctypes

import torch

import decode_attention_11_b200 as tq


def test_missing_arrays_are_null_and_refused_by_the_library():
    """An array that is not there reaches the library as NULL, which says what is missing."""
    p = tq.Params(None, None, None, None, None, None).as_c()
    assert p.Pi is None and p.k_centroids is None and p.v_thresholds is None
    c = tq.Cache.allocate(2, 1, 16, 4, 4, device="cpu")
    whole = c.as_c()
    assert tq.lib().tq_paged_decode_workspace_size(1, 4, ctypes.byref(whole)) > 0
    c.k_codes = c.v_norm = None
    null = c.as_c()
    assert null.k_codes is None and null.v_norm is None and null.k_norm == whole.k_norm
    L, R = tq.lib(), ctypes.byref
    assert L.tq_paged_read(R(p), R(null), None, 0, tq.TQ_F32, None, None, None, None, None) == tq.TQ_ERR_INVALID_ARG
    assert "NULL" in tq.last_error()
    assert L.tq_paged_read(R(p), R(whole), None, 0, tq.TQ_F32, None, None, None, None, None) == tq.TQ_ERR_INVALID_ARG
    assert "NULL" in tq.last_error()


def test_mixed_constants_reach_the_library():
    t = torch.zeros(16)
    p = tq.Params(t, t, t, t, t, t, None, t, t, t, t, (1, 2, 3, 4)).as_c()
    assert p.k_centroids_lo == t.data_ptr() == p.v_thresholds_lo and list(p.outlier_mask) == [1, 2, 3, 4]
