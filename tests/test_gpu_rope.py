"""Rotary positions (tq_rope) on the GPU against the rotation in 64 bits.

Tolerance.  An output is x cos t -+ y sin t.  The angle is exact to about 1e-10 turns in fp64, then
rounded to fp32 half turns (|2r| <= 1: at most 2^-25 half turns, 9.4e-8 rad); sincospi is within 2 ulp of
a value <= 1 (1.2e-7); two roundings of the sum add 2 * 2^-24.  Together at most 3.4e-7 (|x| + |y|);
a bf16 output adds half a step, eps / 2 = 2^-8 of the value."""
import numpy as np
import pytest
import torch

import decode_attention_11_b200 as tq

pytestmark = pytest.mark.gpu


def rotate(x, pos, axis_of_pair, base, style, inverse=False):
    """x [N, H, 128] float64, pos [axes, N]: each pair as a complex number times e^(+-i t)."""
    i = np.arange(64)
    t = pos[np.asarray(axis_of_pair)].T.astype(np.float64) * base ** (-2.0 * i / 128)  # [N, 64]
    turn = np.exp((-1j if inverse else 1j) * t)[:, None]
    a, b = (x[..., :64], x[..., 64:]) if style == tq.TQ_ROPE_HALF else (x[..., 0::2], x[..., 1::2])
    z = (a + 1j * b) * turn
    if style == tq.TQ_ROPE_HALF:
        return np.concatenate([z.real, z.imag], -1), np.abs(a) + np.abs(b)
    out = np.empty_like(x)
    out[..., 0::2], out[..., 1::2] = z.real, z.imag
    return out, np.abs(a) + np.abs(b)


def close(got, x, pos, axis_of_pair, base, style, inverse=False):
    ref, mag = rotate(x.double().cpu().numpy(), pos.cpu().numpy().reshape(-1, pos.shape[-1]), axis_of_pair, base, style, inverse)
    mag = np.concatenate([mag, mag], -1) if style == tq.TQ_ROPE_HALF else np.repeat(mag, 2, -1)
    tol = 3.4e-7 * mag + 1e-12
    if got.dtype == torch.bfloat16:
        tol = tol + (torch.finfo(torch.bfloat16).eps / 2) * (np.abs(ref) + tol)
    err = np.abs(got.double().cpu().numpy() - ref)
    assert (err <= tol).all(), (err - tol).max()


SECTIONS = {1: (64,), 2: (32, 32), 3: (16, 24, 24), 4: (0, 20, 4, 40)}


@pytest.mark.parametrize("N", [1, 3, 257, 1500])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("style", [tq.TQ_ROPE_HALF, tq.TQ_ROPE_PAIR])
@pytest.mark.parametrize("axes", [1, 3, 4])
def test_rope_values(N, dtype, style, axes):
    torch.manual_seed(N + axes)
    Hq, Hkv = (5, 1) if axes == 4 else (8, 2)
    q = torch.randn(N, Hq, 128, device="cuda").to(dtype)
    k = torch.randn(N, Hkv, 128, device="cuda").to(dtype)
    pos = torch.randint(0, 1 << 20, (axes, N), device="cuda", dtype=torch.int32)
    axis = [a for a, s in enumerate(SECTIONS[axes]) for _ in range(s)]
    base = 1e6 if axes == 3 else 1e4
    qo, ko = tq.rope(q, k, pos if axes > 1 else pos[0], sections=SECTIONS[axes], base=base, style=style)
    close(qo, q, pos, axis, base, style)
    close(ko, k, pos, axis, base, style)


def test_rope_interleaved_axes_strides_and_far_positions():
    N, H = 37, 6
    wide = torch.randn(N, H + 3, 256, device="cuda")
    q = wide[:, 1:1 + H, 128:]              # strided heads and tokens
    qkv = torch.randn(N, (H + 4) * 128, device="cuda").to(torch.bfloat16).view(N, H + 4, 128)
    kb = qkv[:, H:H + 2]                    # a slice of a fused projection
    axis = [i % 3 for i in range(64)]
    pos = torch.stack([torch.arange(N) * 50_000_000, -torch.arange(N) * 7, torch.full((N,), 2**31 - 1)]).to(torch.int32).cuda()
    qo, _ = tq.rope(q, None, pos, axis_of_pair=axis)
    # the reference's own angle, pos * freq, is exact to 2^-53 of up to 2^31 rad: 2.4e-7 rad more
    ref, mag = rotate(q.double().cpu().numpy(), pos.cpu().numpy(), axis, 1e4, tq.TQ_ROPE_HALF)
    mag = np.concatenate([mag, mag], -1)
    # far positions: pos * turns carries 2^-53 of up to 3.4e8 turns = 3.8e-8 turns = 2.4e-7 rad here too
    assert (np.abs(qo.double().cpu().numpy() - ref) <= (3.4e-7 + 4 * 2.4e-7) * mag + 1e-12).all()
    _, ko = tq.rope(None, kb, pos[1], inverse=True)
    close(ko, kb, pos[1:2], [0] * 64, 1e4, tq.TQ_ROPE_HALF, inverse=True)


@pytest.mark.parametrize("style", [tq.TQ_ROPE_HALF, tq.TQ_ROPE_PAIR])
def test_rope_gradient(style):
    """The map is linear and orthogonal: its gradient applied to g is the inverse turn of g.  Against the
    formula (above, inverse=True) and against differences: <g, rope(x + d) - rope(x - d)> / 2 = <grad, d>."""
    torch.manual_seed(3)
    N, H = 65, 4
    x, d, g = (torch.randn(N, H, 128, device="cuda") for _ in range(3))
    pos = torch.randint(0, 5000, (2, N), device="cuda", dtype=torch.int32)
    kw = dict(sections=(32, 32), style=style)
    f = lambda t, **k: tq.rope(t, None, pos, **kw, **k)[0]
    grad = f(g, inverse=True)
    close(grad, g, pos, [0] * 32 + [1] * 32, 1e4, style, inverse=True)
    diff = ((f(x + d).double() - f(x - d).double()) / 2 * g.double()).sum(-1)
    want = (grad.double() * d.double()).sum(-1)
    # 128 products; each factor carries at most 3.4e-7 (|x| + |y|) of its pair, |.| below 6 here, three
    # rotations, plus fp32 rounding of x +- d (2^-24 * 12): under 128 * 6 * (3 * 3.4e-7 * 24) = 2e-2;
    # errors of both signs add as a root, so a tenth of that is already far outside
    assert (diff - want).abs().max().item() < 2e-3
    back = f(f(x), inverse=True)
    assert (back - x).abs().max().item() < 6 * 4 * 3.4e-7 * 6


def test_rope_in_place_empty_and_graph():
    N, H = 200, 8
    q = torch.randn(N, H, 128, device="cuda").to(torch.bfloat16)
    pos = torch.arange(N, device="cuda", dtype=torch.int32)
    want, _ = tq.rope(q, None, pos)
    p = q.clone()
    r, _ = tq.rope(p, None, pos, q_out=p)
    assert r is p and torch.equal(p, want)
    one = q[5:6]  # one token, one head: contiguous whatever the strides say
    tq.rope(one, None, pos[5:6], q_out=one)
    assert torch.equal(q[5], want[5])
    q[5] = p.new_tensor(0)
    lone = torch.randn(3, 9, 128, device="cuda")[1:2, 4:5]
    keep = lone.clone()
    tq.rope(lone, None, pos[7:8], q_out=lone)
    assert torch.equal(lone, tq.rope(keep, None, pos[7:8])[0])
    e, _ = tq.rope(q[:0], None, pos[:0])
    assert e.shape == (0, H, 128)
    out = torch.empty_like(q)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        tq.rope(q, None, pos, q_out=out)
    pos.add_(1000)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, tq.rope(q, None, pos)[0])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other, _ = tq.rope(q, None, pos, stream=side)
    side.synchronize()
    assert torch.equal(other, out)
