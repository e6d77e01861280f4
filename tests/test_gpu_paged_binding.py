"""What the Python binding of the paged and rotary calls does besides passing arguments on."""
import pytest
import torch

import decode_attention_11_b200 as tq

pytestmark = pytest.mark.gpu


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def keep_busy(stream, n=60):
    """Some tens of milliseconds of work on `stream`."""
    with torch.cuda.stream(stream):
        a = torch.ones(8192, 8192, device="cuda", dtype=torch.bfloat16)
        b = torch.empty_like(a)
        for _ in range(n):
            torch.mm(a, a, out=b)


def test_check_sees_calls_on_every_stream():
    pt = tq.PageTable.allocate(2, 4, 8, 16)
    seqs, one, far = ints([0]), ints([1]), ints([7])
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(3):
        keep_busy(side)
        tq.pages_reserve(pt, far, one, 1, stream=side)  # no such sequence: recorded when the stream gets there
        with pytest.raises(ValueError, match="out of range"):
            pt.check()
        pt.check()
        # what is recorded right after a check that clears is not lost
        keep_busy(torch.cuda.current_stream(), 5)
        tq.pages_reserve(pt, far, one, 1)
        with pytest.raises(ValueError, match="out of range"):
            pt.check()
        tq.pages_free(pt, far, stream=side)
        with pytest.raises(ValueError, match="out of range"):
            pt.check()
    assert tq.pages_reserve(pt, seqs, one, 1).tolist() == [0]
    pt.check()


# -------------------------------------------------------------------------- rope under autograd

def fused(N, dtype, requires_grad=True):
    """q [N, 6, 128] and k [N, 2, 128] as slices of one projection (strided rows)."""
    torch.manual_seed(N)
    w = torch.randn(N, 10, 128, device="cuda").to(dtype).requires_grad_(requires_grad)
    return w, w[:, :6], w[:, 6:8]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("style", [tq.TQ_ROPE_HALF, tq.TQ_ROPE_PAIR])
@pytest.mark.parametrize("inverse", [False, True])
@pytest.mark.parametrize("N", [0, 1, 37])
def test_rope_gradient_through_autograd(dtype, style, inverse, N):
    """The gradient is the turn back of the outputs' gradients, bit for bit what rope gives for them; what it
    gives is compared with the formula in 64 bits in test_gpu_rope.py."""
    w, q, k = fused(N, dtype)
    pos = torch.randint(0, 5000, (2, N), device="cuda", dtype=torch.int32)
    kw = dict(sections=(40, 24), base=5e5, style=style)
    qo, ko = tq.rope(q, k, pos, inverse=inverse, **kw)
    with torch.no_grad():
        a, b = tq.rope(q, k, pos, inverse=inverse, **kw)
    assert torch.equal(qo, a) and torch.equal(ko, b) and not a.requires_grad
    gq, gk = torch.randn_like(qo), torch.randn_like(ko)
    torch.autograd.backward([qo, ko], [gq, gk])
    wq, wk = tq.rope(gq, gk, pos, inverse=not inverse, **kw)
    want = torch.cat([wq, wk, torch.zeros(N, 2, 128, device="cuda", dtype=dtype)], 1)
    assert torch.equal(w.grad, want)


def test_rope_gradient_against_differences():
    """<g, rope(x + d) - rope(x - d)> / 2 = <grad, d> (the map is linear), in 64 bits over fp32 outputs.  Each of
    the 2 * 128 products of a head's row is off by at most 3.4e-7 (|x| + |y|) times 6 (outputs, gradient) and by the
    rounding of x +- d, |.| below 6: 256 * 6 * 3 * 3.4e-7 * 12 = 1.9e-2 if all errors had one sign."""
    w, q, k = fused(53, torch.float32)
    pos = torch.randint(0, 1 << 20, (53,), device="cuda", dtype=torch.int32)
    d, gq, gk = torch.randn_like(w), torch.randn_like(q), torch.randn_like(k)
    f = lambda x: tq.rope(x[:, :6], x[:, 6:8], pos, axis_of_pair=[0] * 64)
    torch.autograd.backward(f(w), [gq, gk])
    with torch.no_grad():
        (qa, ka), (qb, kb) = f(w + d), f(w - d)
    dq, dk = ((a.double() - b.double()) / 2 for a, b in ((qa, qb), (ka, kb)))
    diff = torch.cat([(dq * gq).sum(-1), (dk * gk).sum(-1)], 1)
    want = (w.grad.double() * d.double()).sum(-1)[:, :8]
    assert (diff - want).abs().max().item() < 1.9e-2 and want.abs().max().item() > 10


def test_rope_gradient_forms():
    w, q, k = fused(20, torch.float32)
    pos = torch.arange(20, device="cuda", dtype=torch.int32)
    # one input, one output used, a gradient with strides of 0
    for out, part in ((tq.rope(q, None, pos)[0], slice(0, 6)), (tq.rope(None, k, pos)[1], slice(6, 8)),
                      (tq.rope(q, k, pos)[1], slice(6, 8)), (tq.rope(q.detach(), k, pos)[1], slice(6, 8)),
                      (tq.rope(q, k.detach(), pos)[0], slice(0, 6))):
        w.grad = None
        out.sum().backward()
        want = tq.rope(torch.ones_like(out), None, pos, inverse=True)[0]
        assert torch.equal(w.grad[:, part], want)
        rest = torch.ones(10, dtype=torch.bool, device="cuda")
        rest[part] = False
        assert (w.grad[:, rest] == 0).all()
    # a gradient that starts off a 16-byte boundary
    out = tq.rope(q, None, pos)[0]
    g = torch.randn(out.numel() + 1, device="cuda")[1:].view_as(out)
    got, = torch.autograd.grad(out, q, g)
    assert torch.equal(got, tq.rope(g.clone(), None, pos, inverse=True)[0])
    # the gradient's own gradient: turned forward again
    out = tq.rope(q, None, pos)[0]
    g = torch.randn_like(out, requires_grad=True)
    got, = torch.autograd.grad(out, q, g, create_graph=True)
    v = torch.randn_like(got)
    second, = torch.autograd.grad(got, g, v)
    assert torch.equal(second, tq.rope(v, None, pos)[0])
    # on a stream of the caller's
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    out = tq.rope(q, None, pos, stream=s)[0]
    torch.cuda.synchronize()
    g = torch.randn_like(out)
    got, = torch.autograd.grad(out, q, g)
    assert torch.equal(got, tq.rope(g, None, pos, inverse=True)[0])
    # outputs of the caller's: refused with a gradient, taken without
    with pytest.raises(ValueError, match="requires a gradient"):
        tq.rope(q, None, pos, q_out=torch.empty(20, 6, 128, device="cuda"))
    with torch.no_grad():
        assert torch.equal(tq.rope(q, None, pos, q_out=torch.empty(20, 6, 128, device="cuda"))[0], out)
    # positions changed before the backward pass: an error, no wrong gradient
    out = tq.rope(q, None, pos)[0]
    pos.add_(1)
    with pytest.raises(RuntimeError):
        out.sum().backward()


# -------------------------------------------------------------------------- numbers past 32 bits

def test_window_past_32_bits_sees_all():
    """A window wider than any sequence shows all tokens, also where its low 32 bits say something else."""
    pool = tq.Cache.allocate(4, 1, 16, 4, 4, 0)
    for n in ("k_codes", "v_codes"):
        getattr(pool, n).random_(0, 256)
    pool.k_norm.fill_(3.0)
    pool.v_norm.fill_(3.0)
    p = tq.Params.create(torch.eye(128).numpy(), None, 4, 4)
    q = torch.randn(1, 4, 128, device="cuda")
    table, lens = torch.arange(4, dtype=torch.int32, device="cuda")[None], ints([60])
    call = lambda w: tq.paged_decode_attn(p, q, pool, table, lens, window=w)
    want = call(0)
    assert not torch.equal(call(5), want)
    for w in (60, 2**31 - 1, 2**31, 2**32 + 5, 2**40 + 5):
        assert torch.equal(call(w), want)
    for w in (-1, -2**32, -2**32 + 5):
        with pytest.raises(tq.TqError):
            call(w)


# -------------------------------------------------------------------------- diagnostics

def test_diagnostics_see_calls_on_every_stream():
    """Error bits and counters are read after what any stream still has to do."""
    g = torch.Generator(device="cuda").manual_seed(3)
    pool = tq.Cache.allocate(40, 4, 64, 4, 4, 0)
    p = tq.Params.create(torch.eye(128).numpy(), None, 4, 4)
    q = torch.randn(1, 4, 128, device="cuda")
    bad, lens = torch.full((1, 4), 10**6, dtype=torch.int32, device="cuda"), ints([60])
    x = torch.randn(2500, 4, 128, generator=g, device="cuda").to(torch.bfloat16)
    slots = torch.arange(2500, dtype=torch.int32, device="cuda")
    side = torch.cuda.Stream()
    tq.reset_device_errors()
    for _ in range(2):
        count = tq.quantize_code_fixups()
        keep_busy(side)
        tq.paged_quantize(p, x, x, pool, slots, stream=side)
        assert tq.quantize_code_fixups() > count
        keep_busy(side)
        tq.paged_decode_attn(p, q, pool, bad, lens, stream=side)
        assert tq.decode_device_errors() == 16
        keep_busy(side)
        tq.paged_decode_attn(p, q, pool, bad, lens, stream=side)
        tq.reset_device_errors()
        torch.cuda.synchronize()
        assert tq.decode_device_errors() == 0


def test_rope_gradient_in_a_graph():
    """Forward and backward captured together: a replay turns the inputs, positions and gradients as they are then."""
    torch.manual_seed(1)
    q = torch.randn(33, 4, 128, device="cuda", requires_grad=True)
    g = torch.randn(33, 4, 128, device="cuda")
    pos = torch.arange(33, dtype=torch.int32, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        out, _ = tq.rope(q, None, pos)
        grad, = torch.autograd.grad(out, q, g)
    for _ in range(2):
        with torch.no_grad():
            q.copy_(torch.randn_like(q))
        g.copy_(torch.randn_like(g))
        pos.add_(1000)
        graph.replay()
        torch.cuda.synchronize()
        with torch.no_grad():
            assert torch.equal(out, tq.rope(q, None, pos)[0])
            assert torch.equal(grad, tq.rope(g, None, pos, inverse=True)[0])
