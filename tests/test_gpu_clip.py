"""The global gradient norm, clipping and the clipped Adam update against
plain 64-bit forms.  Tolerances count roundings: the norm and the coefficient
are formed in fp64 and rounded once to fp32 (u = 2^-24); a clipped value takes
the coefficient's rounding, the product's and that to its type."""
import math

import numpy as np
import pytest
import torch

from gpu_util import B

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
F64 = 1e-8   # of an fp64 sum of up to 2^26 terms, in units of the result
HALF_STEP = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
TINY = {torch.float32: 2.0 ** -150, torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -134}


@pytest.fixture(scope="module")
def b():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    torch.cuda.set_device(0)
    return B()


def gen(seed):
    return torch.Generator("cuda").manual_seed(seed)


def rand(shape, seed, sigma=1.0, dtype=torch.float32):
    return (torch.randn(shape, generator=gen(seed), device="cuda") * sigma).to(dtype)


def norm_of(b, tensors, max_norm, eps=1e-6, st=None):
    clip = torch.full((2,), -1.0, device="cuda")
    ws = torch.randint(255, (b.gs_grad_norm_workspace_size(tensors),), dtype=torch.uint8,
                       generator=gen(99), device="cuda")
    b.gs_grad_norm(tensors, max_norm, clip, ws, eps=eps, dev_status=st)
    return clip


def exact_norm(tensors):
    return math.sqrt(math.fsum(float(t.double().square().sum()) for t in tensors if t.numel()))


def check_clip(clip, tensors, max_norm, eps=1e-6):
    n = exact_norm(tensors)
    c = min(1.0, max_norm / (n + eps)) if n + eps > 0 else 1.0
    assert abs(float(clip[0]) - n) <= (U + F64) * n + 2.0 ** -150
    assert abs(float(clip[1]) - c) <= (U + F64) * c + 2.0 ** -150
    return c


def sets(seed):
    """Lists of tensors: one element, ragged, strided planes, mixed types, many."""
    yield [rand(1, seed)]
    yield [rand(7, seed), rand((3, 5), seed + 1), rand(0, 1), rand((2, 0, 3), 1)]
    yield [rand((59, 1003), seed)[:, :1000], rand((11, 64), seed + 1)[:, :1]]
    yield [rand(100_003, seed, 1e-3, torch.bfloat16), rand((7, 333), seed, 5.0, torch.float16)[:, 1:],
           rand(99, seed)[3:], rand((4, 1), seed, 1.0, torch.float16)]
    yield [rand(1 + 37 * k % 5000, seed + k, 10.0 ** (k % 5 - 3),
                (torch.float32, torch.bfloat16, torch.float16)[k % 3]) for k in range(700)]
    yield [rand((14, 300_001), seed), rand((5, 100_000), seed)[:, 17:99_990],
           rand(2_000_001, seed, 1.0, torch.bfloat16)[1:], rand(3_000_003, seed, 1.0, torch.float16)[3:]]


@pytest.mark.parametrize("which", range(6))
@pytest.mark.parametrize("max_norm", [0.0, 0.5, 1e9])
def test_norm_and_clip(b, which, max_norm):
    src = list(sets(which * 1000))[which]
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    clip = norm_of(b, src, max_norm, st=st)
    c = check_clip(clip, src, max_norm)
    assert torch.equal(clip, norm_of(b, src, max_norm))  # the same bits again
    assert int(st) == 0
    # into other tensors: contiguous ones, one element past an aligned address
    dst = []
    for t in src:
        buf = torch.full((t.numel() + 2,), 3.0, dtype=t.dtype, device="cuda")
        dst.append(buf[1:1 + t.numel()].view(t.shape))
    keep = [t.clone() for t in src]
    b.gs_grad_clip(src, dst, clip)
    for s, d, k in zip(src, dst, keep):
        ref = c * s.double()
        tol = (HALF_STEP[s.dtype] + 2.1 * U + F64) * ref.abs() + TINY[s.dtype]
        assert ((d.double() - ref).abs() <= tol).all()
        assert torch.equal(s, k)
        if d.numel():
            whole = torch.as_strided(d, (d.numel() + 2,), (1,), d.storage_offset() - 1)
            assert whole[0] == 3.0 and whole[-1] == 3.0
    # in place: the same bits
    b.gs_grad_clip(src, src, clip)
    for s, d in zip(src, dst):
        assert torch.equal(s, d)


def test_clip_leaves_the_padding(b):
    buf = rand((9, 70), 5)
    keep = buf.clone()
    view = buf[:, 3:64]
    clip = norm_of(b, [view], 0.25)
    b.gs_grad_clip([view], [view], clip)
    assert torch.equal(buf[:, :3], keep[:, :3]) and torch.equal(buf[:, 64:], keep[:, 64:])
    assert abs(exact_norm([view]) - 0.25) <= 1e-5


def test_norm_of_large_and_small_values(b):
    """Squares that leave fp32's range do not leave the sum's."""
    big = torch.full((1000,), 1e30, device="cuda")
    small = torch.full((1000,), 1e-30, device="cuda")
    for t in (big, small, big.bfloat16(), small.bfloat16(),
              torch.full((999,), 2.0 ** -24, dtype=torch.float16, device="cuda"),
              torch.full((999,), 65504.0, dtype=torch.float16, device="cuda")):
        check_clip(norm_of(b, [t], 1.0, eps=0.0), [t], 1.0, eps=0.0)


def test_norm_of_nothing_and_of_zeros(b):
    for tensors in ([], [torch.empty(0, device="cuda")], [torch.zeros(1000, device="cuda")]):
        clip = norm_of(b, tensors, 1.0)
        assert float(clip[0]) == 0.0 and float(clip[1]) == 1.0
        assert float(norm_of(b, tensors, 0.0, eps=0.0)[1]) == 1.0


@pytest.mark.parametrize("size", [5, 100_000, 9_000_000])
def test_non_finite_gradients_are_flagged(b, size):
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    for dtype in (torch.float32, torch.bfloat16, torch.float16):
        t = rand(size, 3, 1.0, dtype)
        t[size // 2] = float("inf")
        clip = norm_of(b, [t], 1.0, st=st)
        assert float(clip[0]) == math.inf and float(clip[1]) == 0.0 and int(st) == 4
        st.zero_()
        t[size - 1] = float("nan")
        clip = norm_of(b, [rand(10, 1), t], 1.0, st=st)
        assert math.isnan(float(clip[0])) and math.isnan(float(clip[1])) and int(st) == 4
        st.zero_()


def test_clip_of_non_finite_norms(b):
    t = rand(100, 3)
    out = torch.empty_like(t)
    b.gs_grad_clip([t], [out], torch.tensor([math.inf, 0.0], device="cuda"))
    assert (out == 0).all()
    b.gs_grad_clip([t], [out], torch.tensor([math.nan, math.nan], device="cuda"))
    assert torch.isnan(out).all()


def test_norm_past_32_bit_offsets(b):
    n = 2 ** 31 + 4099
    t = torch.zeros(n, dtype=torch.float16, device="cuda")
    t[0], t[n - 1], t[2 ** 31] = 3.0, 4.0, 12.0
    clip = norm_of(b, [t], 1.3, eps=0.0)
    assert float(clip[0]) == 13.0
    b.gs_grad_clip([t], [t], clip)
    want = torch.tensor([3.0, 12.0, 4.0], device="cuda") * clip[1]
    assert torch.equal(t[torch.tensor([0, 2 ** 31, n - 1], device="cuda")], want.half())
    assert int(torch.count_nonzero(t[:1 << 20])) == 1


# ---- Adam on the clipped gradient ----------------------------------------------

LR, B1, B2, EPS = 1e-3, 0.9, 0.999, 1e-8


def adam_exact(p, m, v, g, c, step):
    p, m, v, g = (x.double() for x in (p, m, v, g))
    g = c * g
    m1 = B1 * m + (1 - B1) * g
    v1 = B2 * v + (1 - B2) * g * g
    den = (v1 / (1 - B2 ** step)).sqrt() + EPS
    lr = LR / (1 - B1 ** step)
    # roundings: m has 2 of b1 m and 5 of (1 - b1) c g; v 2 and 10; the
    # quotient takes v's half, and 12 of its own (a fast division has 4)
    em = 7 * U * (B1 * m.abs() + (1 - B1) * g.abs())
    ev = 10 * U * v1
    dp = lr * m1 / den
    ep = lr * em / den + dp.abs() * 20 * U + U * (p.abs() + dp.abs())
    return p - dp, m1, v1, ep, em, ev


@pytest.mark.parametrize("n,P", [(1, 11), (2, 59), (63, 14), (1000, 59), (1003, 23), (50_001, 38)])
@pytest.mark.parametrize("compact", [False, True])
@pytest.mark.parametrize("step", [1, 100])
def test_adam_clipped(b, n, P, compact, step):
    n_pad = (n + 63) // 64 * 64
    p, m = rand((P, n_pad), 1), rand((P, n_pad), 2, 1e-2)
    v = rand((P, n_pad), 3, 1e-2).square()
    if compact:
        pick = torch.rand(n, generator=gen(4), device="cuda") < 0.6
        C = int(pick.sum())
        slot = torch.full((n,), -1, dtype=torch.int32, device="cuda")
        slot[pick] = torch.arange(C, dtype=torch.int32, device="cuda")
        g = rand((P, max(C, 1)), 5, 1e-2)
        dense = torch.where(slot >= 0, g[:, slot.clamp(min=0).long()], 0.0)
        stride = max(C, 1)
    else:
        slot, g, stride = None, rand((P, n_pad), 5, 1e-2), n_pad
        dense = g[:, :n]
    for coef in (1.0, 0.37):
        clip = torch.tensor([1.0, coef], device="cuda")
        args = b.gs_adam_args(LR, B1, B2, EPS, step, 0)
        a = [x.clone() for x in (p, m, v)]
        b.gs_adam_clipped(*a, g, stride, slot, n, n_pad, P, args, clip)
        ref = adam_exact(p[:, :n], m[:, :n], v[:, :n], dense, float(clip[1].double()), step)
        for got, want, tol in zip(a, ref[:3], ref[3:]):
            assert ((got[:, :n].double() - want).abs() <= 1.01 * tol + 2.0 ** -149).all()
        for got, was in zip(a, (p, m, v)):  # behind the last Gaussian
            assert torch.equal(got[:, n:], was[:, n:])
        if coef == 1.0:  # unclipped: the bits of gs_adam
            o = [x.clone() for x in (p, m, v)]
            b.gs_adam(*o, g, stride, slot, n, n_pad, P, args)
            for x, y in zip(a, o):
                assert torch.equal(x, y)


def test_adam_clipped_unaligned_planes(b):
    """Plane strides and addresses that are not multiples of 16 bytes."""
    n, P, n_pad = 1001, 7, 1003
    bufs = [rand(P * n_pad + 1, k, s)[1:] for k, s in ((1, 1.0), (2, 1e-2), (3, 1e-2))]
    bufs[2].square_()
    g = rand(P * 1005 + 3, 4, 1e-2)[3:]
    clip = torch.tensor([1.0, 0.5], device="cuda")
    was = [x.clone() for x in bufs]
    b.gs_adam_clipped(*bufs, g, 1005, None, n, n_pad, P, b.gs_adam_args(LR, B1, B2, EPS, 3, 0), clip)
    view = [x.view(P, n_pad)[:, :n] for x in was]
    ref = adam_exact(*view, g.view(P, 1005)[:, :n], 0.5, 3)
    for got, w, want, tol in zip(bufs, was, ref[:3], ref[3:]):
        assert ((got.view(P, n_pad)[:, :n].double() - want).abs() <= 1.01 * tol + 2.0 ** -149).all()
        assert torch.equal(got.view(P, n_pad)[:, n:], w.view(P, n_pad)[:, n:])


def test_norm_clip_adam_in_a_graph(b):
    """Norm, clipping copy and update captured and replayed with new gradients."""
    n, P = 5000, 14
    p, m = rand((P, n), 1), rand((P, n), 2, 1e-2)
    v = rand((P, n), 3, 1e-2).square()
    g, out = rand((P, n), 4), torch.empty((P, n), device="cuda")
    clip = torch.empty(2, device="cuda")
    tensors, outs = b.tensor_list([g]), b.tensor_list([out])
    ws = torch.empty(b.gs_grad_norm_workspace_size(tensors), dtype=torch.uint8, device="cuda")
    args = b.gs_adam_args(LR, B1, B2, EPS, 5, 0)
    start = [x.clone() for x in (p, m, v)]

    def step(pp, mm, vv):
        b.gs_grad_norm(tensors, 1.0, clip, ws)
        b.gs_grad_clip(tensors, outs, clip)
        b.gs_adam_clipped(pp, mm, vv, g, n, None, n, n, P, args, clip)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(*[x.clone() for x in start])
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(p, m, v)
    for seed, sigma in ((6, 1.0), (7, 1e-6), (8, 100.0)):
        g.copy_(rand((P, n), seed, sigma))
        for x, s in zip((p, m, v), start):
            x.copy_(s)
        graph.replay()
        got = [x.clone() for x in (p, m, v, out, clip)]
        want = [x.clone() for x in start]
        step(*want)
        for x, y in zip(got, want + [out, clip]):
            assert torch.equal(x, y)
        check_clip(got[4], [g], 1.0)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
def test_an_infinite_element_is_clipped_to_zero(b, dtype):
    """Norm, clipping copy and Adam end to end: an infinite norm scales every
    gradient to 0, the infinite ones too; NaN stays NaN."""
    n, P = 1003, 3
    for short in (False, True):
        g = rand((P, n), 11, 1.0, dtype) if not short else rand((n, P + 1), 12, 1.0, dtype)[:, :P]
        g[1, 2], g[2, 0] = math.inf, -math.inf
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        clip = norm_of(b, [g], 1.0, st=st)
        assert float(clip[0]) == math.inf and float(clip[1]) == 0.0 and int(st) == 4
        out = torch.full(g.shape, 3.0, dtype=dtype, device="cuda")
        b.gs_grad_clip([g], [out], clip)
        assert (out == 0).all()
        b.gs_grad_clip([g], [g], clip)
        assert (g == 0).all()
    g = rand((P, n), 13, 1.0, dtype)
    g[1, 2], g[2, 0] = math.inf, math.nan
    clip = norm_of(b, [g], 1.0)
    b.gs_grad_clip([g], [g], clip)
    assert torch.isnan(g).all()


@pytest.mark.parametrize("compact", [False, True])
def test_adam_takes_an_infinite_gradient_as_zero(b, compact):
    n, P, n_pad = 1003, 5, 1024
    p, m = rand((P, n_pad), 1), rand((P, n_pad), 2, 1e-2)
    v = rand((P, n_pad), 3, 1e-2).square()
    g = rand((P, n), 4)
    g[0, 0], g[3, 500], g[4, n - 1] = math.inf, -math.inf, math.inf
    slot = torch.arange(n, dtype=torch.int32, device="cuda").flip(0).contiguous() if compact else None
    clip = norm_of(b, [g], 1.0)
    assert float(clip[1]) == 0.0
    args = b.gs_adam_args(LR, B1, B2, EPS, 7, 0)
    want = [x.clone() for x in (p, m, v)]
    b.gs_adam_clipped(p, m, v, g, n, slot, n, n_pad, P, args, clip)
    b.gs_adam(*want, torch.zeros_like(g), n, slot, n, n_pad, P, args)
    for x, y in zip((p, m, v), want):
        assert torch.isfinite(x).all() and torch.equal(x, y)


def test_clip_of_neighbours_and_of_a_shared_source(b):
    """What is not refused: rows between one another's, neighbouring pieces of
    one buffer in any order, one source for two destinations; more tensors
    than a launch takes."""
    buf = torch.arange(1, 7 * 64 + 1, device="cuda", dtype=torch.float32).view(7, 64)
    keep, clip = buf.clone(), torch.tensor([2.0, 0.5], device="cuda")
    b.gs_grad_clip([buf[:, 10:40], buf[:, :10], buf[:, 40:64]], [buf[:, 10:40], buf[:, :10], buf[:, 40:64]], clip)
    assert torch.equal(buf, 0.5 * keep)
    out = torch.zeros(2, 7, 64, device="cuda")
    b.gs_grad_clip([buf, buf], [out[1], out[0]], clip)
    assert torch.equal(out[0], 0.25 * keep) and torch.equal(out[1], 0.25 * keep)
    flat = torch.arange(1000 * 12, device="cuda", dtype=torch.float32)
    parts = [flat[12 * k:12 * k + 12] for k in torch.randperm(1000).tolist()]
    b.gs_grad_clip(parts, parts, clip)
    assert torch.equal(flat, 0.5 * torch.arange(1000 * 12, device="cuda"))
    with pytest.raises(b.GsError):
        b.gs_grad_clip(parts + parts[:1], parts + parts[:1], clip)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
def test_clip_rounds_the_fp32_product(b, dtype):
    """The fp32 product, then its rounding to the type: bit for bit."""
    t, clip = rand(100_003, 21, 1.0, dtype), torch.tensor([3.0, 1 / 3], device="cuda")
    out = torch.empty_like(t)
    b.gs_grad_clip([t], [out], clip)
    assert torch.equal(out, (t.float() * clip[1]).to(dtype))
