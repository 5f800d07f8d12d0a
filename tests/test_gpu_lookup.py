"""The table lookup and its gradient against plain 64-bit forms.

Tolerances count roundings (u = 2^-24 for fp32): the lookup rounds the product
once in fp32 and once to the output's type; a sum of m terms in any order
differs from the exact one by at most (m - 1) u times the sum of the terms'
sizes, and the scale rounds once more."""
import numpy as np
import pytest
import torch

from gpu_util import B

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
HALF_STEP = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
# half of the smallest subnormal step
TINY = {torch.float32: 2.0 ** -150, torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -134}


@pytest.fixture(scope="module")
def b():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    torch.cuda.set_device(0)
    return B()


def planes(n, cols, dtype, pad=3, fill=0.0):
    """(buffer, view [n][cols]) of a planar buffer with padding behind each plane."""
    buf = torch.full((cols, n + pad), fill, dtype=dtype, device="cuda")
    return buf, buf[:, :n].t()


def layout(x, kind):
    """x [n][cols] on the device as rows, padded rows, offset rows or planes."""
    n, cols = x.shape
    if kind == "rows":
        return x.contiguous()
    if kind == "padded":
        buf = torch.zeros((n, cols + 5), dtype=x.dtype, device="cuda")
        buf[:, :cols] = x
        return buf[:, :cols]
    if kind == "offset":  # starts one element past an aligned address
        buf = torch.zeros(n * cols + 1, dtype=x.dtype, device="cuda")
        buf[1:] = x.reshape(-1)
        return buf[1:].view(n, cols)
    if kind == "planes":
        return x.t().contiguous().t()
    buf, view = planes(n, cols, x.dtype)
    view.copy_(x)
    return view


def gen(seed):
    return torch.Generator("cuda").manual_seed(seed)


def make_ids(n, rows, seed, holes=0.1, hot=0.0):
    g = gen(seed)
    ids = torch.randint(rows, (n,), generator=g, device="cuda", dtype=torch.int32)
    r = torch.rand(n, generator=g, device="cuda")
    ids[r < hot] = rows // 3
    ids[r > 1 - holes] = -1
    return ids


# ---- lookup ------------------------------------------------------------------

@pytest.mark.parametrize("n", [1, 2, 31, 33, 257, 1000, 40_001])
@pytest.mark.parametrize("cols", [1, 3, 4, 12, 27, 48, 130])
@pytest.mark.parametrize("kind", ["rows", "padded", "offset", "planes", "padded_planes"])
def test_lookup(b, n, cols, kind):
    rows = 1 + (n * 7) % 301
    for k, (tt, to) in enumerate([(torch.float32, torch.float32), (torch.bfloat16, torch.float32),
                                  (torch.float16, torch.float16), (torch.float32, torch.bfloat16),
                                  (torch.bfloat16, torch.bfloat16), (torch.float16, torch.bfloat16),
                                  (torch.float32, torch.float16)]):
        table = torch.randn(rows, cols, generator=gen(n + k), device="cuda").to(tt)
        table = layout(table, ("rows", "padded", "offset")[k % 3])
        ids = make_ids(n, rows, n + cols + k)
        out = layout(torch.full((n, cols), 7.0, dtype=to, device="cuda"), kind)
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        scale = (1.0, 0.75, -3.0)[k % 3]
        b.gs_lookup(table, ids, out, scale=scale, dev_status=st)
        ref = torch.where((ids >= 0)[:, None], scale * table.double()[ids.clamp(min=0).long()], 0.0)
        err = (out.double() - ref).abs()
        assert (err <= (HALF_STEP[to] + 2 * U) * ref.abs() + TINY[to]).all()
        assert int(st) == 0


@pytest.mark.parametrize("kind", ["padded", "padded_planes"])
def test_lookup_leaves_the_padding(b, kind):
    n, cols = 77, 12
    table = torch.randn(9, cols, generator=gen(1), device="cuda")
    ids = make_ids(n, 9, 2)
    if kind == "padded":
        buf = torch.full((n + 4, cols + 5), 3.0, device="cuda")
        out = buf[:n, :cols]
    else:
        buf = torch.full((cols + 2, n + 5), 3.0, device="cuda")
        out = buf[:cols, :n].t()
    b.gs_lookup(table, ids, out)
    keep = torch.ones_like(buf, dtype=torch.bool)
    if kind == "padded":
        keep[:n, :cols] = False
    else:
        keep[:cols, :n] = False
    assert (buf[keep] == 3.0).all()


def test_lookup_through_an_index_and_ids_out_of_range(b):
    n, rows, cols = 500, 40, 27
    table = torch.randn(rows, cols, generator=gen(3), device="cuda")
    ids = make_ids(900, rows, 4)
    index = torch.randint(900, (n,), generator=gen(5), device="cuda", dtype=torch.int32)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = b.gs_lookup(table, ids, torch.empty(n, cols, device="cuda"), index=index, dev_status=st)
    got = ids[index.long()]
    ref = torch.where((got >= 0)[:, None], table[got.clamp(min=0).long()], 0.0)
    assert torch.equal(out, ref) and int(st) == 0
    for bad_ids, bad_index in ((rows, 0), (2 ** 31 - 1, 0), (0, 900), (0, -1), (0, 2 ** 31 - 1)):
        ids2, index2 = ids.clone(), index.clone()
        index2[17] = bad_index if bad_index else 3
        if bad_ids:
            ids2[3] = bad_ids
        st.zero_()
        out = b.gs_lookup(table, ids2, torch.empty(n, cols, device="cuda"), index=index2, dev_status=st)
        assert (out[17] == 0).all() and int(st) == 2
        same = (index2 != 3) & (index2 == index)
        assert torch.equal(out[same], ref[same])
        assert b.gs_check(st) == b.GS_ERR_BOUNDS and int(st) == 0


def test_lookup_keeps_non_finite_values_to_their_rows(b):
    table = torch.randn(5, 6, generator=gen(6), device="cuda")
    table[2, 1], table[2, 4] = float("nan"), float("inf")
    ids = torch.tensor([0, 2, -1, 4, 1], dtype=torch.int32, device="cuda")
    out = b.gs_lookup(table, ids, torch.empty(5, 6, device="cuda"), scale=2.0)
    assert torch.isfinite(out[[0, 2, 3, 4]]).all()
    assert torch.isnan(out[1, 1]) and torch.isinf(out[1, 4])


def test_lookup_of_no_rows_launches_nothing(b):
    n0 = b.gs_launch_counter()
    out = torch.empty((0, 4), device="cuda")
    b.gs_lookup(torch.ones(3, 4, device="cuda"), torch.empty(0, dtype=torch.int32, device="cuda"), out)
    assert b.gs_launch_counter() == n0


def test_lookup_past_32_bit_offsets(b):
    """Planes and rows whose element offsets pass 2^31."""
    n, cols, rows = 45_000_001, 48, 7
    table = torch.randn(rows, cols, generator=gen(7), device="cuda").half()
    ids = torch.randint(rows, (n,), generator=gen(8), device="cuda", dtype=torch.int32)
    at = torch.tensor([0, 1, n // 3, n - 2, n - 1], device="cuda")
    for out in (torch.empty((cols, n), dtype=torch.float16, device="cuda").t(),
                torch.empty((n, cols), dtype=torch.float16, device="cuda")):
        b.gs_lookup(table, ids, out)
        assert torch.equal(out[at], table[ids[at].long()])
        del out


# ---- gradient ----------------------------------------------------------------

def exact_grad(g, ids, rows, scale):
    """(sum, sum of sizes, number of terms) per table row in fp64."""
    g = g.double()
    ok = ids >= 0
    at = ids[ok].long()
    z = torch.zeros((rows, g.shape[1]), dtype=torch.float64, device="cuda")
    s = z.clone().index_add_(0, at, g[ok])
    a = z.clone().index_add_(0, at, g[ok].abs())
    m = torch.bincount(at, minlength=rows).double()[:, None]
    return scale * s, abs(scale) * a, m


def run_grad(b, g, ids, rows, **kw):
    dt = kw.pop("dtable", None)
    if dt is None:
        dt = torch.full((rows, g.shape[1]), 5.0, device="cuda")
    ws = torch.randint(255, (b.gs_lookup_bwd_workspace_size(g, rows),), dtype=torch.uint8,
                       generator=gen(11), device="cuda")
    return b.gs_lookup_bwd(g, ids, dt, ws, **kw)


def check_grad(got, ref, slack=0):
    s, a, m = ref
    err = (got.double() - s).abs()
    # m - 1 additions and the scale's product; 1.01 for products of (1 + u)
    assert (err <= 1.01 * (m + 1 + slack) * U * a + 2.0 ** -149).all(), float((err / (a + 1e-300)).max())


@pytest.mark.parametrize("n", [1, 2, 3, 33, 64, 65, 257, 1024, 1025, 5000, 40_001, 300_007])
@pytest.mark.parametrize("cols,kind", [(1, "rows"), (3, "planes"), (4, "rows"), (12, "padded_planes"),
                                       (27, "rows"), (48, "planes"), (48, "rows"), (16, "padded"),
                                       (64, "offset"), (130, "planes"), (128, "rows")])
def test_lookup_gradient(b, n, cols, kind):
    for k, (dtype, rows, hot, holes) in enumerate([
            (torch.float32, 1 + n // 3, 0.0, 0.1), (torch.bfloat16, 1, 0.0, 0.0),
            (torch.float16, 1000, 0.5, 0.02), (torch.float32, 256, 0.9, 0.5),
            (torch.float32, 70_001, 0.0, 0.0)]):
        g = torch.randn(n, cols, generator=gen(n + k), device="cuda").to(dtype)
        ids = make_ids(n, rows, n + cols + k, holes=holes, hot=hot)
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        scale = (0.75, 1.0, -2.0)[k % 3]
        view = layout(g, kind)
        got = run_grad(b, view, ids, rows, scale=scale, dev_status=st)
        check_grad(got, exact_grad(g, ids, rows, scale))
        assert int(st) == 0
        assert torch.equal(got, run_grad(b, view, ids, rows, scale=scale))  # the same bits again


def test_lookup_gradient_is_the_derivative(b):
    """Central differences of sum(w * lookup): linear in the table, so the
    difference is exact but for the rounding of its two fp64 sums."""
    n, rows, cols, scale = 300, 17, 5, 0.75
    table = torch.randn(rows, cols, generator=gen(21), device="cuda")
    w = torch.randn(n, cols, generator=gen(22), device="cuda")
    ids = make_ids(n, rows, 23)
    got = run_grad(b, w, ids, rows, scale=scale)
    s, a, m = exact_grad(w, ids, rows, scale)

    def value(t):
        return (w.double() * b.gs_lookup(t, ids, torch.empty(n, cols, device="cuda"), scale=scale).double()).sum()

    for k, c in ((0, 0), (5, 4), (16, 2)):
        hi, lo = table.clone(), table.clone()
        hi[k, c] += 1.0
        lo[k, c] -= 1.0
        d = (value(hi) - value(lo)) / (hi[k, c].double() - lo[k, c].double())
        # each looked-up value rounds by u of its size (at most 1 + |table|)
        assert abs(float(d - got[k, c])) <= float(2 * U * a[k, c] * (1 + table[k, c].abs())
                                                  + (m[k, 0] + 1) * U * a[k, c]) + 1e-12


def test_lookup_gradient_accumulates_and_keeps_padding(b):
    n, rows, cols = 3000, 50, 12
    g = torch.randn(n, cols, generator=gen(31), device="cuda")
    ids = make_ids(n, rows, 32)
    ids[ids == 7] = 8  # a row that no item uses
    buf = torch.full((rows, cols + 3), 2.0, device="cuda")
    before = torch.randn(rows, cols, generator=gen(33), device="cuda")
    dt = buf[:, :cols]
    dt.copy_(before)
    run_grad(b, g, ids, rows, dtable=dt, scale=0.5, accumulate=True)
    s, a, m = exact_grad(g, ids, rows, 0.5)
    check_grad(dt, (s + before.double(), a + before.double().abs(), m), slack=1)
    assert torch.equal(dt[7], before[7])
    assert (buf[:, cols:] == 2.0).all()
    run_grad(b, g, ids, rows, dtable=dt, scale=0.5)
    check_grad(dt, (s, a, m))
    assert (dt[7] == 0).all() and (buf[:, cols:] == 2.0).all()


@pytest.mark.parametrize("n", [700, 20_000])
def test_lookup_gradient_with_a_kept_order(b, n):
    rows, cols = 333, 27
    ids = make_ids(2 * n, rows, 41)
    index = torch.randperm(2 * n, generator=gen(42), device="cuda")[:n].sort().values.to(torch.int32)
    g = torch.randn(cols, n, generator=gen(43), device="cuda").t()
    ws = torch.empty(b.gs_lookup_bwd_workspace_size(g, rows), dtype=torch.uint8, device="cuda")
    b.gs_lookup_plan(ids, n, rows, cols, ws, index=index)
    for k in range(3):
        gk = g * (k + 1)
        gk = gk.t().contiguous().t()
        got = b.gs_lookup_bwd(gk, ids, torch.empty(rows, cols, device="cuda"), ws, index=index, planned=True)
        check_grad(got, exact_grad(gk, ids[index.long()], rows, 1.0))


@pytest.mark.parametrize("n", [200, 30_000])
def test_lookup_gradient_reads_no_row_without_an_id(b, n):
    """NaN and infinity in rows whose id is negative or out of range."""
    rows, cols = 20, 8
    g = torch.randn(n, cols, generator=gen(51), device="cuda")
    ids = make_ids(n, rows, 52, holes=0.3)
    clean = exact_grad(torch.where((ids >= 0)[:, None], g, 0.0), ids, rows, 1.0)
    g[ids < 0] = float("nan")
    g[(ids < 0).nonzero()[0]] = float("inf")
    check_grad(run_grad(b, g, ids, rows), clean)
    check_grad(run_grad(b, g.t().contiguous().t(), ids, rows), clean)
    wrong = ids.clone()
    wrong[(ids < 0).nonzero()[:2]] = rows
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    check_grad(run_grad(b, g, wrong, rows, dev_status=st), clean)
    assert int(st) == 2
    # every row without an id
    assert (run_grad(b, g, torch.full_like(ids, -1), rows) == 0).all()
    # a NaN in a used row stays in its table row
    ids[5] = 3
    g[5] = float("nan")
    got = run_grad(b, g, ids, rows)
    assert torch.isnan(got[3]).all() and torch.isfinite(got[[0, 1, 2] + list(range(4, rows))]).all()


def test_lookup_gradient_of_no_items(b):
    g = torch.empty((0, 4), device="cuda")
    none = torch.empty(0, dtype=torch.int32, device="cuda")
    dt = torch.ones(3, 4, device="cuda")
    ws = torch.empty(256, dtype=torch.uint8, device="cuda")
    b.gs_lookup_bwd(g, none, dt, ws, accumulate=True)
    assert (dt == 1).all()
    b.gs_lookup_bwd(g, none, dt, ws)
    assert (dt == 0).all()


def test_lookup_gradient_past_32_bit_offsets(b):
    n, cols, rows = 18_000_000, 120, 3
    g = torch.ones((n, cols), dtype=torch.float16, device="cuda")
    ids = torch.arange(n, device="cuda", dtype=torch.int32) % rows
    got = run_grad(b, g, ids, rows)
    # sums of ones are exact in fp32 up to 2^24
    assert (got == n // rows).all()
    del g
    g = torch.ones((cols, n), dtype=torch.float16, device="cuda").t()
    assert (run_grad(b, g, ids, rows) == n // rows).all()


def test_lookup_on_another_stream_and_in_a_graph(b):
    """Captured once and replayed with new inputs; on a side stream."""
    for n, rows, cols in ((50, 9, 16), (20_000, 700, 12)):
        table = torch.randn(rows, cols, generator=gen(61), device="cuda")
        ids = make_ids(n, rows, 62)
        out = torch.empty((cols, n), device="cuda").t()
        dt = torch.empty(rows, cols, device="cuda")
        ws = torch.empty(b.gs_lookup_bwd_workspace_size(out, rows), dtype=torch.uint8, device="cuda")
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        b.gs_lookup(table, ids, out, stream=side)
        b.gs_lookup_bwd(out, ids, dt, ws, stream=side)
        side.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            b.gs_lookup(table, ids, out, scale=0.5)
            b.gs_lookup_bwd(out, ids, dt, ws, scale=2.0)
        for seed in (63, 64):
            table.copy_(torch.randn(rows, cols, generator=gen(seed), device="cuda"))
            ids.copy_(make_ids(n, rows, seed))
            graph.replay()
            got_out, got_dt = out.clone(), dt.clone()
            want_out = b.gs_lookup(table, ids, torch.empty_like(out), scale=0.5)
            assert torch.equal(got_out, want_out)
            assert torch.equal(got_dt, run_grad(b, want_out.t().contiguous().t(), ids, rows, scale=2.0))


def test_lookup_capacity(b):
    g = torch.ones(5000, 8, device="cuda")
    ids = make_ids(5000, 10, 71)
    ws = torch.empty(b.gs_lookup_bwd_workspace_size(g, 10) - 1, dtype=torch.uint8, device="cuda")
    with pytest.raises(b.GsError) as e:
        b.gs_lookup_bwd(g, ids, torch.empty(10, 8, device="cuda"), ws)
    assert e.value.status == b.GS_ERR_CAPACITY


@pytest.mark.parametrize("n", [40, 3001])
@pytest.mark.parametrize("cols", [1500, 2051])
@pytest.mark.parametrize("kind", ["rows", "planes"])
def test_wide_rows(b, n, cols, kind):
    """More columns than a block takes at a time, with few and many table rows."""
    for rows in (10, 1500):
        ids = make_ids(n, rows, n + rows)
        table = torch.randn(rows, cols, generator=gen(81), device="cuda")
        out = layout(torch.zeros(n, cols, device="cuda"), kind)
        b.gs_lookup(table, ids, out)
        assert torch.equal(out, torch.where((ids >= 0)[:, None], table[ids.clamp(min=0).long()], 0.0))
        for dtype in (torch.float32, torch.bfloat16):
            g = torch.randn(n, cols, generator=gen(82), device="cuda").to(dtype)
            check_grad(run_grad(b, layout(g, kind), ids, rows), exact_grad(g, ids, rows, 1.0))


def test_two_calls_at_once(b):
    """Gradients on two streams with workspaces of their own."""
    n, rows, cols = 60_000, 5000, 27
    data = [(torch.randn(n, cols, generator=gen(90 + k), device="cuda"), make_ids(n, rows, 92 + k))
            for k in range(2)]
    out = [torch.empty(rows, cols, device="cuda") for _ in range(2)]
    ws = [torch.empty(b.gs_lookup_bwd_workspace_size(g, rows), dtype=torch.uint8, device="cuda")
          for g, _ in data]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(5):
        for k, (g, ids) in enumerate(data):
            b.gs_lookup_bwd(g, ids, out[k], ws[k], stream=streams[k])
    torch.cuda.synchronize()
    for k, (g, ids) in enumerate(data):
        assert torch.equal(out[k], run_grad(b, g, ids, rows))


def test_kept_order_with_planes_of_a_small_table(b):
    """A gradient in planes that needs no order leaves a kept one as it is."""
    n, rows, cols = 9000, 200, 12
    ids = make_ids(n, rows, 95)
    g = torch.randn(n, cols, generator=gen(96), device="cuda")
    planar = g.t().contiguous().t()
    ws = torch.empty(b.gs_lookup_bwd_workspace_size(planar, rows), dtype=torch.uint8, device="cuda")
    b.gs_lookup_plan(ids, n, rows, cols, ws)
    for _ in range(2):
        for x in (planar, g):
            got = b.gs_lookup_bwd(x, ids, torch.empty(rows, cols, device="cuda"), ws, planned=True)
            check_grad(got, exact_grad(g, ids, rows, 1.0))


@pytest.mark.parametrize("n", [2049, 3000, 40_001])
@pytest.mark.parametrize("pad,start", [(0, 0), (1, 0), (2, 1), (5, 3)])
def test_lookup_gradient_of_16_bit_planes(b, n, pad, start):
    """Planes of 16-bit types that start and follow at odd places, sorted."""
    for dtype, cols, rows in ((torch.bfloat16, 12, 5000), (torch.float16, 27, 1100), (torch.float16, 100, 2000)):
        g = torch.randn(n, cols, generator=gen(n + pad), device="cuda").to(dtype)
        buf = torch.full((cols * (n + pad) + start,), float("nan"), dtype=dtype, device="cuda")
        view = buf[start:].view(cols, n + pad)[:, :n].t()
        view.copy_(g)
        ids = make_ids(n, rows, n + start)
        check_grad(run_grad(b, view, ids, rows, scale=0.5), exact_grad(g, ids, rows, 0.5))


@pytest.mark.parametrize("n,rows,kind", [(300, 40, "rows"), (9000, 40, "planes"), (9000, 40, "rows"),
                                         (9000, 3000, "planes"), (200_000, 3000, "rows")])
def test_gradient_flags_every_index_out_of_range(b, n, rows, kind):
    """In the one-launch, the private-table and the sorted form and in a plan."""
    cols, n_ids = 12, 2 * n
    ids = make_ids(n_ids, rows, 101)
    index = torch.randint(n_ids, (n,), generator=gen(102), device="cuda", dtype=torch.int32)
    g = layout(torch.randint(-8, 9, (n, cols), generator=gen(103), device="cuda").float(), kind)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    for bad in (None, -1, -2, -3, -2 ** 31, n_ids, 2 ** 31 - 1):
        at = index.clone()
        if bad is not None:
            at[[0, n // 2, n - 1]] = bad
        ok = at == index
        got = torch.where(ok, ids[torch.where(ok, at, 0).long()], -1)
        flag = 0 if bad is None else 2
        dt = run_grad(b, g, ids, rows, index=at, dev_status=st)
        assert int(st) == flag, bad
        st.zero_()
        # sums of small integers are exact in any order
        assert torch.equal(dt.double(), exact_grad(g, got, rows, 1.0)[0])
        if n > 2048:
            ws = torch.empty(b.gs_lookup_bwd_workspace_size(g, rows), dtype=torch.uint8, device="cuda")
            b.gs_lookup_plan(ids, n, rows, cols, ws, index=at, dev_status=st)
            assert int(st) == flag, bad
            st.zero_()


@pytest.mark.parametrize("kind", ["rows", "offset", "planes"])
def test_lookup_rounds_the_fp32_product(b, kind):
    """The product of the fp32 scale in fp32, then its rounding to the output's
    type: bit for bit."""
    n, rows, scale = 5000, 700, 1 / 3
    for cols in (12, 27, 48):
        for tt in (torch.float32, torch.float16, torch.bfloat16):
            table = torch.randn(rows, cols, generator=gen(111), device="cuda").to(tt)
            ids = make_ids(n, rows, 112, holes=0.0)
            for to in (torch.float32, torch.float16, torch.bfloat16):
                out = b.gs_lookup(table, ids, layout(torch.zeros(n, cols, dtype=to, device="cuda"), kind), scale=scale)
                product = table.float() * torch.tensor(scale, dtype=torch.float32, device="cuda")
                assert torch.equal(out, product.to(to)[ids.long()])


# ---- exact sums: whole numbers of at most 8 are exact in every type, and so is
# ---- every sum of up to 2^21 of them in fp32, in any order

def whole(n, cols, seed, dtype=torch.float32):
    return torch.randint(-8, 9, (n, cols), generator=gen(seed), device="cuda").to(dtype)


@pytest.mark.parametrize("n", [33, 2048, 2049, 5000, 40_001, 300_007])
@pytest.mark.parametrize("cols,kind", [(1, "rows"), (12, "planes"), (27, "padded_planes"), (27, "rows"), (48, "rows"),
                                       (48, "planes"), (16, "padded"), (64, "offset"), (128, "rows")])
def test_gradient_of_whole_numbers_is_exact(b, n, cols, kind):
    """Every form and type, with rows that a large part of the items use: an
    item dropped, doubled or given to another row changes a sum."""
    for dtype in (torch.float32, torch.float16, torch.bfloat16):
        g = whole(n, cols, n, dtype)
        view = layout(g, kind)
        for rows, hot, holes in ((1, 0.0, 0.0), (1000, 0.5, 0.02), (1024, 0.0, 0.1), (1025, 0.9, 0.0),
                                 (3000, 0.3, 0.1), (70_001, 0.0, 0.0), (70_001, 0.6, 0.1)):
            ids = make_ids(n, rows, n + rows, holes=holes, hot=hot)
            want = exact_grad(g, ids, rows, 2.0)[0]
            got = run_grad(b, view, ids, rows, scale=2.0)
            assert torch.equal(got.double(), want), (dtype, rows, hot)
            got = run_grad(b, view, ids, rows, scale=-1.0, accumulate=True, dtable=got)
            assert torch.equal(got.double(), want / 2), (dtype, rows, hot)


@pytest.mark.parametrize("n", [700, 20_000, 200_000])  # one launch; up to 64 tiles of the sort; more
@pytest.mark.parametrize("rows", [900, 1100, 70_001, (1 << 20) + 7])  # one, two, two and three passes
@pytest.mark.parametrize("kind", ["rows", "planes"])
def test_kept_order_is_the_one_that_is_summed(b, n, rows, kind):
    """A plan made through an index; other ids at the gradient's call show
    whether it goes by the kept order."""
    cols = 12
    ids, others = make_ids(2 * n, rows, 121, hot=0.2), make_ids(2 * n, rows, 122)
    index = torch.randperm(2 * n, generator=gen(123), device="cuda")[:n].to(torch.int32)
    uses_order = n > 2048 and not (kind == "planes" and rows <= 1024)
    by = (ids if uses_order else others)[index.long()]
    ws = torch.empty(b.gs_lookup_bwd_workspace_size(layout(whole(n, cols, 1), kind), rows), dtype=torch.uint8,
                     device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    b.gs_lookup_plan(ids, n, rows, cols, ws, index=index, dev_status=st)
    dt = torch.full((rows, cols), 3.0, device="cuda")
    total = torch.zeros((rows, cols), dtype=torch.float64, device="cuda")
    for k, dtype in enumerate((torch.float32, torch.float16, torch.bfloat16)):
        g = whole(n, cols, 124 + k, dtype)
        total += exact_grad(g, by, rows, 1.0)[0]
        b.gs_lookup_bwd(layout(g, kind), others, dt, ws, index=index, planned=True, accumulate=k > 0, dev_status=st)
        assert torch.equal(dt.double(), total)
    assert int(st) == 0


@pytest.mark.parametrize("n", [20_000, 200_000])
@pytest.mark.parametrize("kind", ["rows", "planes"])
def test_sorted_gradient_in_a_graph(b, n, kind):
    """The sorted form, a plan and a planned gradient, captured and replayed
    with new ids and gradients."""
    rows, cols = 3000, 12
    ids, g = make_ids(n, rows, 131), layout(whole(n, cols, 132), kind)
    dt, kept = torch.empty(rows, cols, device="cuda"), torch.empty(rows, cols, device="cuda")
    size = b.gs_lookup_bwd_workspace_size(g, rows)
    ws, plan = (torch.empty(size, dtype=torch.uint8, device="cuda") for _ in range(2))

    def calls():
        b.gs_lookup_bwd(g, ids, dt, ws, scale=2.0)
        b.gs_lookup_plan(ids, n, rows, cols, plan)
        b.gs_lookup_bwd(g, ids, kept, plan, planned=True)
        b.gs_lookup_bwd(g, ids, kept, plan, planned=True, accumulate=True)

    calls()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        calls()
    for seed in (133, 134, 135):
        ids.copy_(make_ids(n, rows, seed, hot=0.3))
        g.copy_(whole(n, cols, seed))
        ws.fill_(seed)
        plan.fill_(seed)
        graph.replay()
        want = exact_grad(g, ids, rows, 2.0)[0]
        assert torch.equal(dt.double(), want) and torch.equal(kept.double(), want)


@pytest.mark.parametrize("cols", [3, 12, 16, 27, 48, 64, 130])
def test_lookup_into_planes_through_an_index(b, cols):
    """Both kernels, aligned and unaligned tables of each type."""
    n, rows, n_ids = 5001, 300, 9000
    for k, (tt, to) in enumerate([(torch.float32, torch.float32), (torch.bfloat16, torch.float32),
                                  (torch.float16, torch.float16)]):
        for kind in ("rows", "padded", "offset"):
            table = layout(torch.randn(rows, cols, generator=gen(141 + k), device="cuda").to(tt), kind)
            ids = make_ids(n_ids, rows, 142)
            index = torch.randint(n_ids, (n,), generator=gen(143), device="cuda", dtype=torch.int32)
            buf, out = planes(n, cols, to, pad=5, fill=3.0)
            st = torch.zeros(1, dtype=torch.int32, device="cuda")
            b.gs_lookup(table, ids, out, index=index, dev_status=st)
            got = ids[index.long()]
            want = torch.where((got >= 0)[:, None], table[got.clamp(min=0).long()].to(to), 0.0)
            assert torch.equal(out, want) and int(st) == 0 and (buf[:, n:] == 3.0).all()
            for bad in (-1, -2, n_ids, 2 ** 31 - 1):
                at = index.clone()
                at[[0, 77, n - 1]] = bad
                b.gs_lookup(table, ids, out, index=at, dev_status=st)
                assert int(st) == 2 and torch.equal(out, torch.where((at == index)[:, None], want, 0.0))
                st.zero_()


def rest_is_zero(dt, used):
    """No element outside the rows `used` is set."""
    dt[used] = 0.0
    return int(torch.count_nonzero(dt)) == 0


@pytest.mark.parametrize("n", [300, 2049, 200_000])
@pytest.mark.parametrize("rows,cols", [(2 ** 20 + 5, 12), (2 ** 26 + 3, 48), (2 ** 31 - 1, 1)])
def test_large_tables(b, n, rows, cols):
    """Three and four passes of the sort; table offsets past 2^31 elements."""
    used = torch.randint(rows, (64,), generator=gen(151), device="cuda", dtype=torch.int32).unique()
    used = torch.cat([used, torch.tensor([rows - 1, rows - 2, 0], dtype=torch.int32, device="cuda")]).unique()
    pick = torch.randint(len(used), (n,), generator=gen(152), device="cuda", dtype=torch.int32)
    pick[::7] = -1
    ids = torch.where(pick >= 0, used[pick.clamp(min=0).long()], -1)
    for kind in ("rows", "planes"):
        g = whole(n, cols, 153)
        dt = torch.full((rows, cols), 5.0, device="cuda")
        run_grad(b, layout(g, kind), ids, rows, dtable=dt)
        assert torch.equal(dt[used.long()].double(), exact_grad(g, pick, len(used), 1.0)[0])
        assert rest_is_zero(dt, used.long())
        del dt
    table = torch.zeros((rows, cols), dtype=torch.float16, device="cuda")
    table[used.long()] = whole(len(used), cols, 154, torch.float16)
    for kind in ("rows", "planes"):
        out = b.gs_lookup(table, ids, layout(torch.ones(n, cols, device="cuda"), kind))
        assert torch.equal(out, torch.where((ids >= 0)[:, None], table[ids.clamp(min=0).long()].float(), 0.0))


def test_planes_turned_past_32_bit_offsets(b):
    """A gradient in planes of more than 2^31 elements, sorted: turned to rows
    and summed."""
    n, cols, rows = 45_000_001, 48, 3000
    j = torch.arange(n, device="cuda")
    ids = (j * 7919 % rows).to(torch.int32)
    g = torch.empty((cols, n), dtype=torch.float16, device="cuda")
    for c in range(cols):
        g[c] = (j * (c + 3)) % 17 - 8
    got = run_grad(b, g.t(), ids, rows)
    for c in range(cols):
        want = torch.zeros(rows, dtype=torch.float64, device="cuda").index_add_(0, ids.long(), g[c].double())
        assert torch.equal(got[:, c].double(), want), c
