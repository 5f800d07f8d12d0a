"""The view step through a colour codebook and with a clipped gradient: lookup,
render, projection backward, the table's gradient, the norm over both and the
clipped Adam updates, against the CPU oracle's gradient.

The compact gradients are within GRAD_TOL (relative L2 per tensor) of the
oracle's, as in the other parity tests; what follows from them here in fp64
keeps that: the norm moves by at most GRAD_TOL of itself, a clipped gradient
by twice that (its own error and the coefficient's), and a sum of up to m
rows by sqrt(m) times their L2 error (Cauchy-Schwarz)."""
import math

import numpy as np
import pytest
import torch

from gaussian_splatting_differentiable_dgs_b200 import synth
from gpu_util import need_gpu, rel_l2

pytestmark = pytest.mark.gpu

GRAD_TOL = 1e-4
B1, B2 = 0.9, 0.999
GROUPS = [(0, 3), (3, 6), (6, 10), (10, 11), (11, None)]


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    need_gpu()
    torch.cuda.set_device(0)


def scene(n=300, seed=9):
    s, cams = synth.tiny_scene(n=n, width=160, height=120, sh_degree=3, seed=seed, scale_px=(1.0, 12.0))
    return s, cams


def oracle(oracle_mod, sc, params, cam, target):
    return oracle_mod.step(params.astype(np.float64), sc.n, sc.sh_degree, cam, target.astype(np.float64))


def codebook_scene(K=20, scale=0.75, seed=3):
    """A scene whose SH planes are decoded from a table; a few without code."""
    sc, cams = scene()
    rng = np.random.default_rng(seed)
    table = (rng.normal(size=(K, sc.P - 11)) * 0.2).astype(np.float32)
    codes = rng.integers(0, K, sc.n).astype(np.int32)
    codes[rng.random(sc.n) < 0.05] = -1
    params = sc.params.copy()
    decoded = np.where(codes[:, None] >= 0, np.float32(scale) * table[np.maximum(codes, 0)], np.float32(0))
    params[11:, :sc.n] = decoded.T
    return sc, cams, params, table, codes


def table_grad(grad_sh, codes, K, scale):
    out = np.zeros((K, grad_sh.shape[0]))
    ok = codes >= 0
    np.add.at(out, codes[ok], scale * grad_sh.T[ok])
    return out


def check_m(m, ref, coef, tol):
    """Adam's first moment after one step is (1 - b1) c g; `implied` has its
    three fp32 roundings, within 1e-6 of itself."""
    for a, e in GROUPS:
        e = ref.shape[0] if e is None else e
        if e > a and np.linalg.norm(ref[a:e]) > 0:
            assert rel_l2(m[a:e].astype(np.float64) / (1 - B1), coef * ref[a:e]) <= tol + 1e-6, (a, e)


@pytest.mark.parametrize("share", [0.25, 50.0])
@pytest.mark.parametrize("mode", ["bounded", "original"])
def test_clipped_step(oracle_mod, share, mode):
    from gaussian_splatting_differentiable_dgs_b200.step import GaussianModel, Stepper
    sc, cams = scene()
    target = synth.random_image(160, 120, 12) * 0.6
    ref = oracle(oracle_mod, sc, sc.params, cams[0], target)
    g = ref["grad"][:, :sc.n]
    norm = np.linalg.norm(g)
    model = GaussianModel(sc.params, sc.n, sc.sh_degree)
    stp = Stepper(model, budget=200_000, mode=mode, max_grad_norm=share * norm)
    stp.run_view(cams[0], torch.as_tensor(target).cuda())
    stp.check()
    assert abs(stp.last_grad_norm() - norm) <= (GRAD_TOL + 1e-6) * norm
    coef = min(1.0, share * norm / (norm + 1e-6))
    check_m(model.m.cpu().numpy()[:, :sc.n], g, coef, 2 * GRAD_TOL)
    # parameters after the first update move by lr where the gradient is clear
    d = np.abs(model.params.cpu().numpy()[:, :sc.n] - ref["params"][:, :sc.n])
    assert d[np.abs(coef * g) > 1e-3 * np.abs(coef * g).max()].max() <= 2e-5


@pytest.mark.parametrize("max_norm", [None, 0.25, 50.0])
def test_codebook_step(oracle_mod, max_norm):
    from gaussian_splatting_differentiable_dgs_b200.codebook import ColorCodebook
    from gaussian_splatting_differentiable_dgs_b200.step import GaussianModel, Stepper
    scale = 0.75
    sc, cams, params, table, codes = codebook_scene(scale=scale)
    target = synth.random_image(160, 120, 5) * 0.6
    ref = oracle(oracle_mod, sc, params, cams[0], target)
    g = ref["grad"][:, :sc.n]
    want = table_grad(g[11:], codes, len(table), scale)
    norm = math.hypot(np.linalg.norm(g[:11]), np.linalg.norm(want))
    model = GaussianModel(sc.params, sc.n, sc.sh_degree)  # its own colours are replaced
    cb = ColorCodebook(table, codes, scale)
    stp = Stepper(model, budget=200_000, codebook=cb,
                  max_grad_norm=None if max_norm is None else max_norm * norm)
    assert np.array_equal(model.params.cpu().numpy()[11:, :sc.n], params[11:, :sc.n])
    stp.run_view(cams[0], torch.as_tensor(target).cuda())
    stp.check()
    assert abs(stp.last_loss() - ref["loss"]) <= 1e-5 * ref["loss"]
    coef = 1.0 if max_norm is None else min(1.0, max_norm * norm / (norm + 1e-6))
    most = np.bincount(codes[codes >= 0]).max()
    slack = scale * math.sqrt(most) * GRAD_TOL * np.linalg.norm(g[11:])
    got = cb.grad.cpu().numpy().astype(np.float64)
    assert np.linalg.norm(got - want) <= slack + 1e-6 * np.linalg.norm(want)
    tol = GRAD_TOL + slack / np.linalg.norm(want)
    if max_norm is not None:
        assert abs(stp.last_grad_norm() - norm) <= (tol + 1e-6) * norm
    check_m(model.m.cpu().numpy()[:11, :sc.n], g[:11], coef, 2 * tol)
    got_m = cb.m.cpu().numpy().astype(np.float64) / (1 - B1)
    assert rel_l2(got_m, coef * want) <= 2 * tol + 1e-6
    # the SH planes take no update of their own: they are the new table's rows
    assert not model.m[11:].any() and not model.v[11:].any()
    new = cb.table.cpu().numpy()
    assert not np.array_equal(new, table)
    decoded = np.where(codes[:, None] >= 0, np.float32(scale) * new[np.maximum(codes, 0)], np.float32(0))
    assert np.array_equal(model.params.cpu().numpy()[11:, :sc.n], decoded.T)


def test_grouped_codebook_step_matches_the_whole_view():
    from gaussian_splatting_differentiable_dgs_b200.codebook import ColorCodebook
    from gaussian_splatting_differentiable_dgs_b200.step import GaussianModel, Stepper
    sc, cams, params, table, codes = codebook_scene()
    target = torch.as_tensor(synth.random_image(160, 120, 6) * 0.6).cuda()
    out = []
    for grouped in (False, True):
        model, cb = GaussianModel(params, sc.n, sc.sh_degree), ColorCodebook(table, codes, 0.75)
        stp = Stepper(model, budget=200_000, codebook=cb, max_grad_norm=1e-3)
        (stp.run_view_grouped if grouped else stp.run_view)(cams[0], target)
        stp.check()
        assert model.step == 1
        out.append((model.m.cpu().numpy()[:11, :sc.n], cb.m.cpu().numpy(), stp.last_grad_norm()))
    (m0, t0, n0), (m1, t1, n1) = out
    assert rel_l2(m1, m0) <= 2 * GRAD_TOL and rel_l2(t1, t0) <= 2 * GRAD_TOL
    assert abs(n1 - n0) <= 2 * GRAD_TOL * n0


def test_codebook_training_loop_runs():
    """Several views through the prefetcher, with more items than one launch of
    the table's gradient takes; fixed blocks; a view without candidates."""
    from gaussian_splatting_differentiable_dgs_b200.codebook import ColorCodebook
    from gaussian_splatting_differentiable_dgs_b200.step import GaussianModel, Stepper, TargetPrefetcher
    sc, cams = scene(n=6000, seed=2)
    rng = np.random.default_rng(1)
    table = (rng.normal(size=(1500, sc.P - 11)) * 0.2).astype(np.float32)
    cb = ColorCodebook(table, rng.integers(0, 1500, sc.n))
    model = GaussianModel(sc.params, sc.n, sc.sh_degree)
    stp = Stepper(model, codebook=cb, max_grad_norm=0.5, leaf_streams=2)
    targets = [torch.as_tensor(synth.random_image(160, 120, k) * 0.5).pin_memory() for k in range(3)]
    feeder = TargetPrefetcher(targets, stepper=stp)
    for v, target in feeder.iterate([0, 1, 2, 0]):
        stp.run_view(cams[0], target)
        stp.check()
        assert math.isfinite(stp.last_loss()) and stp.last_grad_norm() > 0
    stp.run_view_blocks(cams[0], targets[0].cuda(), blocks=(2, 2))
    stp.check()
    away = synth.Camera(cams[0].R, cams[0].t + np.float32([0, 0, -1e4]), cams[0].fx, cams[0].fy,
                        cams[0].cx, cams[0].cy, cams[0].width, cams[0].height)
    before = cb.table.clone()
    stats = stp.run_view(away, targets[0].cuda())
    stp.check()
    assert stats.n_cand == 0 and stp.last_grad_norm() == 0.0
    assert torch.isfinite(cb.table).all() and not torch.equal(cb.table, before)  # the moments go on
    assert torch.equal(model.params[11:, :sc.n].t(), cb.table[cb.codes.long()])
    img = stp.render(cams[0])
    assert torch.isfinite(img).all()


def test_codebook_refusals():
    from gaussian_splatting_differentiable_dgs_b200.codebook import ColorCodebook
    from gaussian_splatting_differentiable_dgs_b200.step import GaussianModel, Stepper
    sc, cams = scene(n=30)
    model = GaussianModel(sc.params, sc.n, sc.sh_degree)
    table = np.zeros((4, sc.P - 11), np.float32)
    for cb in (ColorCodebook(table[:, :-1], np.zeros(sc.n, np.int32)),
               ColorCodebook(table, np.zeros(sc.n - 1, np.int32))):
        with pytest.raises(ValueError):
            Stepper(model, codebook=cb)
    with pytest.raises(ValueError):
        Stepper(model).last_grad_norm()


def test_codebook_gradient_on_another_stream():
    """Two gradients queued on a side stream, the second with more candidates:
    memory allocated on the current stream in the meantime belongs to neither."""
    from gaussian_splatting_differentiable_dgs_b200 import binding as B
    from gaussian_splatting_differentiable_dgs_b200.codebook import ColorCodebook
    rng = np.random.default_rng(4)
    n, K, cols = 400_000, 3000, 12
    cb = ColorCodebook(np.zeros((K, cols), np.float32), rng.integers(0, K, n), 0.5)
    g = torch.as_tensor(rng.integers(-8, 9, (cols, n)).astype(np.float32)).cuda()
    few = g[:, :100_000].contiguous()
    need = B.gs_lookup_bwd_workspace_size(few.t(), K)
    want = torch.zeros((K, cols), device="cuda").index_add_(0, cb.codes.long(), g.t()) * 0.5
    long = torch.empty(1 << 30, dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        for _ in range(50):  # keeps the side stream busy while the host goes on
            long.fill_(1)
    index = torch.arange(n, dtype=torch.int32, device="cuda")
    side.wait_stream(torch.cuda.current_stream())
    for handle in (side, side.cuda_stream):
        cb.gradient(few, index[:100_000], stream=handle)
        cb.gradient(g, index, stream=handle)
    others = [torch.full((need // 8 * k,), 255, dtype=torch.uint8, device="cuda") for k in range(4, 13)]
    torch.cuda.synchronize()
    assert all(bool((x == 255).all()) for x in others)
    assert torch.equal(cb.grad, want)  # sums of small integers are exact


def test_codebook_workspace_is_in_the_working_set():
    """The gradient's workspace counts in peak_ws_bytes of every view, the later
    ones too: none of it is held between views, where the peak starts from."""
    from gaussian_splatting_differentiable_dgs_b200 import binding as B
    from gaussian_splatting_differentiable_dgs_b200.codebook import ColorCodebook
    from gaussian_splatting_differentiable_dgs_b200.step import GaussianModel, Stepper
    sc, cams = scene(n=60_000, seed=2)
    rng = np.random.default_rng(1)
    cb = ColorCodebook(np.zeros((1500, sc.P - 11), np.float32), rng.integers(0, 1500, sc.n))
    stp = Stepper(GaussianModel(sc.params, sc.n, sc.sh_degree), codebook=cb)
    target = torch.as_tensor(synth.random_image(160, 120, 1) * 0.5).cuda()
    for _ in range(3):
        before = torch.cuda.memory_allocated()
        stats = stp.run_view(cams[0], target)
        stp.check()
        after = torch.cuda.memory_allocated()
        g = torch.empty((sc.P - 11, stats.n_cand), device="cuda").t()
        need = B.gs_lookup_bwd_workspace_size(g, 1500)
        assert stats.n_cand > 10_000 and need > 200 * stats.n_cand
        assert after - before < 1 << 20
        assert stats.peak_ws_bytes >= need + 4 * sc.P * stats.n_cand  # beside the compact gradient
        del g


def test_codebook_step_of_the_whole_image_mode():
    """mode="original" takes the same update as the bounded mode."""
    from gaussian_splatting_differentiable_dgs_b200.codebook import ColorCodebook
    from gaussian_splatting_differentiable_dgs_b200.step import GaussianModel, Stepper
    sc, cams, params, table, codes = codebook_scene()
    target = torch.as_tensor(synth.random_image(160, 120, 6) * 0.6).cuda()
    out = []
    for mode in ("bounded", "original"):
        model, cb = GaussianModel(params, sc.n, sc.sh_degree), ColorCodebook(table, codes, 0.75)
        stp = Stepper(model, budget=200_000, codebook=cb, max_grad_norm=1e-3, mode=mode)
        stp.run_view(cams[0], target)
        stp.check()
        assert not model.m[11:].any()
        new = cb.table.cpu().numpy()
        decoded = np.where(codes[:, None] >= 0, np.float32(0.75) * new[np.maximum(codes, 0)], np.float32(0))
        assert np.array_equal(model.params.cpu().numpy()[11:, :sc.n], decoded.T)
        out.append((model.m.cpu().numpy()[:11, :sc.n], cb.m.cpu().numpy(), stp.last_grad_norm()))
    (m0, t0, n0), (m1, t1, n1) = out
    assert rel_l2(m1, m0) <= 2 * GRAD_TOL and rel_l2(t1, t0) <= 2 * GRAD_TOL
    assert abs(n1 - n0) <= 2 * GRAD_TOL * n0


def test_codebook_gradient_in_a_graph():
    """Captured with a workspace of the graph's own: eager calls and other
    allocations between replays do not share it."""
    from gaussian_splatting_differentiable_dgs_b200.codebook import ColorCodebook
    rng = np.random.default_rng(5)
    n, K, cols = 30_000, 3000, 12
    cb = ColorCodebook(np.zeros((K, cols), np.float32), rng.integers(0, K, 4 * n))
    codes = cb.codes.long()
    whole = lambda k: torch.as_tensor(rng.integers(-8, 9, (cols, k)).astype(np.float32)).cuda()
    exact = lambda g: torch.zeros((K, cols), device="cuda").index_add_(0, codes[:g.shape[1]], g.t())
    g, more = whole(n), whole(4 * n)
    cb.gradient(g)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cb.gradient(g)
    for _ in range(3):
        cb.gradient(more)
        assert torch.equal(cb.grad, exact(more))
        others = [torch.full((1 << k,), 255, dtype=torch.uint8, device="cuda") for k in range(16, 25)]
        g.copy_(whole(n))
        graph.replay()
        assert torch.equal(cb.grad, exact(g))
        assert all(bool((x == 255).all()) for x in others)


def test_grouped_update_is_in_the_working_set(monkeypatch):
    """The grouped schedule's one update sums the codebook's gradient over all
    Gaussians behind the regions: what it takes counts (here 64 MiB more than
    its workspace, far above a region's peak)."""
    from gaussian_splatting_differentiable_dgs_b200 import binding as B
    from gaussian_splatting_differentiable_dgs_b200.codebook import ColorCodebook
    from gaussian_splatting_differentiable_dgs_b200.step import GaussianModel, Stepper
    sc, cams = scene(n=6000, seed=2)
    rng = np.random.default_rng(1)
    cb = ColorCodebook(np.zeros((1500, sc.P - 11), np.float32), rng.integers(0, 1500, sc.n))
    stp = Stepper(GaussianModel(sc.params, sc.n, sc.sh_degree), budget=200_000, codebook=cb)
    target = torch.as_tensor(synth.random_image(160, 120, 1) * 0.5).cuda()
    need = B.gs_lookup_bwd_workspace_size(stp.model.params[11:, :sc.n].t(), 1500)
    gradient = cb.gradient

    def more(*args, **kw):
        held = torch.empty(64 << 20, dtype=torch.uint8, device="cuda")
        gradient(*args, **kw)
        del held

    monkeypatch.setattr(cb, "gradient", more)
    for _ in range(2):
        stats = stp.run_view_grouped(cams[0], target, groups=(3, 3))
        stp.check()
        assert stats.peak_ws_bytes >= (64 << 20) + need + target.numel() * 4
