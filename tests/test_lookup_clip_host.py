"""Refusals of the lookup, norm and clipping calls: all on the host, before
any device work, so none of them needs a GPU."""
import ctypes

import pytest
import torch

from gaussian_splatting_differentiable_dgs_b200 import build


@pytest.fixture(scope="module")
def b():
    build.build()
    from gaussian_splatting_differentiable_dgs_b200 import binding
    return binding


def ref(x):
    return ctypes.byref(x)


def mat(b, rows=4, cols=3, rs=3, cs=1, dtype=0, data=256):
    return b.gs_matrix(data, rows, rs, cs, cols, dtype)


def test_lookup_refusals(b):
    L, n0 = b.lib(), b.gs_launch_counter()

    def call(t, o, ids=256, n_ids=4, index=None):
        return L.gs_lookup(ref(t), ids, n_ids, index, 1.0, ref(o), None, None)

    good = mat(b)
    A, S = b.GS_ERR_ARG, b.GS_ERR_UNSUPPORTED
    assert L.gs_lookup(None, 256, 4, None, 1.0, ref(good), None, None) == A
    assert call(good, mat(b, cols=2, rs=2)) == A                   # columns differ
    assert call(good, mat(b, rs=2)) == A                           # rows overlap
    assert call(good, mat(b, rs=1, cs=3)) == A                     # planes overlap
    assert call(good, mat(b, rs=6, cs=2)) == A                     # neither axis contiguous
    assert call(good, mat(b, rows=-1)) == A
    assert call(good, mat(b, cols=0)) == A
    assert call(good, mat(b, dtype=3)) == A and call(mat(b, dtype=-1), good) == A
    assert call(good, mat(b, data=None)) == A
    assert call(good, mat(b, data=258)) == A                       # misaligned fp32
    assert call(mat(b, data=257, dtype=1), good) == A              # misaligned fp16
    assert call(good, good, ids=None) == A
    assert call(good, good, n_ids=3) == A                          # fewer ids than rows
    assert call(good, good, n_ids=-1) == A
    assert call(good, good, ids=258) == A and call(good, good, index=258) == A
    assert call(mat(b, rows=0), good) == A                         # an empty table
    assert call(mat(b, rs=1, cs=4), good) == S                     # a table in planes
    assert call(good, mat(b, rows=2 ** 31), n_ids=2 ** 31) == S
    wide = mat(b, cols=2 ** 30 + 1, rs=2 ** 31)
    assert call(wide, wide) == S
    assert call(mat(b, rows=0), mat(b, rows=0)) == b.GS_OK
    assert b.gs_launch_counter() == n0


def test_lookup_gradient_refusals(b):
    L, n0 = b.lib(), b.gs_launch_counter()
    A, S, K = b.GS_ERR_ARG, b.GS_ERR_UNSUPPORTED, b.GS_ERR_CAPACITY
    big = 1 << 30

    def call(g, d, ids=256, n_ids=4, index=None, flags=1, ws=256, nb=big):
        return L.gs_lookup_bwd(ref(g), ids, n_ids, index, 1.0, ref(d), flags, ws, nb, None, None)

    good = mat(b)
    assert call(good, good, flags=4) == A
    assert call(good, mat(b, cols=2, rs=2)) == A
    assert call(good, mat(b, rows=0)) == A
    assert call(good, mat(b, rows=2 ** 31)) == A
    assert call(good, mat(b, dtype=1)) == S                        # an fp32 gradient only
    assert call(good, mat(b, rs=1, cs=4)) == S
    assert call(good, good, n_ids=3) == A and call(good, good, ids=None) == A
    assert call(good, good, ws=None) == K and call(good, good, nb=0) == K
    assert call(good, good, ws=384) == A                           # workspace alignment
    assert call(mat(b, rows=2 ** 31), good, n_ids=2 ** 31) == S
    plan = lambda **k: L.gs_lookup_plan(*[{"ids": 256, "n_ids": 4, "index": None, "n": 4, "rows": 4,
                                          "cols": 3, "ws": 256, "nb": big, **k}[x] for x in
                                         ("ids", "n_ids", "index", "n", "rows", "cols", "ws", "nb")],
                                        None, None)
    assert plan(rows=0) == A and plan(cols=0) == A and plan(n=-1) == A and plan(n=5) == A
    assert plan(ws=None) == K and plan(nb=16) == K and plan(ws=264) == A
    assert plan(n=0) == b.GS_OK
    assert L.gs_lookup_bwd_workspace_size(-1, 4, 3, 0) == 0
    assert L.gs_lookup_bwd_workspace_size(4, 0, 3, 0) == 0
    assert L.gs_lookup_bwd_workspace_size(4, 4, 2 ** 30 + 1, 0) == 0
    wide = mat(b, cols=2 ** 30 + 1, rs=2 ** 31)
    assert call(wide, wide) == S and plan(cols=2 ** 30 + 1) == S
    assert 0 < L.gs_lookup_bwd_workspace_size(10, 4, 3, 0) <= L.gs_lookup_bwd_workspace_size(10 ** 6, 4, 3, 1)
    assert b.gs_launch_counter() == n0


def test_norm_and_clip_refusals(b):
    L, n0 = b.lib(), b.gs_launch_counter()
    A, K = b.GS_ERR_ARG, b.GS_ERR_CAPACITY
    T = b.gs_tensor

    def norm(t, max_norm=1.0, eps=0.0, clip=256, ws=256, nb=1 << 20, count=1):
        return L.gs_grad_norm(ref(t) if t is not None else None, count, max_norm, eps, clip, ws, nb, None, None)

    good = T(256, 2, 5, 8, 0, 0)
    assert norm(None) == A and norm(good, count=-1) == A
    for bad in (T(256, 2, 5, 4, 0, 0), T(None, 1, 5, 5, 0, 0), T(258, 1, 5, 5, 0, 0), T(257, 1, 5, 5, 2, 0),
                T(256, -1, 5, 5, 0, 0), T(256, 1, -5, 5, 0, 0), T(256, 1, 5, 5, 3, 0), T(256, 2 ** 40, 2 ** 40, 2 ** 40, 0, 0)):
        assert norm(bad) == A
    for v in (-1.0, float("nan"), float("inf")):
        assert norm(good, max_norm=v) == A and norm(good, eps=v) == A
    assert norm(good, clip=None) == A and norm(good, clip=260) == A
    assert norm(good, ws=None) == K and norm(good, nb=8) == K and norm(good, ws=264) == A
    assert L.gs_grad_norm_workspace_size(-1) == 0 and L.gs_grad_norm_workspace_size(0) > 0

    def clip(s, d, c=256, count=1):
        return L.gs_grad_clip(ref(s), ref(d), count, c, None)

    assert clip(good, T(4096, 2, 5, 8, 1, 0)) == A                 # another type
    assert clip(good, T(4096, 2, 4, 8, 0, 0)) == A                 # another shape
    assert clip(good, T(260, 2, 5, 8, 0, 0)) == A                  # overlapping
    assert clip(good, T(4096, 5, 2, 8, 0, 0)) == A                 # other rows
    assert clip(good, T(256, 2, 5, 9, 0, 0)) == A                  # in place with other strides
    assert clip(good, T(256, 1, 10, 10, 0, 0)) == A
    assert clip(good, good, c=None) == A
    assert clip(T(256, 0, 5, 8, 0, 0), T(256, 0, 5, 8, 0, 0)) == b.GS_OK  # nothing to do
    args = b.gs_adam_args(1e-3, 0.9, 0.999, 1e-8, 1, 0)
    adam = lambda a=args, n=4, pad=4, P=3, clip=256, st=4: L.gs_adam_clipped(256, 256, 256, 256, st, None, n, pad, P, ref(a), clip, None)
    assert adam(clip=None) == A and adam(n=-1) == A and adam(pad=3) == A and adam(P=0) == A and adam(st=3) == A
    assert adam(b.gs_adam_args(1e-3, 0.9, 0.999, 1e-8, 0, 0)) == A
    assert adam(n=0) == b.GS_OK
    assert b.gs_launch_counter() == n0


def test_binding_refuses_what_it_cannot_describe(b):
    f = torch.zeros
    i = f(4, dtype=torch.int32)
    with pytest.raises(ValueError):  # on the CPU
        b.gs_lookup(f(3, 2), i, f(4, 2))
    with pytest.raises(ValueError):
        b.gs_lookup(f(3, 2), i.long(), f(4, 2))
    with pytest.raises(ValueError):
        b.gs_lookup(f(3, 2), i, f(4, 2), index=i[:3])
    with pytest.raises(ValueError):
        b.matrix(f(3))
    with pytest.raises(ValueError):
        b.matrix(f(3, 2, dtype=torch.float64))
    with pytest.raises(ValueError):
        b.tensor_list([f(3, dtype=torch.int32)])
    with pytest.raises(ValueError):
        b.tensor_list([f(4, 6)[:, ::2]])
    with pytest.raises(ValueError):
        b.gs_grad_clip([f(3)], [f(3), f(2)], f(2))
    with pytest.raises(ValueError):
        b.gs_grad_norm([f(3)], 1.0, f(1), f(256, dtype=torch.uint8))


def test_matrix_descriptors(b):
    f = torch.zeros
    d = lambda m: (m.rows, m.cols, m.row_stride, m.col_stride)
    assert d(b.matrix(f(5, 3))) == (5, 3, 3, 1)
    assert d(b.matrix(f(5, 7)[:, :3])) == (5, 3, 7, 1)
    assert d(b.matrix(f(3, 9)[:, :5].t())) == (5, 3, 1, 9)
    assert d(b.matrix(f(1, 9).t())) in ((9, 1, 1, 1), (9, 1, 1, 9))
    assert d(b.matrix(f(5, 4)[:, 1:2])) == (5, 1, 4, 1)
    assert d(b.matrix(f(3, 9)[:, :1].t()))[:2] == (1, 3)
    t = b.tensor_list([f(59, 70)[:, :64], f(4, 5), f(6, 3)[:, :1], f(0), f(2, 3, 4)])
    got = [(x.rows, x.cols, x.row_stride) for x in t.array]
    assert got == [(59, 64, 70), (1, 20, 20), (6, 1, 3), (1, 0, 0), (1, 24, 24)]


def test_codebook_and_stepper_check_their_options():
    """On the host, without device work."""
    import numpy as np
    from gaussian_splatting_differentiable_dgs_b200 import synth
    from gaussian_splatting_differentiable_dgs_b200.codebook import ColorCodebook
    from gaussian_splatting_differentiable_dgs_b200.step import GaussianModel, Stepper
    table = np.zeros((4, 48), np.float32)
    for bad in (np.zeros(3), np.zeros((3, 1), np.int32), np.array([0, 4])):
        with pytest.raises(ValueError):
            ColorCodebook(table, bad, device="cpu")
    with pytest.raises(ValueError):
        ColorCodebook(table[0], np.zeros(3, np.int32), device="cpu")
    cb = ColorCodebook(table, np.array([0, 3, -1]), device="cpu")
    assert cb.codes.dtype == torch.int32 and (cb.rows, cb.cols) == (4, 48)
    sc, _ = synth.tiny_scene(n=4)
    model = GaussianModel(np.asarray(sc.params), sc.n, sc.sh_degree, device="cpu")
    for kw in ({"max_grad_norm": -1.0}, {"max_grad_norm": float("nan")},
               {"max_grad_norm": float("inf")}, {"codebook": cb}):
        with pytest.raises(ValueError):
            Stepper(model, device="cpu", **kw)


def test_codebook_gradient_keeps_no_workspace(b, monkeypatch):
    """Each call's workspace ends with the call: one that outlived it could be
    given up, by a later call that needs more, while its stream still reads it."""
    import weakref
    import numpy as np
    from gaussian_splatting_differentiable_dgs_b200.codebook import ColorCodebook
    cb = ColorCodebook(np.zeros((1500, 12), np.float32), np.zeros(2700, np.int64), device="cpu")
    held = []

    def bwd(g, ids, dtable, ws, **kw):
        assert ws.numel() >= b.gs_lookup_bwd_workspace_size(g, 1500) and dtable is cb.grad
        held.append(weakref.ref(ws))
        return dtable

    monkeypatch.setattr(b, "gs_lookup_bwd", bwd)
    for n in (2100, 2700, 5):
        cb.gradient(torch.empty(12, n), cand_idx=torch.zeros(n, dtype=torch.int32))
    assert [r() for r in held] == [None] * 3


def test_codebook_takes_codes_of_every_integer_type():
    """Negative codes beyond 32 bits mean "no colour" as all negative ones do;
    they do not wrap to a row."""
    import numpy as np
    from gaussian_splatting_differentiable_dgs_b200.codebook import ColorCodebook
    table = np.zeros((4, 48), np.float32)
    far = ColorCodebook(table, np.array([-2 ** 32 + 1, -2 ** 31 - 1, -2 ** 31, -2 ** 63, 3, -1]), device="cpu")
    assert (far.codes < 0).tolist() == [True, True, True, True, False, True] and int(far.codes[4]) == 3
    for dtype in (np.int8, np.int16, np.int32, np.int64, np.uint8, np.uint16, np.uint32):
        cb = ColorCodebook(table, np.array([0, 3, 2], dtype), device="cpu")
        assert cb.codes.tolist() == [0, 3, 2] and cb.codes.dtype == torch.int32
        with pytest.raises(ValueError):
            ColorCodebook(table, np.array([0, np.iinfo(dtype).max], dtype), device="cpu")
    assert ColorCodebook(table, np.array([True, False]), device="cpu").codes.tolist() == [1, 0]
    for bad in (np.array([1j, 0]), np.array([0.0])):
        with pytest.raises(ValueError):
            ColorCodebook(table, bad, device="cpu")


def test_first_use_from_two_threads(b, monkeypatch):
    """A thread that finds the torch names there (_int32 is set) finds all of
    them, at whatever line another thread is setting them."""
    import sys
    for name in ("_int32", "_float32", "_get_device", "_raw_stream"):
        monkeypatch.setattr(b, name, None)
    monkeypatch.setattr(b, "_codes", {})
    seen = []

    def at_line(frame, event, arg):
        seen.append(b._int32 is None or None not in (b._float32, b._get_device, b._raw_stream)
                    and len(b._codes) == 3)
        return at_line

    before = sys.gettrace()
    sys.settrace(lambda frame, event, arg: at_line if frame.f_code is b._torch_names.__code__ else None)
    try:
        b._torch_names()
    finally:
        sys.settrace(before)
    assert len(seen) > 4 and all(seen) and b._int32 is torch.int32


def test_clip_refuses_a_tensor_twice(b):
    """A tensor that two entries of the list write, or one reads and another
    writes, as a parameter that two layers share."""
    import random
    L, n0 = b.lib(), b.gs_launch_counter()
    T = b.gs_tensor
    piece = lambda at, size: T(at, 1, size, size, 0, 0)

    def clip(src, dst, clip):
        return L.gs_grad_clip((T * len(src))(*src), (T * len(dst))(*dst), len(src), clip, None)

    a, c, d = piece(4096, 100), piece(8192, 100), piece(16384, 100)
    rows = T(1 << 20, 4, 10, 30, 0, 0)
    A, nothing = b.GS_ERR_ARG, piece(4096, 0)
    assert clip([a, c, a], [a, c, a], 256) == A                    # in place
    assert clip([a, c], [d, d], 256) == A                          # one destination
    assert clip([a, c], [c, d], 256) == A                          # read by one, written by the other
    assert clip([d, c], [c, a], 256) == A
    assert clip([rows, a, rows], [rows, a, rows], 256) == A
    assert clip([rows, T(1 << 20, 1, 7, 7, 0, 0)], [rows, T(1 << 20, 1, 7, 7, 0, 0)], 256) == A
    for size in (17, 256, 257, 3000):
        many = [piece(1 << 30 | 4096 * k, 1000) for k in range(size)]
        random.Random(1).shuffle(many)
        assert clip(many + [many[7]], many + [many[7]], 256) == A
    # no overlap: only the empty ones get past the checks here, as nothing may launch
    assert clip([nothing, nothing], [nothing, nothing], 256) == b.GS_OK
    assert b.gs_launch_counter() == n0


def test_lookup_gradient_refuses_a_scale_that_is_not_finite(b):
    """Its product with an empty sum would put NaN into rows that no item uses.
    (A workspace of None is refused next, so that nothing launches.)"""
    L, n0, m = b.lib(), b.gs_launch_counter(), mat(b)
    call = lambda scale: L.gs_lookup_bwd(ref(m), 256, 4, None, scale, ref(m), 0, None, 0, None, None)
    for scale in (float("inf"), -float("inf"), float("nan"), 1e39):
        assert call(scale) == b.GS_ERR_ARG
    for scale in (0.0, -3e38, 1e-300):
        assert call(scale) == b.GS_ERR_CAPACITY
    assert b.gs_launch_counter() == n0
