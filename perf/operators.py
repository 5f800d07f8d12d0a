"""The shared colour codebook's lookup and gradient, and the gradient norm with clipping: cases, plain forms, exact values.

Four kinds of case.  "lookup": rows of a table by an index, scaled (the SH coefficients of Gaussians that share a codebook,
or a per-view embedding).  "grad": the table's gradient, rows with the same index summed.  "clip": the global norm over many
gradient tensors and the clipped copies (the raw gradients stay, as density control reads them).  "step": the norm of a
view's gradient and the Adam update that takes the clipped gradient."""
import math

import torch

own = False

F32, F16, BF16 = "float32", "float16", "bfloat16"


def listed():
    return [
        # every Gaussian of the 6M outdoor scene decoded from a codebook of 2^16 colours, SH degree 3, into the model's planes
        _lookup("lookup_6m_sh3", n=6_000_000, rows=65_536, dim=48, table=F32, out=F32, planar=True),
        # a stored codebook in 16 bits, SH degree 2, odd sizes; a few Gaussians without a code
        _lookup("lookup_1m_sh2_bf16", n=1_000_003, rows=4099, dim=27, table=BF16, out=F32, planar=True, holes=0.02),
        # embeddings of a handful of views: latency alone
        _lookup("lookup_views", n=33, rows=1200, dim=32, table=F32, out=F32, planar=False),
        # the codebook's gradient from the candidates of one view of the 6M scene, in the compact planes of the projection backward
        _grad("grad_view_sh3", n=2_500_001, rows=65_536, dim=48, g=F32, planar=True, of=6_000_000),
        # the same on a small scene with few colours
        _grad("grad_view_sh1", n=150_000, rows=1024, dim=12, g=F32, planar=True, of=1_000_000),
        # wide 16-bit rows, an eighth of them with the same index
        _grad("grad_rows_bf16", n=262_145, rows=50_001, dim=128, g=BF16, planar=False, share=0.125),
        # the gradient of a few views' embeddings: latency alone
        _grad("grad_views", n=37, rows=100, dim=16, g=F32, planar=False),
        # the dense gradient of the 6M model at SH degree 3: one strided tensor of 59 planes
        _clip("clip_model_6m", tensors=1, size=354_000_000, planes=59, mixed=False),
        # a model's planes beside a network's tensors of three types
        _clip("clip_mixed_64", tensors=64, size=20_000_003, planes=11, mixed=True),
        # a few small tensors: latency alone
        _clip("clip_small", tensors=5, size=3001, planes=1, mixed=False),
        # one view's update with the compact gradient of its candidates
        _step("step_3m", n=3_000_000, n_cand=1_250_000, planes=59, compact=True),
        # a small model's dense gradient
        _step("step_small", n=2500, n_cand=2500, planes=23, compact=False),
    ]


def _lookup(name, n, rows, dim, table, out, planar, holes=0.0, scale=0.75):
    return {"name": name, "kind": "lookup", "n": n, "rows": rows, "dim": dim, "table": table, "out": out, "planar": planar, "holes": holes, "scale": scale}


def _grad(name, n, rows, dim, g, planar, of=0, share=0.0, holes=0.0, scale=0.75):
    return {"name": name, "kind": "grad", "n": n, "rows": rows, "dim": dim, "g": g, "planar": planar, "of": of, "share": share, "holes": holes, "scale": scale}


def _clip(name, tensors, size, planes, mixed, max_norm=1.0):
    return {"name": name, "kind": "clip", "tensors": tensors, "size": size, "planes": planes, "mixed": mixed, "max_norm": max_norm}


def _step(name, n, n_cand, planes, compact, max_norm=1.0):
    return {"name": name, "kind": "step", "n": n, "n_cand": n_cand, "planes": planes, "compact": compact, "max_norm": max_norm}


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(("lookup", "grad", "clip", "step"))
    dim = rng.choice((3, 12, 27, 48, 16, 32, 64, 128, rng.randint(1, 130)))
    if kind == "lookup":
        table = rng.choice((F32, F16, BF16))
        c = _lookup("", n=_log(rng, 1, min(6_000_000, 280_000_000 // dim)), rows=_log(rng, 1, 200_000), dim=dim, table=table,
                    out=rng.choice((F32, table)), planar=rng.random() < 0.6, holes=rng.choice((0.0, 0.02, 0.5)), scale=rng.choice((1.0, 0.75, 8.0)))
    elif kind == "grad":
        n = _log(rng, 1, min(2_500_000, 120_000_000 // dim))
        c = _grad("", n=n, rows=_log(rng, 1, 200_000), dim=dim, g=rng.choice((F32, F32, F16, BF16)), planar=rng.random() < 0.6,
                  of=rng.choice((0, n + n // 2)), share=rng.choice((0.0, 0.0, 0.1, 0.5)), holes=rng.choice((0.0, 0.02)), scale=rng.choice((1.0, 0.75, 8.0)))
    elif kind == "clip":
        k = rng.randint(1, 200)
        c = _clip("", tensors=k, size=_log(rng, 8 * k, 200_000_000), planes=rng.randint(1, 59), mixed=rng.random() < 0.5, max_norm=rng.choice((1.0, 0.1, 1e4)))
    else:
        n = _log(rng, 1, 2_500_000)
        c = _step("", n=n, n_cand=max(1, int(n * rng.uniform(0.05, 0.9))), planes=rng.choice((14, 23, 38, 59)), compact=rng.random() < 0.6, max_norm=rng.choice((1.0, 0.1, 1e4)))
    del c["name"]
    return c


def _pad(n):
    return max(64, (n + 63) // 64 * 64)


def _parts(case):
    """The element counts of a clip case's tensors: the first is a quarter of the whole in strided planes, the others differ by up to a factor of eight."""
    k, size = case["tensors"], case["size"]
    if k == 1:
        return [size]
    weights = [1 + (37 * i + 11) % 8 for i in range(k - 1)]
    return [size // 4] + [max(1, (size - size // 4) * w // sum(weights)) for w in weights]


def _types(case):
    kinds = (torch.float32, torch.bfloat16, torch.float16) if case["mixed"] else (torch.float32,)
    return [kinds[i % len(kinds)] for i in range(case["tensors"])]


def _slots(grads):
    """Where each tensor lies in the flat buffer of its type: (type, offset), each at a multiple of 64 elements."""
    ends, slots = {}, []
    for g in grads:
        at = ends.get(g.dtype, 0)
        slots.append((g.dtype, at))
        ends[g.dtype] = _pad(at + g.numel())
    return ends, slots


def _flat_sizes(grads):
    return _slots(grads)[0]


def _views(grads, flat):
    """The clipped gradients: views of one flat buffer for each type."""
    ends, slots = _slots(grads)
    by_type = dict(zip(ends, flat))
    return [by_type[t][at: at + g.numel()].view(g.shape) for g, (t, at) in zip(grads, slots)]


def _codes(n, rows, share, holes, gen):
    ids = torch.randint(rows, (n,), generator=gen, device="cuda", dtype=torch.int32)
    pick = torch.rand(n, generator=gen, device="cuda")
    ids = torch.where(pick < share, torch.full_like(ids, rows // 2), ids)
    return torch.where(pick > 1.0 - holes, torch.full_like(ids, -1), ids)


def _normal(shape, gen, sigma, dtype=torch.float32):
    return torch.randn(shape, generator=gen, device="cuda").mul_(sigma).to(dtype)


def prepare(case, seed):
    gen = torch.Generator("cuda").manual_seed(int(seed))
    s = {"case": case, "handles": {}}
    if case["kind"] == "lookup":
        n, dim, out = case["n"], case["dim"], getattr(torch, case["out"])
        s["table"] = _normal((case["rows"], dim), gen, 0.3, getattr(torch, case["table"]))
        s["ids"] = _codes(n, case["rows"], 0.0, case["holes"], gen)
        buf = torch.zeros((dim, _pad(n)) if case["planar"] else (n, dim), dtype=out, device="cuda")
        s["out"] = buf[:, :n].t() if case["planar"] else buf
    elif case["kind"] == "grad":
        n, dim, of = case["n"], case["dim"], case["of"]
        s["ids"] = _codes(max(n, of), case["rows"], case["share"], case["holes"], gen)
        # the candidates of a view: an ascending choice of the Gaussians
        s["index"] = torch.randperm(of, generator=gen, device="cuda")[:n].sort().values.to(torch.int32) if of else None
        # gradients of rows differ by orders of magnitude, as pixels do that they cover
        g = torch.randn((dim, n) if case["planar"] else (n, dim), generator=gen, device="cuda")
        size = torch.randn(n, generator=gen, device="cuda").mul_(1.5).exp_().mul_(1e-3)
        s["g"] = (g.mul_(size).t() if case["planar"] else g.mul_(size[:, None])).to(getattr(torch, case["g"]))
        s["dtable"] = torch.empty((case["rows"], dim), dtype=torch.float32, device="cuda")
    elif case["kind"] == "clip":
        sizes, types = _parts(case), _types(case)
        cols = max(1, sizes[0] // case["planes"])
        first = [_normal((case["planes"], _pad(cols)), gen, 1e-2, types[0])[:, :cols]]
        s["grads"] = first + [_normal((m,), gen, 10.0 ** (i % 4 - 4), t) for i, (m, t) in enumerate(zip(sizes[1:], types[1:]))]
        s["flat"] = [torch.zeros(m, dtype=t, device="cuda") for t, m in _flat_sizes(s["grads"]).items()]
        s["clipped"] = _views(s["grads"], s["flat"])
    else:
        n, planes, n_cand = case["n"], case["planes"], case["n_cand"]
        shape = (planes, _pad(n))
        s["params"], s["m"] = _normal(shape, gen, 1.0), _normal(shape, gen, 1e-3)
        s["v"] = _normal(shape, gen, 1e-3).square_()
        if case["compact"]:
            chosen = torch.randperm(n, generator=gen, device="cuda")[:n_cand].sort().values
            s["slot"] = torch.full((n,), -1, dtype=torch.int32, device="cuda")
            s["slot"][chosen] = torch.arange(n_cand, dtype=torch.int32, device="cuda")
            s["g"] = _normal((planes, n_cand), gen, 1e-3)
        else:
            s["slot"], s["g"] = None, _normal(shape, gen, 1e-3)
    return s


# Adam's settings and the number of the update: those of the view step
LR, BETA1, BETA2, EPS, STEP = 1e-3, 0.9, 0.999, 1e-8, 100
NORM_EPS = 1e-6


def run(s):
    kind = s["case"]["kind"]
    if own:
        return {"lookup": _own_lookup, "grad": _own_grad, "clip": _own_clip, "step": _own_step}[kind](s)
    return {"lookup": _plain_lookup, "grad": _plain_grad, "clip": _plain_clip, "step": _plain_step}[kind](s)


# ---- the framework's calls ------------------------------------------------------------------------------------------

def _own_lookup(s):
    from gaussian_splatting_differentiable_dgs_b200 import binding as B
    B.gs_lookup(s["table"], s["ids"], s["out"], scale=s["case"]["scale"])
    return s["out"]


def _own_grad(s):
    from gaussian_splatting_differentiable_dgs_b200 import binding as B
    if "ws" not in s["handles"]:  # the workspace that a training program keeps
        s["handles"]["ws"] = torch.empty(B.gs_lookup_bwd_workspace_size(s["g"], s["dtable"].shape[0]), dtype=torch.uint8, device="cuda")
    B.gs_lookup_bwd(s["g"], s["ids"], s["dtable"], s["handles"]["ws"], scale=s["case"]["scale"], index=s["index"])
    return s["dtable"]


def _own_norm_handles(B, s, grads):
    if not s["handles"]:  # the list of tensors and the workspace that a training program keeps
        tensors = B.tensor_list(grads)
        ws = torch.empty(B.gs_grad_norm_workspace_size(tensors), dtype=torch.uint8, device="cuda")
        s["handles"] = {"grads": tensors, "ws": ws, "clip": torch.empty(2, dtype=torch.float32, device="cuda")}
    return s["handles"]


def _own_clip(s):
    from gaussian_splatting_differentiable_dgs_b200 import binding as B
    h = _own_norm_handles(B, s, s["grads"])
    if "clipped" not in h:
        h["clipped"] = B.tensor_list(s["clipped"])
    B.gs_grad_norm(h["grads"], s["case"]["max_norm"], h["clip"], h["ws"], eps=NORM_EPS)
    B.gs_grad_clip(h["grads"], h["clipped"], h["clip"])
    return {"norm": h["clip"][0], "clipped": s["flat"]}


def _own_step(s):
    from gaussian_splatting_differentiable_dgs_b200 import binding as B
    n, planes, n_pad = s["case"]["n"], s["case"]["planes"], s["params"].shape[1]
    g = s["g"] if s["slot"] is not None else s["g"][:, :n]
    h = _own_norm_handles(B, s, [g])
    B.gs_grad_norm(h["grads"], s["case"]["max_norm"], h["clip"], h["ws"], eps=NORM_EPS)
    B.gs_adam_clipped(s["params"], s["m"], s["v"], s["g"], s["g"].shape[1], s["slot"], n, n_pad, planes,
                      B.gs_adam_args(LR, BETA1, BETA2, EPS, STEP, 0), h["clip"])
    return {"norm": h["clip"][0], "params": s["params"][:, :n], "m": s["m"][:, :n], "v": s["v"][:, :n]}


# ---- the plain forms ------------------------------------------------------------------------------------------------

def _plain_lookup(s):
    ids = s["ids"].long()
    if s["case"]["planar"]:
        planes = s["table"].float().t()[:, ids.clamp(min=0)] * s["case"]["scale"]
        return torch.where(ids >= 0, planes, 0.0).to(s["out"].dtype).t()
    rows = s["table"].float()[ids.clamp(min=0)] * s["case"]["scale"]
    return torch.where((ids >= 0)[:, None], rows, 0.0).to(s["out"].dtype)


def _plain_grad(s):
    c = s["case"]
    ids = s["ids"].long() if s["index"] is None else s["ids"].long()[s["index"].long()]
    ids = torch.where(ids >= 0, ids, c["rows"])[: c["n"]]  # rows without an index go to one row more, which is dropped
    # one index's sum over so many rows that 32 bits lose too much is taken in 64
    wide = torch.float64 if c["n"] * max(c["share"], 1.0 / c["rows"]) > 20_000 else torch.float32
    total = torch.zeros((c["rows"] + 1, c["dim"]), dtype=wide, device="cuda").index_add_(0, ids, s["g"].to(wide))
    return (total[: c["rows"]] * c["scale"]).float()


def _plain_norm(s, grads):
    norm = torch.stack([g.float().square().sum(dtype=torch.float64) for g in grads]).sum().sqrt()
    return norm.float(), (s["case"]["max_norm"] / (norm + NORM_EPS)).clamp(max=1.0).float()


def _plain_clip(s):
    norm, coef = _plain_norm(s, s["grads"])
    _ = [torch.mul(g.float(), coef, out=c) for g, c in zip(s["grads"], s["clipped"])]
    return {"norm": norm, "clipped": s["flat"]}


def _plain_step(s):
    n = s["case"]["n"]
    g = s["g"] if s["slot"] is not None else s["g"][:, :n]
    norm, coef = _plain_norm(s, [g])
    if s["slot"] is not None:
        g = torch.where(s["slot"] >= 0, g[:, s["slot"].clamp(min=0).long()], 0.0)
    g = g * coef
    p, m, v = s["params"][:, :n], s["m"][:, :n], s["v"][:, :n]
    m.mul_(BETA1).add_(g, alpha=1.0 - BETA1)
    v.mul_(BETA2).add_(g.square(), alpha=1.0 - BETA2)
    p.sub_(LR / (1.0 - BETA1**STEP) * m / ((v / (1.0 - BETA2**STEP)).sqrt() + EPS))
    return {"norm": norm, "params": p, "m": m, "v": v}


# ---- in 64 bits -----------------------------------------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    if case["kind"] == "lookup":
        table = torch.cat([s["table"].double(), torch.zeros((1, case["dim"]), dtype=torch.float64, device="cuda")])
        return torch.index_select(table, 0, s["ids"].remainder(case["rows"] + 1)).mul_(case["scale"])
    if case["kind"] == "grad":
        ids = s["ids"] if s["index"] is None else torch.index_select(s["ids"], 0, s["index"])
        ids = ids[: case["n"]]
        order = torch.argsort(ids)  # each index's rows behind one another, then differences of running sums over short stretches
        ids, rows, out = ids[order].long(), s["g"], torch.zeros((case["rows"], case["dim"]), dtype=torch.float64, device="cuda")
        for a in range(0, case["n"], 1 << 18):
            part = ids[a: a + (1 << 18)]
            sums = torch.cumsum(torch.index_select(rows, 0, order[a: a + (1 << 18)]).double(), 0)
            last = torch.nonzero(torch.cat([part[1:] != part[:-1], part.new_ones(1, dtype=torch.bool)])).reshape(-1)
            upto = sums[last]
            piece = upto - torch.cat([torch.zeros_like(upto[:1]), upto[:-1]])
            there = part[last] >= 0
            out[part[last][there]] += piece[there]
        return out.mul_(case["scale"])
    if case["kind"] == "clip":
        norm = math.sqrt(math.fsum(float(g.double().pow(2).sum()) for g in s["grads"]))
        coef = min(1.0, case["max_norm"] / (norm + NORM_EPS))
        flat = [torch.zeros(m, dtype=torch.float64, device="cuda") for m in _flat_sizes(s["grads"]).values()]
        for view, g in zip(_views(s["grads"], flat), s["grads"]):
            view[...] = g.double() * coef
        return {"norm": torch.tensor(norm, dtype=torch.float64), "clipped": flat}
    n = case["n"]
    g = s["g"][:, : case["n_cand"]] if case["compact"] else s["g"][:, :n]
    norm = math.sqrt(math.fsum(float(row.double().pow(2).sum()) for row in g))
    g = g.double() * min(1.0, case["max_norm"] / (norm + NORM_EPS))
    if case["compact"]:
        full = torch.zeros((case["planes"], n), dtype=torch.float64, device="cuda")
        full[:, torch.nonzero(s["slot"] >= 0).reshape(-1)] = g
        g = full
    m = BETA1 * s["m"][:, :n].double() + (1.0 - BETA1) * g
    v = BETA2 * s["v"][:, :n].double() + (1.0 - BETA2) * g * g
    p = s["params"][:, :n].double() - LR * (m / (1.0 - BETA1**STEP)) / (torch.sqrt(v / (1.0 - BETA2**STEP)) + EPS)
    return {"norm": torch.tensor(norm, dtype=torch.float64), "params": p, "m": m, "v": v}


def work(case):
    size = {F32: 4, F16: 2, BF16: 2}
    if case["kind"] == "lookup":
        n, dim = case["n"], case["dim"]
        return {"bytes": 4 * n + min(n, case["rows"]) * dim * size[case["table"]] + n * dim * size[case["out"]], "flops": n * dim}
    if case["kind"] == "grad":
        n, dim = case["n"], case["dim"]
        return {"bytes": (8 if case["of"] else 4) * n + n * dim * size[case["g"]] + 4 * case["rows"] * dim, "flops": n * dim}
    if case["kind"] == "clip":
        sizes = _parts(case)
        sizes[0] = max(1, sizes[0] // case["planes"]) * case["planes"]
        return {"bytes": sum(2 * m * t.itemsize for m, t in zip(sizes, _types(case))), "flops": 3 * sum(sizes)}
    n, planes, n_cand = case["n"], case["planes"], case["n_cand"] if case["compact"] else case["n"]
    return {"bytes": 24 * planes * n + 4 * planes * n_cand + (4 * n if case["compact"] else 0), "flops": planes * (2 * n_cand + 14 * n)}
