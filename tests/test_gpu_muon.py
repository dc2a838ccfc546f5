"""GPU parity of the Muon step against its oracle, through the C ABI: the
per-element passes bit for bit, the Newton-Schulz products within what their
documented precision costs, and the whole step with AdamW on the other
parameters."""

import numpy as np
import pytest
import torch

import fully_sharded_amd as F
from oracle import fsdp_oracle as O
from oracle import muon_oracle as M
from tests.gpu_util import assert_bitexact, to_dev, to_host
from workloads.configs import ADAMW

pytestmark = pytest.mark.gpu
DEV = "cuda"
TORCH = {"bf16": torch.bfloat16, "f32": torch.float32}
ODD = [(33, 7), (5,), (3, 2, 7), (9, 1), (1, 33), (130, 66), (2,), (17, 129)]


@pytest.fixture(autouse=True)
def _gpu(request):
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    F.lib()
    print(f"[gpu] {request.node.name}", flush=True)
    yield
    torch.cuda.synchronize()
    torch.cuda.empty_cache()


def values(rng, n, sigma, dtype):
    return M.cast((rng.standard_normal(n) * sigma).astype(np.float32), dtype)


def at_offset(a, off):
    """A device copy of `a` that begins `off` elements into its allocation."""
    t = to_dev(np.concatenate([np.zeros(off, a.dtype), a]))
    return t[off:]


# --------------------------------------------------------------- momentum
@pytest.mark.parametrize("nesterov", [True, False])
@pytest.mark.parametrize("gdt,udt", [("bf16", "bf16"), ("f32", "f32"), ("bf16", "f32"),
                                     ("f32", "bf16")])
@pytest.mark.parametrize("R,layout", [(1, "flat"), (2, "per_param"), (3, "per_param"),
                                      (4, "flat"), (5, "per_param"), (8, "per_param"),
                                      (16, "flat")])
def test_momentum_bit_exact(R, layout, gdt, udt, nesterov):
    rng = np.random.default_rng(R * 8 + len(gdt) + 2 * len(udt) + nesterov)
    po = O.plan_layout(ODD, R, layout)
    params = [0, 2, 5, 7] if R != 3 else [0, 2, 3, 4, 5, 7]
    mask, place = M.chosen_mask(ODD, params), M.shard_map(po)
    grads = [values(rng, po.T, 1e-2, gdt) for _ in range(R)]
    m0 = values(rng, po.R * po.S, 1e-2, "f32")
    u0 = values(rng, po.T, 1.0, udt)
    hp = dict(F.MUON, momentum=0.9, nesterov=nesterov)
    new, u = M.momentum(M.mean(grads), m0[place], 0.9, nesterov)
    m1, u1 = m0.copy(), u0.copy()
    m1[place[mask]] = new[mask]
    u1[mask] = M.cast(u, udt)[mask]
    mu = F.Muon(F.Plan(ODD, R, layout), params)
    for off in (0, 1):       # aligned buffers, and ones off the vector grid
        m, upd = at_offset(m0, off), at_offset(u0, off)
        F.fsdp_muon_momentum(mu, hp, [at_offset(g, off) for g in grads], m, upd)
        assert_bitexact(to_host(m), m1, "m")
        assert_bitexact(to_host(upd), u1, "update")


@pytest.mark.parametrize("layout", ["per_param", "flat"])
def test_momentum_of_the_reduced_gradient(layout):
    rng = np.random.default_rng(5)
    R = 3
    plan = F.Plan(ODD, R, layout)
    mu = F.Muon(plan)
    n = plan.R * plan.S
    grads = [to_dev(values(rng, plan.T, 1e-2, "bf16")) for _ in range(R)]
    red = torch.zeros(n, device=DEV)
    F.fsdp_reduce_scatter_avg(plan, grads, red)
    m0 = torch.randn(n, device=DEV)
    got = []
    for g, rep in ((grads, True), (red, False)):
        m, u = m0.clone(), torch.zeros(plan.T, device=DEV)
        F.fsdp_muon_momentum(mu, F.MUON, g, m, u, grads_are_replicas=rep)
        got.append((to_host(m), to_host(u)))
    assert_bitexact(got[0][0], got[1][0], "m")
    assert_bitexact(got[0][1], got[1][1], "update")


# ------------------------------------------------------------------ apply
@pytest.mark.parametrize("scale", ["none", "aspect", "rms"])
@pytest.mark.parametrize("odt,pdt", [("bf16", "bf16"), ("f32", "f32"), ("bf16", "f32"),
                                     ("f32", "bf16")])
@pytest.mark.parametrize("R,layout", [(1, "per_param"), (3, "per_param"), (4, "flat"),
                                      (7, "per_param")])
def test_apply_bit_exact(R, layout, odt, pdt, scale):
    rng = np.random.default_rng(R * 8 + len(odt) + 2 * len(pdt))
    po = O.plan_layout(ODD, R, layout)
    params = [7, 0, 2, 5]
    mask, place = M.chosen_mask(ODD, params), M.shard_map(po)
    x = values(rng, po.T, 0.1, odt)
    p0 = values(rng, po.R * po.S, 0.1, "f32")
    out0 = values(rng, po.R * po.S, 1.0, pdt)
    p1, out1 = p0.copy(), out0.copy()
    for p, at, r, c in M.matrices(ODD):
        if p in params:
            w = place[at:at + r * c]
            p1[w] = M.apply(p0[w], M.widen(x[at:at + r * c]), 0.02, 0.1,
                            M.scale_of(r, c, scale))
            out1[w] = M.cast(p1[w], pdt)
    mu = F.Muon(F.Plan(ODD, R, layout), params)
    hp = dict(F.MUON, lr=0.02, weight_decay=0.1, scale=scale)
    for off in (0, 1):
        master, out = at_offset(p0, off), at_offset(out0, off)
        F.fsdp_muon_apply(mu, hp, at_offset(x, off), master, out)
        assert_bitexact(to_host(master), p1, "master")
        assert_bitexact(to_host(out), out1, "param")


# ----------------------------------------------------------- orthogonalise
def spectrum(rng, r, c, kind):
    if kind == "white":
        return rng.standard_normal((r, c))
    if kind == "low":
        return 0.1 * rng.standard_normal((r, c)) + \
            rng.standard_normal((r, 2)) @ rng.standard_normal((2, c))
    k = min(r, c)
    q, _ = np.linalg.qr(rng.standard_normal((r, k)))
    p, _ = np.linalg.qr(rng.standard_normal((c, k)))
    return (q / np.arange(1, k + 1)) @ p.T


def check(got, u, dtype, steps=5, eps=1e-7, poly=M.POLY, what=""):
    """The library's precision, imitated on the CPU, is off the definition by
    `off` (rms over the matrix): roundings at the same places, but with
    other sums, may be three times that off, a single entry (some five sigma
    of many small errors) 16 times; the result's own rounding adds half a
    step of its type at most.

    Where a matrix has few rows, `off` is no average but one draw, so what
    the last step alone can add comes on top, spread over the m rows.  It is
    X' = (a + y) X with y = b A + c A^2, 0.68 <= a + y near A = 1, A <= 1.45.
    With operands of relative error r = 2^-11 (f32: 2^-22), an entry of A
    moves y by |b + 2 c A| A r <= 4.78 * 1.45 r = 6.9 r, which is 6.9 / 0.68
    = 10 r of the result.  In fp32, b A, c A^2 and their sum add (6.9 + 4.3
    + 3) 2^-24 = 3.6 * 2^-22, which is 5.3 * 2^-22 of the result, and the
    residual's parts and a + y another 2 * 2^-22: below 18 * 2^-22 in all.

    An entry is held to its part of that at the scale of the larger of the
    rms and itself: where k of N entries hold all of a matrix (one, in a
    matrix of one entry), rms = |entry| sqrt(k / N) and a relative error e of
    those entries is an `off` of e rms, so an entry is off by e |entry| =
    (off / rms) |entry|, not by off."""
    want = M.orthogonalize(u, steps, eps, poly)
    model = M.orthogonalize_rounded(u, steps, eps, poly, split=dtype == "f32")
    rms = np.sqrt((want ** 2).mean())
    off = np.sqrt(((model - want) ** 2).mean())
    half = 2.0 ** -8 if dtype == "bf16" else 2.0 ** -24
    few = 10 * 2.0 ** -11 if dtype == "bf16" else 18 * 2.0 ** -22
    floor = few / np.sqrt(min(u.shape)) * rms
    d = M.widen(got).astype(np.float64) - want
    rel = np.sqrt((d ** 2).mean())
    print(f"[gpu]   {what} {u.shape}: off {rel / rms:.2e}, imitation {off / rms:.2e}", flush=True)
    assert rel <= half * rms + 3 * off + floor, (what, rel / rms, off / rms)
    scale = np.maximum(np.abs(want), rms) / rms
    assert (np.abs(d) <= half * np.abs(want) + (16 * off + 4 * floor) * scale).all(), what


def run_ortho(shapes, us, udt, odt, hp=None, in_place=False, off=0):
    """us: one fp32 array per parameter (1-D ones too).  Checks that nothing
    outside the matrices is written; returns the used update (fp32 values)
    and the results, per matrix."""
    plan = F.Plan(shapes, 1, "per_param")
    mu = F.Muon(plan)
    flat = M.cast(np.concatenate([u.reshape(-1) for u in us]).astype(np.float32), udt)
    update = at_offset(flat, off)
    ortho = update if in_place else torch.full((plan.T + off,), 7.0, dtype=TORCH[odt],
                                               device=DEV)[off:]
    ws = mu.workspace(TORCH[udt], TORCH[odt])
    ws.fill_(0xff)           # NaN in every type
    F.fsdp_orthogonalize(mu, hp or F.MUON, update, ortho, ws)
    got = to_host(ortho)
    if not in_place:
        assert_bitexact(to_host(update), flat, "update")
    mask = M.chosen_mask(shapes, mu.params)
    seven = M.cast(np.full(plan.T, 7.0, np.float32), odt)
    assert_bitexact(got[~mask], (flat if in_place else seven)[~mask], "outside")
    vals = M.widen(flat)
    return [(vals[at:at + r * c].reshape(r, c), got[at:at + r * c].reshape(r, c))
            for _, at, r, c in M.matrices(shapes)]


SIDES = [(1, 1), (1, 5), (5, 1), (2, 2), (63, 64), (64, 64), (65, 64), (65, 191), (100, 333),
         (333, 100), (128, 128), (129, 129), (257, 255), (40, 1025), (1025, 40), (320, 960)]


@pytest.mark.parametrize("kind", ["white", "low", "steep"])
@pytest.mark.parametrize("udt,odt", [("bf16", "bf16"), ("f32", "f32"), ("f32", "bf16"),
                                     ("bf16", "f32")])
@pytest.mark.parametrize("r,c", SIDES)
def test_one_matrix(r, c, udt, odt, kind):
    rng = np.random.default_rng(r * 1000 + c)
    (u, got), = run_ortho([(r, c)], [spectrum(rng, r, c, kind) * 1e-3], udt, odt)
    check(got, u, odt, what=kind)


@pytest.mark.parametrize("udt,odt", [("bf16", "bf16"), ("f32", "f32")])
@pytest.mark.parametrize("shapes", [[(3, 9001)], [(20000, 70)], [(130, 12345)], [(25000, 300)], [(512, 29200), (60, 200)],
                                    [(40, 300), (17,), (64, 30000), (90, 80)]])
def test_long_sums_in_parts(shapes, udt, odt):
    """A's few tiles have their sums cut into parts, beside others that do not."""
    rng = np.random.default_rng(sum(s[0] for s in shapes))
    us = [rng.standard_normal(s) for s in shapes]
    for off in (0, 1):
        for u, got in run_ortho(shapes, us, udt, odt, off=off):
            check(got, u, odt, what=f"{udt} {odt}")


@pytest.mark.parametrize("udt,odt,in_place", [("bf16", "bf16", False), ("bf16", "bf16", True),
                                              ("f32", "f32", True), ("f32", "bf16", False)])
def test_unit_of_many_matrices(udt, odt, in_place):
    rng = np.random.default_rng(11)
    shapes = [(512, 512), (33,), (512, 700), (1,), (700, 130), (3, 5, 7), (1, 9), (200, 64),
              (2, 1), (3,)]
    us = [rng.standard_normal(s) * 10.0 ** (k - 5) for k, s in enumerate(shapes)]
    for off in (0, 1):
        for k, (u, got) in enumerate(run_ortho(shapes, us, udt, odt, in_place=in_place, off=off)):
            check(got, u, odt, what=f"matrix {k}")


def test_steps_coefficients_and_eps():
    rng = np.random.default_rng(12)
    u = rng.standard_normal((96, 160)) * 1e-3
    for steps, eps, poly in ((1, 1e-7, M.POLY), (2, 1e-7, M.POLY), (3, 1e-2, M.POLY),
                             (8, 1e-7, M.POLY), (16, 1e-7, (1.5, -0.5, 0.0)),
                             (4, 1e-7, (2.0, -1.5, 0.5)), (5, 1e3, M.POLY)):
        hp = dict(F.MUON, steps=steps, eps=eps, coefficients=poly)
        for dt in ("bf16", "f32"):
            (v, got), = run_ortho([(96, 160)], [u], dt, dt, hp)
            check(got, v, dt, steps, eps, poly, what=f"{steps} steps, eps {eps}, {poly[0]}")


def test_every_magnitude():
    """The norm's square leaves fp32's range; the result does not depend on it
    while eps does not matter."""
    rng = np.random.default_rng(13)
    u = rng.standard_normal((70, 90))
    for mag in (1e-30, 1e-10, 1e10, 1e30, 2e37):
        for dt in ("bf16", "f32"):
            hp = dict(F.MUON, eps=1e-40)
            (v, got), = run_ortho([(70, 90)], [u * mag], dt, dt, hp)
            check(got, v, dt, eps=1e-40, what=f"magnitude {mag}")


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_zeros_infinities_and_nan(dt):
    """Zeros give zeros; a matrix with one infinity or NaN gives NaN
    throughout; neighbours in the unit are not touched by either."""
    rng = np.random.default_rng(14)
    shapes = [(70, 90), (64, 64), (70, 90), (90, 70), (33, 200)]
    us = [rng.standard_normal(s) for s in shapes]
    us[1][:] = 0
    us[2][3, 5] = np.inf
    us[3][80, 2] = np.nan
    out = run_ortho(shapes, us, dt, dt)
    check(out[0][1], out[0][0], dt, what="first")
    check(out[4][1], out[4][0], dt, what="last")
    assert (M.widen(out[1][1]) == 0).all()
    assert np.isnan(M.widen(out[2][1])).all() and np.isnan(M.widen(out[3][1])).all()
    # low-rank and repeated rows, a single entry
    us = [np.ones((70, 90)), np.outer(np.arange(64), np.ones(64)), np.zeros((70, 90)),
          np.eye(90, 70), np.ones((33, 200))]
    us[2][69, 89] = -3.0
    for k, (u, got) in enumerate(run_ortho(shapes, us, dt, dt)):
        check(got, u, dt, what=f"degenerate {k}")


def test_same_bits_every_time_and_on_every_stream():
    rng = np.random.default_rng(15)
    shapes = [(512, 512), (300, 1100), (1100, 300)]
    plan = F.Plan(shapes, 1, "flat")
    mu = F.Muon(plan)
    sets = []
    for k in range(3):
        u = to_dev(values(rng, plan.T, 1e-3, "bf16"))
        sets.append((u, torch.empty_like(u), mu.workspace()))
    want = []
    for u, o, ws in sets:
        F.fsdp_orthogonalize(mu, F.MUON, u, o, ws)
        want.append(to_host(o))
        o.zero_()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    for _ in range(3):
        for (u, o, ws), s in zip(sets, streams):
            F.fsdp_orthogonalize(mu, F.MUON, u, o, ws, stream=s)
    torch.cuda.synchronize()
    for (u, o, ws), w in zip(sets, want):
        assert_bitexact(to_host(o), w, "stream")
    # one workspace, one stream, one call after the other
    ws = sets[0][2]
    for u, o, _ in sets:
        o.zero_()
        F.fsdp_orthogonalize(mu, F.MUON, u, o, ws)
    for (u, o, _), w in zip(sets, want):
        assert_bitexact(to_host(o), w, "shared workspace")


# ------------------------------------------------------------- whole steps
def unit(rng, shapes, R, layout, pdt="bf16"):
    plan = F.Plan(shapes, R, layout)
    full = rng.uniform(-0.1, 0.1, plan.T).astype(np.float32)
    master = torch.empty(plan.R * plan.S, device=DEV)
    F.fsdp_shard_pack(plan, to_dev(full), master)
    param = torch.empty(plan.R * plan.S, dtype=TORCH[pdt], device=DEV)
    F.fsdp_shard_pack(plan, to_dev(full), param)
    return plan, dict(master=master, m=torch.zeros_like(master), v=torch.zeros_like(master),
                      param=param)


BLOCK = [(96, 96), (96,), (96, 260), (260, 96), (8, 3, 5), (7,)]


@pytest.mark.parametrize("R,layout,gdt,pdt", [(4, "per_param", "bf16", "bf16"),
                                              (3, "per_param", "bf16", "f32"),
                                              (8, "flat", "f32", "bf16"),
                                              (1, "flat", "bf16", "bf16"),
                                              (5, "per_param", "f32", "f32")])
def test_step_equals_its_parts_and_adamw(R, layout, gdt, pdt):
    """Three steps in one call each, the parameters gathered after each, equal
    the separate calls on the chosen matrices and AdamW's step on the others,
    bit for bit."""
    rng = np.random.default_rng(R)
    plan, a = unit(rng, BLOCK, R, layout, pdt)
    b = {k: t.clone() for k, t in a.items()}
    c = {k: t.clone() for k, t in a.items()}
    params = [0, 3, 4]
    mu = F.Muon(plan, params)
    po = O.plan_layout(BLOCK, R, layout)
    chosen = np.zeros(R * po.S, bool)
    chosen[M.shard_map(po)[M.chosen_mask(BLOCK, params)]] = True
    chosen = torch.from_numpy(chosen).to(DEV)
    ws, ws1 = mu.step_workspace(), mu.workspace()
    ws.fill_(0xff)
    update = torch.zeros(plan.T, dtype=torch.bfloat16, device=DEV)
    ortho = torch.zeros_like(update)
    recv = [torch.empty(plan.T, dtype=TORCH[pdt], device=DEV) for _ in range(R)]
    for t in range(1, 4):
        grads = [to_dev(values(rng, plan.T, 1e-3, gdt)) for _ in range(R)]
        F.fsdp_muon_shard_step(mu, F.MUON, grads, a["master"], a["m"], a["param"], ws,
                               adamw=ADAMW, step=t, v=a["v"])
        F.fsdp_muon_momentum(mu, F.MUON, grads, b["m"], update)
        F.fsdp_orthogonalize(mu, F.MUON, update, ortho, ws1)
        F.fsdp_muon_apply(mu, F.MUON, ortho, b["master"], b["param"])
        F.fsdp_adamw_shard_step(plan, ADAMW, t, grads, c["master"], c["m"], c["v"], c["param"])
        for k in ("master", "m", "v", "param"):
            want = torch.where(chosen, b[k], c[k])
            assert_bitexact(to_host(a[k]), to_host(want), f"{k}, step {t}")
        F.fsdp_gather_unflatten(plan, a["param"], recv)
        for x, s in zip(plan.unflatten(recv[R - 1]), BLOCK):
            assert x.shape == s and torch.isfinite(x).all()


def test_step_without_adamw_leaves_the_others():
    rng = np.random.default_rng(21)
    plan, a = unit(rng, BLOCK, 3, "per_param")
    mu = F.Muon(plan, [2])
    for t in a.values():
        t.copy_(torch.randn_like(t.float()))        # padding and all
    before = {k: to_host(t) for k, t in a.items()}
    po = O.plan_layout(BLOCK, 3, "per_param")
    chosen = np.zeros(3 * po.S, bool)
    chosen[M.shard_map(po)[M.chosen_mask(BLOCK, [2])]] = True
    grads = [to_dev(values(rng, plan.T, 1e-3, "bf16")) for _ in range(3)]
    F.fsdp_muon_shard_step(mu, F.MUON, grads, a["master"], a["m"], a["param"],
                           mu.step_workspace())
    assert_bitexact(to_host(a["v"]), before["v"], "v")
    for k in ("master", "m", "param"):
        got = to_host(a[k])
        assert_bitexact(got[~chosen], before[k][~chosen], k)
        assert (got[chosen] != before[k][chosen]).mean() > 0.5, k


def test_captured_and_replayed():
    """A captured step and a captured orthogonalisation of the same workspace,
    replayed with eager work between, equal eager calls on a copy."""
    rng = np.random.default_rng(22)
    plan, a = unit(rng, BLOCK, 4, "per_param")
    b = {k: t.clone() for k, t in a.items()}
    mu = F.Muon(plan)
    plan.prepare()
    mu.prepare()
    grads = [to_dev(values(rng, plan.T, 1e-3, "bf16")) for _ in range(4)]
    ws, ws2 = mu.step_workspace(), mu.step_workspace()
    u = to_dev(values(rng, plan.T, 1e-3, "bf16"))
    o, o2 = torch.zeros_like(u), torch.zeros_like(u)
    one = F.bind_muon_shard_step(mu, F.MUON, grads, a["master"], a["m"], a["param"], ws,
                                 adamw=ADAMW, v=a["v"])
    orth = F.bind_orthogonalize(mu, F.MUON, u, o, ws[:mu.workspace_bytes()[0]])
    s = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=s):
        one(1)
        orth()
    for t in range(4):
        for g in grads:                         # other gradients each time, in place
            g.copy_(to_dev(values(rng, plan.T, 1e-3, "bf16")))
        u.copy_(to_dev(values(rng, plan.T, 1e-3, "bf16")))
        graph.replay()
        torch.cuda.synchronize()
        F.fsdp_muon_shard_step(mu, F.MUON, grads, b["master"], b["m"], b["param"], ws2,
                               adamw=ADAMW, step=1, v=b["v"])
        F.fsdp_orthogonalize(mu, F.MUON, u, o2, ws2[:mu.workspace_bytes()[0]])
        for k in a:
            assert_bitexact(to_host(a[k]), to_host(b[k]), f"{k}, replay {t}")
        assert_bitexact(to_host(o), to_host(o2), f"ortho, replay {t}")


@pytest.mark.parametrize("odt", ["bf16", "f32"])
@pytest.mark.parametrize("shape", [(20000, 70), (512, 29200)])
def test_sums_in_parts_captured_and_on_two_streams(shape, odt):
    rng = np.random.default_rng(24)
    plan = F.Plan([shape], 1, "flat")
    mu = F.Muon(plan)
    mu.prepare()
    dt = TORCH[odt]
    sets = [(torch.zeros(plan.T, dtype=dt, device=DEV), torch.zeros(plan.T, dtype=dt, device=DEV),
             mu.workspace(dt, dt)) for _ in range(3)]
    graph = torch.cuda.CUDAGraph()
    s = torch.cuda.Stream()
    calls = [F.bind_orthogonalize(mu, F.MUON, *x) for x in sets]
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=s):
        calls[0]()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for t in range(3):
        u = to_dev(values(rng, plan.T, 1e-3, odt))
        for x in sets:
            x[0].copy_(u)
            x[2].fill_(0xff)
        torch.cuda.synchronize()
        graph.replay()
        for c, st in zip(calls[1:], streams):
            c(st)
        torch.cuda.synchronize()
        want = to_host(sets[1][1])
        assert np.isfinite(M.widen(want)).all()
        assert_bitexact(to_host(sets[0][1]), want, f"replay {t}")
        assert_bitexact(to_host(sets[2][1]), want, f"stream {t}")


def test_other_devices_and_bad_workspaces_are_refused():
    plan = F.Plan([(8, 8)], 1, "flat")
    mu = F.Muon(plan)
    u = torch.zeros(64, dtype=torch.bfloat16, device=DEV)
    ws = mu.workspace()
    with pytest.raises(F.FsdpError):
        F.fsdp_orthogonalize(mu, F.MUON, u, torch.zeros_like(u), ws[:-256])
    with pytest.raises(F.FsdpError):
        F.fsdp_orthogonalize(mu, F.MUON, u, torch.zeros(64, device=DEV), ws)
    with pytest.raises(ValueError):
        F.fsdp_orthogonalize(mu, F.MUON, u[:32], u[32:], ws)
    with pytest.raises(ValueError):
        F.fsdp_orthogonalize(mu, F.MUON, u.view(8, 8).t(), torch.zeros_like(u), ws)
