"""Host-side checks of the Muon calls (no GPU): the choice of parameters, the
work items, the workspace's size, and every entry point's refusals, which come
before any device call."""

import ctypes

import numpy as np
import pytest
import torch

import fully_sharded_amd as F
from fully_sharded_amd import binding as B
from oracle import fsdp_oracle as O
from oracle import muon_oracle as M
from workloads.configs import ADAMW

SHAPES = [(6, 4), (5,), (3, 2, 7), (9, 1), (1, 33)]
BASE = 1 << 40   # an address that is never touched: every call here is refused


def handle(plan, params):
    h = ctypes.c_void_p()
    arr = (ctypes.c_int32 * max(1, len(params)))(*params)
    return B.lib().fsdp_muon_plan(plan.handle, len(params), arr, ctypes.byref(h)), h


def test_choice_of_parameters():
    plan = F.Plan(SHAPES, 3, "per_param")
    assert F.Muon(plan).params == [0, 2, 3, 4]
    assert F.Muon(plan, [3, 0]).params == [3, 0]
    for bad in ([], [1], [0, 0], [5], [-1], [0, 1]):
        st, h = handle(plan, bad)
        assert st == -1 and not h.value, bad
    assert B.lib().fsdp_muon_plan(None, 1, (ctypes.c_int32 * 1)(0),
                                  ctypes.byref(ctypes.c_void_p())) == -1
    assert B.lib().fsdp_muon_plan(plan.handle, 1, (ctypes.c_int32 * 1)(0), None) == -1
    st, h = handle(F.Plan([((1 << 30) + 1, 1), (2, 2)], 1, "flat"), [0])
    assert st == -2 and not h.value
    B.lib().fsdp_muon_destroy(None)


def test_plan_may_go_first():
    plan = F.Plan(SHAPES, 2, "flat")
    st, h = handle(plan, [0, 2])
    assert st == 0
    del plan
    n = ctypes.c_int64()
    assert B.lib().fsdp_muon_work_items(h, 0, None, 0, ctypes.byref(n)) == 0 and n.value >= 2
    B.lib().fsdp_muon_destroy(h)


@pytest.mark.parametrize("layout", ["per_param", "flat"])
@pytest.mark.parametrize("R", [1, 2, 3, 8, 13])
def test_work_items_cover_the_chosen_elements_once(R, layout):
    rng = np.random.default_rng(R)
    for shapes, params in [(SHAPES, [0, 2, 3, 4]), (SHAPES, [4, 2]),
                           ([(40, 90), (7,), (1, 3000), (33, 3, 3), (2,)], [3, 0])] + [
            ([(int(rng.integers(1, 60)), int(rng.integers(1, 90))) for _ in range(5)], [1, 3])]:
        po = O.plan_layout(shapes, R, layout)
        place = M.shard_map(po)
        mask = M.chosen_mask(shapes, params)
        mu = F.Muon(F.Plan(shapes, R, layout), params)
        for space in (0, 1):
            got = np.full(po.T, -1, np.int64)
            ends = -1
            for dst, src, n in mu.work_items(space):
                assert 0 < n <= 1024 and dst // 1024 == (dst + n - 1) // 1024 and dst > ends
                ends = dst + n - 1
                flat, shard = (src, dst) if space == 0 else (dst, src)
                assert (got[flat:flat + n] == -1).all()
                got[flat:flat + n] = shard + np.arange(n)
            assert np.array_equal(got[mask], place[mask]) and (got[~mask] == -1).all()


def test_work_items_refusals():
    mu = F.Muon(F.Plan(SHAPES, 2, "flat"))
    L, n = B.lib(), ctypes.c_int64()
    buf = (ctypes.c_int64 * 3)()
    assert L.fsdp_muon_work_items(None, 0, None, 0, ctypes.byref(n)) == -1
    assert L.fsdp_muon_work_items(mu.handle, 2, None, 0, ctypes.byref(n)) == -1
    assert L.fsdp_muon_work_items(mu.handle, 0, None, 0, None) == -1
    assert L.fsdp_muon_work_items(mu.handle, 0, buf, 0, ctypes.byref(n)) == -1


def test_workspace_sizes():
    shapes = [(512, 512), (7,), (100, 700)]
    mu = F.Muon(F.Plan(shapes, 4, "per_param"))
    one, step = mu.workspace_bytes()
    f32, step2 = mu.workspace_bytes(torch.float32, torch.float32)
    assert one % 256 == 0 and step % 256 == 0 and f32 > one and step == step2
    assert step - one >= 2 * mu.plan.T
    L = B.lib()
    assert L.fsdp_muon_workspace(mu.handle, 7, 1, None, None) == -1
    assert L.fsdp_muon_workspace(mu.handle, 1, 7, None, None) == -1
    assert L.fsdp_muon_workspace(None, 1, 1, None, None) == -1
    assert L.fsdp_muon_workspace(mu.handle, 1, 1, None, None) == 0


def hparams(**over):
    d = dict(F.MUON, **over)
    a, b, c = d["coefficients"]
    scale = d["scale"] if isinstance(d["scale"], int) else {"none": 0, "aspect": 1,
                                                            "rms": 2}[d["scale"]]
    return B.MuonHParams(d["lr"], d["momentum"], d["weight_decay"], d["eps"], a, b, c,
                         d["steps"], int(d["nesterov"]), scale)


class Calls:
    """The four entry points with addresses that lie 256 MiB apart; `over`
    replaces arguments."""

    def __init__(self, R=2, layout="per_param"):
        self.plan = F.Plan(SHAPES, R, layout)
        self.mu = F.Muon(self.plan)
        self.ws, self.step_ws = self.mu.workspace_bytes()

    @staticmethod
    def at(k):
        return BASE + (k << 28)

    def grads(self, over):
        arr = (ctypes.c_void_p * self.plan.R)(*[self.at(20 + q) for q in range(self.plan.R)])
        for q, p in over.items():
            arr[q] = p
        return arr

    def momentum(self, hp=None, g=None, gdt=1, rep=1, m=None, u=None, udt=1, mu=True):
        return B.lib().fsdp_muon_momentum(
            self.mu.handle if mu else None, ctypes.byref(hp or hparams()),
            self.grads(g or {}), gdt, rep, self.at(1) if m is None else m,
            self.at(2) if u is None else u, udt, None)

    def ortho(self, hp=None, u=None, udt=1, o=None, odt=1, w=None, n=None, mu=True):
        return B.lib().fsdp_orthogonalize(
            self.mu.handle if mu else None, ctypes.byref(hp or hparams()),
            self.at(1) if u is None else u, udt, self.at(2) if o is None else o, odt,
            self.at(3) if w is None else w, self.ws if n is None else n, None)

    def apply(self, hp=None, o=None, odt=1, p=None, out=None, pdt=1, mu=True):
        return B.lib().fsdp_muon_apply(
            self.mu.handle if mu else None, ctypes.byref(hp or hparams()),
            self.at(1) if o is None else o, odt, self.at(2) if p is None else p,
            self.at(3) if out is None else out, pdt, None)

    def step(self, hp=None, adamw=True, t=1, g=None, gdt=1, p=None, m=None, v=None, out=None,
             pdt=1, w=None, n=None, mu=True):
        a = B.AdamWHParams(*[ADAMW[k] for k in ("lr", "beta1", "beta2", "eps", "weight_decay")])
        if isinstance(adamw, B.AdamWHParams):
            a = adamw
        return B.lib().fsdp_muon_shard_step(
            self.mu.handle if mu else None, ctypes.byref(hp or hparams()),
            ctypes.byref(a) if adamw else None, t, self.grads(g or {}), gdt,
            self.at(1) if p is None else p, self.at(2) if m is None else m,
            self.at(3) if v is None else v, self.at(4) if out is None else out, pdt,
            self.at(5) if w is None else w, self.step_ws if n is None else n, None)


BAD_HP = [dict(lr=-1.0), dict(lr=float("nan")), dict(momentum=1.0), dict(momentum=-0.1),
          dict(weight_decay=-1.0), dict(eps=0.0), dict(eps=1e-301), dict(eps=float("inf")),
          dict(coefficients=(17.0, 0.0, 0.0)), dict(coefficients=(1.0, float("nan"), 0.0)),
          dict(coefficients=(1.0, 0.0, -16.5)), dict(steps=0), dict(steps=17),
          dict(scale=3), dict(scale=-1)]


@pytest.mark.parametrize("bad", BAD_HP)
def test_hyper_parameters_are_checked(bad):
    c, h = Calls(), hparams(**bad)
    assert c.momentum(hp=h) == c.ortho(hp=h) == c.apply(hp=h) == c.step(hp=h) == -1


def test_nesterov_flag_is_checked():
    c, h = Calls(), hparams()
    h.nesterov = 2
    assert c.momentum(hp=h) == c.step(hp=h) == -1


def test_momentum_refusals():
    c = Calls()
    at = c.at
    T, n = c.plan.T, c.plan.R * c.plan.S
    assert c.momentum(mu=False) == -1
    for over in (dict(gdt=2), dict(udt=-1), dict(rep=2), dict(rep=0, gdt=1), dict(m=0),
                 dict(u=0), dict(g={1: 0}), dict(m=at(1) + 2), dict(u=at(2) + 1),
                 dict(g={0: at(20) + 1}),
                 dict(u=at(1)),                     # on the momentum
                 dict(u=at(1) + 4 * n - 2),         # on its last element
                 dict(u=at(20)), dict(m=at(21)),    # on a gradient
                 dict(m=at(20) + (2 * T - 1) // 4 * 4)):
        assert c.momentum(**over) == -1, over


def test_orthogonalize_refusals():
    c = Calls()
    at, T = c.at, c.plan.T
    assert c.ortho(mu=False) == -1
    for over in (dict(udt=2), dict(odt=5), dict(u=0), dict(o=0), dict(w=0), dict(n=c.ws - 1),
                 dict(n=0), dict(n=-1), dict(w=at(3) + 128), dict(u=at(1) + 1),
                 dict(o=at(2) + 1), dict(odt=0, o=at(2) + 2),
                 dict(odt=0),                       # the workspace for bf16 results is too small
                 dict(o=at(1), odt=0, n=1 << 27),   # in place, another type
                 dict(o=at(1) + 2), dict(o=at(1) + 2 * T - 2),
                 dict(u=at(3)), dict(o=at(3) + c.ws - 2)):
        assert c.ortho(**over) == -1, over


def test_apply_refusals():
    c = Calls()
    at, T, n = c.at, c.plan.T, c.plan.R * c.plan.S
    assert c.apply(mu=False) == -1
    for over in (dict(odt=2), dict(pdt=2), dict(o=0), dict(p=0), dict(out=0), dict(o=at(1) + 1),
                 dict(p=at(2) + 2), dict(out=at(3) + 1), dict(p=at(1)), dict(out=at(1)),
                 dict(out=at(2) + 4 * n - 2), dict(o=at(3) + 2 * n - 2)):
        assert c.apply(**over) == -1, over


def test_step_refusals():
    c = Calls()
    at, n = c.at, c.plan.R * c.plan.S
    bad_adam = B.AdamWHParams(1e-3, 1.0, 0.999, 1e-8, 0.0)
    assert c.step(mu=False) == -1
    for over in (dict(t=0), dict(adamw=bad_adam), dict(v=0), dict(p=0), dict(m=0), dict(out=0),
                 dict(w=0), dict(gdt=3), dict(pdt=3), dict(g={0: 0}), dict(n=c.step_ws - 1),
                 dict(w=at(5) + 64), dict(m=at(1)), dict(v=at(2) + 4 * n - 4), dict(out=at(3)),
                 dict(w=at(4)), dict(w=at(20)), dict(p=at(21)), dict(adamw=False, m=at(1)),
                 dict(p=at(1) + 1), dict(v=at(3) + 2)):
        assert c.step(**over) == -1, over


def test_binding_refuses_before_the_library():
    plan = F.Plan(SHAPES, 2, "per_param")
    mu = F.Muon(plan)
    T, n = plan.T, plan.R * plan.S
    g = [torch.zeros(T, dtype=torch.bfloat16) for _ in range(2)]
    bf = torch.zeros(T, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="GPU tensor"):
        F.fsdp_muon_momentum(mu, F.MUON, g, torch.zeros(n), bf)
    with pytest.raises(ValueError, match="GPU tensor"):
        F.fsdp_orthogonalize(mu, F.MUON, bf, bf, torch.zeros(1 << 20, dtype=torch.uint8))
    with pytest.raises(ValueError, match="GPU tensor"):
        F.fsdp_muon_apply(mu, F.MUON, bf, torch.zeros(n), torch.zeros(n))
    with pytest.raises(ValueError, match="replicas"):
        F.bind_muon_momentum(mu, F.MUON, g[:1], torch.zeros(n), bf)
    with pytest.raises(ValueError):
        F.bind_muon_momentum(mu, F.MUON, [g[0], g[1].float()], torch.zeros(n), bf)
    with pytest.raises(TypeError):
        F.bind_muon_momentum(mu, F.MUON, [x.half() for x in g], torch.zeros(n), bf)
    with pytest.raises(ValueError):
        F.bind_muon_momentum(mu, F.MUON, torch.zeros(n - 1), torch.zeros(n), bf,
                             grads_are_replicas=False)
    with pytest.raises(ValueError, match="scale"):
        F.bind_muon_apply(mu, dict(F.MUON, scale="l2"), bf, torch.zeros(n), torch.zeros(n))
    with pytest.raises(ValueError):
        F.bind_orthogonalize(mu, F.MUON, bf, bf, torch.zeros(1 << 20))
    with pytest.raises(ValueError, match="AdamW"):
        F.bind_muon_shard_step(mu, F.MUON, g, torch.zeros(n), torch.zeros(n), torch.zeros(n),
                               torch.zeros(1 << 20, dtype=torch.uint8), adamw=ADAMW)


def test_oracle_polynomial_on_singular_values():
    """The oracle against the definition by singular values."""
    rng = np.random.default_rng(3)
    for r, c in ((5, 9), (9, 5), (1, 4), (6, 6)):
        u = rng.standard_normal((r, c))
        p, s, q = np.linalg.svd(u / (np.linalg.norm(u) + 1e-7), full_matrices=False)
        for _ in range(5):
            s = M.POLY[0] * s + M.POLY[1] * s ** 3 + M.POLY[2] * s ** 5
        # each step multiplies relative errors by at most a few: 5 steps of
        # float64 products of sides below 10
        np.testing.assert_allclose(M.orthogonalize(u), (p * s) @ q, rtol=0, atol=1e-11)
