"""GPU parity of the AdamW step with the float64 oracle.

Bounds, in half steps e = 2^-24 of fp32: each moment is two products and a
sum (3 e of the magnitudes that enter), the square one rounding more; the
parameter takes the rounding of its decay and of the difference (2 e of its
magnitude) and the update's own: the moment's error, and about a dozen
roundings.  8-bit moments: the code and scale must be ones that a value
inside the fp32 bound gives under the element's own random bits (both are
monotone in the value); where the bound crosses no border that is exact."""
import numpy as np
import pytest
import torch

import mxfp4_block_scaled_fp4q_amd as fq
from oracle import blocks as ob
from gpu_helpers import dev

pytestmark = pytest.mark.gpu

E = ob.EPS32
HYPER = dict(lr=3e-3, beta1=0.9, beta2=0.95, eps=1e-8)


class Problem:
    """Tensors of an AdamW step in guarded flat buffers, and their float64 values."""

    def __init__(self, sizes, bits, gdt, copy, seed=0, start=True, scale=1e-3):
        rng = np.random.default_rng(seed)
        self.sizes, self.bits = sizes, bits
        self.at, n = [], 64
        for k in sizes:
            self.at.append(n)
            n += (k + 31) // 32 * 32 + 64
        self.n = n

        def flat(dtype, fill):
            return torch.full((n,), fill, dtype=dtype, device="cuda")

        def cut(t, block=1):
            return [t[a // block:a // block + (k + block - 1) // block] for a, k in zip(self.at, sizes)]
        self.p, self.g = flat(torch.float32, 7.0), flat(gdt, float("nan"))
        self.c = flat(torch.bfloat16, 5.0) if copy else None
        state = torch.float32 if bits == 32 else torch.uint8
        self.m, self.v = flat(state, 3), flat(state, 3)
        self.ms = self.vs = None
        if bits == 8:
            self.ms, self.vs = (torch.full((n // 32,), 3, dtype=torch.uint8, device="cuda") for _ in range(2))
        self.P, self.G, self.M, self.V = cut(self.p), cut(self.g), cut(self.m), cut(self.v)
        self.C = cut(self.c) if copy else None
        self.MS, self.VS = (cut(self.ms, 32), cut(self.vs, 32)) if bits == 8 else (None, None)
        for i, k in enumerate(sizes):
            self.P[i].copy_(torch.from_numpy(rng.normal(0, 0.02, k).astype(np.float32)))
            self.G[i].copy_(torch.from_numpy(rng.normal(0, scale, k).astype(np.float32)))
            if bits == 32:
                self.M[i].copy_(torch.from_numpy((rng.normal(0, scale / 3, k) * start).astype(np.float32)))
                self.V[i].copy_(torch.from_numpy((rng.normal(0, scale, k) ** 2 * start).astype(np.float32)))
            else:
                nb = (k + 31) // 32
                # any finite code, zeros among them; scales over a wide range
                m = rng.integers(0, 127, k) | (rng.integers(0, 2, k) << 7)
                self.M[i].copy_(torch.from_numpy((m * start).astype(np.uint8)))
                self.V[i].copy_(torch.from_numpy((rng.integers(0, 105, k) * start).astype(np.uint8)))
                for s in (self.MS[i], self.VS[i]):
                    s.copy_(torch.from_numpy((rng.integers(95, 112, nb) * start).astype(np.uint8)))

    def plan(self, wd):
        return fq.adamw_plan(self.P, self.G, self.M, self.V, self.MS, self.VS, copies=self.C, weight_decay=wd)

    def values(self):
        """Per tensor (p, g, m, v) in float64."""
        out = []
        for i in range(len(self.sizes)):
            p, g = (t[i].double().cpu().numpy() for t in (self.P, self.G))
            if self.bits == 32:
                m, v = (t[i].double().cpu().numpy() for t in (self.M, self.V))
            else:
                m = ob.decode8(self.M[i].cpu().numpy(), self.MS[i].cpu().numpy())
                v = ob.decode8(self.V[i].cpu().numpy(), self.VS[i].cpu().numpy()) ** 2
            out.append((p, g, m, v))
        return out

    def guards_intact(self):
        mask = np.ones(self.n, bool)
        for a, k in zip(self.at, self.sizes):
            mask[a:a + k] = False
        ok = (self.p.cpu().numpy()[mask] == 7.0).all()
        ok &= (self.m.cpu().numpy()[mask] == 3).all() and (self.v.cpu().numpy()[mask] == 3).all()
        if self.c is not None:
            ok &= (self.c.float().cpu().numpy()[mask] == 5.0).all()
        if self.bits == 8:
            mb = np.ones(self.n // 32, bool)
            for a, k in zip(self.at, self.sizes):
                mb[a // 32:a // 32 + (k + 31) // 32] = False
            ok &= (self.ms.cpu().numpy()[mb] == 3).all() and (self.vs.cpu().numpy()[mb] == 3).all()
        return bool(ok)


def check8(codes, scales, x, err, u, what):
    """Codes and scale bytes of the values x +- err under random bits u;
    returns how many codes the bound leaves open."""
    n = len(x)
    pad = -n % 32

    def blocks(a):
        return np.pad(a, (0, pad)).reshape(-1, 32)
    ax, e = np.abs(x), err
    amax = blocks(ax + e).max(1), blocks(np.maximum(ax - e, 0)).max(1)
    lo, hi = ob.e4m3_scale_byte(amax[1]), ob.e4m3_scale_byte(amax[0])
    s = scales.astype(np.int64)
    assert ((s >= lo) & (s <= hi)).all(), f"{what}: scale"
    unit = np.repeat(2.0 ** (s - 127.0), 32)[:n]
    top = 256.0  # a block on the border of two scales may hold its largest at 256 itself
    c0 = ob.sr_e4m3(np.minimum(np.maximum(ax - e, 0) / unit, top), u)
    c1 = ob.sr_e4m3(np.minimum((ax + e) / unit, top), u)
    mag = codes.astype(np.int64) & 127
    bad = ~((mag >= c0) & (mag <= c1))
    assert not bad.any(), (f"{what}: {int(bad.sum())} codes; first {int(np.argwhere(bad)[0])}: "
                           f"got {mag[bad][0]} of [{c0[bad][0]}, {c1[bad][0]}]")
    neg = (codes >> 7) == 1
    clear = ax > e
    assert (neg[clear] == (x[clear] < 0)).all(), f"{what}: sign"
    return int((c0 != c1).sum())


def step_check(prob, wd, step, seed=11, grad_scale=None):
    before = prob.values()
    wds = wd if isinstance(wd, list) else [wd] * len(prob.sizes)
    gs = None if grad_scale is None else torch.tensor(grad_scale, device="cuda")
    fq.adamw_step(prob.plan(wd), step=step, seed=seed, grad_scale=gs, **HYPER)
    torch.cuda.synchronize()
    assert prob.guards_intact(), "wrote outside its tensors"
    base, opened, total = 0, 0, 0
    b1, b2 = HYPER["beta1"], HYPER["beta2"]
    f = 1.0 if grad_scale is None else float(np.float32(grad_scale))
    for i, (p, g, m, v) in enumerate(before):
        k = prob.sizes[i]
        wp, wm, wv, parts, den = ob.adamw(p, g, m, v, step=step, wd=wds[i], grad_scale=f, **HYPER)
        what = f"tensor {i} of {len(before)} ({k} elements, {prob.bits} bits)"
        em = 5 * E * parts + 2.0 ** -149
        ev = 8 * E * wv + 2.0 ** -149
        up = np.abs(HYPER["lr"] * wm / (1 - b1 ** step) / den)
        # the root's relative error is half of v's; below the normal range the root is not that exact
        tol = 3 * E * np.abs(p) + 20 * E * up + HYPER["lr"] * em / (1 - b1 ** step) / den
        got = prob.P[i].double().cpu().numpy()
        bad = ~(np.abs(got - wp) <= tol)
        assert not bad.any(), f"{what}: param {int(bad.sum())}, first {np.argwhere(bad)[0]}"
        if prob.C is not None:
            assert torch.equal(prob.C[i], prob.P[i].bfloat16()), f"{what}: copy"
        if prob.bits == 32:
            assert (np.abs(prob.M[i].double().cpu().numpy() - wm) <= em).all(), f"{what}: exp_avg"
            assert (np.abs(prob.V[i].double().cpu().numpy() - wv) <= ev).all(), f"{what}: exp_avg_sq"
        else:
            w = ob.philox_words(base + np.arange(k), step, seed).astype(np.int64)
            r = np.sqrt(wv)
            er = 6 * E * r + 2.0 ** -74
            opened += check8(prob.M[i].cpu().numpy(), prob.MS[i].cpu().numpy(), wm, em, w & 0xFFFF,
                             what + " exp_avg")
            opened += check8(prob.V[i].cpu().numpy(), prob.VS[i].cpu().numpy(), r, er, w >> 16,
                             what + " root")
            total += 2 * k
            base += (k + 31) // 32 * 32
    if total >= 1000:  # the bound crosses a border of the 2^16 fractions rarely
        assert opened <= 0.01 * total, (opened, total)


GRADS = [torch.float32, torch.bfloat16]
LISTS = [[1], [2, 3], [31, 32, 33], [4095, 4096, 4097], [0, 5, 0, 8193], [100] * 150, [40000, 1, 7777]]


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("gdt", GRADS)
@pytest.mark.parametrize("sizes", LISTS, ids=lambda s: "x".join(map(str, s[:4])) + f"_{len(s)}")
def test_step(sizes, gdt, bits):
    step_check(Problem(sizes, bits, gdt, copy=True, seed=len(sizes)), 0.1, step=3)
    step_check(Problem(sizes, bits, gdt, copy=False, seed=5), [0.01 * (i % 3) for i in range(len(sizes))],
               step=1000)


@pytest.mark.parametrize("bits", [32, 8])
def test_first_step_from_zero_state(bits):
    step_check(Problem([300, 4100], bits, torch.float32, copy=True, start=False), 0.1, step=1)


@pytest.mark.parametrize("bits", [32, 8])
def test_grad_scale_and_small_gradients(bits):
    step_check(Problem([5000], bits, torch.bfloat16, copy=False), 0.0, step=7, grad_scale=0.37)
    step_check(Problem([5000], bits, torch.float32, copy=False, scale=1e-12), 0.1, step=2)


def test_steps_in_a_row_follow_the_oracle():
    prob = Problem([700, 33], 8, torch.float32, copy=True, start=False)
    for step in range(1, 6):
        step_check(prob, 0.1, step)
        for g in prob.G:
            g.mul_(-0.7)


def test_zero_gradients_of_a_zero_state_only_decay():
    p = torch.randn(1000, device="cuda")
    for bits in (8, 32):
        q = p.clone()
        m, v, ms, vs = fq.adamw_state(q, bits)
        scales = ([ms], [vs]) if bits == 8 else ()
        plan = fq.adamw_plan([q], [torch.zeros_like(q)], [m], [v], *scales, weight_decay=0.5)
        fq.adamw_step(plan, lr=0.1, step=1)
        assert torch.equal(q, p * np.float32(1 - 0.05)) and not m.any() and not v.any()


def test_non_finite_gradients():
    """32-bit: the element alone; 8-bit: the element's parameter, and the
    states of its block of 32 (scale byte 0xFF, zero codes)."""
    for bad in (float("inf"), float("nan")):
        for bits in (32, 8):
            prob = Problem([200], bits, torch.float32, copy=False)
            prob.G[0][40] = bad
            fq.adamw_step(prob.plan(0.1), step=2, **HYPER)
            p = torch.isnan(prob.P[0]).cpu().numpy()
            assert p.nonzero()[0].tolist() == [40]
            if bits == 8:
                for codes, s in ((prob.M[0], prob.MS[0]), (prob.V[0], prob.VS[0])):
                    s, c = s.cpu().numpy(), codes.cpu().numpy()
                    assert s[1] == 255 and not c[32:64].any() and (np.delete(s, 1) < 255).all()
                # and the block's parameters are NaN from the next step on
                prob.G[0][40] = 0.0
                fq.adamw_step(prob.plan(0.1), step=3, **HYPER)
                p = torch.isnan(prob.P[0]).cpu().numpy()
                assert p.nonzero()[0].tolist() == list(range(32, 64))


def test_stochastic_states_average_out():
    """Many steps of one gradient from zero: the 8-bit moments follow the
    32-bit ones on average over elements that share the gradient."""
    n, g0 = 32 * 2000, 1e-3
    p = [torch.zeros(n, device="cuda") for _ in range(2)]
    g = torch.full((n,), g0, device="cuda")
    s32, s8 = fq.adamw_state(p[0], 32), fq.adamw_state(p[1], 8)
    a = fq.adamw_plan([p[0]], [g], [s32[0]], [s32[1]])
    b = fq.adamw_plan([p[1]], [g], [s8[0]], [s8[1]], [s8[2]], [s8[3]])
    steps = 40
    for t in range(1, steps + 1):
        for plan in (a, b):
            fq.adamw_step(plan, lr=1e-3, beta1=0.9, beta2=0.99, step=t, seed=5)
    m = ob.decode8(s8[0].cpu().numpy(), s8[2].cpu().numpy())
    # each rounding moves a value by at most 1/8 of itself without bias; what
    # is left after 40 steps of beta 0.9 has a spread below 1/8 of the mean
    # times sqrt(1 / (1 - 0.81)), over 64000 elements
    want = float(s32[0][0])
    assert abs(m.mean() - want) < 6 * want / 8 * np.sqrt(1 / 0.19) / np.sqrt(n)
    assert m.std() > 0


def test_other_stream_and_graph_replays():
    def run(bits, how):
        prob = Problem([5000, 37, 64], bits, torch.bfloat16, copy=True)
        plan = prob.plan(0.1)
        if how == "graph":
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                fq.adamw_step(plan, step=4, **HYPER)
        for _ in range(3):
            if how == "graph":
                graph.replay()
                torch.cuda.synchronize()
                torch.randn(1000, device="cuda").sum().item()
            elif how == "stream":
                side = torch.cuda.Stream()
                side.wait_stream(torch.cuda.current_stream())
                fq.adamw_step(plan, step=4, stream=side, **HYPER)
                side.synchronize()
            else:
                fq.adamw_step(plan, step=4, **HYPER)
        torch.cuda.synchronize()
        return [t.clone() for t in (prob.p, prob.m, prob.v, prob.c)]
    for bits in (8, 32):
        want = run(bits, "plain")
        for how in ("stream", "graph"):
            assert all(torch.equal(a, b) for a, b in zip(run(bits, how), want)), (bits, how)


@pytest.mark.parametrize("gdt", GRADS)
@pytest.mark.parametrize("bits", [32, 8])
def test_table_gives_the_same_bits_as_arguments(bits, gdt):
    """One launch that reads a table, and launches of 44 tensors each."""
    sizes = [1 + (i * 977) % 9000 for i in range(97)] + [0, 3 * 4096 + 5]

    def run(table):
        prob = Problem(sizes, bits, gdt, copy=True)
        plan = prob.plan([0.1 * (i % 2) for i in range(len(sizes))])
        assert plan.table is not None and plan.chunks == sum((k + 4095) // 4096 for k in sizes)
        if not table:
            plan.table = None
        for step in (1, 2):
            fq.adamw_step(plan, step=step, seed=9, **HYPER)
        torch.cuda.synchronize()
        assert prob.guards_intact()
        return [t for t in (prob.p, prob.m, prob.v, prob.c, prob.ms, prob.vs) if t is not None]
    for a, b in zip(run(True), run(False)):
        assert torch.equal(a, b)


def test_8bit_states_are_the_formula_in_fp32_bit_for_bit():
    """Every product, sum and root of the moments is rounded once, to nearest, so
    codes and scale bytes are those of the formula in fp32: a root that is a unit
    off changes a code in some hundred thousand.  Zeros and values whose squares
    are subnormal are among them."""
    f = np.float32
    n, step, seed = (1 << 23) + 13, 40, 99
    prob = Problem([n], 8, torch.float32, False, seed=5)
    prob.V[0][: 4096].zero_()
    prob.G[0][: 2048].mul_(1e-17)
    prob.G[0][2048:3000].zero_()
    b = [t[0].cpu().numpy() for t in (prob.G, prob.M, prob.V, prob.MS, prob.VS)]
    fq.adamw_step(prob.plan(0.1), step=step, seed=seed, **HYPER)
    torch.cuda.synchronize()
    g, r = b[0], ob.decode8(b[2], b[4]).astype(f)
    a1, a2 = f(1 - HYPER["beta1"]), f(1 - HYPER["beta2"])
    m = f(HYPER["beta1"]) * ob.decode8(b[1], b[3]).astype(f) + a1 * g
    r = np.sqrt(f(HYPER["beta2"]) * (r * r) + a2 * g * g)
    assert m.dtype == r.dtype == f
    w = ob.philox_words(np.arange(n), step, seed)
    for what, x, u, codes, scales in (("m", m, w & np.uint64(0xFFFF), prob.M, prob.MS),
                                      ("r", r, w >> np.uint64(16), prob.V, prob.VS)):
        ax = np.abs(x).astype(np.float64)
        s = ob.e4m3_scale_byte(np.pad(ax, (0, -n % 32)).reshape(-1, 32).max(1))
        assert np.array_equal(scales[0].cpu().numpy(), s), f"{what}: scale bytes"
        c = ob.sr_e4m3(ax / np.repeat(2.0 ** (s - 127.0), 32)[:n], u.astype(np.int64))
        got = codes[0].cpu().numpy()
        bad = (got & 127) != c
        assert not bad.any(), f"{what}: {int(bad.sum())} codes; first at {int(np.argmax(bad))}"
        assert np.array_equal(got >> 7, np.signbit(x).astype(np.uint8)), f"{what}: signs"
