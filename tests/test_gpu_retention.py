"""The retention operators on the GPU against the 64-bit reference.

Tolerances, as relative L2 errors.  fp32 tensors and fp32 states: a value is a sum of
at most L * headdim (< 2^17) products; with rounding 2^-24 an operation and errors that
add like a random walk that is below 2^-24 * 2^8.5 = 2.2e-5, and sums are blocked, so
2e-5 (F32).  bf16 outputs: the output, the products inside a block and the state as an
operand are each rounded once to bf16 (at most 2^-9 relative each): 2^-9 * sqrt(3) =
3.4e-3, so 4e-3 (BF16).  States of bf16 inputs keep fp32 precision: F32."""
from __future__ import annotations

import pytest
import torch

import mamba2_ssd_selective_gb300 as ssd
from tests import retention_ref as ref

pytestmark = pytest.mark.gpu

F32, BF16 = 2e-5, 4e-3
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from mamba2_ssd_selective_gb300.build import build

    build()
    ssd.load()


def close(got, want, tol, what=""):
    got, want = got.detach().double().cpu(), want.double()
    assert got.shape == want.shape, what
    assert torch.isfinite(got).all(), what
    err = (got - want).norm() / want.norm().clamp(min=1e-30)
    assert err <= tol, f"{what}: {err:.2e} > {tol:.2e}"


def rounded(want, dtype):
    """Tolerance of an output that is rounded once: 2^-9 for bf16, or the error of the 64-bit result itself rounded to
    bf16 where that is more (a norm that hangs on few values: up to 2^-8), with 1% for roundings that fp32 turns."""
    if dtype == "f32":
        return F32
    want = want.double()
    return max(2 ** -9, 1.01 * float((want.bfloat16().double() - want).norm() / want.norm().clamp(min=1e-30)))


class Case:
    """Random inputs of one shape: q, k, v are views of one projection output."""

    def __init__(self, lens, H, K, dk, dv, dtype="bf16", packed=True, seed=0, decay=None):
        g = torch.Generator().manual_seed(seed)
        R = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
        self.lens, self.H, self.K, self.dk, self.dv, self.dtype, self.packed = lens, H, K, dk, dv, dtype, packed
        self.T, self.n = sum(lens), len(lens)
        tt = TYPES[dtype]
        self.qkv = R(self.T, (H + K) * dk + K * dv).to(tt)
        self.do = R(self.T, H * dv).to(tt)
        self.init, self.dfin = R(self.n, H, dk, dv), R(self.n, H, dk, dv)
        self.decay = torch.log1p(-torch.exp2(-1 - 9 * torch.rand(H, generator=g))) if decay is None else decay
        self.cu = torch.tensor([0] + lens).cumsum(0).to(torch.int32)
        self.scale = dk ** -0.5

    def parts(self, dev):
        return self.qkv.to(dev).split([self.H * self.dk, self.K * self.dk, self.K * self.dv], dim=1)

    def runner(self):
        return ssd.LinearAttnRunner(self.n, self.T if self.packed else self.lens[0], self.H, self.dk, self.dv,
                                    nheads_kv=self.K, dtype=self.dtype, packed=self.packed)

    def gpu(self, init=True, backward=True, runner=None):
        r = runner or self.runner()
        q, k, v = self.parts("cuda")
        cu = self.cu.cuda() if self.packed else None
        s0 = self.init.cuda() if init else None
        decay = self.decay.cuda()
        o, fin = r.forward(q, k, v, decay, initial_state=s0, cu_seqlens=cu)
        g = {}
        if backward:
            g = r.backward(q, k, v, decay, self.do.cuda(), initial_state=s0,
                           dfinal_state=self.dfin.cuda() if init else None, cu_seqlens=cu)
        torch.cuda.synchronize()
        assert ssd.ssd_device_status(r.workspace) == 0
        return o, fin, g

    def ref(self, init=True):
        q, k, v = (x.reshape(self.T, -1, d) for x, d in zip(self.parts("cpu"), (self.dk, self.dk, self.dv)))
        return ref.linear_attn(q, k, v, self.decay, self.scale, self.lens, self.init if init else None,
                               self.do.view(self.T, self.H, self.dv), self.dfin if init else None)

    def check(self, init=True):
        o, fin, g = self.gpu(init)
        ro, rfin, rdq, rdk, rdv, rdinit = self.ref(init)
        tol = BF16 if self.dtype == "bf16" else F32
        flat = lambda x: x.reshape(self.T, -1)  # noqa: E731
        close(o, flat(ro), tol, "o")
        close(fin, rfin, F32, "final state")
        close(g["dq"], flat(rdq), tol, "dq")
        close(g["dk"], flat(rdk), tol, "dk")
        close(g["dv"], flat(rdv), tol, "dv")
        if init:
            close(g["dinitial_state"], rdinit, F32, "dinitial_state")
        else:
            assert g["dinitial_state"] is None


# ------------------------------------------------------------------ linear attention

@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("L", [1, 2, 31, 32, 33, 63, 64, 65, 128, 200])
def test_lengths(L, dtype):
    Case([L, L], 2, 2, 64, 64, dtype, packed=False, seed=L).check(init=L % 2 == 0)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dk,dv", [(8, 8), (128, 128), (64, 128), (128, 64), (72, 40), (96, 120), (136, 64), (64, 256),
                                   (256, 200)])
def test_widths(dk, dv, dtype):
    Case([70, 129], 2, 1, dk, dv, dtype, seed=dk + dv).check()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("H,K", [(1, 1), (6, 6), (6, 3), (8, 1)])
def test_shared_heads(H, K, dtype):
    Case([100, 37], H, K, 64, 64, dtype, seed=H).check()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("lens", [[0, 1, 0, 64, 65, 0], [1] * 40, [0, 0, 5], [300, 1, 129, 0, 63]])
def test_packed_sequences(lens, dtype):
    Case(lens, 2, 2, 64, 64, dtype, seed=len(lens)).check()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("lens,packed", [([1500], False), ([700, 700], False), ([3, 1400, 0, 257], True),
                                         ([5000], False), ([3, 8000, 0, 257], True)])
def test_sequences_cut_into_segments(lens, packed, dtype):
    c = Case(lens, 2, 2, 64, 72, dtype, packed=packed, seed=11)
    if max(lens) > 4000:  # a shorter one is cut only where that pays
        # the segments' states are in the workspace, so that this case takes the path it is meant for
        assert ssd.ssd_linear_attn_workspace_size(c.runner().dims, False) > 2 * 2 * 64 * 72 * 4
    c.check()
    c.check(init=False)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_strong_and_absent_decay(dtype):
    decay = torch.tensor([0.0, -float("inf"), -30.0, -1.0, -1e-4])
    Case([150], 5, 5, 64, 64, dtype, seed=5, decay=decay).check()
    # cut into segments
    Case([900], 5, 5, 8, 8, dtype, seed=6, decay=decay).check()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_decays_about_the_reach_of_inverse_powers(dtype):
    """lam^64 about 2^-40, where the tensor-core path changes how it weighs scores, and on both sides of it."""
    decay = torch.tensor([-0.2, -0.43, -0.4332, -0.4333, -0.44, -0.8])
    Case([200, 64, 7], 6, 2, 64, 64, dtype, seed=31, decay=decay).check()
    Case([129], 6, 6, 128, 128, dtype, seed=32, decay=decay).check()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_other_sequences_do_not_see_nan(dtype):
    lens = [33, 40, 70]
    c = Case(lens, 2, 2, 64, 64, dtype, seed=8)
    clean = c.gpu()
    c.qkv[33:73] = float("nan")
    c.do[33:73] = float("inf")
    o, fin, g = c.gpu()
    for got, want in ((o, clean[0]), (g["dq"], clean[2]["dq"]), (g["dk"], clean[2]["dk"]), (g["dv"], clean[2]["dv"])):
        assert torch.equal(got[:33], want[:33]) and torch.equal(got[73:], want[73:])
    for got, want in ((fin, clean[1]), (g["dinitial_state"], clean[2]["dinitial_state"])):
        assert torch.equal(got[0], want[0]) and torch.equal(got[2], want[2])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_repeats_give_equal_bits(dtype):
    c = Case([500, 3, 400], 6, 2, 64, 64, dtype, seed=9)
    a, b = c.gpu(), c.gpu()
    for x, y in zip([a[0], a[1], *a[2].values()], [b[0], b[1], *b[2].values()]):
        assert torch.equal(x, y)


def test_rows_outside_every_sequence_are_not_written():
    c = Case([40, 30], 2, 2, 64, 64, seed=4)
    r = c.runner()
    q, k, v = c.parts("cuda")
    cu = torch.tensor([5, 40, 60], dtype=torch.int32, device="cuda")  # rows 0-4 and 60-69 belong to none
    out = torch.full((70, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    o, fin = r.forward(q, k, v, c.decay.cuda(), cu_seqlens=cu, out=out)
    assert (o[:5] == 7).all() and (o[60:] == 7).all() and (o[5:60] != 7).any()
    # bounds outside the rows are clamped
    bad = torch.tensor([-100, 1 << 30, -5], dtype=torch.int32, device="cuda")
    r.forward(q, k, v, c.decay.cuda(), cu_seqlens=bad, out=out)
    torch.cuda.synchronize()


def test_batched_layout_and_output_stride():
    c = Case([90, 90, 90], 4, 2, 64, 64, packed=False, seed=2)
    q, k, v = (x.view(3, 90, -1) for x in c.qkv.cuda().view(3, 90, -1).split([256, 128, 128], dim=2))
    buf = torch.zeros(3, 90, 512, dtype=torch.bfloat16, device="cuda")
    o, _ = c.runner().forward(q, k, v, c.decay.cuda(), out=buf[:, :, 128:384], final_state=False)
    want = c.ref(init=False)[0].reshape(270, 256)
    close(buf[:, :, 128:384].reshape(270, 256), want, BF16)
    assert (buf[:, :, :128] == 0).all() and (buf[:, :, 384:] == 0).all()


@pytest.mark.parametrize("dtype", ["f32"])
def test_gradients_against_differences(dtype):
    """The pass is linear in q, k, v and the initial state, each alone, so a difference over a whole direction is
    exact up to rounding: F32 relative to the root of the summed squares of the loss's terms."""
    c = Case([130, 70], 4, 2, 40, 64, dtype, seed=21)
    r = c.runner()
    cu, decay, do, dfin = c.cu.cuda(), c.decay.cuda(), c.do.cuda(), c.dfin.cuda()
    x = [t.contiguous() for t in c.parts("cuda")] + [c.init.cuda()]
    g = r.backward(*x[:3], decay, do, initial_state=x[3], dfinal_state=dfin, cu_seqlens=cu)
    gen = torch.Generator(device="cuda").manual_seed(1)
    for i, name in enumerate(("dq", "dk", "dv", "dinitial_state")):
        e = torch.randn(x[i].shape, generator=gen, device="cuda")

        def loss(sign):
            a = list(x)
            a[i] = x[i] + sign * e
            o, fin = r.forward(*a[:3], decay, initial_state=a[3], cu_seqlens=cu)
            terms = torch.cat([(o.double() * do).flatten(), (fin.double() * dfin).flatten()])
            return terms.sum(), terms.norm()

        (lp, norm), (lm, _) = loss(1), loss(-1)
        want = (g[name].double() * e).sum()
        assert abs((lp - lm) / 2 - want) <= F32 * norm, name


def test_side_stream_and_graph():
    c = Case([200], 4, 4, 64, 64, packed=False, seed=13)
    r = c.runner()
    q, k, v = c.parts("cuda")
    decay = c.decay.cuda()
    want, fin = r.forward(q, k, v, decay)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got, gfin = r.forward(q, k, v, decay)
    side.synchronize()
    assert torch.equal(got, want) and torch.equal(gfin, fin)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got, gfin = r.forward(q, k, v, decay)
    got.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(got, want) and torch.equal(gfin, fin)


# ------------------------------------------------------------------ single tokens

@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dk,dv,H,K", [(64, 64, 4, 4), (128, 128, 6, 2), (8, 40, 1, 1), (256, 256, 2, 1),
                                       (72, 200, 3, 3)])
def test_steps_continue_a_prompt(dk, dv, H, K, dtype):
    """A prompt, then its next tokens one at a time, give what one longer prompt gives."""
    rows, L, more = 3, 20, 5
    c = Case([L + more] * rows, H, K, dk, dv, dtype, packed=False, seed=dk)
    ro, rfin = c.ref(init=False)[:2]
    ro = ro.view(rows, L + more, -1)
    x = [t.reshape(rows, L + more, -1) for t in c.parts("cuda")]
    decay = c.decay.cuda()
    prompt = ssd.LinearAttnRunner(rows, L, H, dk, dv, nheads_kv=K, dtype=dtype)
    tok = ssd.LinearAttnRunner(rows, 1, H, dk, dv, nheads_kv=K, dtype=dtype)
    _, fin = prompt.forward(*(t[:, :L].reshape(rows * L, -1) for t in x), decay)
    cache = torch.full((7, H, dk, dv), 3.0, device="cuda")
    slots = torch.tensor([5, 0, 2], dtype=torch.int32, device="cuda")
    cache[slots.long()] = fin
    tol = BF16 if dtype == "bf16" else F32
    for t in range(L, L + more):
        o = tok.step(*(y[:, t] for y in x), decay, cache, slot_idx=slots)
        close(o, ro[:, t], tol, f"token {t}")
    close(cache[slots.long()], rfin, F32, "state")
    assert (cache[[1, 3, 4, 6]] == 3).all()


def test_step_rows_without_a_slot():
    c = Case([1, 1, 1, 1], 2, 2, 64, 64, packed=False, seed=3)
    cache = torch.randn(3, 2, 64, 64, device="cuda")
    before = cache.clone()
    slots = torch.tensor([-1, 2, 3, 1], dtype=torch.int32, device="cuda")  # 3 is past the cache
    o = c.runner().step(*c.parts("cuda"), c.decay.cuda(), cache, slot_idx=slots)
    assert (o[0] == 0).all() and (o[2] == 0).all() and (o[1] != 0).any()
    assert torch.equal(cache[0], before[0]) and not torch.equal(cache[2], before[2])


# ------------------------------------------------------------------ group norm

def gn_case(n, m, C, G, act, dtype, seed=0, affine=True, shift=0.5):
    g = torch.Generator().manual_seed(seed)
    tt = TYPES[dtype]
    R = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    x, dy = (R(n, m, C) * 1.5 + shift).to(tt), R(n, m, C).to(tt)
    w, b = (R(C) * 0.3 + 1, R(C) * 0.3) if affine else (None, None)
    z = R(n, m, C).to(tt) if act == "gate" else None
    return x, dy, w, b, z


def gn_check(n, m, C, G, act, dtype, seed=0, affine=True, shift=0.5):
    x, dy, w, b, z = gn_case(n, m, C, G, act, dtype, seed, affine, shift)
    y, mean, rstd, dx, dw, db, dz = ref.group_norm(x, G, w, b, z, act, 1e-5, dy)
    r = ssd.GroupNormRunner(n, m, C, G, act, dtype)
    d = lambda t: None if t is None else t.cuda()  # noqa: E731
    gy, gmean, grstd = r.forward(d(x), d(w), d(b), z=d(z))
    g = r.backward(d(dy), d(x), d(w), d(b), gmean, grstd, z=d(z))
    # one rounding of the output; fp32: sums of < 2^17 terms, x - mean loses |mean| / std ~ 1
    close(gy, y, rounded(y, dtype), "y")
    close(gmean, mean, F32, "mean")
    close(grstd, rstd, F32, "rstd")
    # groups of one value: dx is zero but for rounding
    if m * C // G > 1:
        close(g["dx"], dx, rounded(dx, dtype), "dx")
    close(g["dbias"], db, F32, "dbias")
    if m * C // G > 1:
        close(g["dweight"], dw, F32, "dweight")
    if act == "gate":
        close(g["dz"], dz, rounded(dz, dtype), "dz")
    else:
        assert g["dz"] is None


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("act", ["none", "silu", "gate"])
@pytest.mark.parametrize("n,m,C,G", [(37, 1, 512, 8), (5, 1, 128, 1), (9, 1, 96, 1), (3, 7, 40, 5), (2, 300, 64, 2),
                                     (2, 33, 30, 3), (4, 1, 4096, 1), (1, 1000, 24, 1), (300, 1, 60, 20)])
def test_group_norm(n, m, C, G, act, dtype):
    gn_check(n, m, C, G, act, dtype, seed=n + m + C)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n,m,C,G", [(1, 5000, 64, 4), (3, 2047, 72, 9), (2, 1, 32768, 2), (1, 40000, 8, 1),
                                     (70000, 1, 16, 2), (6, 1, 9, 9), (130, 40, 7, 1)])
def test_group_norm_large_and_odd(n, m, C, G, dtype):
    gn_check(n, m, C, G, "silu", dtype, seed=7, affine=(n % 2 == 0))


def test_group_norm_large_mean():
    """The mean is 1000 times the deviation: sums of squares would leave nothing of it in fp32."""
    n, m, C, G = 3, 500, 64, 4
    x = gn_case(n, m, C, G, "none", "f32", 5)[0] / 1.5 + 1000.0
    y, mean, rstd = ref.group_norm(x, G)
    gy, gmean, grstd = ssd.GroupNormRunner(n, m, C, G, "none", "f32").forward(x.cuda())
    # x itself is stored to 2^-24 * 1000, and the mean rounds likewise: 2 * 6e-5 of the deviation
    close(gy, y, 1.2e-4, "y")
    close(gmean, mean, F32, "mean")
    close(grstd, rstd, 1.2e-4, "rstd")


def test_group_norm_constant_input():
    x = torch.full((4, 3, 64), 2.5, device="cuda")
    y, mean, rstd = ssd.GroupNormRunner(4, 3, 64, 2, "none", "f32").forward(x)
    assert (y == 0).all() and (mean == 2.5).all()
    close(rstd, torch.full((4, 2), 1e-5).rsqrt(), F32)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("m", [1, 600])
@pytest.mark.parametrize("pad", [8, 3])
def test_group_norm_row_strides(m, pad, dtype):
    """Views into wider rows; a stride that is not a multiple of 8 elements moves element by element."""
    n, C, G = 4, 128, 4
    x, dy, w, b, z = gn_case(n, m, C, G, "gate", dtype, 17)
    wide = lambda t: torch.nn.functional.pad(t, (0, pad)).cuda()[..., :C]  # noqa: E731
    r = ssd.GroupNormRunner(n, m, C, G, "gate", dtype)
    buf = torch.zeros(n, m, C + pad, dtype=TYPES[dtype], device="cuda")
    y, mean, rstd = r.forward(wide(x), w.cuda(), b.cuda(), z=wide(z), out=buf[..., :C])
    ry, _, _, rdx, rdw, rdb, rdz = ref.group_norm(x, G, w, b, z, "gate", 1e-5, dy)
    tol = 2 ** -9 if dtype == "bf16" else F32
    close(y, ry, tol, "y")
    assert (buf[..., C:] == 0).all()
    g = r.backward(wide(dy), wide(x), w.cuda(), b.cuda(), mean, rstd, z=wide(z))
    for name, want, t in (("dx", rdx, tol), ("dz", rdz, tol), ("dweight", rdw, F32), ("dbias", rdb, F32)):
        close(g[name], want, t, name)


def test_group_norm_nan_stays_in_its_group():
    x, dy, w, b, _ = gn_case(3, 50, 64, 4, "silu", "bf16", 19)
    r = ssd.GroupNormRunner(3, 50, 64, 4, "silu")
    clean, _, _ = r.forward(x.cuda(), w.cuda(), b.cuda())
    x[1, 7, 20] = float("nan")
    y, _, _ = r.forward(x.cuda(), w.cuda(), b.cuda())
    bad = torch.zeros(3, 50, 64, dtype=torch.bool)
    bad[1, :, 16:32] = True
    assert torch.isnan(y.cpu()[bad]).all() and torch.equal(y.cpu()[~bad], clean.cpu()[~bad])


def test_group_norm_gradient_against_differences():
    """Central differences of the fp32 forward in random directions: rounding 2^-24 |y| over 2 h and h^2 / 6 of third
    derivatives of order one, both as random-walk sums, stay below 1e-3 of the terms' norm at h = 1e-2."""
    n, m, C, G, h = 2, 30, 48, 3, 1e-2
    x, dy, w, b, z = (t.cuda() for t in gn_case(n, m, C, G, "gate", "f32", 23))
    r = ssd.GroupNormRunner(n, m, C, G, "gate", "f32")
    _, mean, rstd = r.forward(x, w, b, z=z)
    g = r.backward(dy, x, w, b, mean, rstd, z=z)
    gen = torch.Generator(device="cuda").manual_seed(2)
    args = {"dx": x, "dweight": w, "dbias": b, "dz": z}
    for name in args:
        e = torch.randn(args[name].shape, generator=gen, device="cuda")

        def loss(sign):
            a = dict(args)
            a[name] = a[name] + sign * h * e
            return r.forward(a["dx"], a["dweight"], a["dbias"], z=a["dz"])[0].double() * dy

        diff = (loss(1) - loss(-1)) / (2 * h)
        want = (g[name].double() * e).sum()
        assert abs(diff.sum() - want) <= 1e-3 * diff.norm(), name
