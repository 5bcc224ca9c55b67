"""The AdamW step over many tensors, its 8-bit states, and the norm of all gradients, against their definitions
in 64 bits.

Tolerances, with u = 2^-24:
- m = beta1 m + (1 - beta1) g', g' = g c: the constants, c (a sum of squares within 80 u, a root, a sum and a
  quotient) and four operations are each rounded once, so m is within 8 u (90 u where gradients are clipped) of
  the sum of its terms' magnitudes, v within twice that, and its root within that (half of v's relative error,
  and its own rounding);
- the update is a quotient of those, with a reciprocal of 2 units in the last place and constants of its own:
  within 16 u plus the errors of m and the root, relative to the sum of m's terms' magnitudes over the
  denominator; the parameter adds 2 u of its magnitude, and its own rounding (2^-8 relative in bf16; one unit,
  2^-7, where it is random);
- rounded states are compared with the grid: within one spacing at the value before rounding, plus that
  value's error.  Where the inputs are small integers times powers of two, so that fp32 is exact, codes
  are compared bit for bit.
"""
import pytest

import lowbit_ref as ref
from gpu_common import gq_module

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

U = 2.0 ** -24
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


@pytest.fixture(scope="module")
def gq():
    return gq_module()


def flat(n, g, scale, dtype=torch.float32, shift=0):
    """Normal numbers, `shift` elements into a buffer."""
    out = torch.empty(n + shift, dtype=dtype, device="cuda")[shift:]
    out.copy_(torch.randn(n, generator=g, device="cuda") * scale)
    return out


def values(gq, states, sizes):
    out = tuple([torch.empty(n, device="cuda") for n in sizes] for _ in range(2))
    gq.gq_adamw_values(states, out=out)
    return out


def random_state(n, g, size):
    """An 8-bit state with codes of every kind."""
    from allreduce_compatible_gradient_gb300 import Adam8
    room = (n + 31) // 32 * 32
    m = torch.randint(0, 256, (room,), generator=g, device="cuda", dtype=torch.uint8)
    m = torch.where(m % 128 == 127, 0, m).to(torch.uint8)
    v = torch.randint(0, 256, (room,), generator=g, device="cuda", dtype=torch.uint8)
    m[n:] = 0
    v[n:] = 0
    e = torch.empty((room // 32, 2), dtype=torch.uint8, device="cuda")
    k = torch.frexp(torch.tensor(size))[1].item()
    e[:, 0], e[:, 1] = 127 + k - 9, 127 + k - 19
    e += torch.randint(0, 3, (room // 32, 2), generator=g, device="cuda", dtype=torch.uint8)
    return Adam8(m, v, e)


def decode(s, n):
    """The values of a state, from its bytes."""
    m = s.m[:n].view(torch.float8_e4m3fn).double()
    c = s.v[:n].long()
    r = torch.where(c < 16, c, (16 + c % 16) << (c // 16 - 1).clamp(min=0)).double()
    e = s.exps.long().repeat_interleave(32, dim=0)[:n]
    unit = torch.where(e == 255, float("nan"), ref.two(e - 127))
    return m * unit[:, 0], r * unit[:, 1]


SIZES = [[1], [8], [31, 32, 33], [256, 1, 8192, 8193, 7], [100000], [5, 0, 70000, 16384], [33] * 40,
         [129 + i for i in range(300)]]
KW = dict(lr=2e-3, betas=(0.9, 0.99), eps=1e-8, weight_decay=0.02)


def step_case(gq, sizes, param, grad, eight, seed, shift=0, clip=None, step=7, counter=False):
    g = torch.Generator(device="cuda").manual_seed(sum(sizes) + shift)
    p = [flat(n, g, 0.5, TYPES[param], shift) for n in sizes]
    d = [flat(n, g, 0.01, TYPES[grad], shift) for n in sizes]
    if eight:
        states = [random_state(n, g, 0.01) for n in sizes]
        old = [decode(s, n) for s, n in zip(states, sizes)]
        old = [(m, r * r) for m, r in old]
    else:
        states = [(flat(n, g, 0.004, shift=shift), flat(n, g, 1e-4, shift=shift).square_()) for n in sizes]
        old = [(m.double(), v.double()) for m, v in states]
    before = [t.double() for t in p]
    norm = None
    if clip is not None:
        norm = gq.gq_tensors_norm(d)
        want = torch.stack([t.double().square().sum() for t in d]).sum().sqrt()
        assert abs(norm.double() - want) <= 80 * U * want
        c = min(1.0, clip / (float(want) + 1e-6))
    else:
        c = 1.0
    number = torch.tensor([step], device="cuda") if counter else step
    gq.gq_adamw_step(p, d, states, number, norm=norm, max_norm=clip, seed=seed, **KW)
    b1, b2 = KW["betas"]
    lost = 90 if clip is not None else 8
    for i, n in enumerate(sizes):
        if n == 0:
            continue
        grad64 = d[i].double()
        np_, nm, nv = ref.adamw(before[i], grad64, *old[i], step, KW["lr"], KW["betas"], KW["eps"],
                                KW["weight_decay"], c)
        terms = b1 * old[i][0].abs() + (1 - b1) * (grad64 * c).abs()
        tm, tr = lost * U * terms, lost * U * nv.sqrt()
        den = nv.sqrt() / (1 - b2 ** step) ** 0.5 + KW["eps"]
        rel = (16 + 2 * lost) * U + (1e-6 if counter else 0.0)  # expm1 of a rounded exponent
        tp = 2 * U * before[i].abs() + KW["lr"] / (1 - b1 ** step) * rel * terms / den
        if param == "f32":
            tp = tp + U * np_.abs()
        else:
            tp = tp + (2.0 ** -7 if seed is not None else 2.0 ** -8) * np_.abs()
        got = p[i].double()
        assert ((got - np_).abs() <= tp).all(), ((got - np_).abs() / tp).max()
        if not eight:
            assert ((states[i][0].double() - nm).abs() <= tm + 1e-45).all()
            assert ((states[i][1].double() - nv).abs() <= 2 * lost * U * nv + 1e-45).all()
            continue
        assert not states[i].m[n:].any() and not states[i].v[n:].any()
        gm, gr = decode(states[i], n)
        vm, vr = values(gq, [states[i]], [n])
        assert torch.equal(vm[0].double(), gm) and torch.equal(vr[0].double(), gr)
        step_of = 1.0 if seed is not None else 0.5
        _, _, sm = ref.on_grid(nm.abs(), ref.E4M3_MOST, 3, -9, None, False)
        _, _, sr = ref.on_grid(nv.sqrt(), ref.ROOT_MOST, 4, 0, None, True)
        # a value near a power of two may be rounded on the side of the wider spacing; a root is kept from 0
        assert ((gm - nm).abs() <= step_of * 2 * sm + tm).all()
        kept = (gr > 0) | (nv == 0)
        assert kept.all() and ((gr - nv.sqrt()).abs() <= torch.maximum(step_of * 2 * sr, sr) + tr).all()


@pytest.mark.parametrize("sizes", SIZES, ids=lambda s: "%dx%d" % (len(s), max(s)))
@pytest.mark.parametrize("param,grad", [("f32", "f32"), ("f32", "bf16"), ("bf16", "bf16"), ("bf16", "f32")])
@pytest.mark.parametrize("eight,seed", [(False, None), (True, None), (True, 5), (False, 5)])
def test_step(gq, sizes, param, grad, eight, seed):
    step_case(gq, sizes, param, grad, eight, seed)


@pytest.mark.parametrize("shift", [1, 2, 4, 8, 11])
@pytest.mark.parametrize("eight", [False, True])
def test_step_alignments(gq, shift, eight):
    step_case(gq, [70001, 40], "f32", "f32", eight, None, shift)
    step_case(gq, [9000], "bf16", "bf16", eight, 3, shift)


@pytest.mark.parametrize("eight", [False, True])
def test_step_clipped(gq, eight):
    step_case(gq, [5000, 33, 100], "f32", "f32", eight, None, clip=0.1)     # norm about 0.7
    step_case(gq, [5000, 33, 100], "f32", "bf16", eight, 9, clip=100.0)     # below the limit


@pytest.mark.parametrize("step", [1, 2, 1000, 10 ** 6])
def test_step_counted_on_the_device(gq, step):
    step_case(gq, [3000], "f32", "f32", True, 4, step=step, counter=True)
    step_case(gq, [3000], "f32", "f32", False, None, step=step, counter=True)
    step_case(gq, [3000], "bf16", "f32", False, 4, step=step)


def exact_case(n, seed):
    """A gradient and a state for which beta1 = 1/2, beta2 = 3/4 make m, v and its root exact in fp32: r is a
    small integer, v = r^2 = 3/4 r0^2 + 1/4 g^2 with r0 = g = r."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = torch.randint(0, 2048, (n,), generator=g, device="cuda").float()
    r *= 2.0 ** -torch.randint(0, 8, (n,), generator=g, device="cuda").float()
    m = torch.randint(-2048, 2048, (n,), generator=g, device="cuda").float() * 2.0 ** -6
    return r, m


@pytest.mark.parametrize("n", [32, 1000, 20001])
@pytest.mark.parametrize("seed", [None, 0, 2 ** 63 + 11])
def test_codes_bit_for_bit(gq, n, seed):
    """Two steps' worth of rounding on values that fp32 holds exactly: from fp32 states through a state of 8 bits.
    The first step starts from zeros: m = g / 2, v = g^2 / 4, root |g| / 2."""
    r, _ = exact_case(n, n)
    g = torch.where(torch.rand(n, device="cuda") < 0.5, -r, r)
    p = torch.zeros(n, device="cuda")
    state = gq.gq_adamw_state(n)
    big = 2 ** 40 + 3
    gq.gq_adamw_step([p], [g], [state], big, lr=1e-3, betas=(0.5, 0.75), seed=seed, first=6)
    h = [None] * 2 if seed is None else [ref.words(n, 18 + k, seed, big, "cuda") for k in range(2)]
    qm, em, _ = ref.on_grid(g.double().abs() / 2, ref.E4M3_MOST, 3, -9, h[0], False)
    qr, er, _ = ref.on_grid(g.double().abs() / 2, ref.ROOT_MOST, 4, 0, h[1], True)
    m, root = decode(state, n)
    assert torch.equal(state.exps[:, 0].long(), em) and torch.equal(state.exps[:, 1].long(), er)
    assert torch.equal(m, torch.sign(g.double()) * qm) and torch.equal(root, qr)


def test_random_rounding_is_unbiased(gq):
    """The mean over 4,000 steps' words of m, the root and a bf16 parameter is the value itself, within 5
    standard deviations of the mean (at most half a spacing each) and the 2^-17 of a spacing of 16-bit numbers."""
    n, times = 64, 4000
    g = torch.Generator(device="cuda").manual_seed(1)
    d = torch.rand(n, generator=g, device="cuda") + 0.5
    total = [torch.zeros(n, device="cuda", dtype=torch.float64) for _ in range(3)]
    for t in range(1, times + 1):
        s, p = gq.gq_adamw_state(n), torch.full((n,), 1.0, device="cuda", dtype=torch.bfloat16)
        gq.gq_adamw_step([p], [d], [s], 10 ** 6 + t, lr=0.003, betas=(0.5, 0.75), weight_decay=0.5, seed=3)
        m, r = decode(s, n)
        for a, b in zip(total, (m, r, p.double())):
            a += b
    m, r = d.double() / 2, d.double() / 2
    want = [m, r, 1.0 * (1 - 0.003 * 0.5) - 0.003 * m / (r + 1e-8)]
    spacing = [ref.spacing(m / 2.0 ** -9, 3, -9) * 2.0 ** -9, ref.spacing(r / 2.0 ** -19, 4, 0) * 2.0 ** -19,
               torch.full_like(m, 2.0 ** -8)]
    for a, b, s in zip(total, want, spacing):
        off = (a / times - b).abs()
        assert (off <= s * (5 * 0.5 / times ** 0.5 + 2.0 ** -17) + 1e-6 * b.abs()).all(), (off / s).max()


def test_small_roots_are_kept(gq):
    """A root too small for its block's grid keeps the smallest code, also rounded at random; zeros stay."""
    g = torch.full((32,), 1e-20, device="cuda")
    g[0], g[1] = 1e4, 0.0
    for seed in (None, 1, 2, 3):
        s = gq.gq_adamw_state(32)
        p = torch.zeros(32, device="cuda")
        gq.gq_adamw_step([p], [g], [s], 1, betas=(0.9, 0.75), seed=seed)
        assert (s.v[2:] == 1).all() and s.v[1] == 0 and s.v[0] > 200
        assert p.isfinite().all()


def test_norm(gq):
    g = torch.Generator(device="cuda").manual_seed(2)
    for sizes in ([1], [0, 3], [7, 16384, 16385, 1], [3] * 600, [1 << 22, 5], [1 << 20], [(1 << 20) + 1], [1 << 21],
                  [4097] * 200, [4096] * 256, [100, 0, 900000, 4095]):
        for dtype in TYPES.values():
            t = [flat(n, g, 3.0, dtype, shift=i % 3) for i, n in enumerate(sizes)]
            want = torch.stack([x.double().square().sum() for x in t]).sum().sqrt()
            got = gq.gq_tensors_norm(t)
            assert got.shape == (1,) and got.dtype == torch.float32
            assert abs(got.double() - want) <= 80 * U * want
            assert torch.equal(got, gq.gq_tensors_norm(t))
            ws = torch.full((gq.gq_tensors_norm_workspace_bytes(len(t)),), 255, dtype=torch.uint8, device="cuda")
            assert torch.equal(got, gq.gq_tensors_norm(t, ws=ws))
    assert gq.gq_tensors_norm([torch.empty(0, device="cuda")]).item() == 0.0
    x = torch.ones(100, device="cuda")
    for bad in (float("nan"), float("inf"), -float("inf"), 1e30):
        x[50] = bad
        assert not gq.gq_tensors_norm([x]).isfinite().any()


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_step_without_a_finite_norm_changes_nothing(gq, bad):
    for eight in (False, True):
        g = torch.Generator(device="cuda").manual_seed(2)
        p, d = flat(1000, g, 1.0), flat(1000, g, 1.0)
        d[500] = bad
        s = random_state(1000, g, 1.0) if eight else (flat(1000, g, 1.0), flat(1000, g, 1.0).abs())
        before = [t.clone() for t in (p, *s)]
        gq.gq_adamw_step([p], [d], [s], 3, norm=gq.gq_tensors_norm([d]), max_norm=1.0)
        assert all(torch.equal(a, b) for a, b in zip(before, (p, *s)))


def test_gradients_that_are_not_finite(gq):
    """Without a norm they reach their own element and, in 8 bits, the states of its block."""
    g = torch.Generator(device="cuda").manual_seed(2)
    p, d = flat(100, g, 1.0), flat(100, g, 1.0)
    d[40] = float("nan")
    s = gq.gq_adamw_state(100)
    gq.gq_adamw_step([p], [d], [s], 1)
    assert p[40].isnan() and p.isnan().sum() == 1
    m, r = values(gq, [s], [100])
    bad = torch.zeros(100, dtype=torch.bool, device="cuda")
    bad[32:64] = True
    assert torch.equal(m[0].isnan(), bad) and torch.equal(r[0].isnan(), bad)
    assert (s.exps[1] == 255).all()


def test_step_captured_in_a_graph(gq):
    """A captured step with the norm, a step number on the device and random words follows the eager one."""
    g = torch.Generator(device="cuda").manual_seed(4)
    p0 = [flat(n, g, 0.5) for n in (3000, 100)]
    d = [flat(n, g, 0.01) for n in (3000, 100)]

    def fresh():
        return [t.clone() for t in p0], [gq.gq_adamw_state(t.numel()) for t in p0]

    p, s = fresh()
    number = torch.ones(1, dtype=torch.int64, device="cuda")

    def once():
        gq.gq_adamw_step(p, d, s, number, norm=gq.gq_tensors_norm(d), max_norm=0.2, seed=8)
        number.add_(1)

    graph = torch.cuda.CUDAGraph()
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        gq.gq_tensors_norm(d)
    torch.cuda.current_stream().wait_stream(stream)
    with torch.cuda.graph(graph):
        once()
    for _ in range(5):
        graph.replay()
    captured = [t.clone() for t in p] + [x.clone() for t in s for x in t]
    assert number.item() == 6
    p, s = fresh()
    number.fill_(1)
    for _ in range(5):
        once()
    eager = p + [x for t in s for x in t]
    assert all(torch.equal(a, b) for a, b in zip(captured, eager))


def test_steps_count_as_changes_in_place(gq):
    """A backward pass that saved a parameter before the step refuses to run after it."""
    w = torch.randn(64, device="cuda", requires_grad=True)
    loss = (w * w).sum()
    gq.gq_adamw_step([w.detach()], [torch.ones(64, device="cuda")], [gq.gq_adamw_state(64)], 1)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()


def test_step_on_another_stream(gq):
    g = torch.Generator(device="cuda").manual_seed(4)
    p, d = [flat(100000, g, 0.5)], [flat(100000, g, 0.01)]
    q = [p[0].clone()]
    gq.gq_adamw_step(p, d, [gq.gq_adamw_state(100000)], 1)
    s = gq.gq_adamw_state(100000)
    torch.cuda.synchronize()
    stream = torch.cuda.Stream()
    gq.gq_adamw_step(q, d, [s], 1, stream=stream)
    stream.synchronize()
    assert torch.equal(p[0], q[0])
