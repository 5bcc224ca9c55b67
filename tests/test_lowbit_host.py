"""8-bit floating point and the optimizer's step on a machine without a GPU: what the C entry points refuse before
any device call, their size queries, and the tests' own definitions against worked examples."""
import ctypes

import pytest

torch = pytest.importorskip("torch")

import lowbit_ref as ref  # noqa: E402

fake = 1 << 20  # aligned, never read


@pytest.fixture(scope="module")
def L():
    from allreduce_compatible_gradient_gb300 import _binding, _build
    _build.build_library()
    if torch.cuda.is_available():
        pytest.skip("fake pointers: run only where no GPU can be reached")
    return _binding.lib()


def test_sizes(L):
    import allreduce_compatible_gradient_gb300 as gq
    assert [gq.gq_fp8_code_pitch(c) for c in (0, 1, 16, 17, 4096)] == [0, 16, 16, 32, 4096]
    assert gq.gq_fp8_exp_bytes(1, 1) == 512 and gq.gq_fp8_exp_bytes(129, 513) == 4 * 512
    assert gq.gq_fp8_exp_bytes(0, 5) == 0 and gq.gq_fp8_exp_bytes(-1, 5) == 0 and gq.gq_fp8_exp_bytes(5, 0) == 0
    # rows of codes, and exponents behind them; none where x is put into 8 bits on its way
    assert gq.gq_fp8_linear_workspace_bytes(5000, 700, 4096) == 5000 * 704 + 40 * 2 * 512
    assert gq.gq_fp8_linear_workspace_bytes(1, 4096, 4096) == 0 == gq.gq_fp8_linear_workspace_bytes(0, 64, 64)
    one = gq.gq_tensors_norm_workspace_bytes(1)
    assert one > 0 and gq.gq_tensors_norm_workspace_bytes(257) == 2 * one
    assert gq.gq_tensors_norm_workspace_bytes(-1) == 0
    with pytest.raises(ValueError):
        gq.gq_adamw_state(-1, device="cpu")
    s = gq.gq_adamw_state(33, device="cpu")
    assert s.m.numel() == s.v.numel() == 64 and s.exps.shape == (2, 2) and not any(t.any() for t in s)


def test_quantisation_refuses(L):
    def quant(x=fake, dt=0, rows=4, cols=64, ld=64, block=1, codes=fake, exps=fake, exps_t=None):
        return L.gq_fp8_quantize(x, dt, rows, cols, ld, block, codes, exps, exps_t, None)
    assert quant(rows=0) == 0 and quant(rows=0, codes=None) == 0
    for bad in (dict(x=None), dict(x=fake + 2), dict(dt=2), dict(rows=-1), dict(cols=0), dict(ld=63), dict(block=2),
                dict(block=0), dict(exps_t=fake), dict(block=128, exps_t=fake + 8), dict(codes=None),
                dict(codes=fake + 8), dict(exps=None), dict(exps=fake + 8), dict(rows=1 << 31),
                dict(rows=(1 << 31) - 1, cols=1 << 30, ld=1 << 30)):
        assert quant(**bad) == 1, bad

    def dequant(codes=fake, exps=fake, rows=4, cols=64, out=fake, dt=1, ld=64):
        return L.gq_fp8_dequantize(codes, exps, rows, cols, out, dt, ld, None)
    assert dequant(rows=0) == 0
    for bad in (dict(codes=None), dict(exps=fake + 4), dict(out=None), dict(out=fake + 1), dict(dt=3), dict(ld=10)):
        assert dequant(**bad) == 1, bad


def test_products_refuse(L):
    def linear(x=None, dt=1, ldx=64, xc=fake, xe=fake, rows=4, cols=64, wc=fake, we=fake, outs=32, bias=None, y=fake,
               ydt=1, ldy=32):
        return L.gq_fp8_linear(x, dt, ldx, xc, xe, rows, cols, wc, we, outs, bias, y, ydt, ldy, None)
    assert linear(rows=0) == 0
    for bad in (dict(xc=None), dict(xe=None), dict(xc=fake + 8), dict(xe=fake + 4), dict(wc=None), dict(we=fake + 1),
                dict(x=fake + 1), dict(x=fake, dt=2), dict(x=fake, ldx=63), dict(rows=-1), dict(rows=1 << 30),
                dict(cols=0), dict(cols=1 << 30), dict(outs=0), dict(outs=1 << 30), dict(bias=fake + 2),
                dict(y=None), dict(y=fake + 1), dict(ydt=2), dict(ldy=31)):
        assert linear(**bad) == 1, bad

    def dgrad(dy=None, rows=4, outs=32, wc=fake, we=fake, cols=64, dx=fake, dt=1, ld=64):
        return L.gq_fp8_linear_dgrad(dy, 1, outs, fake, fake, rows, outs, wc, we, cols, dx, dt, ld, None)
    assert dgrad(rows=0) == 0
    for bad in (dict(dy=fake + 1), dict(wc=None), dict(we=None), dict(dx=None), dict(dt=2), dict(ld=63), dict(outs=0),
                dict(cols=1 << 30)):
        assert dgrad(**bad) == 1, bad


def test_the_step_refuses(L):
    P, N = ctypes.c_void_p * 2, ctypes.c_int64 * 2
    good = dict(count=2, p=P(fake, fake + 4096), pdt=0, g=P(fake, fake), gdt=0, m=P(fake, fake), v=P(fake, fake),
                e=None, n=N(10, 20), step=1, step_dev=None, lr=1e-3, b1=0.9, b2=0.999, eps=1e-8, wd=0.1, norm=None,
                most=-1.0, rnd=0, first=0)

    def step(**kw):
        a = good | kw
        return L.gq_adamw_step(a["count"], a["p"], a["pdt"], a["g"], a["gdt"], a["m"], a["v"], a["e"], a["n"],
                               a["step"], a["step_dev"], a["lr"], a["b1"], a["b2"], a["eps"], a["wd"], a["norm"],
                               a["most"], a["rnd"], 0, a["first"], None)
    assert step(count=0, p=None, g=None, m=None, v=None, n=None) == 0
    assert step(n=N(0, 0), p=P(None, None)) == 0             # tensors without elements: nothing is read
    nan = float("nan")
    for bad in (dict(count=-1), dict(p=None), dict(p=P(None, fake)), dict(p=P(fake + 2, fake)), dict(pdt=2),
                dict(gdt=3), dict(g=P(fake, None)), dict(m=P(fake + 2, fake)), dict(v=P(None, fake)), dict(n=N(-1, 5)),
                dict(n=N(1 << 34, 5)), dict(step=0), dict(step_dev=fake + 4), dict(b1=1.0), dict(b2=-0.1),
                dict(b1=nan), dict(eps=-1e-8), dict(eps=nan), dict(lr=nan), dict(wd=float("inf")), dict(rnd=2),
                dict(first=-1), dict(first=1 << 30), dict(norm=fake + 2), dict(e=P(fake, None)),
                dict(e=P(fake, fake + 1)), dict(e=P(fake, fake), m=P(fake + 8, fake))):
        assert step(**bad) == 1, bad

    def norm(count=2, t=P(fake, fake), n=N(10, 20), dt=0, out=fake, ws=fake, size=1 << 20):
        return L.gq_tensors_norm(count, t, n, dt, out, ws, size, None)
    for bad in (dict(t=None), dict(t=P(fake, None)), dict(t=P(fake + 2, fake)), dict(n=N(5, -1)), dict(dt=2),
                dict(out=None), dict(out=fake + 1), dict(count=-1)):
        assert norm(**bad) == 1, bad
    assert norm(ws=None) == 7 and norm(size=64) == 7 and norm(ws=fake + 8) == 7

    def values(count=2, m=P(fake, fake), e=P(fake, fake), n=N(10, 20), out=P(fake, fake), dt=1):
        return L.gq_adamw_values(count, m, m, e, n, out, out, dt, None)
    assert values(count=0) == 0
    for bad in (dict(m=None), dict(m=P(fake, fake + 8)), dict(e=P(fake + 1, fake)), dict(out=P(None, fake)),
                dict(out=P(fake + 1, fake)), dict(dt=2), dict(n=N(1, -1))):
        assert values(**bad) == 1, bad


def test_the_definitions_by_hand():
    """Worked examples of the formats: exponents at their borders, ties, subnormal codes, roots that are kept."""
    x = torch.tensor([[448.0, 17.0, 19.0, 2.0 ** -10, 3 * 2.0 ** -10, -18.0]])
    q, e = ref.fp8(x, 1)
    assert e.tolist() == [[127]] and q.tolist() == [[448.0, 16.0, 20.0, 0.0, 2.0 ** -8, -18.0]]
    q, e = ref.fp8(torch.tensor([[449.0, 1.0]]), 1)
    assert e.tolist() == [[128]] and ref.values(q, e, 1).tolist() == [[448.0, 1.0]]
    q, e = ref.fp8(torch.tensor([[float("inf"), 1.0]]), 1)
    assert e.tolist() == [[255]] and q.tolist() == [[0.0, 0.0]]
    q, e = ref.fp8(torch.zeros(200, 3), 128)
    assert e.tolist() == [[1], [1]] and not q.any()
    top = ref.ROOT_MOST
    v, e, s = ref.on_grid(torch.tensor([top, 1.0, 0.4, 0.0, 33.0], dtype=torch.float64), top, 4, 0, None, True)
    assert e.tolist() == [127] and v.tolist() == [top, 1.0, 1.0, 0.0, 32.0] and s.tolist()[4] == 2.0
    v, _, _ = ref.on_grid(torch.tensor([top, 33.0], dtype=torch.float64), top, 4, 0,
                          torch.tensor([65535.0, 32768.0], dtype=torch.float64), True)
    assert v.tolist() == [top, 34.0]  # 16.5 spacings and 0.5 + 2^-17


def test_step_by_hand():
    """The first step from zeros moves by lr along the gradient's sign."""
    p, m, v = ref.adamw(torch.tensor([1.0, -2.0]), torch.tensor([0.5, -4.0]), torch.zeros(2), torch.zeros(2), 1, 0.1,
                        (0.9, 0.99), 0.0, 0.5)
    assert torch.allclose(p, torch.tensor([0.95 - 0.1, -1.9 + 0.1], dtype=torch.float64), atol=1e-12)
    assert torch.allclose(m, torch.tensor([0.05, -0.4], dtype=torch.float64), atol=1e-12)
    assert torch.allclose(v, torch.tensor([0.0025, 0.16], dtype=torch.float64), atol=1e-12)
