"""Products in 8-bit floating point and AdamW as a training program uses them: the layers, the optimizer, both
with everything else of a step."""
import copy
import importlib.util
import io
import os
import threading

import pytest

import lowbit_ref as ref
from gpu_common import gq_module

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def gq():
    return gq_module()


@pytest.fixture(scope="module")
def layers(gq):
    from allreduce_compatible_gradient_gb300 import act8_layers
    return act8_layers


@pytest.fixture(scope="module")
def adamw(gq):
    from allreduce_compatible_gradient_gb300 import adamw
    return adamw


def block_of(layers, width=96, hidden=200, dtype=torch.float32, **kw):
    torch.manual_seed(3)
    block = layers.MlpBlock8(width, hidden, seed=5, device="cuda", products="e4m3", **kw)
    with torch.no_grad():
        for p in block.parameters():
            p += 0.1 * torch.randn_like(p)
    return block.to(dtype)


# ---- the layers ------------------------------------------------------------------------------

@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_block_is_its_operators(gq, layers, dtype):
    """Output and gradients bit for bit from the operators called one by one."""
    block = block_of(layers)
    x = torch.randn((2, 75, 96), device="cuda").to(dtype).requires_grad_()
    r = torch.randn((2, 75, 96), device="cuda").to(dtype)
    out = block(x)
    got = torch.autograd.grad((out * r).sum(), [x, *block.parameters()])
    with torch.no_grad():
        nw, nb, w1, b1, w2, b2 = (p.detach() for p in block.parameters())
        f1, f2 = gq.gq_fp8_quantize(w1, tiles=True), gq.gq_fp8_quantize(w2, tiles=True)
        (s0, t0), (s1, t1) = block.words(0), block.words(1)
        y, _, rstd, act = gq.gq_layernorm_forward(x.detach(), nw, nb, seed=s0, step=t0)
        u = gq.gq_fp8_linear(y, f1, bias=b1)
        h, act_u = gq.gq_gelu_forward(u, seed=s1, step=t1)
        assert torch.equal(out, x + gq.gq_fp8_linear(h, f2, bias=b2))
        d = r.view(-1, 96)
        du, h = gq.gq_gelu_backward(gq.gq_fp8_linear_dgrad(d, f2), act_u, need_output=True)
        dw1, db1 = gq.gq_linear_wgrad(du, act, scale=nw, shift=nb)
        dx, dnw, dnb = gq.gq_layernorm_backward(gq.gq_fp8_linear_dgrad(du, f1), nw, rstd, act=act)
    want = [dx.view(x.shape) + r, dnw, dnb, dw1, db1]
    for g, w in zip(got, want):
        assert torch.equal(g, w.view(g.shape))
    assert torch.equal(got[6], d.sum(0, dtype=torch.float32))


def test_block_near_exact_gradients(layers):
    """Operands in e4m3 are within 2^-4 of their elements, 0.026 in the mean square each (a rounding spread evenly
    over a spacing of 1/8 to 1/16); two operands and two products behind one another leave about 0.04 to 0.08
    of a gradient's norm."""
    block = block_of(layers)
    x = torch.randn((2, 75, 96), device="cuda", requires_grad=True)
    r = torch.randn((2, 75, 96), device="cuda")
    got = torch.autograd.grad((block(x) * r).sum(), [x, *block.parameters()])
    p = {k: v.detach().double().requires_grad_() for k, v in block.named_parameters()}
    z = x.detach().double().requires_grad_()
    y = torch.nn.functional.layer_norm(z, (96,), p["norm_weight"], p["norm_bias"], block.eps)
    h = torch.nn.functional.gelu(y @ p["w1"].t() + p["b1"])
    want = torch.autograd.grad(((z + h @ p["w2"].t() + p["b2"]) * r.double()).sum(), [z, *p.values()])
    for g, w in zip(got, want):
        assert (g.double() - w).norm() < 0.1 * w.norm()


def test_product_gradient_against_differences(gq):
    """gq_fp8_linear is linear in the values of its operands: the change of its result along a direction, from
    values that e4m3 holds exactly, is the gradient's product with the direction."""
    g = torch.Generator(device="cuda").manual_seed(7)
    x, v = (torch.randint(-8, 9, (70, 300), generator=g, device="cuda").float() for _ in range(2))
    w = gq.gq_fp8_quantize(torch.randint(-8, 9, (130, 300), generator=g, device="cuda").float(), tiles=True)
    dy = torch.randint(-8, 9, (70, 130), generator=g, device="cuda").float()
    # 2 x and 2 (x + v), 2 (x - v) are integers of at most 32: all of them are e4m3 numbers where even above 16
    x, v = 2 * x, 2 * v
    up, down = x + v, x - v
    for t in (x, up, down):
        assert torch.equal(gq.gq_fp8_dequantize(gq.gq_fp8_quantize(t), out_dtype=torch.float32), t)
    f = lambda t: (gq.gq_fp8_linear(t, w).double() * dy.double()).sum()  # noqa: E731
    dx = gq.gq_fp8_linear_dgrad(dy, w).double()
    assert (f(up) - f(down)) / 2 == (dx * v.double()).sum()


def test_block_frozen_and_without_gradients(layers):
    block = block_of(layers)
    x = torch.randn((33, 96), device="cuda")
    with torch.no_grad():
        assert block(x).shape == x.shape
    for name, p in block.named_parameters():
        p.requires_grad_(name in ("b2", "norm_bias"))
    block(x).sum().backward()
    assert block.b2.grad is not None and block.norm_bias.grad is not None and block.w1.grad is None


def test_block_bf16_parameters_and_no_rows(layers):
    block = block_of(layers, dtype=torch.bfloat16)
    x = torch.randn((5, 96), device="cuda", dtype=torch.bfloat16)
    block(x).float().sum().backward()
    assert all(p.grad.dtype == torch.bfloat16 for p in block.parameters())
    assert block(x[:0]).shape == (0, 96)


def test_block_captured_while_an_eager_graph_lives(layers):
    """Forward and backward pass captured with an eager graph of the same parameters alive; the replay is the
    eager pass."""
    block = block_of(layers)
    x, r = (torch.randn((64, 96), device="cuda") for _ in range(2))
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        eager = (block(x) * r).sum()
        want = torch.autograd.grad(eager, list(block.parameters()), retain_graph=True)
        # a copy whose leaves have no eager graph: a captured backward pass waits for its leaves' streams
        twin = copy.deepcopy(block)
        twin.seed = block.seed
        torch.autograd.grad((twin(x) * r).sum(), list(twin.parameters()))
    torch.cuda.current_stream().wait_stream(stream)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        got = torch.autograd.grad((twin(x) * r).sum(), list(twin.parameters()))
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_two_threads_on_two_streams(gq):
    """Calls of both forms from two threads, each with a stream and tensors of its own."""
    g = torch.Generator(device="cuda").manual_seed(7)
    cases = [(3, 640, 300), (300, 1000, 500), (2600, 520, 2100)]
    args = [(torch.randn((t, k), generator=g, device="cuda").bfloat16(),
             gq.gq_fp8_quantize(torch.randn((n, k), generator=g, device="cuda"), tiles=True)) for t, k, n in cases]
    want = [gq.gq_fp8_linear(x, w) for x, w in args]
    back = [gq.gq_fp8_linear_dgrad(y, w) for y, (_, w) in zip(want, args)]
    torch.cuda.synchronize()
    bad = []

    def work():
        stream = torch.cuda.Stream()
        for _ in range(30):
            for (x, w), y, d in zip(args, want, back):
                z = gq.gq_fp8_linear(x, w, stream=stream)
                e = gq.gq_fp8_linear_dgrad(y, w, stream=stream)
                stream.synchronize()
                if not torch.equal(z, y) or not torch.equal(e, d):
                    bad.append(x.shape)

    threads = [threading.Thread(target=work) for _ in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad


@pytest.mark.parametrize("rows,cols,outs", [(1, 700, 300), (200, 700, 300), (4200, 300, 1100)])
def test_products_captured_in_graphs(gq, rows, cols, outs):
    """A call of every form captured and replayed on new inputs, two graphs in turn."""
    g = torch.Generator(device="cuda").manual_seed(7)
    w = gq.gq_fp8_quantize(torch.randn((outs, cols), generator=g, device="cuda"), tiles=True)
    x = torch.randn((rows, cols), generator=g, device="cuda").bfloat16()
    graphs = []
    gq.gq_fp8_linear_dgrad(gq.gq_fp8_linear(x, w), w)
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            y = gq.gq_fp8_linear(x, w)
            d = gq.gq_fp8_linear_dgrad(y, w)
        graphs.append((graph, y, d))
    for k in range(4):
        x.copy_(torch.randn((rows, cols), generator=g, device="cuda"))
        graph, y, d = graphs[k % 2]
        graph.replay()
        want = gq.gq_fp8_linear(x, w)
        assert torch.equal(y, want) and torch.equal(d, gq.gq_fp8_linear_dgrad(want, w))


def test_overlapping_calls_keep_their_inputs(gq):
    """Weights written by the launch right before a product, in a loop that nothing waits in: each product sees
    the weight of its turn, in every form."""
    g = torch.Generator(device="cuda").manual_seed(7)
    for rows, cols, outs in ((1, 1024, 512), (200, 1024, 512), (4200, 512, 1100)):
        x = torch.randn((rows, cols), generator=g, device="cuda").bfloat16()
        fx = gq.gq_fp8_quantize(x)
        ws = [torch.randn((outs, cols), generator=g, device="cuda") for _ in range(8)]
        want = []
        for w in ws:
            f = gq.gq_fp8_quantize(w, tiles=True)
            torch.cuda.synchronize()
            want.append(gq.gq_fp8_linear(x, f))
            torch.cuda.synchronize()
        for source in (x, fx):
            got = [gq.gq_fp8_linear(source, gq.gq_fp8_quantize(w, tiles=True)) for w in ws]
            assert all(torch.equal(a, b) for a, b in zip(got, want))


# ---- the optimizer ---------------------------------------------------------------------------

def parameters(dtype=torch.float32, seed=1):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return [torch.nn.Parameter(torch.randn(s, generator=g, device="cuda").to(dtype))
            for s in ((64, 33), (33,), (1,), (5000,))]


def with_gradients(params, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    for p in params:
        p.grad = (torch.randn(p.shape, generator=g, device="cuda") * 0.1).to(p.dtype)
    return params


def test_optimizer_follows_torch(adamw):
    """Twenty steps with fp32 states beside torch's AdamW in fp64: a step's rounding is within 3 units of fp32, and
    the steps add up."""
    ours = parameters()
    theirs = [torch.nn.Parameter(p.detach().double()) for p in ours]
    a = adamw.AdamW(ours, lr=1e-2, weight_decay=0.1, states="f32")
    b = torch.optim.AdamW(theirs, lr=1e-2, weight_decay=0.1)
    for k in range(20):
        with_gradients(ours, k)
        for p, q in zip(ours, theirs):
            q.grad = p.grad.double()
        a.step()
        b.step()
    for p, q in zip(ours, theirs):
        assert ((p.double() - q).abs() <= 20 * (3 * 2.0 ** -24 * q.abs() + 1e-2 * 32 * 2.0 ** -24)).all()


@pytest.mark.parametrize("states", ["8bit", "f32"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_optimizer_is_its_operator(gq, adamw, states, dtype):
    """Two parameter groups, one parameter without a gradient, clipping: bit for bit what the calls give."""
    ours = with_gradients(parameters(dtype), 5)
    ours[2].grad = None
    twins = [p.detach().clone() for p in ours]
    opt = adamw.AdamW([dict(params=ours[:2]), dict(params=ours[2:], lr=5e-4, weight_decay=0.0)], lr=1e-2,
                      states=states, max_norm=0.5, seed=9)
    kept = [gq.gq_adamw_state(p.numel()) if states == "8bit" else
            tuple(torch.zeros(p.shape, device="cuda") for _ in range(2)) for p in ours]
    for step in range(1, 4):
        opt.step()
        norm = gq.gq_tensors_norm([ours[i].grad for i in (0, 1, 3)])
        kw = dict(norm=norm, max_norm=0.5, seed=opt.key)
        gq.gq_adamw_step(twins[:2], [p.grad for p in ours[:2]], kept[:2], step, lr=1e-2, **kw)
        gq.gq_adamw_step(twins[3:], [ours[3].grad], kept[3:], step, lr=5e-4, weight_decay=0.0, first=2, **kw)
        assert all(torch.equal(p, t) for p, t in zip(ours, twins))
    for p, s in zip(ours, kept):
        if p.grad is not None:
            assert all(torch.equal(a, b) for a, b in zip(opt.state[p].values(), s))
    assert not opt.state[ours[2]]


def test_optimizer_keys_are_its_own(adamw, layers):
    """No seed of a gradient (below 2^63) and no key of a block, named or not."""
    keys = {adamw.AdamW(parameters(), seed=s).key for s in (0, 1, (1 << 31) - 1)}
    assert len(keys) == 3 and all(1 << 63 < k < 1 << 64 for k in keys)
    named = max(1 << 63 | 2 * s + 1 for s in (0, (1 << 62) - (1 << 32) - 1))
    unnamed = 1 << 63 | 2 * ((1 << 62) - 1 - (1 << 24))  # of the block made after 16 million others
    assert all(named < k < unnamed for k in keys)


@pytest.mark.parametrize("states", ["8bit", "f32"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_optimizer_continues_from_a_file(adamw, states, dtype):
    def made():
        params = parameters(dtype)
        return params, adamw.AdamW(params, states=states, max_norm=1.0)

    ours, a = made()
    for k in range(3):
        with_gradients(ours, k)
        a.step()
    f = io.BytesIO()
    torch.save((a.state_dict(), [p.detach() for p in ours]), f)
    f.seek(0)
    theirs, b = made()
    saved, values = torch.load(f)
    b.load_state_dict(saved)
    with torch.no_grad():
        for p, v in zip(theirs, values):
            p.copy_(v)
    for k in range(3, 6):
        with_gradients(ours, k)
        with_gradients(theirs, k)
        a.step()
        b.step()
    assert all(torch.equal(p, q) for p, q in zip(ours, theirs))
    for p, q in zip(ours, theirs):
        assert all(x.dtype == y.dtype and torch.equal(x, y) for x, y in zip(a.state[p].values(), b.state[q].values()))


def test_optimizer_of_both_types(adamw):
    """Parameters of both types in one group; the norm is over all of them."""
    ours = with_gradients(parameters() + parameters(torch.bfloat16, 2), 3)
    opt = adamw.AdamW(ours, states="f32", max_norm=0.25, random=False, weight_decay=0.0)
    norm = torch.stack([p.grad.double().square().sum() for p in ours]).sum().sqrt()
    before = [p.detach().double() for p in ours]
    opt.step()
    for p, b in zip(ours, before):
        g = p.grad.double() * 0.25 / norm
        m = opt.state[p]["m"].double()
        assert ((m - 0.1 * g).abs() <= 100 * 2.0 ** -24 * g.abs()).all()
        want = b - 1e-3 * g / (g.abs() + 1e-8)
        step = 2.0 ** -8 if p.dtype == torch.bfloat16 else 2.0 ** -23
        assert ((p.double() - want).abs() <= step * want.abs() + 1e-6).all()


def test_optimizer_captured_in_a_graph(adamw):
    """Three replays of a captured step are three eager ones."""
    ours, theirs = with_gradients(parameters(), 1), with_gradients(parameters(), 1)
    a = adamw.AdamW(ours, max_norm=0.1, capturable=True)
    b = adamw.AdamW(theirs, max_norm=0.1, capturable=True)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        a.step()
    torch.cuda.current_stream().wait_stream(stream)
    b.step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        a.step()
    for _ in range(3):
        graph.replay()
        b.step()
    assert a.param_groups[0]["step"].item() == 4
    assert all(torch.equal(p, q) for p, q in zip(ours, theirs))
    assert all(torch.equal(x, y) for p, q in zip(ours, theirs) for x, y in zip(a.state[p].values(), b.state[q].values()))


def test_optimizer_captured_from_made_states(adamw):
    """Captured before any step: refused without states, and with them the replays count from 1."""
    ours, theirs = with_gradients(parameters(), 1), with_gradients(parameters(), 1)
    a, b = (adamw.AdamW(p, capturable=True) for p in (ours, theirs))
    graph = torch.cuda.CUDAGraph()
    with pytest.raises(RuntimeError, match="before a step is captured"):
        with torch.cuda.graph(graph):
            a.step()
    a.make_states()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        a.step()
    for _ in range(3):
        graph.replay()
        b.step()
    assert a.param_groups[0]["step"].item() == 3
    assert all(torch.equal(p, q) for p, q in zip(ours, theirs))


def test_optimizer_copies(adamw):
    """A deep copy goes on like the original, clipping and words included."""
    ours = with_gradients(parameters(torch.bfloat16), 1)
    a = adamw.AdamW(ours, max_norm=0.1, seed=3)
    a.step()
    b = copy.deepcopy(a)
    twins = with_gradients([p for g in b.param_groups for p in g["params"]], 1)
    a.step()
    b.step()
    assert all(p is not q and torch.equal(p, q) for p, q in zip(ours, twins))


def test_optimizer_refuses(adamw):
    for bad in (dict(states="4bit"), dict(betas=(1.0, 0.9)), dict(betas=(0.9, -0.1)), dict(eps=-1.0),
                dict(max_norm=-1.0), dict(seed=-1), dict(seed=1 << 31)):
        with pytest.raises(ValueError):
            adamw.AdamW(parameters(), **bad)
    p = torch.nn.Parameter(torch.zeros(4, 4, device="cuda").t()[:, :2])
    p.grad = torch.ones_like(p)
    with pytest.raises(ValueError):
        adamw.AdamW([p]).step()
    p = torch.nn.Parameter(torch.zeros(4, device="cuda", dtype=torch.float16))
    p.grad = torch.ones_like(p)
    with pytest.raises(TypeError):
        adamw.AdamW([p]).step()


def test_training_example_runs(gq):
    """Products in 8-bit floating point, gradients through Global-QSGD, AdamW in 8 bits: every loss is a number."""
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "train_mlp8.py")
    spec = importlib.util.spec_from_file_location("train_mlp8", path)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    losses = example.train(workers=2, steps=4, width=64, hidden=128, tokens=100, products="e4m3", optimizer="adamw8")
    assert len(losses) == 4 and all(v == v and v < float("inf") for v in losses)


# ---- refusals on the GPU's side of the package ---------------------------------------------------

def test_refusals(gq):
    x = torch.randn((40, 300), device="cuda")
    w = torch.randn((70, 300), device="cuda")
    f, rows = gq.gq_fp8_quantize(w, tiles=True), gq.gq_fp8_quantize(w)
    c, e, t = f.codes, f.exps, f.exps_t
    whole = gq.Fp8(c, e, 300, exps_t=t)
    assert torch.equal(gq.gq_fp8_linear(x, whole), gq.gq_fp8_linear(x, f))
    with pytest.raises(ValueError):
        gq.Fp8(c[:, :300], e, 300)
    with pytest.raises(ValueError):
        gq.Fp8(c, e[:, :, :16], 300)
    with pytest.raises(ValueError):
        gq.Fp8(c, e, 300, exps_t=t[:1])
    with pytest.raises(TypeError):
        gq.Fp8(c, e.float(), 300)
    with pytest.raises(ValueError):
        gq.gq_fp8_linear(x, gq.Fp8(c.cpu(), e, 300))
    with pytest.raises(ValueError):
        gq.gq_fp8_linear(x[:, :299], f)                      # another depth
    with pytest.raises(ValueError):
        gq.gq_fp8_linear(f, f)                               # tokens in tiles
    with pytest.raises(ValueError):
        gq.gq_fp8_linear_dgrad(x[:, :70].contiguous(), rows)  # no exponents of the transposed matrix
    with pytest.raises(TypeError):
        gq.gq_fp8_linear(x.half(), f)
    with pytest.raises(TypeError):
        gq.gq_fp8_linear(x, f, out_dtype=torch.float16)
    with pytest.raises(TypeError):
        gq.gq_fp8_linear(x, w)
    with pytest.raises(TypeError):
        gq.gq_fp8_linear(x, f, bias=torch.zeros(70, device="cuda", dtype=torch.bfloat16))
    with pytest.raises(ValueError):
        gq.gq_fp8_linear(x, f, bias=torch.zeros(71, device="cuda"))
    with pytest.raises(ValueError):
        gq.gq_fp8_linear(x.cpu(), f)
    for shape in ((1, 300), (40, 2, 300), ()):               # not that of its rows
        q = gq.gq_fp8_quantize(x)
        with pytest.raises(ValueError):
            gq.gq_fp8_linear(gq.Fp8(q.codes, q.exps, 300, shape=shape), f)
    with pytest.raises(ValueError):
        gq.gq_fp8_quantize(x.t()[::2])
    with pytest.raises(ValueError):
        gq.gq_fp8_dequantize(f, out=torch.empty((70, 299), device="cuda"))

    p, g = torch.zeros(100, device="cuda"), torch.ones(100, device="cuda")
    s = gq.gq_adamw_state(100)
    pair = (torch.zeros(100, device="cuda"), torch.zeros(100, device="cuda"))
    step = gq.gq_adamw_step
    for bad in (dict(step=0), dict(betas=(1.0, 0.9)), dict(eps=-1.0), dict(max_norm=1.0), dict(first=-1),
                dict(norm=torch.ones(2, device="cuda")), dict(seed=-1), dict(seed=1 << 64),
                dict(step=torch.ones(1, device="cuda", dtype=torch.int64).cpu())):
        with pytest.raises((ValueError, TypeError)):
            step([p], [g], [s], bad.pop("step", 1), **bad)
    for params, grads, states in (([p], [g, g], [s]), ([p], [g[:99]], [s]), ([p], [g], [gq.gq_adamw_state(200)]),
                                  ([p, p], [g, g], [s, gq.gq_adamw_state(100)]), ([p, g], [g, g], [s, s]),
                                  ([p[::2]], [g[::2]], [gq.gq_adamw_state(50)]), ([p], [g.cpu()], [s]),
                                  ([p, p + 1], [g, g], [s, pair]), ([p.half()], [g], [s]),
                                  ([p], [g], [(pair[0], pair[1].double())]), ([p], [g], [pair[0]])):
        with pytest.raises((ValueError, TypeError)):
            step(params, grads, states, 1)
    assert not p.any() and not s.m.any()
    with pytest.raises(ValueError):
        gq.gq_tensors_norm([])
    with pytest.raises(TypeError):
        gq.gq_tensors_norm([p, p.bfloat16()])
    with pytest.raises(TypeError):
        gq.gq_tensors_norm(p)
    with pytest.raises(ValueError):
        gq.gq_adamw_values([s], out=([torch.empty(50, device="cuda")], [torch.empty(50, device="cuda")]))
    step([], [], [], 1)
