"""Checkpoints as Python objects, and the layers over them in the uses of a training program: copies,
second derivatives, memory, frozen parameters, seeds."""
import copy
import pickle

import pytest

from gpu_common import gq_module

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def gq():
    return gq_module()


# ---- a checkpoint follows its tensors --------------------------------------------------------

def everywhere(gq, act, dy):
    """What every operator that reads a checkpoint makes of it."""
    rstd = torch.ones(act.rows, device="cuda")
    return [gq.gq_act_dequantize(act), *gq.gq_layernorm_backward(dy, None, rstd, act=act),
            *gq.gq_gelu_backward(dy, act, need_output=True), *gq.gq_linear_wgrad(dy, act)]


@pytest.mark.parametrize("made", ["by a call", "from tensors"])
@pytest.mark.parametrize("duplicate", [copy.deepcopy, lambda a: pickle.loads(pickle.dumps(a))],
                         ids=["deepcopy", "pickle"])
def test_a_copied_checkpoint_is_read_from_its_own_memory(gq, duplicate, made):
    """The original is overwritten, not freed: its copy still reads as before."""
    x = torch.randn((40, 96), device="cuda")
    dy = torch.randn((40, 96), device="cuda")
    act = gq.gq_act_quantize(x)
    if made == "from tensors":
        act = gq.Act8(act.codes.clone(), act.exps.clone(), 96)
    want = everywhere(gq, act, dy)
    other = duplicate(act)
    act.codes.zero_()
    act.exps.fill_(1)
    assert other.shape == act.shape and other.rows == 40 and other.cols == 96
    for a, b in zip(everywhere(gq, other, dy), want):
        assert torch.equal(a, b)
    assert not gq.gq_act_dequantize(act).any()


def test_a_checkpoint_follows_new_storage(gq):
    """codes and exponents given new storage are read from there (the old one stays allocated)."""
    x = torch.randn((8, 64), device="cuda")
    a, b = gq.gq_act_quantize(x), gq.gq_act_quantize(2 * x.flip(0))
    codes, exps = a.codes.clone(), a.exps.clone()
    old = codes.detach(), exps.detach()
    act = gq.Act8(codes, exps, 64)
    codes.data, exps.data = b.codes.clone(), b.exps.clone()
    assert torch.equal(gq.gq_act_dequantize(act), gq.gq_act_dequantize(b))
    assert old[0].numel() and old[1].numel()


def test_a_checkpoint_whose_tensors_no_longer_hold_it_is_refused(gq):
    x = torch.randn((8, 64), device="cuda")
    made = gq.gq_act_quantize(x)
    for part in (0, 1):
        parts = [made.codes.clone(), made.exps.clone()]
        keep = [p.detach() for p in parts]
        act = gq.Act8(*parts, 64)
        parts[part].data = parts[part][:7].clone()  # a row short
        with pytest.raises(ValueError):
            gq.gq_act_dequantize(act)
        assert keep[part].numel()
        parts[part].data = made.codes.cpu() if part == 0 else made.exps.cpu()
        with pytest.raises(ValueError):
            gq.gq_act_dequantize(act)


# ---- the layers ------------------------------------------------------------------------------

@pytest.fixture(scope="module")
def layers(gq):
    from allreduce_compatible_gradient_gb300 import act8_layers
    return act8_layers


def block_of(layers, width=96, hidden=200, **kw):
    torch.manual_seed(3)
    block = layers.MlpBlock8(width, hidden, device="cuda", **kw)
    with torch.no_grad():
        for p in block.parameters():
            p += 0.1 * torch.randn_like(p)
    return block


def exact_gradients(block, x, r):
    """Autograd's, in fp64, of sum(block(x) r)."""
    p = {k: v.detach().double().requires_grad_() for k, v in block.named_parameters()}
    x = x.detach().double().requires_grad_()
    y = torch.nn.functional.layer_norm(x, x.shape[-1:], p["norm_weight"], p["norm_bias"], block.eps)
    h = torch.nn.functional.gelu(y @ p["w1"].t() + p["b1"], approximate=block.approximate)
    out = x + h @ p["w2"].t() + p["b2"]
    return dict(zip(["x", *p], torch.autograd.grad((out * r.double()).sum(), [x, *p.values()])))


@pytest.fixture
def calls(layers, monkeypatch):
    """(name, arguments, result) of every operator that the layers call."""
    seen = []

    def record(name):
        call = getattr(layers.ops, name)

        def recorded(*a, **kw):
            out = call(*a, **kw)
            seen.append((name, a, kw, out))
            return out
        monkeypatch.setattr(layers.ops, name, recorded)
    for name in ("gq_layernorm_forward", "gq_layernorm_backward", "gq_gelu_forward", "gq_gelu_backward",
                 "gq_linear_wgrad"):
        record(name)
    return seen


def test_a_second_derivative_is_refused(layers):
    """The operators of the backward pass are not differentiable: a gradient penalty is refused, not
    computed without their part."""
    block, x = block_of(layers), torch.randn((10, 96), device="cuda", requires_grad=True)
    g, = torch.autograd.grad(block(x).square().sum(), x, create_graph=True)
    with pytest.raises(RuntimeError, match="once_differentiable"):
        g.square().sum().backward()


def test_checkpoints_are_freed_by_the_backward_pass(layers):
    """As autograd's saved tensors are: not when the loss goes, which most loops hold into the next step."""
    block = block_of(layers, 256, 1024)
    x = torch.randn((4096, 256), device="cuda", dtype=torch.bfloat16)
    saved = 4096 * (256 + 1024)  # bytes of codes

    def step():
        loss = block(x).float().sum()
        loss.backward()
        return loss
    step()  # gradients and library workspaces are there from here on
    torch.cuda.synchronize()
    before = torch.cuda.memory_allocated()
    loss = step()
    assert torch.cuda.memory_allocated() - before < saved / 4
    assert loss.isfinite()


def test_saved_tensor_hooks_see_the_checkpoints(layers):
    """Offloaded to the host and brought back, they give the same gradients."""
    block = block_of(layers)
    x = torch.randn((150, 96), device="cuda", dtype=torch.bfloat16)
    sizes = []

    def gradients():
        return torch.autograd.grad(block(x).float().square().sum(), list(block.parameters()))

    def pack(t):
        sizes.append(t.nbytes)
        return t.cpu()
    want = gradients()
    with torch.autograd.graph.saved_tensors_hooks(pack, lambda t: t.cuda()):
        got = gradients()
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    # codes of 96 and of round_up(200, 32) bytes a row, 16 exponent bytes a row each
    assert sizes.count(150 * (96 + 16)) == 1 and sizes.count(150 * (224 + 16)) == 1


def test_a_graph_that_is_kept_gives_the_same_gradients_again(layers):
    block = block_of(layers)
    loss = block(torch.randn((20, 96), device="cuda")).square().sum()
    first = torch.autograd.grad(loss, list(block.parameters()), retain_graph=True)
    for a, b in zip(first, torch.autograd.grad(loss, list(block.parameters()))):
        assert torch.equal(a, b)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_bf16_parameters(layers, dtype):
    """Gradients of a block whose parameters are bf16: 2 % of the norm as in the fp32 block's test, and
    2^-8 for their own rounding."""
    block = block_of(layers, seed=5).bfloat16()
    x = torch.randn((2, 75, 96), device="cuda").to(dtype).requires_grad_()
    r = torch.randn((2, 75, 96), device="cuda")
    got = torch.autograd.grad((block(x).float() * r).sum(), [x, *block.parameters()])
    for g, p, (name, w) in zip(got, [x, *block.parameters()], exact_gradients(block, x, r).items()):
        assert g.dtype == p.dtype and g.shape == p.shape
        assert (g.double() - w).norm() < (0.02 + 2.0 ** -8) * w.norm(), name


def test_no_checkpoints_without_a_backward_pass(layers, calls):
    """Under no_grad, and where nothing requires a gradient; the outputs are the same."""
    block, x = block_of(layers), torch.randn((70, 96), device="cuda", dtype=torch.bfloat16)

    def checkpoints():
        made = [out[-1] is not None for name, _, _, out in calls if name.endswith("forward")]
        calls.clear()
        return made
    want = block(x)
    assert checkpoints() == [True, True]
    with torch.no_grad():
        assert torch.equal(block(x), want)
    assert checkpoints() == [False, False]
    block.requires_grad_(False)
    assert torch.equal(block(x), want)
    assert checkpoints() == [False, False]
    block.b2.requires_grad_()  # whose gradient needs no activation
    assert torch.equal(block(x), want)
    assert checkpoints() == [False, False]
    block.w2.requires_grad_()
    assert torch.equal(block(x), want)
    assert checkpoints() == [False, True]


@pytest.mark.parametrize("wanted,called", [
    (["b2"], []), (["w2"], ["gelu"]), (["b1"], ["gelu"]), (["w1"], ["gelu", "wgrad"]),
    (["w1", "b1"], ["gelu", "wgrad"]), (["norm_weight"], ["gelu", "norm"]), (["norm_bias", "w2"], ["gelu", "norm"]),
    (["x"], ["gelu", "norm"]), (["x", "b1", "b2"], ["gelu", "norm"]),
    (["norm_weight", "norm_bias", "w1", "b1", "w2", "b2"], ["gelu", "wgrad", "norm"])])
def test_frozen_parameters_cost_no_gradient(layers, calls, wanted, called):
    """Only what requires a gradient gets one, the same one as when all do, and operators whose results
    nobody wants are not called."""
    block = block_of(layers)
    x = torch.randn((70, 96), device="cuda", dtype=torch.bfloat16, requires_grad=True)
    r = torch.randn((70, 96), device="cuda")
    leaves = dict(x=x, **dict(block.named_parameters()))

    def gradients():
        names = [k for k, v in leaves.items() if v.requires_grad]
        loss = (block(x).float() * r).sum()
        return dict(zip(names, torch.autograd.grad(loss, [leaves[k] for k in names])))
    want = gradients()
    for k, v in leaves.items():
        v.requires_grad_(k in wanted)
    calls.clear()
    got = gradients()
    assert set(got) == set(wanted)
    for k, g in got.items():
        # (a bias' gradient alone is a plain sum, of another order)
        exact = k != "b1" or "w1" in wanted
        assert torch.equal(g, want[k]) if exact else torch.allclose(g, want[k], rtol=1e-3, atol=1e-4)
    short = {"gq_gelu_backward": "gelu", "gq_linear_wgrad": "wgrad", "gq_layernorm_backward": "norm"}
    assert [short[n] for n, *_ in calls if n in short] == called


# ---- random words ------------------------------------------------------------------------------

def errors(calls, gq):
    """Rounding errors of the checkpoints made since the last time, in steps of their blocks."""
    out = []
    for name, a, kw, got in calls:
        if name == "gq_gelu_forward" and got[1] is not None:
            act = got[1]
            step = torch.ldexp(torch.ones((), device="cuda"), act.exps[:, :act.codes.shape[1] // 32].int() - 127)
            step = step.repeat_interleave(32, dim=1)[:, :act.cols]
            out.append((gq.gq_act_dequantize(act, out_dtype=torch.float32) - a[0].float()) / step)
    calls.clear()
    return out


def test_blocks_do_not_share_their_rounding(gq, layers, calls):
    """Two blocks made alike, ranks and steps of one: errors of 70 x 200 roundings of the same numbers are
    uncorrelated within 5 / sqrt(14,000), where the same words make them equal."""
    a, b = (layers.MlpBlock8(96, 200, device="cuda") for _ in range(2))
    b.load_state_dict(a.state_dict())
    x = torch.randn((70, 96), device="cuda")
    a(x), b(x)
    a.rank = 1
    a(x)
    a.step = 1
    a(x)
    got = errors(calls, gq)
    assert len(got) == 4
    for i in range(4):
        for j in range(i):
            e, f = got[i] - got[i].mean(), got[j] - got[j].mean()
            assert abs((e * f).sum() / (e.norm() * f.norm())) < 5 / 14000 ** 0.5
    a(x)
    assert torch.equal(errors(calls, gq)[0], got[3])  # the same words again


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_inputs_of_any_strides(layers, dtype):
    """A transposed matrix, a broadcast row, every second column: as their contiguous copies."""
    block = block_of(layers)
    base = torch.randn((96, 40), device="cuda").to(dtype)
    for x in (base.t(), base.t()[:1].expand(40, 96), torch.randn((40, 192), device="cuda").to(dtype)[:, ::2],
              base.t().reshape(2, 20, 96).transpose(0, 1)):
        results = []
        for v in (x, x.contiguous()):
            v = v.detach().requires_grad_()
            out = block(v)
            results.append([out, *torch.autograd.grad(out.float().square().sum(), [v, *block.parameters()])])
        for a, b in zip(*results):
            assert torch.equal(a, b)


def test_gradient_of_the_second_weight_is_not_rounded_to_bf16(layers, calls):
    """An fp32 parameter's gradient from bf16 operands carries the error of their sum alone, which the
    tensor cores may truncate 2^-22 of the largest partial sum per 16 products; nothing of bf16's 2^-9."""
    block = block_of(layers)
    x = torch.randn((150, 96), device="cuda", dtype=torch.bfloat16)
    r = torch.randn((150, 96), device="cuda").bfloat16()
    dw2, db2 = torch.autograd.grad((block(x) * r).sum(), [block.w2, block.b2])
    h, = [out[1] for name, _, _, out in calls if name == "gq_gelu_backward"]
    d, h = r.double(), h.double()
    mag = d.abs().t() @ h.abs()
    assert dw2.dtype == db2.dtype == torch.float32
    assert ((dw2.double() - d.t() @ h).abs() <= (150 / 16 + 32) * 2.0 ** -22 * mag).all()
    assert ((db2.double() - d.sum(0)).abs() <= 190 * 2.0 ** -24 * d.abs().sum(0)).all()


# ---- infinities ------------------------------------------------------------------------------

WIDTHS = [1, 8, 40, 96, 200, 256, 264, 512, 520, 768, 1000, 1024, 1030, 2048, 2056, 3000, 4096, 5000, 8192, 8200, 9001]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("cols", WIDTHS)
def test_layernorm_of_an_infinity(gq, cols, dtype):
    """The mean of a row that holds an infinity is that infinity, wherever it stands; its rstd and outputs
    are NaN.  The other rows are as without it."""
    x = torch.randn((9, cols), device="cuda").to(dtype)
    y0, mean0, rstd0, _ = gq.gq_layernorm_forward(x)
    x[2, 0], x[5, cols - 1], x[7, cols // 2] = float("inf"), float("-inf"), float("inf")
    y, mean, rstd, act = gq.gq_layernorm_forward(x)
    assert mean[[2, 5, 7]].tolist() == [float("inf"), float("-inf"), float("inf")]
    rest = [0, 1, 3, 4, 6, 8]
    assert y[[2, 5, 7]].isnan().all() and rstd[[2, 5, 7]].isnan().all()
    assert gq.gq_act_dequantize(act)[[2, 5, 7]].isnan().all()
    assert torch.equal(y[rest], y0[rest]) and torch.equal(mean[rest], mean0[rest])
    assert torch.equal(rstd[rest], rstd0[rest])


@pytest.mark.parametrize("source", ["codes", "input"])
@pytest.mark.parametrize("cols", WIDTHS[1:])
def test_layernorm_backward_of_an_infinite_gradient(gq, cols, source):
    """dx of its row follows the formula's own infinities and NaNs; other rows and columns are finite."""
    x = torch.randn((9, cols), device="cuda")
    x[4] = x[4].abs()
    w = 0.5 + torch.rand(cols, device="cuda")
    _, mean, rstd, act = gq.gq_layernorm_forward(x, w)
    dy = torch.randn((9, cols), device="cuda")
    dy[4, 0] = float("inf")
    if source == "codes":
        got = gq.gq_layernorm_backward(dy, w, rstd, act=act)
        hat = gq.gq_act_dequantize(act, out_dtype=torch.float32).double()
    else:
        got = gq.gq_layernorm_backward(dy, w, rstd, x=x, mean=mean)
        hat = (x - mean[:, None]).double() * rstd.double()[:, None]
    g = dy.double() * w.double()
    want = rstd.double()[:, None] * (g - g.mean(1, keepdim=True) - hat * (g * hat).mean(1, keepdim=True))
    for kind in (torch.isnan, torch.isposinf, torch.isneginf):
        assert torch.equal(kind(got[0]), kind(want))
    others = [0, 1, 2, 3, 5, 6, 7, 8]
    assert got[0][others].isfinite().all()
    assert got[2][0].isinf() and got[2][1:].isfinite().all() and got[1][1:].isfinite().all()


# ---- launches that overlap -------------------------------------------------------------------

def test_sums_of_an_overlapping_launch_are_its_own(gq):
    """Back to back calls in one workspace, whose launches start before those ahead of them have ended:
    every result is that of the call alone, bit for bit."""
    shapes = [(600, 384, 256), (5000, 520, 264), (130, 70, 33)]
    for rows, outs, cols in shapes:
        x = torch.randn((rows, cols), device="cuda")
        act, shift = gq.gq_act_quantize(x), torch.randn(cols, device="cuda")
        rstd = torch.rand(rows, device="cuda")
        grads = [torch.randn((rows, outs), device="cuda").bfloat16() * 10.0 ** i for i in range(4)]
        dys = [torch.randn((rows, cols), device="cuda").bfloat16() * 10.0 ** i for i in range(4)]
        want = []
        for g, d in zip(grads, dys):
            one = [*gq.gq_linear_wgrad(g, act, shift=shift), *gq.gq_layernorm_backward(d, None, rstd, act=act)]
            torch.cuda.synchronize()
            want.append(one)
        ws = [torch.empty(gq.gq_linear_wgrad_workspace_bytes(grads[0], cols), dtype=torch.uint8, device="cuda"),
              torch.empty(gq.gq_layernorm_workspace_bytes(rows, cols), dtype=torch.uint8, device="cuda")]
        got = []
        for i in range(40):
            got.append([*gq.gq_linear_wgrad(grads[i % 4], act, shift=shift, ws=ws[0]),
                        *gq.gq_layernorm_backward(dys[i % 4], None, rstd, act=act, ws=ws[1])])
        for i, one in enumerate(got):
            for a, b in zip(one, want[i % 4]):
                assert torch.equal(a, b)


@pytest.mark.parametrize("shape,ok", [([2, 20, 96], True), (torch.Size([40, 96]), True), (None, False), (7, False),
                                      ([40, "96"], False), ([40, 95], False), ([-1, 96], False), ([3840], False)])
def test_a_checkpoints_shape_may_be_any_sequence(gq, shape, ok):
    """`shape` is an attribute that a program can set: a list is taken, what is no shape is refused."""
    act = gq.gq_act_quantize(torch.randn((40, 96), device="cuda"))
    act.shape = shape
    if ok:
        assert gq.gq_act_dequantize(act).shape == torch.Size(shape)
    else:
        with pytest.raises((TypeError, ValueError, RuntimeError)):
            gq.gq_act_dequantize(act)


# ---- workspaces ------------------------------------------------------------------------------

@pytest.mark.parametrize("rows,cols", [(1, 8200), (9, 8193), (1030, 9000), (40, 16384), (300, 8192)])
def test_layernorm_backward_stays_in_its_workspace(gq, rows, cols):
    x = torch.randn((rows, cols), device="cuda").bfloat16()
    _, _, rstd, act = gq.gq_layernorm_forward(x)
    n = gq.gq_layernorm_workspace_bytes(rows, cols)
    full = torch.full((n + 8192,), 77, dtype=torch.uint8, device="cuda")
    want = gq.gq_layernorm_backward(x, None, rstd, act=act)
    got = gq.gq_layernorm_backward(x, None, rstd, act=act, ws=full[4096:-4096])
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    assert (full[:4096] == 77).all() and (full[-4096:] == 77).all()


# ---- other uses ------------------------------------------------------------------------------

@pytest.mark.parametrize("shape", [(0, 96), (2, 0, 96), (96,), (1, 96), (3, 1, 96)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_inputs_without_rows_and_single_rows(layers, shape, dtype):
    block = block_of(layers)
    x = torch.randn(shape, device="cuda").to(dtype).requires_grad_()
    out = block(x)
    got = torch.autograd.grad(out.float().sum(), [x, *block.parameters()])
    assert out.shape == x.shape
    for g, p in zip(got, [x, *block.parameters()]):
        assert g.shape == p.shape and g.isfinite().all()
        assert x.numel() or not g.any()


@pytest.mark.parametrize("reentrant", [True, False])
def test_recomputed_blocks_give_the_same_gradients(layers, reentrant):
    """torch.utils.checkpoint over a block: the first pass or the second makes the checkpoints."""
    from torch.utils.checkpoint import checkpoint
    block = block_of(layers)
    x = torch.randn((40, 96), device="cuda", requires_grad=True)
    want = torch.autograd.grad(block(x).square().sum(), [x, *block.parameters()])
    checkpoint(block, x, use_reentrant=reentrant).square().sum().backward()
    for p, w in zip([x, *block.parameters()], want):
        assert torch.equal(p.grad, w)


def test_a_captured_step_replays(layers):
    block = block_of(layers)
    x = torch.randn((40, 96), device="cuda", requires_grad=True)

    def step():
        return torch.autograd.grad(block(x).square().sum(), [x, *block.parameters()])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        want = step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for g in got:
        g.zero_()
    graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)
