"""Paths of the activation operators that need sizes, alignments or callers of their own: chains of
accumulations in the weight gradient, vectors that are not 16-byte aligned, calls on several streams and
from several threads, the layers under the gradients' communication hook.

Tolerances as in test_gpu_activations.py, where its header derives them.
"""
import datetime
import socket
import threading

import numpy as np
import pytest

import activation_ref as ref
from gpu_common import gq_module
from test_gpu_activations import U, host, inputs, near, tensor, types

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def gq():
    return gq_module()


# ---- chains of the weight gradient -----------------------------------------------------------

def wgrad_case(gq, rows, outs, cols, dtype, extra=0):
    g = torch.Generator(device="cuda").manual_seed(rows + outs)
    x = torch.randn((rows, cols), generator=g, device="cuda")
    full = torch.zeros((rows, outs + extra), device="cuda", dtype=types(torch, dtype))
    full[:, :outs] = torch.randn((rows, outs), generator=g, device="cuda") * 1e-2
    scale = 1 + 0.3 * torch.randn(cols, generator=g, device="cuda")
    shift = torch.randn(cols, generator=g, device="cuda")
    return full[:, :outs], gq.gq_act_quantize(x), scale, shift


# tile: 512 for pairs of blocks; own, left: whole tiles of each share, and tiles that they divide
CHAINS = [(7000, 4096, 2600, "bf16", "f32", False, 0, 512, True, True),
          (7000, 4096, 2601, "bf16", "bf16", True, 0, 512, True, True),   # rows of dw that are not aligned
          (9000, 2048, 4096, "bf16", "bf16", True, 3, 512, True, False),  # packed dy
          (16384, 100, 8192, "bf16", "f32", True, 0, 128, False, True),
          (16384, 64, 4096, "f32", "f32", False, 0, 128, False, True),    # three parts of dy
          (12800, 70, 20000, "bf16", "f32", True, 0, 128, True, True)]


@pytest.mark.parametrize("rows,outs,cols,dtype,out,affine_part,extra,tile,own,left", CHAINS)
def test_linear_wgrad_of_several_chains(gq, rows, outs, cols, dtype, out, affine_part, extra, tile, own, left):
    """Tiles whose steps take more than one accumulation, whole or divided between shares, against a
    64-bit product; the plan says that they are such."""
    dy, act, scale, shift = wgrad_case(gq, rows, outs, cols, dtype, extra)
    plan = gq.gq_linear_wgrad_plan(dy, cols)
    assert plan["tile_outs"] == tile and plan["longest"] > plan["chain"]
    assert (plan["own"] > 0) == own and (plan["left"] > 0) == left
    kw = dict(scale=scale, shift=shift) if affine_part else {}
    dw, db = gq.gq_linear_wgrad(dy, act, out_dtype=types(torch, out), **kw)
    v, d = gq.gq_act_dequantize(act, out_dtype=torch.float32).double(), dy.double()
    s64 = scale.double() if affine_part else torch.ones(cols, device="cuda", dtype=torch.float64)
    h64 = shift.double() if affine_part else torch.zeros_like(s64)
    want = (d.t() @ v) * s64 + torch.outer(d.sum(0), h64)
    steps = 3 * rows if dtype == "f32" else rows
    bias = d.abs().sum(0)
    tolb = (rows + 40) * U * bias
    tol = ((steps / 16 + 32) * 2.0 ** -22 + 4 * U) * (d.abs().t() @ v.abs()) * s64.abs() + \
        torch.outer(tolb + 4 * U * bias, h64.abs()) + (2.0 ** -8 if out == "bf16" else U) * want.abs()
    assert ((dw.double() - want).abs() <= tol).all()
    assert ((db.double() - d.sum(0)).abs() <= tolb).all()
    again, _ = gq.gq_linear_wgrad(dy, act, out_dtype=types(torch, out), **kw)
    assert torch.equal(dw, again)


def test_linear_wgrad_error_is_that_of_short_chains(gq):
    """The error of one accumulation grows with its length: 5.8e-6 of the result's norm over 256 steps of
    such inputs, so 2.2e-6 over the 96 of a chain.  Within 1.5 times that; chains of 150 steps, or a single
    one, are not."""
    rows, outs, cols = 16384, 4096, 4096
    dy, act, _, _ = wgrad_case(gq, rows, outs, cols, "bf16")
    plan = gq.gq_linear_wgrad_plan(dy, cols)
    assert plan["longest"] == 256 and plan["own"] > 0 and plan["left"] > 0
    dw, _ = gq.gq_linear_wgrad(dy, act)
    want = dy.double().t() @ gq.gq_act_dequantize(act, out_dtype=torch.float32).double()
    assert (dw.double() - want).norm() <= 1.5 * 5.8e-6 / 256 * 96 * want.norm()


def test_linear_wgrad_special_values_in_later_chains(gq):
    """A NaN block and an infinite gradient among the last tokens reach what they touch, and nothing else."""
    dy, act, _, shift = wgrad_case(gq, 16384, 100, 8192, "bf16")
    act.exps[16300, 5] = 255
    act.codes[16300, 160:192] = 0
    dy[16000, 7] = float("inf")
    dw, db = gq.gq_linear_wgrad(dy, act, shift=shift)
    assert dw[:, 160:192].isnan().all()
    assert not dw[7].isfinite().any() and db[7].isinf()
    rest = [i for i in range(100) if i != 7]
    assert dw[rest][:, :160].isfinite().all() and dw[rest][:, 192:].isfinite().all()
    assert db[rest].isfinite().all()


@pytest.mark.parametrize("rows,outs,cols", [
    (4096, 1024, 4096), (4096, 4096, 1024), (1024, 768, 768), (384, 768, 768), (100, 4096, 4096), (20000, 700, 700)])
def test_linear_wgrad_plan_adds_up(gq, rows, outs, cols):
    """Tiles and shares of ordinary sizes: every step in one share, and the result is the product."""
    dy, act, _, _ = wgrad_case(gq, rows, outs, cols, "bf16")
    p = gq.gq_linear_wgrad_plan(dy, cols)
    tiles = -(-outs // p["tile_outs"]) * -(-cols // p["tile_cols"])
    assert p["own"] * p["shares"] + p["left"] == tiles and p["steps"] == -(-rows // 64)
    dw, _ = gq.gq_linear_wgrad(dy, act)
    v, d = gq.gq_act_dequantize(act, out_dtype=torch.float32).double(), dy.double()
    assert ((dw.double() - d.t() @ v).abs() <= (rows / 16 + 32) * 2.0 ** -22 * (d.abs().t() @ v.abs())).all()


# ---- vectors that are not 16-byte aligned ----------------------------------------------------

def shifted(t, by=1):
    """t's values in memory that begins `by` elements behind a 16-byte boundary."""
    full = torch.empty(t.numel() + 8, dtype=t.dtype, device="cuda")
    assert full.data_ptr() % 16 == 0
    full[by:by + t.numel()] = t
    return full[by:by + t.numel()]


@pytest.mark.parametrize("vectors", ["f32", "bf16"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,cols", [(3, 8), (400, 96), (9, 256), (400, 768), (19, 1024), (320, 4096), (3, 8192),
                                       (2, 8200), (2, 16384)])
def test_layernorm_with_unaligned_vectors(gq, rows, cols, dtype, vectors):
    """weight, bias, dweight and dbias of aligned rows, one element behind an aligned address."""
    x, xv = tensor(torch, inputs(rows, cols, rows + cols), dtype)
    dy, dyv = tensor(torch, inputs(rows, cols, rows + 3 * cols, 1e-2), dtype)
    r = np.random.default_rng(cols)
    w, b = (shifted(torch.tensor(a, dtype=torch.float32, device="cuda").to(types(torch, vectors)))
            for a in (1 + 0.3 * r.standard_normal(cols), 0.5 * r.standard_normal(cols)))
    wv, bv = host(w), host(b)
    y, mean, rstd, act = gq.gq_layernorm_forward(x, w, b)
    wy, wm, wr, hat = ref.layernorm(xv, wv, bv, 1e-5)
    size = np.abs(xv).mean(axis=1)
    dm = ((cols + 2) * U * size + U * np.abs(xv).max(axis=1)) * wr
    rel = (cols + 8) * U + 2 * dm
    tol = np.abs(hat * wv) * (rel[:, None] + 4 * U) + np.abs(wv) * dm[:, None] + 2 * U * np.abs(bv)
    near(host(y), wy, tol, dtype)
    near(host(mean), wm, (cols + 2) * U * size, "f32")
    near(host(rstd), wr, rel * wr, "f32")
    # through the C interface, so that the sums' addresses are unaligned too
    L, kind = gq.lib(), {"f32": 0, "bf16": 1}
    dx = torch.empty_like(dy)
    dw, db = (shifted(torch.zeros(cols, device="cuda", dtype=types(torch, vectors))) for _ in range(2))
    n = gq.gq_layernorm_workspace_bytes(rows, cols)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    assert L.gq_layernorm_backward(dy.data_ptr(), kind[dtype], rows, cols, cols, w.data_ptr(), kind[vectors],
                                   rstd.data_ptr(), act.codes.data_ptr(), act.exps.data_ptr(), None, 0, None,
                                   dx.data_ptr(), cols, dw.data_ptr(), db.data_ptr(), kind[vectors],
                                   ws.data_ptr(), n, torch.cuda.current_stream().cuda_stream) == 0
    hat, rv = ref.values(act.codes.cpu().numpy(), act.exps.cpu().numpy(), cols), host(rstd)
    wx, ww, wb = ref.layernorm_backward(dyv, wv, rv, hat)
    g = np.abs(dyv * wv)
    m1, m2 = g.mean(axis=1, keepdims=True), (g * np.abs(hat)).mean(axis=1, keepdims=True)
    n = (cols + 8) * U
    tol = rv[:, None] * (4 * U * g + n * m1 + np.abs(hat) * n * m2 + 4 * U * (m1 + np.abs(hat) * m2))
    near(host(dx), wx, tol, dtype)
    n = (rows + 40) * U
    near(host(dw), ww, n * (np.abs(dyv) * np.abs(hat)).sum(axis=0), vectors)
    near(host(db), wb, n * np.abs(dyv).sum(axis=0), vectors)


@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("rows,outs,cols", [(1, 8, 8), (70, 40, 96), (500, 256, 264), (2100, 1024, 1024),
                                            (4096, 1024, 4096)])
def test_linear_wgrad_with_unaligned_vectors(gq, rows, outs, cols, out):
    """scale, shift and dbias one element behind an aligned address: the same bits as aligned ones give."""
    dy, act, scale, shift = wgrad_case(gq, rows, outs, cols, "bf16")
    t = types(torch, out)
    want, wb = gq.gq_linear_wgrad(dy, act, scale=scale, shift=shift, out_dtype=t)
    for s, h in ((shifted(scale), shift), (scale, shifted(shift)), (shifted(scale, 3), shifted(shift, 2))):
        got, db = gq.gq_linear_wgrad(dy, act, scale=s, shift=h, out_dtype=t)
        assert torch.equal(got, want) and torch.equal(db, wb)
    got, _ = gq.gq_linear_wgrad(dy, act, scale=shifted(scale), out_dtype=t)
    assert torch.equal(got, gq.gq_linear_wgrad(dy, act, scale=scale, out_dtype=t)[0])


# ---- streams and threads ---------------------------------------------------------------------

def step_of(gq, i):
    """A call of every operator on inputs of its own; its results."""
    g = torch.Generator(device="cuda").manual_seed(i)
    x = torch.randn((700 + i, 512), generator=g, device="cuda").bfloat16()
    dy = torch.randn((700 + i, 384), generator=g, device="cuda").bfloat16()
    w = torch.randn(512, generator=g, device="cuda")

    def run(**kw):
        y, mean, rstd, act = gq.gq_layernorm_forward(x, w, w, seed=i, step=i, **kw)
        h, ga = gq.gq_gelu_forward(y, **kw)
        du, h2 = gq.gq_gelu_backward(h, ga, need_output=True, **kw)
        return [y, mean, rstd, h, du, h2, gq.gq_act_dequantize(act, **kw),
                *gq.gq_layernorm_backward(du, w, rstd, act=act, **kw),
                *gq.gq_linear_wgrad(dy, act, scale=w, shift=w, **kw)]
    return run


def test_calls_on_two_streams_at_once(gq):
    runs = [step_of(gq, i) for i in range(2)]
    want = [run() for run in runs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in runs]
    got = []
    for _ in range(20):
        got.append([run(stream=s) for run, s in zip(runs, streams)])
    torch.cuda.synchronize()
    for both in got:
        for a, b in zip(both, want):
            assert all(torch.equal(p, q) for p, q in zip(a, b))


def test_calls_from_several_threads(gq):
    runs = [step_of(gq, i) for i in range(4)]
    want = [run() for run in runs]
    torch.cuda.synchronize()
    failures = []

    def work(i):
        try:
            s = torch.cuda.Stream()
            for _ in range(20):
                got = runs[i](stream=s)
                s.synchronize()
                assert all(torch.equal(p, q) for p, q in zip(got, want[i]))
        except BaseException as e:  # noqa: B036 - reported below
            failures.append((i, e))
    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failures, failures


# ---- the layers under the communication hook -------------------------------------------------

def test_layers_under_the_communication_hook(gq):
    """Two blocks in DistributedDataParallel (one rank): their gradients arrive through the hook, each
    within a level of its bucket's largest magnitude."""
    import torch.distributed as dist
    from allreduce_compatible_gradient_gb300 import comm_hook
    from allreduce_compatible_gradient_gb300.act8_layers import MlpBlock8
    with socket.socket() as s:
        s.bind(("127.0.0.1", 0))
        port = s.getsockname()[1]
    dist.init_process_group("nccl", init_method="tcp://127.0.0.1:%d" % port, rank=0, world_size=1,
                            timeout=datetime.timedelta(seconds=60))
    try:
        torch.manual_seed(0)
        model = torch.nn.Sequential(*[MlpBlock8(96, 200, device="cuda") for _ in range(2)])
        x = torch.randn((64, 96), device="cuda", dtype=torch.bfloat16)
        plain = torch.autograd.grad(model(x).float().square().mean(), list(model.parameters()))
        ddp = torch.nn.parallel.DistributedDataParallel(model, device_ids=[0])
        comm_hook.register(ddp, scheme=gq.LINEAR, s=127, q=gq.NORM_INF, p=gq.NORM_INF, seed=0)
        ddp(x).float().square().mean().backward()
        top = max(g.abs().max() for g in plain)
        for p, g in zip(model.parameters(), plain):
            assert ((p.grad - g).abs() <= top / 127 + 1e-6 * top).all()
        assert max(p.grad.abs().max() for p in model.parameters()) >= top * (126 / 127)
    finally:
        dist.destroy_process_group()
