"""A launch that CUDA refuses is an error of its call, and of no other."""
import os
import subprocess
import sys

import pytest

from gpu_common import gq_module

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


def calls(gq):
    """Calls that launch in every way: their results are compared before and after."""
    g = torch.Generator(device="cuda").manual_seed(1)
    randn = lambda *size: torch.randn(size, generator=g, device="cuda")  # noqa: E731
    made = {}
    for rows, cols, outs in ((3, 640, 300), (300, 1000, 500), (9000, 520, 2100)):
        w, x = gq.gq_fp8_quantize(randn(outs, cols), tiles=True), randn(rows, cols)
        x8 = gq.gq_fp8_quantize(x)
        made["linear of 8 bits, %d rows" % rows] = lambda x8=x8, w=w: gq.gq_fp8_linear(x8, w)
        made["linear, %d rows" % rows] = lambda x=x, w=w: gq.gq_fp8_linear(x, w)
    for rows in (0, 200, 5000):
        dy, x = randn(rows, 256), randn(rows, 384)
        act, rstd, weight = gq.gq_act_quantize(x), torch.ones(rows, device="cuda"), randn(384)
        made["weight gradient, %d rows" % rows] = lambda dy=dy, act=act: torch.cat(
            [v.view(-1) for v in gq.gq_linear_wgrad(dy, act)])
        d = randn(rows, 384)
        made["layer norm backward, %d rows" % rows] = lambda d=d, act=act, rstd=rstd, weight=weight: torch.cat(
            [v.view(-1) for v in gq.gq_layernorm_backward(d, weight, rstd, act=act)])
    p = [randn(1000) for _ in range(3)]
    made["norm"] = lambda: gq.gq_tensors_norm(p)
    made["quantise"] = lambda: gq.gq_fp8_quantize(p[0].view(10, 100)).data[:1120]
    ws = gq.gq_workspace("cuda")
    for n, d in ((4, 4096), (4, 3_000_001)):
        grads = randn(n, d)
        made["mean of %d" % d] = lambda grads=grads: gq.gq_allreduce_mean(
            grads, gq.NORM_INF, gq.NORM_INF, gq.LINEAR, 127, 5, 1, ws=ws)
    return made


def refuse_and_go_on():
    """Launches into a capture that has ended early (a synchronisation inside it) are refused on the host: each by
    itself, and a right call behind it is right."""
    gq = gq_module()
    made = calls(gq)
    want = {name: call() for name, call in made.items()}
    torch.cuda.synchronize()
    wrong = []
    for name, call in made.items():
        with pytest.raises(RuntimeError):  # the capture's own end
            with torch.cuda.graph(torch.cuda.CUDAGraph()):
                with pytest.raises(RuntimeError):
                    torch.cuda.synchronize()
                with pytest.raises(gq.GQError):
                    call()
                raise RuntimeError("the capture is over")
        for other in ("norm", name):
            try:
                if not torch.equal(made[other](), want[other]):
                    wrong.append((name, other))
            except gq.GQError as e:
                wrong.append((name, other, str(e)))
    torch.cuda.synchronize()
    assert not wrong, wrong


def test_the_call_after_a_refused_launch():
    """In a process of its own: torch's random numbers stay in a capture that has not ended well."""
    gq_module()
    done = subprocess.run([sys.executable, os.path.abspath(__file__)], capture_output=True, text=True, timeout=300)
    assert done.returncode == 0 and "all right" in done.stdout, done.stdout + done.stderr


if __name__ == "__main__":
    sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
    refuse_and_go_on()
    print("all right")
