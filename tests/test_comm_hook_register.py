"""comm_hook.register on a DistributedDataParallel model: what torch checks of a hook when it is attached."""
import datetime
import socket

import pytest

torch = pytest.importorskip("torch")


def test_the_hook_is_accepted():
    import torch.distributed as dist
    import allreduce_compatible_gradient_gb300 as gq
    from allreduce_compatible_gradient_gb300 import comm_hook
    with socket.socket() as s:
        s.bind(("127.0.0.1", 0))
        port = s.getsockname()[1]
    dist.init_process_group("gloo", init_method="tcp://127.0.0.1:%d" % port, rank=0, world_size=1,
                            timeout=datetime.timedelta(seconds=30))
    try:
        ddp = torch.nn.parallel.DistributedDataParallel(torch.nn.Linear(4, 4))
        state = comm_hook.register(ddp, scheme=gq.EXP, s=4, q=gq.NORM_INF, p=gq.NORM_INF, seed=0)
        assert isinstance(state, comm_hook.GlobalQSGDState) and state.s == 4
    finally:
        dist.destroy_process_group()
