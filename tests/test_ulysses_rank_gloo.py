"""UlyssesRank.step and backward_step on CPU ranks over gloo: the exchanges
are the product's (nccl_all_to_all), the local phases plain torch in 64 bits.
Output and gradients are those of the unsharded problem."""
import datetime
import os
import socket
import sys

import pytest
import torch.multiprocessing as mp

HERE = os.path.dirname(os.path.abspath(__file__))


def _free_port():
    with socket.socket() as s:
        s.bind(("127.0.0.1", 0))
        return s.getsockname()[1]


def _rank_main(rank, world, port, queue, args):
    sys.path[:0] = [os.path.dirname(HERE), HERE]
    import torch
    import torch.distributed as dist

    import test_ulysses_rank_cpu as plain
    import video_dit_sequence_b200 as sp
    os.environ.update(MASTER_ADDR="127.0.0.1", MASTER_PORT=str(port))
    dist.init_process_group("gloo", rank=rank, world_size=world,
                            timeout=datetime.timedelta(seconds=60))
    try:
        plain._play(setattr)
        torch.set_num_threads(2)
        B, N, H, D = args
        shape = sp.Shape(B, N, H, D, world)
        exchange, worst = sp.nccl_all_to_all(), 0.0
        ulysses = sp.UlyssesRank(shape)
        lse = torch.empty(shape.head_group().lse_shape)
        for seed in (1, 2):   # the buffers of the first step are the second's
            q, k, v, do = plain._inputs(shape, seed)
            out = ulysses.step(q[rank], k[rank], v[rank], exchange, lse=lse)
            grads = ulysses.backward_step(do[rank], lse, exchange)
            o, full = torch.empty_like(q), torch.empty(shape.lse_shape)
            plain._attend(q, k, v, o, shape, lse=full)
            want = [torch.empty_like(q) for _ in range(3)]
            plain._attend_backward(q, k, v, o, full, do, *want, shape)
            # the same 64-bit formula on a head group: sums in another order can
            # only turn the last rounding to bf16 (one step, 2^-7 of the value)
            for got, ref in zip([out] + grads, [o] + want):
                ref = ref[rank].double()
                worst = max(worst, ((got.double() - ref).abs() / (ref.abs() + 1e-12)).max().item())
        queue.put((rank, worst))
        dist.barrier()
    finally:
        dist.destroy_process_group()


@pytest.mark.timeout(180)
@pytest.mark.parametrize("world,args", [(2, (2, 37, 4, 64)), (4, (1, 50, 8, 64)), (4, (2, 9, 4, 64))])
def test_there_and_back_over_gloo(world, args):
    ctx = mp.get_context("spawn")
    queue, port = ctx.Queue(), _free_port()
    procs = [ctx.Process(target=_rank_main, args=(r, world, port, queue, args)) for r in range(world)]
    for p in procs:
        p.start()
    for p in procs:
        p.join(150)
        assert p.exitcode == 0
    got = dict(queue.get(timeout=5) for _ in range(world))
    assert sorted(got) == list(range(world))
    assert all(w <= 2.0 ** -7 for w in got.values()), got
