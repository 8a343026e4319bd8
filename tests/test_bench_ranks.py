"""The multi-rank host logic of bench.py on CPU: two gloo ranks (replicas, no data-path collective).

bench.py under torchrun gives every rank its own batch (weak scaling); the ranks meet only to
combine the timings.  The whole-job time is the slowest rank's and the processed units are the sum
over ranks.  This runs that very function over a world of 2 on the gloo backend.
"""
import os
import socket

import pytest
import torch
import torch.distributed as dist
import torch.multiprocessing as mp

import bench


def _free_port():
    with socket.socket() as s:
        s.bind(("127.0.0.1", 0))
        return s.getsockname()[1]


def _rank(rank, world, port, out):
    os.environ.update(MASTER_ADDR="127.0.0.1", MASTER_PORT=str(port), RANK=str(rank), WORLD_SIZE=str(world),
                      LOCAL_RANK=str(rank))
    w, r, lr = bench.dist_setup()
    assert (w, r, lr) == (world, rank, rank)
    dist.init_process_group("gloo", rank=rank, world_size=world)
    try:
        # rank r: 10 + r ms for K steps, e2e 3 + 2r ms, units 1000 * (r + 1)
        res = bench.aggregate_over_ranks(torch, 10.0 + rank, 3.0 + 2 * rank, 1000.0 * (rank + 1), 7.0 * (rank + 1),
                                         torch.device("cpu"))
        out[rank] = res
    finally:
        dist.destroy_process_group()


def test_aggregate_over_two_gloo_ranks():
    world, port = 2, _free_port()
    with mp.get_context("spawn").Manager() as m:  # no fork of this multi-threaded process
        out = m.dict()
        mp.spawn(_rank, args=(world, port, out), nprocs=world, join=True)
        res = dict(out)
    for r in range(world):
        total_ms, e2e_ms, units, e2e_units = res[r]
        assert total_ms == 11.0 and e2e_ms == 5.0        # the slowest rank's times
        assert units == 3000.0 and e2e_units == 21.0     # summed over the replicas


def test_dist_setup_defaults_to_one_rank(monkeypatch):
    for k in ("WORLD_SIZE", "RANK", "LOCAL_RANK"):
        monkeypatch.delenv(k, raising=False)
    assert bench.dist_setup() == (1, 0, 0)


def test_the_line_stays_short():
    """Standard output gets every key of the contract and no table per launch."""
    launch = {"name": "s0.down", "kernel": "cb::stem_tc_kernel", "us": 91.2, "roofline": {"frac": 0.5}}
    keys = ("metric", "value", "unit", "n_gpus", "steps", "warmup", "ms_per_step", "higher_is_better", "scaling",
            "vs_baseline", "dtype", "data", "config", "e2e", "gpu_launches", "clocks", "roofline")
    line = {k: k for k in keys}
    line.update(launches=[launch] * 40, kernel_shares={"k": launch}, timing={"launches": "x" * 200},
                configs={f"cfg{i}": {"value": 711047.277, "unit": "images/s", "launches": [launch] * 40} for i in range(10)})
    short = bench.short_line(line)
    assert all(short[k] == k for k in keys)
    assert short["configs"]["cfg3"] == [711047.277, "images/s"]
    assert len(bench.json.dumps(short)) < 2000 and "launches" in line
