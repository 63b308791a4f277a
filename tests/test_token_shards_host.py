"""The 8-bit gather of token shards (column_parallel.gather_tokens) on gloo
ranks with uneven, empty and equal shards: codes and scales arrive bit by bit
in rank order."""
import os
import socket
import sys

import pytest
import torch
import torch.distributed as dist
import torch.multiprocessing as mp

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

from rotated_w4_linear_b200.column_parallel import gather_tokens  # noqa: E402


def _state(counts, features=144):
    g = torch.Generator().manual_seed(7)
    codes = torch.randint(0, 256, (sum(counts), features), dtype=torch.uint8, generator=g)
    return codes.view(torch.float8_e4m3fn), torch.rand(sum(counts), 2, generator=g)


def _free_port():
    with socket.socket() as sk:
        sk.bind(("127.0.0.1", 0))
        return sk.getsockname()[1]


def _rank(rank, world, port, counts, out):
    sys.path.insert(0, ROOT)
    os.environ.update(MASTER_ADDR="127.0.0.1", MASTER_PORT=str(port))
    dist.init_process_group("gloo", rank=rank, world_size=world)
    try:
        Q, S = _state(counts)
        lo = sum(counts[:rank])
        mine = slice(lo, lo + counts[rank])
        q, s = gather_tokens(Q[mine], S[mine], counts)
        with pytest.raises(ValueError):                     # refused before anything is sent
            gather_tokens(Q[mine], S[mine], [c + 1 for c in counts])
        torch.save((q.view(torch.uint8), s), os.path.join(out, f"{rank}.pt"))
    finally:
        dist.destroy_process_group()


@pytest.mark.parametrize("counts", [[3, 5], [4, 0, 1], [2, 2]])
def test_shards_arrive_in_rank_order(tmp_path, counts):
    world = len(counts)
    mp.spawn(_rank, args=(world, _free_port(), counts, str(tmp_path)), nprocs=world, join=True)
    Q, S = _state(counts)
    for r in range(world):
        q, s = torch.load(tmp_path / f"{r}.pt")
        assert torch.equal(q, Q.view(torch.uint8)) and torch.equal(s, S)
