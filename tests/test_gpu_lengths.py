"""Lengths that a block table cannot hold, in both caches: flagged, the other requests right, and the work of the
claiming request bounded by its row of the table (the planner's tile counts, the first words of the workspace)."""

import numpy as np
import pytest
import torch

import workloads
from oracle import layout as olayout

from harness import GpuState
from test_gpu_faults import BAD_PAGE_ID, _check_others
from test_gpu_q4 import Q4State

pytestmark = pytest.mark.gpu

HUGE = [2 ** 40, 2 ** 63 - 1]


def tiles(lens, N, I, P, max_pages):
    """Tile prefix sums of the (request, shard) units, every unit at most as long as its row of the table."""
    per = [-(-min(int(olayout.count(r, S, N, I)), max_pages * P) // 64) for S in lens for r in range(N)]
    return np.concatenate([[0], np.cumsum(per)]).tolist()


@pytest.mark.parametrize("name,over", [("tiny", dict(B=3, S=1000)), ("ragged", dict(B=4, S=3000, S_min=400)),
                                       ("k3", dict(B=3, S=4109))])
@pytest.mark.parametrize("length", ["one past"] + HUGE)
def test_bf16_length_beyond_the_table(name, over, length):
    import context_sharded_mla_gb300 as dcp
    st = GpuState(workloads.config(name, **over))
    d, cfg = st.dec, st.cfg
    lens = [int(s) for s in st.S]
    lens[1] = cfg.N * cfg.P * st.max_pages + 1 if length == "one past" else length
    dcp.dcp_mla_decode_partial(d.layout, 0, cfg.N, st.q, d.arena, d.pool_pages, st.bt, st.max_pages,
                               torch.tensor(lens, device="cuda"), d.scale, d.lse_base, d.o_part, d.lse_part, d.workspace,
                               d.status)
    d.merge()
    torch.cuda.synchronize()
    assert int(d.status.item()) == BAD_PAGE_ID
    _check_others(st, *(x.double().cpu().numpy() for x in (d.o, d.lse, d.o_part, d.lse_part)), 1)
    U = cfg.B * cfg.N
    assert d.workspace[:4 * (U + 1)].view(torch.int32).tolist() == tiles(lens, cfg.N, cfg.I, cfg.P, st.max_pages)


@pytest.mark.parametrize("H", [16, 8])
@pytest.mark.parametrize("length", [2 * 16 * 13 + 1] + HUGE)
def test_q4_work_of_a_length_beyond_the_table(length, H):
    st = Q4State([50, 400, 90], H, 2, 2, 1, 16, seed=33, junk=False)
    st.lens = [50, length, 90]
    st.run()
    assert int(st.status.item()) == BAD_PAGE_ID
    st.check(reqs=[0, 2], status=BAD_PAGE_ID)
    assert st.ws[:4 * 7].view(torch.int32).tolist() == tiles(st.lens, 2, 1, 16, 13)
