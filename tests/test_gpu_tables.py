"""Block tables on the GPU against the oracle: every array equal, step after step; refusals that change nothing;
and the tables driving a 4-bit decode."""

import random

import numpy as np
import pytest
import torch

import workloads
from oracle import attention, cache_q4, tables

from harness import to_f64

pytestmark = pytest.mark.gpu


def _dcp():
    import context_sharded_mla_gb300 as dcp
    return dcp


class Both:
    """The GPU arrays and the oracle's lists, moved together."""

    def __init__(self, B, cap, most, N, I, P, T, head=0, stride_pad=0, fields=True):
        dcp = _dcp()
        self.lay, self.dims = dcp.Layout(N, I, P), (N, I, P)
        self.B, self.most, self.T = B, most, T
        dev = "cuda"
        ring = list(range(cap))
        ring = ring[-head:] + ring[:-head] if head else ring
        self.lens, self.table, self.ring, self.head, self.count = [0] * B, [[-1] * most for _ in range(B)], ring, head, cap
        self.seq = torch.zeros(B, dtype=torch.int64, device=dev)
        self.bt = torch.full((B, most + stride_pad), -1, dtype=torch.int32, device=dev)
        if stride_pad:
            self.bt[:, most:] = 77
        self.free = torch.tensor(ring, dtype=torch.int32, device=dev)
        self.state = torch.tensor([head, cap], dtype=torch.int64, device=dev)
        self.cu = torch.full((B + 1,), -9, dtype=torch.int64, device=dev)
        self.status = torch.zeros(1, dtype=torch.int32, device=dev)
        self.out = {}
        if T is not None:
            for k, dt in (("pos", torch.int64), ("req", torch.int32), ("owner", torch.int32), ("row", torch.int64),
                          ("slot", torch.int64)):
                if fields or k in ("pos", "req"):
                    self.out[k] = torch.full((T,), -7, dtype=dt, device=dev)

    def step(self, new, stream=None):
        dcp = _dcp()
        self.status.zero_()
        new_d = torch.tensor(new, dtype=torch.int64, device="cuda")
        torch.cuda.synchronize()
        dcp.dcp_block_tables(self.lay, self.seq, new_d, self.bt, self.most, self.free, self.state, self.cu, self.status,
                             **self.out, stream=stream)
        torch.cuda.synchronize()
        self.head, self.count, tokens, cu, status = tables.update(
            self.lens, list(new), self.table, self.most, self.ring, self.head, self.count, *self.dims, T=self.T)
        assert int(self.status.item()) == status
        assert self.seq.tolist() == self.lens
        assert self.bt[:, :self.most].tolist() == self.table
        assert bool((self.bt[:, self.most:] == 77).all())
        assert self.free.tolist() == self.ring
        assert self.state.tolist() == [self.head, self.count]
        assert self.cu.tolist() == cu
        for i, k in enumerate(("pos", "req", "owner", "row", "slot")):
            if k in self.out:
                want = [t[i] for t in tokens] + [-1] * (self.T - len(tokens))
                assert self.out[k].tolist() == want, k
        return status


@pytest.mark.parametrize("N,I,P", [(1, 1, 8), (4, 1, 16), (3, 2, 8), (8, 8, 64)])
@pytest.mark.parametrize("B", [1, 7, 130])
def test_random_steps(N, I, P, B):
    rng = random.Random(B * 1000 + N)
    most = 6
    cap = max(4, 3 * B)
    st = Both(B, cap, most, N, I, P, T=B * most * N * P, head=rng.randrange(cap), stride_pad=rng.randrange(3))
    done = 0
    for k in range(12):
        new = [rng.choice([0, a, min(a + rng.randrange(4), most * N * P), rng.randrange(most * N * P + 1)]) for a in st.lens]
        if k % 3 == 0:
            new = [min(n, N * P) for n in new]
        done += st.step(new) == 0
    assert done >= 4


def test_many_requests():
    """More requests than the scanning block has threads, short and long token lists."""
    B = 2500
    rng = random.Random(4)
    st = Both(B, 2 * B, 4, 2, 1, 8, T=4000, fields=True)
    assert st.step([rng.randrange(2) for _ in range(B)]) == 0
    st.out = {k: torch.full((60000,), -7, dtype=v.dtype, device="cuda") for k, v in st.out.items()}
    st.T = 60000
    assert st.step([rng.choice([0, 1, 17, 30]) for _ in range(B)]) == 0
    assert st.step([rng.choice([0, 16, 64]) for _ in range(B)]) in (0, 128)
    assert st.step([0] * B) == 0
    assert st.count == 2 * B


def test_long_prompt_and_exact_capacity():
    st = Both(2, 1000, 600, 4, 1, 16, T=600 * 64)
    assert st.step([0, 600 * 64]) == 0               # every entry of the list a token
    assert st.step([400 * 64, 0]) == 0               # 400 free pages left, all taken; 600 come back behind them
    assert st.step([400 * 64, 1]) == 0
    assert st.step([0, 0]) == 0


def test_refusals_leave_everything():
    B, N, P = 3, 2, 8
    st = Both(B, 5, 4, N, 1, P, T=40, head=3)
    assert st.step([5, 17, 0]) == 0
    assert st.step([5, 17, 33]) == 128               # 3 pages needed, 2 free
    assert st.step([5, -1, 0]) == 16
    assert st.step([5, 17, 65]) == 2 | 0
    assert st.step([5, 17, 1 << 62]) == 16
    assert st.step([5, 17 + 41, 0]) in (128 | 256, 256)
    st.state[1] = st.count = 4                       # two held by requests, four free, of five: giving back overflows
    assert st.step([0, 0, 0]) == 512
    st.state[1] = st.count = 6
    assert st.step([5, 17, 0]) == 512
    st.state[0] = st.head = 5
    st.state[1] = st.count = 1
    assert st.step([5, 17, 0]) == 512


def test_bad_page_in_the_table():
    st = Both(2, 6, 3, 1, 1, 8, T=11)            # the first step's 11 tokens
    assert st.step([8, 3]) == 0
    st.bt[1, 0] = 99
    dcp = _dcp()
    dcp.dcp_block_tables(st.lay, st.seq, torch.tensor([8, 5], device="cuda"), st.bt, 3, st.free, st.state, st.cu,
                         st.status, **st.out)
    assert int(st.status.item()) == 4 and st.out["slot"].tolist() == [-1] * 11
    assert st.out["pos"].tolist() == [3, 4] + [-1] * 9
    st.status.zero_()
    dcp.dcp_block_tables(st.lay, st.seq, torch.tensor([8, 0], device="cuda"), st.bt, 3, st.free, st.state, st.cu,
                         st.status)
    assert int(st.status.item()) == 4 and st.bt[1, 0].item() == -1 and st.state.tolist()[1] == 5


def test_without_token_list_and_with_some_arrays():
    st = Both(4, 20, 5, 2, 1, 8, T=None)
    assert st.step([3, 40, 0, 16]) == 0
    st = Both(4, 20, 5, 2, 1, 8, T=70, fields=False)
    assert st.step([3, 40, 0, 16], stream=torch.cuda.Stream()) == 0


@pytest.mark.parametrize("T", [64, 6000])
def test_captured_steps(T):
    """One captured update, replayed with other target lengths."""
    dcp = _dcp()
    st = Both(5, 60, 12, 2, 1, 8, T=T)
    new = torch.zeros(5, dtype=torch.int64, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        dcp.dcp_block_tables(st.lay, st.seq, new, st.bt, st.most, st.free, st.state, st.cu, st.status, **st.out)
    for want in ([3, 0, 9, 17, 1], [4, 1, 0, 20, 1], [0, 64, 0, 0, 1]):
        new.copy_(torch.tensor(want))
        graph.replay()
        torch.cuda.synchronize()
        st.head, st.count, tokens, cu, status = tables.update(st.lens, want, st.table, st.most, st.ring, st.head,
                                                              st.count, *st.dims, T=T)
        assert int(st.status.item()) == status == 0
        assert st.bt.tolist() == st.table and st.free.tolist() == st.ring and st.cu.tolist() == cu
        assert st.out["slot"].tolist() == [t[4] for t in tokens] + [-1] * (T - len(tokens))


@pytest.mark.parametrize("cache", ["q4", "bf16"])
def test_serving_loop(cache):
    """Tables, append, partials and merge as a serving loop runs them: prompts, decode steps, a verify step whose
    drafts are rejected, a request that ends and one that takes its pages; each step against fp64 attention over
    the tokens given so far."""
    from context_sharded_mla_gb300.step import BlockTables, ShardedMlaDecoder
    dcp = _dcp()
    B, H, N, I, P = 3, 16, 4, 2, 16
    lay = dcp.Layout(N, I, P)
    tab = BlockTables(lay, B, pool_pages=9, max_pages=6, max_tokens=400)
    dec = ShardedMlaDecoder(lay, B, 1, H, 9, 6, workloads.SCALE, 0, torch.float32, cache=cache)
    gen = torch.Generator().manual_seed(8)
    seqs = [np.zeros((0, 576)) for _ in range(B)]

    def grow(lens):
        old = [len(s) for s in seqs]
        n = sum(max(0, x - a) for x, a in zip(lens, old))
        rows = torch.randn(n, 576, generator=gen).to(torch.bfloat16)
        pos, req = tab.update(torch.tensor(lens, device="cuda"))
        held = rows
        if cache == "q4":
            codes, scales = cache_q4.quantise(to_f64(rows[:, :512]))
            held = cache_q4.unpack(cache_q4.pack(codes, scales,
                                                 rows[:, 512:].contiguous().view(torch.int16).numpy().view(np.uint16)))
            pad = torch.cat([rows, torch.zeros(400 - n, 576, dtype=torch.bfloat16)])   # a padded batch
            dec.append(pad.cuda(), pos, req, tab.block_table)
        else:
            held = to_f64(rows)
            dec.append(rows.cuda(), pos[:n].contiguous(), req[:n].contiguous(), tab.block_table)
        at = 0
        for b in range(B):
            k = max(0, lens[b] - old[b])
            seqs[b] = np.concatenate([seqs[b][:lens[b]], held[at:at + k]])
            at += k

    def decode():
        q = torch.randn(B, 1, H, 576, generator=gen).to(torch.bfloat16)
        o, lse = dec.decode(q.cuda(), tab.block_table, tab.seq_lens)
        torch.cuda.synchronize()
        for b in range(B):
            if not len(seqs[b]):
                continue
            ro, rl = attention._softmax_attend(to_f64(q)[b, 0], seqs[b], workloads.SCALE, 0)
            x = workloads.SCALE * to_f64(q)[b, 0] @ seqs[b].T
            w = np.exp(x - rl[:, None])
            ds = 576 * 2.0 ** -23 * workloads.SCALE * (np.abs(to_f64(q)[b, 0]) @ np.abs(seqs[b]).T).max(1)
            tol = (2.0 ** -8 + 4 * ds + 2.0 ** -15)[:, None] * (w @ np.abs(seqs[b][:, :512]))
            assert np.all(np.abs(to_f64(o)[b, 0] - ro) <= tol)
            assert np.all(np.abs(to_f64(lse)[b, 0] - rl) <= 2 * ds + 2.0 ** -19 * np.maximum(1, np.abs(rl)))

    grow([100, 65, 1])
    decode()
    for _ in range(3):
        grow([len(s) + 1 for s in seqs])
        decode()
    here = [len(s) for s in seqs]
    grow([n + 4 for n in here])                      # drafts ...
    grow([n + 1 for n in here])                      # ... of which one each is accepted
    decode()
    grow([0, here[1] + 1, here[2] + 1])              # a request ends
    grow([180, here[1] + 2, here[2] + 2])            # another takes its place
    decode()
    assert tab.status_bits() == 0 and dec.status_bits() in (0, 16)   # 16: the decode of an empty request
