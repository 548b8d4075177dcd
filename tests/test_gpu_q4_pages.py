"""Bad entries of the block table in the 4-bit partial decode: the keys on such a page are flagged and carry no weight,
in both of its kernels and whatever the pools hold, and a call repeats itself bit for bit."""

import numpy as np
import pytest
import torch

from oracle import attention, layout as olayout

from harness import to_f64
from test_gpu_q4 import Q4State, SCALE

pytestmark = pytest.mark.gpu

BAD_PAGE_ID = 4


def check_without(st, b, bad):
    """Request b against attention over the rows that are not on the pages `bad` (indices in its table)."""
    o, lse, q = to_f64(st.o), to_f64(st.lse), to_f64(st.q)
    S = st.lens[b]
    for r in range(st.begin, st.end):
        rho = np.arange(int(olayout.count(r, S, st.N, st.I)))
        rho = rho[~np.isin(rho // st.P, bad)]
        K = st.values[r - st.begin, st.bt[b][rho // st.P] * st.P + rho % st.P]
        at = olayout.global_pos(r, rho, st.N, st.I)
        for t in range(st.q_len):
            seen = K[at <= S - st.q_len + t]
            go, gl = o[r - st.begin, b, t], lse[r - st.begin, b, t]
            if not len(seen):
                assert np.all(go == 0) and np.all(np.isneginf(gl)), (b, r, t)
                continue
            ro, rl = attention._softmax_attend(q[b, t], seen, SCALE, 2 if st.base else 0)
            x = SCALE * q[b, t] @ seen.T
            w = np.exp(x - x.max(1, keepdims=True))
            w /= w.sum(1, keepdims=True)
            # the bounds of the partial decode's own tests (test_gpu_q4.py)
            ds = 576 * 2.0 ** -23 * SCALE * (np.abs(q[b, t]) @ np.abs(seen).T).max(1)
            tol = (2.0 ** -8 + 2 * ds + 2.0 ** -16)[:, None] * (w @ np.abs(seen[:, :512]))
            tol = tol + 2.0 ** -110 * np.abs(seen[:, :512]).sum(0)
            assert np.all(np.abs(go - ro) <= tol), (b, r, t, float((np.abs(go - ro) - tol).max()))
            assert np.all(np.abs(gl - rl) <= 1.5 * ds + 2.0 ** -20 * np.maximum(1, np.abs(rl))), (b, r, t)


# table entries of request 1 that are bad, of the pages its length uses
@pytest.mark.parametrize("P,lens,bad", [
    (16, [500, 700, 90], [0]), (16, [500, 700, 90], [21]), (16, [500, 700, 90], [3, 4, 5, 6, 10]),
    (8, [500, 700, 90], [7, 43]), (64, [500, 700, 90], [2]), (128, [500, 1500, 90], [1, 5]),
    (16, [500, 60, 90], [0, 1]), (64, [9000, 20000, 5], [0, 1, 100, 101, 156]),
])
@pytest.mark.parametrize("H,q_len", [(16, 1), (17, 1), (4, 3), (96, 1), (128, 2)])
@pytest.mark.parametrize("junk", [True, False])
def test_keys_on_bad_pages_carry_no_weight(P, lens, bad, H, q_len, junk):
    st = Q4State(lens, H, q_len, 2, 1, P, seed=5 + P, junk=junk, base=1)
    good = st.bt.copy()
    for i, k in enumerate(bad):
        assert st.bt[1, k] >= 0
        st.bt[1, k] = (st.pool + 3, -1, -2, 2 ** 31 - 1, -2 ** 31)[i % 5]
    outs = []
    for _ in range(3):
        st.status.zero_()
        st.o.fill_(float("nan"))
        st.lse.fill_(float("nan"))
        st.run()
        assert int(st.status.item()) == BAD_PAGE_ID
        outs.append((st.o.clone(), st.lse.clone()))
    assert all(torch.equal(outs[0][0], o) and torch.equal(outs[0][1], l) for o, l in outs[1:])
    st.check(reqs=[0, 2], status=BAD_PAGE_ID)
    check_without(st, 1, bad)
    st.status.zero_()                                   # and nothing of it is left behind
    st.bt = good
    st.run()
    st.check()
