"""Views with equally strided rows, where a dimension of extent 1 has a stride that says nothing."""

import pytest
import torch

import context_sharded_mla_gb300 as dcp


class OnGpu(torch.Tensor):
    """A host tensor that passes for a CUDA one: only strides are looked at."""
    is_cuda = property(lambda self: True)


def host(*shape):
    return torch.zeros(*shape, dtype=torch.bfloat16).as_subclass(OnGpu)


def cases(make):
    """(view [..., 192], the distance of its rows in elements)"""
    return [
        (make(5, 1024)[:, :192].unsqueeze(1), 1024),                # one head of a projection's output
        (make(5, 6, 256)[:, 2:3, :192], 1536),                      # one head of several
        (make(1, 5, 192).transpose(0, 1), 192),                     # the head's dimension was the first
        (make(1, 5, 448).transpose(0, 1)[..., 64:256], 448),
        (make(1, 1, 256)[..., :192], 192),                          # one row: no distance
        (make(7, 256)[3:4, :192].unsqueeze(0), 192),
        (make(5, 6, 256)[:, :, :192], 256),
        (make(5, 6, 256)[2:3, :, :192], 256),
        (make(5, 6, 256)[:0, :, :192], 192),                        # no rows
        (make(3, 1, 2, 1, 256)[..., :192], 256),
        (make(4, 192), 192),
    ]


@pytest.mark.parametrize("i", range(len(cases(host))))
def test_distance_of_rows(i):
    view, want = cases(host)[i]
    assert dcp._rows(view, "q", 192) == want


@pytest.mark.parametrize("view", [
    lambda: host(6, 5, 256).transpose(0, 1)[..., :192], lambda: host(5, 1, 6, 256).transpose(0, 2)[..., :192],
    lambda: host(4, 6, 256)[:, :3, :192], lambda: host(5, 192, 2)[..., 0].unsqueeze(1)])
def test_rows_that_are_not_equally_strided(view):
    with pytest.raises(ValueError):
        dcp._rows(view(), "q", 192)


@pytest.mark.gpu
@pytest.mark.parametrize("i", range(len(cases(host))))
def test_calls_on_views_give_what_they_give_on_copies(i):
    g = torch.Generator(device="cuda").manual_seed(i)
    view, _ = cases(lambda *s: torch.randn(*s, generator=g, device="cuda").to(torch.bfloat16))[i]
    flat = view.contiguous()
    if view.dim() == 3:
        T, H = view.shape[:2]
        pos = torch.arange(T, device="cuda") * 1000
        freq = (10000.0 ** (-torch.arange(0, 64, 2, device="cuda") / 64)).float()
        out = [torch.zeros(T, H, 192, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
        for x, o in zip((view, flat), out):
            dcp.dcp_q_norm_rope(x, pos, o, gamma=torch.ones(192, device="cuda"), inv_freq=freq)
        assert torch.equal(*out) and (T == 0 or bool(out[0].any()))
    H = view.shape[-2]
    w = torch.randn(H, 128, 512, generator=g, device="cuda").to(torch.bfloat16)
    out = [torch.zeros(*view.shape[:-1], 576, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    for x, o in zip((view, flat), out):
        dcp.dcp_absorb_q(x[..., :128], x[..., 128:], w, o)
    assert torch.equal(*out) and (view.numel() == 0 or bool(out[0].any()))


@pytest.mark.gpu
def test_one_row_of_a_wide_projection_is_appended():
    """kv [1, 576]: the distance of one row to the next does not matter."""
    wide = torch.randn(1, 1601, device="cuda").to(torch.bfloat16)
    arena = torch.zeros(1, 8, 576, dtype=torch.bfloat16, device="cuda")
    zero = torch.zeros(1, dtype=torch.int64, device="cuda")
    i32 = torch.zeros(1, dtype=torch.int32, device="cuda")
    dcp.dcp_kv_norm_rope_append(dcp.Layout(1, 1, 8), 0, 1, wide[:, 1024:1600], zero, i32, i32[None], 1, arena, 1, i32.clone())
    assert torch.equal(arena[0, 0], wide[0, 1024:1600])
