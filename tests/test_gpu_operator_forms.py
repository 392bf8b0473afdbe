"""The forms of the adapters' and the router's kernels that sizes choose between, each at
sizes that reach it: against fp64, after a launch that left infinities in LDS, and with a
token that holds an infinity."""
import pytest
import torch

from gpu_util import digest, say
from test_gpu_lora import case, run, verify

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def B():
    from mixture_experts_layer_plan_amd import binding
    return binding


def leave_infinities_in_lds(B):
    """Rank 128 with infinite weights: its stages of 32 KiB fill with them on every CU."""
    T, hi, ho, n = 2048, 64, 7168, 1
    s = B.lora_shape(T, hi, ho, n, 128)
    u8 = dict(dtype=torch.uint8, device="cuda")
    bf = dict(dtype=torch.bfloat16, device="cuda")
    plan = torch.empty(B.moe_lora_plan_bytes(s), **u8)
    B.moe_lora_plan(s, torch.zeros(T, dtype=torch.int32, device="cuda"), plan)
    y = torch.zeros(T, ho, **bf)
    B.moe_lora_bf16(s, plan, torch.ones(T, hi, **bf), torch.ones(n, 128, hi, **bf),
                    torch.full((n, ho, 128), float("inf"), **bf), torch.ones(n, device="cuda"), y, y,
                    None, torch.empty(B.moe_lora_workspace_bytes(s, False), **u8))


# 64-row tiles of two column blocks a workgroup, then 128-row tiles, of y and of dx
@pytest.mark.parametrize("T,hi,ho,n,r", [(600, 64, 7168, 4, 96), (600, 7168, 64, 4, 96), (1000, 64, 7168, 8, 96),
                                         (600, 64, 7168, 4, 72), (600, 64, 7168, 4, 120), (1100, 64, 6656, 1, 96),
                                         (1100, 6656, 64, 1, 96), (1100, 64, 6656, 1, 88), (1100, 6656, 64, 1, 128)])
def test_ranks_past_64(B, T, hi, ho, n, r):
    say(f"lora forms T={T} {hi}->{ho} n={n} r={r}")
    c = case(T, hi, ho, n, r, "all")
    leave_infinities_in_lds(B)
    got = run(B, c)
    verify(c, got)
    assert digest(*run(B, c, base="inplace", fill=0)) == digest(*got)


@pytest.mark.parametrize("T,hi,ho,n,r", [(1100, 64, 6656, 1, 72), (1100, 64, 6656, 1, 96), (1100, 64, 6656, 1, 128),
                                         (1100, 6656, 64, 1, 96), (2300, 64, 6912, 1, 64), (2300, 13824, 64, 1, 16),
                                         (1000, 64, 7168, 8, 16), (1000, 64, 7168, 8, 64), (1000, 64, 7168, 8, 96),
                                         (1000, 7168, 64, 8, 96), (96, 264, 520, 32, 24), (50, 72, 264, 20, 16)])
def test_an_infinite_token_spoils_its_own_rows(B, T, hi, ho, n, r):
    """A token's infinity reaches its own y (dx) and the gradients it enters, nothing else,
    wherever the token lies in its tile."""
    say(f"lora with inf T={T} {hi}->{ho} n={n} r={r}")
    c = case(T, hi, ho, n, r, "all")
    clean = run(B, c)
    group = [t for t in range(T) if c["idx"][t] == c["idx"][0]]
    a = int(c["idx"][0])
    others = [i for i in range(n) if i != a]
    for t in {group[min(100, len(group) - 1)], group[-1]}:
        rows = torch.arange(T, device="cuda") != t
        cols = torch.arange(hi, device="cuda") != 9
        cx = dict(c, x=c["x"].clone())
        cx["x"][t, 9] = float("inf")
        y, dx, da, db = run(B, cx)
        assert torch.equal(y[rows], clean[0][rows]) and not torch.isfinite(y[t]).any()
        assert torch.equal(dx, clean[1]) and torch.equal(da[:, :, cols], clean[2][:, :, cols])
        assert torch.equal(da[others], clean[2][others]) and torch.equal(db[others], clean[3][others])
        cy = dict(c, dy=c["dy"].clone())
        cy["dy"][t, 9] = float("-inf")
        y, dx, da, db = run(B, cy)
        assert torch.equal(dx[rows], clean[1][rows]) and not torch.isfinite(dx[t]).any()
        keep = torch.arange(ho, device="cuda") != 9
        assert torch.equal(y, clean[0]) and torch.equal(db[:, keep], clean[3][:, keep])
        assert torch.equal(da[others], clean[2][others]) and torch.equal(db[others], clean[3][others])
