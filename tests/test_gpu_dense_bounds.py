"""What linear and gated layers write and spread (GPU): workspaces of just the size that was asked for, with memory behind them
that stays as it is; infinite inputs and weights, which stay in their rows and columns."""
import math

import pytest
import torch

import mxfp4_precision_numerics_amd as mxq
from test_gpu_dense_calls import SIZES
from test_gpu_dense_layers import ACTS, BF, DEV, F32, act, mm, rn

pytestmark = pytest.mark.gpu
MORE = [(16, 32768, 1424), (40, 4096, 11264), (128, 4104, 11280), (512, 4096, 4096), (2000, 2880, 1008), (2048, 2056, 4112),
        (8192, 1024, 512), (300, 8200, 1040), (1100, 1416, 10000)]
BEHIND = 1 << 20


@pytest.mark.parametrize("T,H,N", SIZES + MORE, ids=lambda v: str(v))
def test_what_lies_behind_a_workspace_stays(T, H, N):
    x, w, dy, z = rn(T, H, seed=1), rn(N, H, seed=2, std=1 / math.sqrt(H)), rn(T, N, seed=3), rn(T, N, seed=4)
    I = N // 2
    dh = dy[:, :I].contiguous()
    y, h, dx, dw, db = (torch.empty(*s, dtype=d, device=DEV) for s, d in (((T, N), BF), ((T, I), BF), ((T, H), BF), ((N, H), F32),
                                                                          ((N,), F32)))
    def workspace(n):
        room = torch.full((n + BEHIND,), 0xA5, dtype=torch.uint8, device=DEV)
        rooms.append((room, n))
        return room[:n]
    rooms = []
    back, gback = mxq.linear_workspace(T, H, N, True), mxq.gated_linear_workspace(T, H, I, True)
    mxq.linear(x, w, y, workspace=workspace(mxq.linear_workspace(T, H, N)))
    mxq.gated_linear(x, w, h, workspace=workspace(mxq.gated_linear_workspace(T, H, I)))
    mxq.linear_backward(x, w, dy, dx, dw, db, activation=mxq.ACT_SILU, z=z, workspace=workspace(back))
    mxq.linear_backward(x, w, dy, dx, dw, db, workspace=workspace(back))
    mxq.linear_backward(x, w, dy, dx, workspace=workspace(back))
    mxq.linear_backward(x, w, dy, dw=dw, workspace=workspace(back))
    mxq.gated_linear_backward(x, w, dh, dx, dw, z=z, workspace=workspace(gback))
    mxq.gated_linear_backward(x, w, dh, dx, dw, workspace=workspace(gback))
    torch.cuda.synchronize()
    for k, (room, n) in enumerate(rooms):
        assert bool((room[n:] == 0xA5).all()), k


@pytest.mark.parametrize("name", list(ACTS))
@pytest.mark.parametrize("T,H,N", SIZES, ids=lambda v: str(v))
def test_infinities_stay_in_their_rows_and_columns(T, H, N, name):
    """A token with one infinite entry, a row of weights with another: what they reach is what the definition in 64 bits gives,
    a number, an infinity or a NaN; all else is as without them, bit for bit."""
    x, w = rn(T, H, seed=1), rn(N, H, seed=2, std=1 / math.sqrt(H))
    ws = torch.empty(max(mxq.linear_workspace(T, H, N), mxq.gated_linear_workspace(T, H, N // 2)), dtype=torch.uint8, device=DEV)
    I, t, f = N // 2, T // 2, N // 2 - 3
    outs = []
    for bad in (False, True):
        if bad:
            x[t, H // 3], w[f, H // 5] = float("inf"), float("-inf")
        y, h = torch.empty(T, N, device=DEV), torch.empty(T, I, dtype=BF, device=DEV)
        mxq.linear(x, w, y, activation=ACTS[name], workspace=ws)
        mxq.gated_linear(x, w, h, activation=ACTS[name], workspace=ws)
        outs.append((y, h))
    z = mm(x, w)
    for (clean, got), want in zip(zip(*outs), (act(z, name), act(z[:, :I], name) * z[:, I:])):
        hit = torch.zeros(got.shape, dtype=torch.bool, device=DEV)
        hit[t], hit[:, f] = True, True
        assert torch.equal(got[~hit], clean[~hit])
        got, want = got[hit].double(), want[hit]
        assert torch.equal(got.isnan(), want.isnan()) and torch.equal(got.isinf(), want.isinf())
        assert torch.equal(got[got.isinf()], want[want.isinf()])
