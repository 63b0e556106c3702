"""GPU parity of expert routing: the choice, its weights and the sorted map
against the 64-bit form, over group edges (31 / 32 / 33 tokens), expert
counts around the wave width, ties, masks and strides."""
import numpy as np
import pytest
import torch

from oracle import serving as S
from gpu_util import dev

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def F():
    assert torch.cuda.is_available(), "GPU tests need a ROCm GPU"
    import fp8_block_scaled_02_amd as fp8w
    fp8w.lib()
    return fp8w


def _check(F, x, k, score="softmax", bias=None, renorm=True, scale=1.0, **kw):
    r = F.fp8w_route_experts(x, k, score=score, bias=bias, renorm=renorm, scale=scale, **kw)
    torch.cuda.synchronize()
    ids, w, slots, rows, offsets = S.route(x.float().cpu().numpy(), k, score,
                                           None if bias is None else bias.cpu().numpy(), renorm, scale)
    assert np.array_equal(r.ids.cpu().numpy(), ids)
    assert np.array_equal(r.offsets.cpu().numpy(), offsets)
    assert np.array_equal(r.slots.cpu().numpy(), slots)
    assert np.array_equal(r.rows.cpu().numpy(), rows)
    # a weight is an exponential (its argument rounded at the size of the
    # logits' spread; beyond 104 the term is zero in fp32) over a sum of at
    # most E of them
    xs = x.float().cpu().numpy().astype(np.float64)
    span = min(np.where(np.isfinite(xs), np.abs(xs), 0).max(), 104.0) if xs.size else 0
    tol = (2 * span + x.shape[1] + 16) * 2.0 ** -23
    assert (np.abs(r.weights.cpu().numpy() - w) <= tol * np.abs(w) + 1e-37).all()
    return r


@pytest.mark.parametrize("t", [0, 1, 2, 31, 32, 33, 64, 257, 1000])
@pytest.mark.parametrize("e,k", [(1, 1), (8, 2), (60, 6), (128, 8)])
def test_group_edges(F, t, e, k):
    g = torch.Generator(device="cuda").manual_seed(t * 1000 + e)
    _check(F, torch.randn(t, e, generator=g, device=dev()), k)


@pytest.mark.parametrize("e,k", [(2, 2), (63, 5), (64, 64), (65, 3), (127, 1), (129, 8), (256, 8), (257, 7),
                                 (512, 10), (1023, 16), (1024, 64)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_expert_counts(F, e, k, score):
    g = torch.Generator(device="cuda").manual_seed(e)
    for renorm in (True, False):
        _check(F, torch.randn(37, e, generator=g, device=dev()) * 2, k, score, renorm=renorm, scale=2.5)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("t", [5, 70])
def test_selection_bias(F, score, t):
    g = torch.Generator(device="cuda").manual_seed(11 + t)
    x = torch.randn(t, 72, generator=g, device=dev())
    x[0, 3:] = -np.inf
    _check(F, x, 6, score, bias=torch.randn(72, generator=g, device=dev()))


@pytest.mark.parametrize("t", [9, 100])
def test_ties_go_to_the_lower_expert(F, t):
    g = torch.Generator(device="cuda").manual_seed(t)
    x = torch.randint(-2, 3, (t, 96), generator=g, device=dev()).to(torch.bfloat16)
    x[0] = 0
    x[1] = torch.where(x[1] == 0, torch.tensor(-0.0, device=dev()), x[1]).to(torch.bfloat16)   # -0 equals +0
    _check(F, x, 8)


@pytest.mark.parametrize("t", [6, 65])
def test_masked_experts(F, t):
    g = torch.Generator(device="cuda").manual_seed(t)
    x = torch.randn(t, 40, generator=g, device=dev())
    x[torch.rand(t, 40, generator=g, device=dev()) < 0.9] = -np.inf
    x[0] = -np.inf                                    # nothing left
    x[1], x[1, 39] = -np.inf, -3e38                   # one expert, far down
    x[2] = torch.finfo(torch.float32).min             # the lowest value everywhere is no mask
    x[3, :20] = float("nan")
    x[4], x[4, 7], x[4, 9] = -np.inf, float("nan"), 0.0
    _check(F, x, 5)
    _check(F, x, 5, "sigmoid", renorm=False)


def test_large_logits_and_underflowing_scores(F):
    x = torch.tensor([[1e4, 1e4 - 1, -1e4], [-200.0, -201.0, -202.0], [88.0, 3.0, -88.0]], device=dev())
    _check(F, x, 2)
    r = F.fp8w_route_experts(x, 2, score="sigmoid")   # sigmoid(-200) is below fp32: no weight, not NaN
    assert torch.isfinite(r.weights).all() and r.weights[1].tolist() == [0.0, 0.0]


def test_strided_rows_and_types(F):
    g = torch.Generator(device="cuda").manual_seed(3)
    wide = torch.randn(50, 90, generator=g, device=dev())
    for dtype in (torch.float32, torch.bfloat16):
        _check(F, wide.to(dtype)[:, 7:71], 4)
        _check(F, wide.to(dtype)[3:4, 5:6], 1)


def test_many_groups(F):
    g = torch.Generator(device="cuda").manual_seed(8)
    t, e, k = 20000, 33, 3
    x = torch.randn(t, e, generator=g, device=dev()) + torch.randn(e, generator=g, device=dev())
    r = F.fp8w_route_experts(x, k)
    ids = r.ids.long()
    assert torch.equal(ids, torch.sort(x, dim=1, descending=True, stable=True).indices[:, :k])
    order = torch.sort(ids.reshape(-1), stable=True).indices
    assert torch.equal(r.rows.long(), order // k)
    assert torch.equal(r.slots.reshape(-1)[order].long(), torch.arange(t * k, device=dev()))
    assert torch.equal(r.offsets[1:].long(), torch.bincount(ids.reshape(-1), minlength=e).cumsum(0))


def test_another_stream_and_graph_replays(F):
    g = torch.Generator(device="cuda").manual_seed(21)
    x = torch.randn(48, 64, generator=g, device=dev())
    want = [v.clone() for v in F.fp8w_route_experts(x, 4)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = F.fp8w_route_experts(x, 4, stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    buf = [torch.empty_like(v) for v in want]
    ws = torch.empty(F.lib().fp8w_route_experts_workspace_bytes(48, 64), dtype=torch.uint8, device=dev())
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        F.fp8w_route_experts(x, 4, ids=buf[0], weights=buf[1], slots=buf[2], rows=buf[3], offsets=buf[4], workspace=ws)
    for i in range(3):
        for b in buf:
            b.fill_(-7)
        ws.fill_(255)
        x.copy_(torch.randn(48, 64, generator=g, device=dev()))
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(buf, F.fp8w_route_experts(x, 4))), i
