"""Operands and results that lie past 4 GiB of their tensors: rows of x and
of y of the grouped products, rows that are summed, rows of logits."""
import pytest
import torch

from gpu_util import dev

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def F():
    assert torch.cuda.is_available(), "GPU tests need a ROCm GPU"
    import fp8_block_scaled_02_amd as fp8w
    fp8w.lib()
    return fp8w


@pytest.mark.parametrize("act", ["none", "swiglu"])
@pytest.mark.parametrize("many", [5, 60, 300])
def test_rows_of_x(F, act, many):
    """Slots that name the first and the last rows of 5 GB."""
    k, n, rows = 8192, 128, 330000
    x = torch.zeros(rows, k, dtype=torch.bfloat16, device=dev())
    x[-many:] = torch.randn(many, k, device=dev()).to(torch.bfloat16)
    near = x[-many:].contiguous()
    q = F.Fp8Experts.quantize(torch.randn(1, n, k, device=dev()).to(torch.bfloat16))
    off = torch.tensor([0, many], dtype=torch.int32, device=dev())
    at = torch.arange(rows - many, rows, dtype=torch.int32, device=dev())
    assert torch.equal(q.matmul(x, off, at, act), q.matmul(near, off, None, act))


@pytest.mark.parametrize("k,n", [(64, 2048), (128, 3000)])
def test_rows_of_y(F, k, n):
    """The last expert's slots lie past 4 GiB of y."""
    slots = 1100000
    y = torch.zeros(slots, n, dtype=torch.bfloat16, device=dev())
    x = torch.randn(64, k, device=dev()).to(torch.bfloat16)
    q = F.Fp8Experts.quantize(torch.randn(3, n, k, device=dev()).to(torch.bfloat16), "row")
    off = torch.tensor([slots - 300, slots - 300, slots - 200, slots], dtype=torch.int32, device=dev())
    at = torch.zeros(slots, dtype=torch.int32, device=dev())
    at[-300:] = torch.arange(300, device=dev()).int() % 64
    q.matmul(x, off, at, y=y)
    want = q.matmul(x, torch.tensor([0, 0, 100, 300], dtype=torch.int32, device=dev()), at[-300:].contiguous(),
                    y=torch.empty(300, n, dtype=torch.bfloat16, device=dev()))
    assert not y[:-300].any()
    # the same products, of another kernel (by the average of all slots)
    assert (y[-300:].float() - want.float()).abs().max() <= 2.0 ** -7 * want.float().abs().max()


@pytest.mark.parametrize("n", [2048, 2049])
def test_rows_that_are_summed(F, n):
    rows = 1100000
    y = torch.zeros(rows, n, dtype=torch.bfloat16, device=dev())
    y[-9:] = torch.randn(9, n, device=dev()).to(torch.bfloat16)
    near = y[-9:].contiguous()
    slots = torch.tensor([[0, 8, -1], [3, 4, 5], [9, 8, 7]], dtype=torch.int32, device=dev())
    w = torch.rand(3, 3, device=dev())
    far = torch.where((slots >= 0) & (slots < 9), slots + rows - 9, -1).int()
    assert torch.equal(F.fp8w_combine_experts(y, w, far), F.fp8w_combine_experts(near, w, slots))


@pytest.mark.parametrize("dtype,t", [(torch.bfloat16, 30000), (torch.float32, 15000)])
@pytest.mark.parametrize("top", [0, 6])
def test_rows_of_logits(F, dtype, t, top):
    v = 80001
    x = torch.zeros(t, v, dtype=dtype, device=dev())
    x[:, 0] = 9.0
    x[-3:] = torch.randn(3, v, device=dev()).to(dtype)
    target = torch.full((t,), v - 1, dtype=torch.int32, device=dev())
    far = F.fp8w_logprobs(x, target, top)
    near = F.fp8w_logprobs(x[-3:].contiguous(), target[-3:].contiguous(), top)
    assert torch.equal(far.top_ids[-3:], near.top_ids)
    for a, b in ((far.logprob, near.logprob), (far.entropy, near.entropy), (far.top_logprobs, near.top_logprobs)):
        assert torch.allclose(a[-3:], b, rtol=1e-5, atol=1e-5)       # segments of 3 rows are joined in another order


def test_rows_of_router_logits(F):
    wide = torch.zeros(70, 1 << 25, dtype=torch.bfloat16, device=dev())
    x = torch.randn(70, 64, device=dev()).to(torch.bfloat16)
    wide[:, :64] = x
    for a, b in zip(F.fp8w_route_experts(wide[:, :64], 5), F.fp8w_route_experts(x, 5)):
        assert torch.equal(a, b)
