"""The gradient through relu where pre is NaN, an infinity or a zero, in both
kernels and by columns: NaN stays NaN, everything else is exact."""
import pytest

from launch_util import only_tiles

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("with_mul", [False, True])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("m,n,k,tiles", [(5, 70, 32, False), (200, 128, 64, False),
                                         (1100, 3136, 64, True), (4224, 4331, 4608, True)])
def test_slope(mx, m, n, k, tiles, dtype, with_mul):
    import torch
    gen = torch.Generator(device="cuda").manual_seed(m)
    t = torch.float32 if dtype == "f32" else torch.bfloat16
    a = mx.quantize(torch.randn(m, k, generator=gen, device="cuda").bfloat16(), 1)
    b = mx.quantize(torch.randn(k, n, generator=gen, device="cuda").bfloat16(), 0)
    pre = torch.randn(m, n, generator=gen, device="cuda").to(t)
    special = torch.tensor([float("nan"), -float("nan"), float("inf"), -float("inf"), 0.0, -0.0],
                           device="cuda").to(t)
    at = torch.randint(0, n, (m, 12), generator=gen, device="cuda")
    pre.scatter_(1, at, special.repeat(2).expand(m, 12).contiguous())
    pre[:, n - 1] = float("nan")            # the last column, which may be its 64 columns' last
    mul = torch.full((m, n), 2.0, device="cuda").to(t) if with_mul else None

    def call():
        return mx.linear_act_backward(a, b, pre, "relu", mul=mul, out_dtype=dtype)
    assert only_tiles(call) == tiles
    got = call()
    # the product by itself: times 2 and 1 every rounding is the same
    g = mx.linear_act_backward(a, b, torch.zeros_like(pre), "none", out_dtype=dtype)
    dz, dmul = got if with_mul else (got, None)
    nan = pre.isnan()
    assert torch.equal(dz.isnan(), nan)
    want = torch.where(pre > 0, g if mul is None else g * mul, torch.zeros_like(g))
    assert torch.equal(dz[~nan], want[~nan])
    if with_mul:
        assert dmul[nan].isnan().all()
