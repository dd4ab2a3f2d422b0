"""A step whose rate is not finite is left out, as one whose gradients' scale is not."""
import math

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("needs a GPU", allow_module_level=True)

import trellis_quantized_moe_gb300 as X  # noqa: E402
import test_gpu_adamw as T  # noqa: E402


@pytest.mark.parametrize("codes", [False, True])
@pytest.mark.parametrize("lr,weight_decay,scale", [
    (1e-2, 0.1, math.nan), (1e-2, 0.0, math.nan), (1e-2, 0.1, math.inf), (1e-2, 0.0, math.inf), (1e-2, 0.1, -math.inf),
    (0.0, 0.0, math.inf), (1e30, 1e30, None), (1e20, 1e20, None), (1.0, 0.0, 3e38), (1.0, 1e3, 1e37)])
def test_a_rate_that_is_not_finite_leaves_the_step_out(lr, weight_decay, scale, codes):
    """3e38 by 1 - 0.9^5 = 0.41 is above the largest float, 3.4e38; so is 1e37 times 1e3."""
    s = T.State([300, 20], "bf16", codes=codes, master=True)
    before = s.clone()
    kw = {} if scale is None else dict(lr_scale=torch.tensor([scale], device="cuda"))
    s.go(lr=lr, weight_decay=weight_decay, **kw)
    torch.cuda.synchronize()
    assert T.same(before, s.lists()) and int(s.step) == 4 and X.exl3_workspace_error(s.ws) == 0
    if scale is not None:                              # the next one is made
        kw["lr_scale"].fill_(0.5)
        s.go(lr=1e-2, weight_decay=weight_decay, **kw)
        if 5e-3 * weight_decay <= 1:
            T.check_step(s, before, 4, lr=1e-2, weight_decay=weight_decay, lr_scale=0.5)
        else:
            # check_step's 3 u |p| hold for a decay factor of at most one; this is 1 - 5, which rounds by four times that.
            # The move is 5e-3 / 0.41 * m / (14 sqrt(v)), m / sqrt(v) at most 5 / 0.5: below 0.01, the decay about 10.
            torch.cuda.synchronize()
            want = before[-1][0].double() * (1 - 5e-3 * weight_decay)
            assert int(s.step) == 5 and float((s.mw[0].double() - want).abs().max()) < 0.02


@pytest.mark.parametrize("scale", [0.0, -0.5])
def test_other_rates_make_the_step(scale):
    s = T.State([300, 20], "f32")
    before = s.clone()
    s.go(**T.HYPER, lr_scale=torch.tensor([scale], device="cuda"))
    T.check_step(s, before, 4, **T.HYPER, lr_scale=scale)
