"""Optimiser states that round at random: what the host refuses (no GPU is needed)."""
import ctypes

import pytest

import __graft_entry__

__graft_entry__.build()
import trellis_quantized_moe_gb300 as X  # noqa: E402
from trellis_quantized_moe_gb300 import binding as B  # noqa: E402

P = 1 << 20          # an aligned address that nothing dereferences


@pytest.mark.parametrize("scales", [(None, None), (P, None), (None, P)])
def test_random_states_need_scales(scales):
    t = B.exl3_adamw_tensors(P, P, P, P, *scales, None, P, P, 3, 2, 1, 1, X.EXL3_E4M3_RANDOM)
    assert B.lib().exl3_adamw(ctypes.byref(t), 1e-3, 0.9, 0.99, 1e-8, 0.1, P, P, P, P, 256, None) == -1


@pytest.mark.parametrize("what", ["param_dtype", "grad_dtype"])
def test_no_other_tensor_is_rounded_at_random(what):
    t = B.exl3_adamw_tensors(P, P, P, P, P, P, None, P, P, 3, 2, 1, 1, X.EXL3_E4M3_RANDOM)
    setattr(t, what, X.EXL3_E4M3_RANDOM)
    assert B.lib().exl3_adamw(ctypes.byref(t), 1e-3, 0.9, 0.99, 1e-8, 0.1, P, P, P, P, 256, None) == -3
    assert B.lib().exl3_dispatch(P, X.EXL3_E4M3_RANDOM, 4, 2, 64, P, P, None) == -3


def test_tables_know_the_rounding():
    torch = pytest.importorskip("torch")
    p = [torch.zeros(300), torch.zeros(5)]
    c = [t.to(torch.float8_e4m3fn) for t in p]
    s = [torch.zeros(2), torch.zeros(1)]
    make = lambda **kw: X.DeviceAdamW(p, p, c, c, m_scale=s, v_scale=s, **kw).struct().state_dtype
    assert (make(), make(rounding="nearest"), make(rounding="random")) == (5, 5, 6)
    for args, kw in (((p, p, c, c), dict(m_scale=s, v_scale=s, rounding="up")), ((p, p, p, p), dict(rounding="random")),
                     ((p, p, c, c), dict(rounding="random"))):
        with pytest.raises(ValueError):
            X.DeviceAdamW(*args, **kw)
