"""8-bit optimiser states that are rounded at random: each step against its formulas, the mean, and long runs.

What a step computes is what the states rounded to the nearest get, with the same
errors before the rounding; a code is one of the two neighbours of what it stands for."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("needs a GPU", allow_module_level=True)

import trellis_quantized_moe_gb300 as X  # noqa: E402
import test_gpu_adamw as T  # noqa: E402

U, BLOCK = T.U, T.BLOCK


def neighbours(lo, hi):
    """The largest e4m3 value at or below lo and the smallest at or above hi."""
    step = lambda y: 2.0 ** np.maximum(np.floor(np.log2(np.maximum(np.abs(y), 2.0 ** -30))) - 3, -9)
    return np.clip(np.floor(lo / step(lo)) * step(lo), -448, 448), np.clip(np.ceil(hi / step(hi)) * step(hi), -448, 448)


def check_codes(codes, scale, x, err, positive):
    if not x.size:
        return
    top, top_err = np.abs(T.blocks(x)).max(axis=1), T.blocks(err).max(axis=1)
    assert np.all(np.abs(scale.double().cpu().numpy() - top / 448) <= 1.01 * (top_err + 2 * U * top) / 448 + 2.0 ** -126)
    inv = T.spread(np.where(top > 0, 448 / np.where(top > 0, top, 1), 0), x.size)
    rel = T.spread(top_err / np.where(top > 0, top, 1), x.size) + 4 * U
    # below 2^-6 the sum with 2^-6 rounds once more, by at most 2^-30
    off = 1.01 * (err * inv + np.abs(x) * inv * rel) + 2.0 ** -30
    lo, hi = x * inv - off, x * inv + off
    if positive:
        lo, hi = (np.where((x > 0) & (y < 2.0 ** -9), 2.0 ** -9, y) for y in (lo, hi))
    lo, hi = neighbours(lo, hi)
    got = codes.cpu().double().numpy()
    zero = x == 0
    assert np.all(got[zero] == 0)
    assert np.all((lo <= got) & (got <= hi) | zero)


@pytest.fixture
def random(monkeypatch):
    """The tests of the states that round to the nearest, with states that round at random."""
    nearest = X.DeviceAdamW

    def make(*args, m_scale=None, **kw):
        return nearest(*args, m_scale=m_scale, rounding="random" if m_scale is not None else "nearest", **kw)

    monkeypatch.setattr(X, "DeviceAdamW", make)
    monkeypatch.setattr(T, "check_codes", check_codes)


@pytest.mark.parametrize("param,grad,master", T.KINDS)
def test_step(random, param, grad, master):
    T.test_step(param, grad, master, True)


@pytest.mark.parametrize("sizes", [[5], [300000], [1] * 3000, [0, 0, 4], [256] * 700 + [255] * 700, [0]])
def test_groups_of_tensors(random, sizes):
    T.test_groups_of_tensors(sizes, True)


def test_large_tensor(random):
    T.test_large_tensor()


@pytest.mark.parametrize("step", [0, 2 ** 31 - 3])
def test_scalars(random, step):
    T.test_scalars(dict(lr=1e-3, betas=(0.99, 0.9999), eps=1e-3), step, True)


def test_a_scale_that_is_not_finite(random):
    T.test_a_scale_that_is_not_finite_leaves_the_step_out(float("nan"))


@pytest.mark.parametrize("which", ["numel", "null", "scale"])
def test_bad_tables(random, which):
    T.test_bad_tables_write_nothing(which)


def test_grouping_and_streams_keep_the_bits(random):
    T.test_grouping_and_streams_keep_the_bits(True)


def test_steps_back_to_back(random):
    T.test_steps_back_to_back_are_the_steps_with_waits(True)


def test_special_values(random):
    T.test_special_values(True)
    T.test_codes_of_a_wide_block()
    T.test_a_subnormal_v_counts(True)


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_a_gradient_that_is_not_finite_stays_visible(random, bad):
    T.test_a_gradient_that_is_not_finite_stays_visible(True, bad)


def test_replays_round_like_eager_steps(random):
    """The random bits follow the step count on the device, not the capture; another count gives others."""
    sizes = [30000, 257, 77]
    a, b = (T.State(sizes, "bf16", codes=True, master=True, seed=2, step=0, fresh=True) for _ in range(2))
    for s in (a, b):
        s.go(**T.HYPER)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        b.go(**T.HYPER)
    for _ in range(5):
        a.go(**T.HYPER)
        graph.replay()
    torch.cuda.synchronize()
    assert T.same(a.lists(), b.lists()) and int(a.step) == int(b.step) == 6
    c = T.State(sizes, "bf16", codes=True, master=True, seed=2, step=7)
    d = T.State(sizes, "bf16", codes=True, master=True, seed=2, step=8)
    for s in (c, d):
        s.go(**T.HYPER)
    torch.cuda.synchronize()
    assert not torch.equal(c.m[0].view(torch.uint8), d.m[0].view(torch.uint8))


class Run:
    """One tensor under the given states, fresh."""

    def __init__(self, n, rounding):
        zero = lambda dt=torch.float32, n=n: torch.zeros(n, device="cuda").to(dt)
        self.p, self.g, self.codes = zero(), zero(), rounding is not None
        kind = torch.float8_e4m3fn if self.codes else torch.float32
        self.m, self.v = zero(kind), zero(kind)
        self.ms, self.vs = (zero(n=-(-n // BLOCK)) for _ in range(2))
        kw = dict(m_scale=[self.ms], v_scale=[self.vs], rounding=rounding) if self.codes else {}
        self.t = X.DeviceAdamW([self.p], [self.g], [self.m], [self.v], **kw)
        self.step = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.ws = torch.empty(X.exl3_adamw_workspace_bytes(), dtype=torch.uint8, device="cuda")

    def go(self, g, **kw):
        self.g.copy_(g)
        X.exl3_adamw(self.t, self.step, self.ws, lr=1e-3, **kw)

    def states(self):
        """m and sqrt(v) in float64."""
        if not self.codes:
            return self.m.double(), self.v.double().sqrt()
        return tuple(c.double() * s.double().repeat_interleave(BLOCK)[:c.numel()] for c, s in ((self.m, self.ms), (self.v, self.vs)))


@pytest.mark.parametrize("ratio", [0.9, 0.51, 0.07, 3e-3, 2e-5, 1e-6])
def test_the_mean_is_kept(ratio):
    """2^20 elements of `ratio` times their block's largest: a code's mean is what it stands for.  A rounding
    between neighbours q apart has a standard deviation of q / 2 at most: five of the mean's, and the errors before
    it (2^-20 of the value, 2^-29 below 2^-6) and the last of its 20 bits.  Every place of a warp's 256 too (4096 of each)."""
    n = 1 << 20
    a = Run(n, "random")
    g = torch.full((n,), ratio, device="cuda")
    g[::BLOCK] = 1.0
    g[BLOCK // 2::BLOCK] *= -1
    a.go(g)
    m, root = a.states()
    for got, want, floor in ((m / a.ms.double().repeat_interleave(BLOCK), g.double() * 448, 0.0),
                             (root / a.vs.double().repeat_interleave(BLOCK), g.double().abs() * 448, 2.0 ** -9)):
        y = max(ratio * 448, floor)
        q = 2.0 ** max(np.floor(np.log2(y)) - 3, -9)
        off = (got - want.sign() * y).view(-1, BLOCK)[:, 1:]
        err = 2.0 ** -19 * y + 2.0 ** -29 + 2.0 ** -20 * q
        assert abs(float(off.mean())) <= 2.5 * q / off.numel() ** 0.5 + err
        assert bool((off.mean(dim=0).abs() <= 3 * q / off.shape[0] ** 0.5 + err).all())


@pytest.mark.parametrize("change", [1 / 20, 4.0])
def test_a_long_run_follows_the_gradients(change):
    """After 1500 steps half of the elements' gradients change their size; 5000 more, five times what v
    remembers.  Against float32 states of the same gradients, on average over either half.

    A step moves s = sqrt(v) by up to 1 - sqrt(beta2) = 0.0005 s, rounded between codes at most s / 8 apart: it adds at
    most 0.0005 / 8 s^2 to the variance of s and nothing to its mean.  Where s stays, deviations
    shrink by 0.001 of them a step: a variance of 0.03 s^2; where it falls 20-fold in ln 20 / 0.0005 steps, 0.37.  The mean
    of g^2 / s is above g^2 / mean by the variance, and half of it is what s is too large: 0.19 at
    most.  (To the nearest: 8 times too large, and 2.8 times beside gradients that grew.)"""
    n = 1 << 15
    gen = torch.Generator(device="cuda").manual_seed(1)
    size = torch.exp(1.5 * torch.randn(n, generator=gen, device="cuda")) * 1e-3
    half = torch.rand(n, generator=gen, device="cuda") < 0.5
    a, b = Run(n, "random"), Run(n, None)
    for i in range(6500):
        if i == 1500:
            size = torch.where(half, size * change, size)
        g = torch.randn(n, generator=gen, device="cuda") * size
        a.go(g)
        b.go(g)
        if i in (1499, 2200, 4000, 6499):
            (m, s), (m32, s32) = a.states(), b.states()
            ratio = s / s32
            for part in (half, ~half):
                assert 0.95 < float(ratio[part].mean()) < 1.19
            # m: a mean of ten steps, each rounded by up to an eighth
            assert float((m - m32).norm() / m32.norm()) < 0.125


def test_an_element_whose_gradients_stop_comes_to_rest():
    """With beta1 = 0.95 codes of m from 1 to 10 times 2^-9, and more, round to the nearest back to themselves.  At
    random their mean is 0.95^400 of at most 448 after 400 steps, 2.9e-4 times 2^-9: of 8192 elements 2.4 are not zero, at most."""
    n = 1 << 14
    gen = torch.Generator(device="cuda").manual_seed(2)
    a = Run(n, "random")
    stop = torch.arange(n, device="cuda") % 2 == 1
    for i in range(500):
        g = torch.randn(n, generator=gen, device="cuda")
        a.go(torch.where(stop, 0.0, g) if i >= 100 else g, betas=(0.95, 0.999))
    m, s = a.states()
    assert int((m[stop] != 0).sum()) <= 20
    assert float((m[~stop] != 0).double().mean()) > 0.99
    # and v: 1 - 0.999^100 of the gradients' square, then 0.999^400 of that, beside 1 - 0.999^500
    want = ((1 - 0.999 ** 100) * 0.999 ** 400 / (1 - 0.999 ** 500)) ** 0.5
    assert abs(float(s[stop].mean() / s[~stop].mean()) - want) < 0.1
