"""Adapters at the sizes their tensor-core kernels are made for, against float64.

Every CTA's share of these batches wraps the kernels' rings, accumulators and
buffers of h more than twice, spans several tiles, and holds items with and
without a product.  The references are computed on the GPU in float64; the
tolerances are the elementwise bounds of test_gpu_lora.py: a product summed in
fp32 over K terms errs by at most D(K) * 2^-23 * sum |terms|, h and dh are kept
in two parts (u^2 of the value), every output rounds once (u)."""
import math

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("needs a GPU", allow_module_level=True)

import trellis_quantized_moe_gb300 as X  # noqa: E402

_T = {"f16": torch.float16, "bf16": torch.bfloat16}
_U = {"f16": 2.0 ** -11, "bf16": 2.0 ** -8}
_TINY = {"f16": 2.0 ** -25, "bf16": 1e-38}


def _acc(K):
    return (K / 16 + 32) * 2.0 ** -23


class Large:
    """A batch made on the GPU: `groups` is a list of (adapter or -1, rows), in row order."""

    def __init__(self, groups, ranks, fin, fout, dtype, seed=0, max_rank=None, x=1.0, dy=0.1, A=1.0, B=0.1,
                 shuffle=False):
        g = torch.Generator(device="cuda").manual_seed(seed)
        dt = _T[dtype]

        def rnd(*shape, scale=1.0):
            return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dt)

        ids = torch.cat([torch.full((n,), a, dtype=torch.int32) for a, n in groups]).cuda()
        if shuffle:
            ids = ids[torch.randperm(len(ids), generator=g, device="cuda")].contiguous()
        self.ids, self.M, self.N, self.fin, self.fout, self.dtype = ids, len(ids), len(ranks), fin, fout, dtype
        self.scales = [(2.0, -0.5, 1.0)[i % 3] for i in range(self.N)]
        self.A = [rnd(r, fin, scale=A / math.sqrt(fin)) for r in ranks]
        self.B = [rnd(r, fout, scale=B) for r in ranks]
        self.x, self.base = rnd(self.M, fin, scale=x), rnd(self.M, fout)
        self.dy, self.dx_base = rnd(self.M, fout, scale=dy), rnd(self.M, fin, scale=dy)
        self.ad = X.DeviceAdapters(self.A, self.B, self.scales, max_rank)
        byte = lambda n: torch.randint(0, 255, (n,), dtype=torch.uint8, device="cuda")
        self.plan = byte(X.exl3_lora_plan_bytes(self.M, self.N))
        self.ws = byte(X.exl3_lora_workspace_bytes(self.M, self.N, fin, fout, self.ad.max_rank))
        nan = float("nan")
        self.y, self.dx = torch.full_like(self.base, nan), torch.full_like(self.x, nan)
        self.h = torch.full((self.M, self.ad.h_cols), nan, dtype=dt, device="cuda")
        self.dA = [torch.full_like(a, nan) for a in self.A]
        self.dB = [torch.full_like(b, nan) for b in self.B]
        self.grads = X.DeviceAdapters(self.dA, self.dB, self.scales, max_rank)

    def run(self, base="given"):
        """base: "given", "null" or "in place", of y and of dx alike."""
        b, db = self.base, self.dx_base
        if base == "in place":
            b, db = self.y.copy_(b), self.dx.copy_(db)
        elif base == "null":
            b = db = None
        X.exl3_lora_plan(self.ids, self.N, self.plan)
        X.exl3_lora_forward(self.x, self.plan, self.ad, self.y, self.ws, base=b, h=self.h)
        assert X.exl3_workspace_error(self.ws) == 0
        X.exl3_lora_backward(self.dy, self.x, self.h, self.plan, self.ad, self.grads, self.ws, dx=self.dx,
                             dx_base=db)
        assert X.exl3_workspace_error(self.plan) == 0 and X.exl3_workspace_error(self.ws) == 0
        return self

    def outputs(self):
        return [self.y, self.dx] + self.dA + self.dB


def _bounded(got, want, err, what):
    assert bool(torch.isfinite(got).all()), what
    if got.numel():
        excess = float(((got.double() - want).abs() - err).max())
        assert excess <= 0, f"{what}: {excess:.3e} over the bound"


def check(b, base=True, floor=None):
    """`floor`: absolute error that h and dh may carry beside their relative one."""
    u, tiny = _U[b.dtype], _TINY[b.dtype]
    floor = tiny if floor is None else floor
    for a in [-1] + list(range(b.N)):
        on = torch.nonzero(b.ids == a).squeeze(1)
        y = b.base[on].double() if base else torch.zeros(len(on), b.fout, dtype=torch.float64, device="cuda")
        dx = b.dx_base[on].double() if base else torch.zeros(len(on), b.fin, dtype=torch.float64, device="cuda")
        if a < 0:
            assert torch.equal(b.y[on].double(), y) and torch.equal(b.dx[on].double(), dx)
            continue
        A, B, s, x, dy = b.A[a].double(), b.B[a].double(), b.scales[a], b.x[on].double(), b.dy[on].double()
        h = x @ A.T
        eh = _acc(b.fin) * (x.abs() @ A.abs().T)
        eh += u * u * (h.abs() + eh) + floor
        dh = s * (dy @ B.T)
        edh = _acc(b.fout) * abs(s) * (dy.abs() @ B.abs().T)
        edh += u * u * (dh.abs() + edh) + floor
        r, k = A.shape[0], _acc(len(on))
        y += s * (h @ B)
        e = abs(s) * ((eh + _acc(r) * h.abs()) @ B.abs())
        _bounded(b.y[on], y, e + u * (y.abs() + e) * 1.01 + tiny, f"y of {a}")
        dx += dh @ A
        e = (edh + _acc(r) * dh.abs()) @ A.abs()
        _bounded(b.dx[on], dx, e + u * (dx.abs() + e) * 1.01 + tiny, f"dx of {a}")
        for got, want, e, what in ((b.dA[a], dh.T @ x, (edh + k * dh.abs()).T @ x.abs(), "dA"),
                                   (b.dB[a], s * (h.T @ dy), abs(s) * ((eh + k * h.abs()).T @ dy.abs()), "dB")):
            _bounded(got, want, e + u * (want.abs() + e) * 1.01 + tiny, f"{what} of {a}")


# An adapter of rank 0 before and between ranked ones.  A CTA's share is 18 to
# 34 items, a run of items without a product 7 * 40 and more: shares end and
# begin inside such runs, and go on with a product after more items without one
# than the ring has slots, twice over.
@pytest.mark.parametrize("base", ["given", "null", "in place"])
@pytest.mark.parametrize("rows,rank,dtype", [(8192, 128, "bf16"), (8192, 40, "f16"), (16384, 16, "f16")])
def test_rank_zero_before_and_between(rows, rank, dtype, base):
    q = rows // 8
    groups = [(0, q - 24), (1, 2 * q), (2, q + 131), (3, 3 * q), (-1, 77), (4, q - 184)]
    b = Large(groups, [0, rank, 0, rank // 2, rank], 5120, 5120, dtype, seed=rows + rank).run(base)
    check(b, base != "null")


def test_rank_zero_between_short_runs():
    """Many changes between items with and without a product inside each share."""
    groups = [(e, 128 * (1 + e % 3) - (e % 2) * 40) for e in range(30)]
    b = Large(groups, [0 if e % 2 == 0 else 16 for e in range(30)], 256, 1024, "bf16", seed=3).run()
    check(b)


# f16 with small h or dh, as at the start of a fine-tuning (B near zero), with
# small gradients or with small activations.  The two parts of h and dh hold 22
# bits down to 2^-14 and 2^-36 absolute below; with an absolute error of 2^-25 these
# gradients are 0.1 to 0.3% off.  Bound, of the Frobenius norm: one
# rounding of every element (u, or half the subnormal spacing), 2^-15 for sums
# of up to 4096 terms in fp32 (random signs: sqrt(4096) roundings of 2^-24 and
# the partial sums' are 2^-18; 8 times that), and 2^-36 in every h and dh.
_SMALL = [dict(B=1e-5, dy=2e-2, A=1000.0), dict(B=1e-4, dy=1e-3, A=1000.0), dict(x=1e-3, A=1e-2, B=50.0)]


def check_norms(b):
    u, tiny, floor = 2.0 ** -11, 2.0 ** -25, 2.0 ** -36
    for a in range(b.N):
        on = torch.nonzero(b.ids == a).squeeze(1)
        A, B, s, x, dy = b.A[a].double(), b.B[a].double(), b.scales[a], b.x[on].double(), b.dy[on].double()
        h, dh = x @ A.T, s * (dy @ B.T)
        one = torch.ones_like(h)
        for got, want, spread, what in ((b.y[on], s * (h @ B), one @ B.square(), "y"),
                                        (b.dx[on], dh @ A, one @ A.square(), "dx"),
                                        (b.dA[a], dh.T @ x, one.T @ x.square(), "dA"),
                                        (b.dB[a], s * (h.T @ dy), s * s * (one.T @ dy.square()), "dB")):
            rounding = torch.clamp(u * want.abs(), min=tiny)
            bound = float(rounding.norm() + 2.0 ** -15 * want.norm() + floor * spread.sqrt().norm())
            off = float((got.double() - want).norm())
            assert off <= bound, f"{what} of {a}: {off / float(want.norm()):.2e}, {bound / float(want.norm()):.2e} allowed"


@pytest.mark.parametrize("sizes", _SMALL, ids=["small B", "small dy", "small x"])
@pytest.mark.parametrize("groups,ranks,fin,fout", [
    ([(0, 300)], [8], 4096, 1408), ([(0, 150), (1, 250)], [100, 30], 1536, 1024),
    ([(0, 2000), (1, 1100)], [8, 40], 1536, 2048), ([(1, 1300), (0, 1000)], [128, 70], 2048, 1024)])
def test_small_values_keep_their_bits(groups, ranks, fin, fout, sizes):
    check_norms(Large(groups, ranks, fin, fout, "f16", seed=len(ranks), **sizes).run("null"))


def _spread(n, rows):
    return [(e, rows + 7 * (e % 5) - 14) for e in range(n)]


# Shares of many stages (wide inputs), of many tiles (128 wide: the buffers of h
# and the first product's accumulators) and of many short items (hundreds of
# adapters: the gradients' accumulators), at ranks up to 16, 64 and 128.
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("groups,ranks,fin,fout", [
    ([(0, 3000), (1, 5192)], [64, 128], 5120, 1536),
    ([(0, 3000), (1, 5192)], [60, 33], 1536, 5120),
    (_spread(16, 1024), [16] * 16, 5120, 1536),
    ([(0, 61000), (1, 39001)], [16, 9], 128, 128),
    ([(0, 61000), (1, 39001)], [64, 40], 128, 256),
    ([(0, 61000), (1, 39001)], [128, 70], 256, 128),
    (_spread(200, 40), [100, 128, 3, 90] * 50, 2048, 2048),
    (_spread(200, 40), [64, 50, 3, 33] * 50, 2048, 1024),
])
def test_large_batches(groups, ranks, fin, fout, dtype):
    b = Large(groups, ranks, fin, fout, dtype, seed=fin + len(ranks), shuffle=len(ranks) == 16).run()
    check(b, floor=2.0 ** -36 if dtype == "f16" else None)
    first = [t.clone() for t in b.outputs()]
    b.run()
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(first, b.outputs()))
