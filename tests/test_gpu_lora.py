"""Adapters on the GPU against their definition in float64.

Tolerances are elementwise bounds of the arithmetic: u = half an ulp of the
activation type (relative); a product summed in fp32 over K terms errs by at
most D(K) * 2^-23 * sum |terms| with D(K) = K / 16 + 32 roundings in a row (a
chain of 16-term steps and what joins its parts); h and dh are kept as a rounded
value and the rounded rest (u^2), the output rounds once (u)."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("needs a GPU", allow_module_level=True)

import trellis_quantized_moe_gb300 as X  # noqa: E402
from trellis_quantized_moe_gb300.binding import (  # noqa: E402
    DERR_PLAN, DERR_ROUTE_ID, DERR_TABLE, Exl3Error)

_T = {"f16": torch.float16, "bf16": torch.bfloat16}
_U = {"f16": 2.0 ** -11, "bf16": 2.0 ** -8}
_TINY = {"f16": 2.0 ** -25, "bf16": 1e-38}


def _f64(t):
    return t.double().cpu().numpy()


def _acc(K):
    return (K / 16 + 32) * 2.0 ** -23


_PAD = 0


@pytest.fixture(autouse=True, params=["few", "many"])
def rows(request):
    """Every test runs as written, and with 1100 more rows that have no adapter:
    batches of more than 1024 rows take the tensor-core kernels."""
    global _PAD
    _PAD = 1100 if request.param == "many" else 0
    yield request.param
    _PAD = 0


class Batch:
    """Rows with their adapters, and every buffer the calls take."""

    def __init__(self, ids, ranks, fin, fout, dtype="bf16", seed=0, id64=False, max_rank=None, pad=None):
        ids = np.concatenate([np.asarray(ids, np.int64), np.full(_PAD if pad is None else pad, -1, np.int64)])
        g = torch.Generator().manual_seed(seed)
        dt = _T[dtype]

        def rnd(*shape, scale=1.0):
            return (torch.randn(*shape, generator=g) * scale).to(dt).cuda()

        self.ids_np = np.asarray(ids, np.int64)
        self.M, self.N, self.fin, self.fout, self.dtype = len(ids), len(ranks), fin, fout, dtype
        self.ids = torch.from_numpy(self.ids_np if id64 else self.ids_np.astype(np.int32)).cuda()
        self.scales = [(2.0, -0.5, 1.0)[i % 3] for i in range(self.N)]
        self.A = [rnd(r, fin, scale=fin ** -0.5) for r in ranks]
        self.B = [rnd(r, fout, scale=0.1) for r in ranks]
        self.x, self.base = rnd(self.M, fin), rnd(self.M, fout)
        self.dy, self.dx_base = rnd(self.M, fout, scale=0.1), rnd(self.M, fin, scale=0.1)
        self.ad = X.DeviceAdapters(self.A, self.B, self.scales, max_rank)
        self.plan = torch.randint(0, 255, (X.exl3_lora_plan_bytes(self.M, self.N),), dtype=torch.uint8,
                                  device="cuda")
        self.ws = torch.randint(0, 255, (X.exl3_lora_workspace_bytes(self.M, self.N, fin, fout, self.ad.max_rank),),
                                dtype=torch.uint8, device="cuda")
        nan = float("nan")
        self.y, self.dx = torch.full_like(self.base, nan), torch.full_like(self.x, nan)
        self.h = torch.full((self.M, self.ad.h_cols), nan, dtype=dt, device="cuda")
        self.dA = [torch.full_like(a, nan) for a in self.A]
        self.dB = [torch.full_like(b, nan) for b in self.B]
        self.grads = X.DeviceAdapters(self.dA, self.dB, self.scales, max_rank)

    def make_plan(self, stream=None):
        X.exl3_lora_plan(self.ids, self.N, self.plan, stream=stream)

    def forward(self, stream=None, **kw):
        d = dict(base=self.base, h=self.h)
        d.update(kw)
        X.exl3_lora_forward(self.x, self.plan, self.ad, self.y, self.ws, stream=stream, **d)

    def backward(self, stream=None, **kw):
        d = dict(dx=self.dx, dx_base=self.dx_base)
        d.update(kw)
        X.exl3_lora_backward(self.dy, self.x, self.h, self.plan, self.ad, d.pop("grads", self.grads), self.ws,
                             stream=stream, **d)

    def all(self, stream=None):
        self.make_plan(stream)
        self.forward(stream)
        self.backward(stream)
        torch.cuda.synchronize()
        assert X.exl3_workspace_error(self.plan) == 0 and X.exl3_workspace_error(self.ws) == 0
        return self

    def outputs(self):
        return [self.y, self.dx] + self.dA + self.dB


def _bounded(got, want, err, what):
    g = _f64(got)
    assert np.all(np.isfinite(g)), what
    excess = np.abs(g - want) - err
    assert not g.size or excess.max() <= 0, f"{what}: {excess.max():.3e} over the bound"


def check(b, forward=True, dx=True, grads=True, base=True, dx_base=True):
    u, tiny = _U[b.dtype], _TINY[b.dtype]
    x, dy = _f64(b.x), _f64(b.dy)
    y = _f64(b.base) if base else np.zeros((b.M, b.fout))
    dxw = _f64(b.dx_base) if dx_base else np.zeros((b.M, b.fin))
    ey, edx = np.zeros_like(y), np.zeros_like(dxw)
    for a in range(b.N):
        on = np.flatnonzero(b.ids_np == a)
        A, B, s = _f64(b.A[a]), _f64(b.B[a]), b.scales[a]
        r = A.shape[0]
        xa, ga = x[on], dy[on]
        h = xa @ A.T
        eh = _acc(b.fin) * (np.abs(xa) @ np.abs(A).T)
        eh += u * u * (np.abs(h) + eh) + tiny
        dh = s * (ga @ B.T)
        edh = _acc(b.fout) * abs(s) * (np.abs(ga) @ np.abs(B).T)
        edh += u * u * (np.abs(dh) + edh) + tiny
        y[on] += s * (h @ B)
        ey[on] += abs(s) * ((eh + _acc(r) * np.abs(h)) @ np.abs(B))
        dxw[on] += dh @ A
        edx[on] += (edh + _acc(r) * np.abs(dh)) @ np.abs(A)
        if grads:
            dA, dB = dh.T @ xa, s * (h.T @ ga)
            k = _acc(len(on))
            eA = (edh + k * np.abs(dh)).T @ np.abs(xa)
            eB = abs(s) * ((eh + k * np.abs(h)).T @ np.abs(ga))
            _bounded(b.dA[a], dA, eA + u * (np.abs(dA) + eA) * 1.01 + tiny, f"dA[{a}]")
            _bounded(b.dB[a], dB, eB + u * (np.abs(dB) + eB) * 1.01 + tiny, f"dB[{a}]")
    if forward:
        _bounded(b.y, y, ey + u * (np.abs(y) + ey) * 1.01 + tiny, "y")
    if dx:
        _bounded(b.dx, dxw, edx + u * (np.abs(dxw) + edx) * 1.01 + tiny, "dx")


def _ids(M, N, seed, idle=0.2):
    rng = np.random.default_rng(seed)
    ids = rng.integers(0, N, M)
    ids[rng.random(M) < idle] = -1
    return ids


# --------------------------------------------------------------------------- plan
def _plan_words(b):
    p = b.plan.cpu().numpy().view(np.int32)
    at = lambda o, n: p[o // 4:o // 4 + n]
    up = lambda v: (v + 255) // 256 * 256
    off = 256
    perm = up(off + (b.N + 2) * 4)
    tiles = up(perm + b.M * 4)
    small = up(tiles + (b.M // 128 + b.N + 1) * 16)
    return p[:64], at(off, b.N + 2), at(perm, b.M), at(tiles, 4 * p[4]).reshape(-1, 4), \
        at(small, 4 * p[5]).reshape(-1, 4)


@pytest.mark.parametrize("M,N", [(0, 1), (1, 1), (5, 3), (33, 2), (1024, 7), (1025, 1024), (5000, 40), (40000, 300)])
@pytest.mark.parametrize("id64", [False, True])
@pytest.mark.parametrize("rows", ["few"], indirect=True)
def test_plan_is_the_stable_grouping(M, N, id64):
    b = Batch.__new__(Batch)
    b.ids_np, b.M, b.N = _ids(M, N, M + N), M, N
    b.ids = torch.from_numpy(b.ids_np if id64 else b.ids_np.astype(np.int32)).cuda()
    b.plan = torch.randint(0, 255, (X.exl3_lora_plan_bytes(M, N),), dtype=torch.uint8, device="cuda")
    b.make_plan()
    torch.cuda.synchronize()
    hdr, off, perm, tiles, small = _plan_words(b)
    key = np.where(b.ids_np < 0, N, b.ids_np)
    assert hdr[0] == 0 and np.array_equal(perm, np.argsort(key, kind="stable"))
    assert np.array_equal(off, np.concatenate([[0], np.cumsum(np.bincount(key, minlength=N + 1))]))
    for t, size in ((tiles, 128), (small, 8)):
        want = [(a if a < N else -1, s, min(size, off[a + 1] - s), 0) for a in range(N + 1)
                for s in range(off[a], off[a + 1], size)]
        assert np.array_equal(t, np.array(want, np.int32).reshape(-1, 4))


# --------------------------------------------------------------------------- values
SHAPES = [
    # M, ranks, in, out
    (1, [16], 128, 128), (1, [1], 5120, 1536), (2, [3, 128], 1408, 640), (7, [8, 5, 17], 256, 384),
    (16, [4], 384, 128), (17, [12, 64], 1536, 256), (40, [9] * 24, 640, 1408), (129, [16], 128, 2048),
    (130, [33, 2], 2048, 128), (300, [100, 1, 31, 64, 16], 1152, 896), (513, [128], 896, 1152),
    (1000, [16, 16, 24], 640, 768), (1030, [64, 7], 384, 1664), (2500, [128, 48, 3], 512, 384),
]


@pytest.mark.parametrize("M,ranks,fin,fout", SHAPES)
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_forward_and_backward(M, ranks, fin, fout, dtype):
    b = Batch(_ids(M, len(ranks), M, idle=0.0 if M < 3 else 0.15), ranks, fin, fout, dtype, seed=M,
              id64=M % 2 == 0).all()
    check(b)


@pytest.mark.parametrize("M", [7, 8, 9, 127, 128, 129, 255, 257, 1024, 1025, 1281])
def test_one_adapter_at_tile_edges(M):
    check(Batch([0] * M, [24], 256, 256, "bf16", seed=M).all())


@pytest.mark.parametrize("M,N", [(60, 1024), (900, 700), (1500, 1024)])
def test_many_adapters(M, N):
    rng = np.random.default_rng(M)
    ranks = [int(r) for r in rng.integers(0, 20, N)]
    b = Batch(_ids(M, N, M), ranks, 128, 256, "f16", seed=M, max_rank=20).all()
    check(b)
    used = set(b.ids_np.tolist())
    assert all(not b.dA[a].any() and not b.dB[a].any() for a in range(N) if a not in used)


def test_long_contiguous_requests():
    rng = np.random.default_rng(3)
    ids = np.repeat([2, -1, 0, 2, 1, -1], [400, 30, 700, 129, 1, 60])
    check(Batch(ids, [16, 8, 40], 1536, 1024, "bf16", seed=9).all())
    check(Batch(rng.permutation(ids), [16, 8, 40], 1536, 1024, "f16", seed=9).all())


def test_adapters_without_rows_get_zero_gradients():
    b = Batch([3, 3, 1], [8, 16, 4, 32, 20], 256, 128).all()
    check(b)
    for a in (0, 2, 4):
        assert not b.dA[a].any() and not b.dB[a].any()


def test_no_row_has_an_adapter():
    b = Batch([-1] * 200, [8, 16], 256, 128).all()
    assert torch.equal(b.y, b.base) and torch.equal(b.dx, b.dx_base)
    assert not any(g.any() for g in b.dA + b.dB)


def test_idle_batches_after_failed_calls():
    """A call of rows without adapters right after one whose tables were bad: no error is left over."""
    good = Batch([-1] * 50, [8, 8], 256, 128)
    bad = Batch([0, 1] * 25, [8, 8], 256, 128)
    bad.ws = good.ws
    good.make_plan()
    bad.make_plan()
    bad.ad.t_A[1] = 0
    for _ in range(20):
        bad.forward()
        good.forward()
        bad.backward()
        good.backward()
    torch.cuda.synchronize()
    assert X.exl3_workspace_error(good.ws) == 0
    assert torch.equal(good.y, good.base) and torch.equal(good.dx, good.dx_base)
    assert not any(g.any() for g in good.dA + good.dB)


def test_rank_zero_changes_nothing():
    b = Batch([0, 1, 1, 0, -1] * 30, [0, 8], 256, 128).all()
    check(b)
    rows = b.ids_np == 0
    assert torch.equal(b.y[rows], b.base[rows])


def test_empty_batch():
    b = Batch([], [8, 3], 256, 128, pad=0)
    b.make_plan()
    b.forward()
    b.backward()
    torch.cuda.synchronize()
    assert not any(g.any() for g in b.dA + b.dB)


def test_max_rank_above_the_ranks():
    check(Batch(_ids(50, 3, 1), [3, 8, 5], 256, 384, max_rank=100).all())


@pytest.mark.parametrize("M", [3, 200])
def test_optional_tensors(M):
    ids = _ids(M, 2, 0)
    full = Batch(ids, [8, 16], 256, 384, seed=4).all()
    b = Batch(ids, [8, 16], 256, 384, seed=4)
    b.make_plan()
    b.forward(h=None)
    torch.cuda.synchronize()
    assert torch.equal(b.y, full.y)
    b.forward(base=None)
    b.backward(dx_base=None)
    torch.cuda.synchronize()
    check(b, base=False, dx_base=False)
    for g, w in zip(b.dA + b.dB, full.dA + full.dB):
        assert torch.equal(g, w)
        g.fill_(float("nan"))
    b.dx.fill_(float("nan"))
    b.backward(dx=None, dx_base=None)
    torch.cuda.synchronize()
    assert all(torch.equal(g, w) for g, w in zip(b.dA + b.dB, full.dA + full.dB)) and torch.isnan(b.dx).all()
    [g.fill_(7.0) for g in b.dA + b.dB]
    X.exl3_lora_backward(b.dy, None, None, b.plan, b.ad, None, b.ws, dx=b.dx, dx_base=b.dx_base)
    torch.cuda.synchronize()
    assert torch.equal(b.dx, full.dx) and all((g == 7.0).all() for g in b.dA + b.dB)


@pytest.mark.parametrize("M", [5, 300])
def test_in_place(M):
    ids = _ids(M, 3, 2)
    full = Batch(ids, [8, 16, 40], 384, 512, seed=4).all()
    b = Batch(ids, [8, 16, 40], 384, 512, seed=4)
    b.make_plan()
    b.y.copy_(b.base)
    b.forward(base=b.y)
    b.dx.copy_(b.dx_base)
    b.backward(dx_base=b.dx)
    torch.cuda.synchronize()
    assert all(torch.equal(g, w) for g, w in zip(b.outputs(), full.outputs()))


@pytest.mark.parametrize("M", [6, 40, 400])
def test_nan_stays_in_its_row_and_adapter(M):
    ids = np.array([0, 1, -1, 2, 1, 0] * (M // 6 + 1))[:M]
    clean = Batch(ids, [8, 16, 24], 256, 384, seed=4).all()
    b = Batch(ids, [8, 16, 24], 256, 384, seed=4)
    b.x[2] = b.dy[2] = float("nan")                    # a row without an adapter
    b.x[1] = float("inf")                              # a row of adapter 1
    b.dy[1] = float("nan")
    b.make_plan()
    b.forward()
    b.backward()
    torch.cuda.synchronize()
    other = torch.ones(b.M, dtype=torch.bool)
    other[1] = False
    assert torch.equal(b.y[other], clean.y[other]) and torch.equal(b.dx[other], clean.dx[other])
    assert not torch.isfinite(b.y[1]).any() and not torch.isfinite(b.dx[1]).any()
    for a in (0, 2):
        assert torch.equal(b.dA[a], clean.dA[a]) and torch.equal(b.dB[a], clean.dB[a])
    assert torch.isnan(b.dA[1]).all() and torch.isnan(b.dB[1]).all()


def test_nan_weights_stay_with_their_adapter():
    ids = _ids(300, 3, 6)
    clean = Batch(ids, [8, 16, 24], 256, 384, seed=4).all()
    b = Batch(ids, [8, 16, 24], 256, 384, seed=4)
    b.A[1].fill_(float("nan"))
    b.B[1].fill_(float("nan"))
    b.make_plan()
    b.forward()
    b.backward()
    torch.cuda.synchronize()
    other = torch.from_numpy(b.ids_np != 1)
    assert torch.equal(b.y[other], clean.y[other]) and torch.equal(b.dx[other], clean.dx[other])
    for a in (0, 2):
        assert torch.equal(b.dA[a], clean.dA[a]) and torch.equal(b.dB[a], clean.dB[a])


def test_gradients_against_differences():
    """Central differences of sum(dy * y) in float64 along random directions of x, A and B."""
    b = Batch(_ids(60, 2, 3), [5, 16], 256, 128, "f16", seed=5).all()
    x, dy = _f64(b.x), _f64(b.dy)

    def objective(x, A, B):
        v = 0.0
        for a in range(b.N):
            on = b.ids_np == a
            v += b.scales[a] * float(((x[on] @ A[a].T @ B[a]) * dy[on]).sum())
        return v

    A, B = [_f64(t) for t in b.A], [_f64(t) for t in b.B]
    rng = np.random.default_rng(0)
    vx = rng.normal(size=x.shape)
    vA, vB = [rng.normal(size=a.shape) for a in A], [rng.normal(size=v.shape) for v in B]
    h = 1e-3
    zero = [np.zeros_like(a) for a in A], [np.zeros_like(v) for v in B]
    grad_x = _f64(b.dx) - _f64(b.dx_base)
    # every 16-bit rounding of a gradient element (and of dx's base sum) is at
    # most u of its size; they add up like the direction's random signs, 6 sigma
    for got, size, dx_, dA_, dB_ in (
            ((grad_x * vx).sum(), _f64(b.dx), vx, *zero),
            (sum((_f64(g) * v).sum() for g, v in zip(b.dA, vA)), np.concatenate([_f64(g) for g in b.dA]), 0 * vx, vA, zero[1]),
            (sum((_f64(g) * v).sum() for g, v in zip(b.dB, vB)), np.concatenate([_f64(g) for g in b.dB]), 0 * vx, zero[0], vB)):
        up = objective(x + h * dx_, [a + h * v for a, v in zip(A, dA_)], [a + h * v for a, v in zip(B, dB_)])
        dn = objective(x - h * dx_, [a - h * v for a, v in zip(A, dA_)], [a - h * v for a, v in zip(B, dB_)])
        assert abs((up - dn) / (2 * h) - got) <= 6 * 3 * _U["f16"] * np.linalg.norm(size)


# --------------------------------------------------------------------------- how it is called
@pytest.mark.parametrize("M", [1, 30, 700])
def test_same_bits_every_time_on_other_streams_and_in_a_graph(M):
    ids, ranks = _ids(M, 3, 5, idle=0.1 if M > 1 else 0.0), [16, 8, 64]
    a = Batch(ids, ranks, 1536, 640, seed=8).all()
    side = torch.cuda.Stream()
    b = Batch(ids, ranks, 1536, 640, seed=8)
    torch.cuda.synchronize()
    b.all(side)
    assert all(torch.equal(g, w) for g, w in zip(a.outputs(), b.outputs()))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        b.make_plan(side)
        b.forward(side)
        b.backward(side)
    for rep in range(2):
        for t in b.outputs():
            t.fill_(float("nan"))
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(s, w) for s, w in zip(a.outputs(), b.outputs()))


def test_graph_of_copies_and_calls():
    """Calls captured right after copies and memsets."""
    ids = _ids(70, 3, 5)
    a = Batch(ids, [16, 8, 40], 384, 640, seed=8).all()
    b = Batch(ids, [16, 8, 40], 384, 640, seed=8)
    x, dy = b.x.clone(), b.dy.clone()
    b.make_plan()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        b.x.copy_(x)
        b.forward()
        b.dy.copy_(dy)
        b.dx.zero_()
        b.backward()
    for _ in range(2):
        b.x.zero_()
        b.dy.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(s, w) for s, w in zip(a.outputs(), b.outputs()))


def test_one_plan_serves_projections_of_other_sizes():
    ids = _ids(77, 4, 1)
    a, b = Batch(ids, [8] * 4, 256, 384, seed=1), Batch(ids, [16, 2, 40, 9], 1024, 128, "f16", seed=2)
    a.make_plan()
    b.plan = a.plan
    for t in (a, b):
        t.forward()
        t.backward()
    torch.cuda.synchronize()
    check(a)
    check(b)


def _zero_filled(b, bits):
    b.forward()
    torch.cuda.synchronize()
    assert X.exl3_workspace_error(b.ws) & bits and not b.y.any() and not torch.isnan(b.y).any()
    b.backward()
    torch.cuda.synchronize()
    assert X.exl3_workspace_error(b.ws) & bits and not b.dx.any() and not torch.isnan(b.dx).any()


@pytest.mark.parametrize("M", [10, 300])
@pytest.mark.parametrize("bad", [3, -2])
def test_bad_id(M, bad):
    ids = _ids(M, 3, 0)
    ids[M // 2] = bad
    b = Batch(ids, [8, 8, 8], 256, 128)
    b.make_plan()
    assert X.exl3_workspace_error(b.plan) == DERR_ROUTE_ID
    _zero_filled(b, DERR_ROUTE_ID)


@pytest.mark.parametrize("M", [10, 300])
def test_a_plan_of_another_batch(M):
    b, o = Batch(_ids(M, 2, 0), [8, 8], 256, 128), Batch(_ids(M + 1, 2, 0), [8, 8], 256, 128)
    o.make_plan()
    b.plan = o.plan
    _zero_filled(b, DERR_PLAN)
    b.plan = torch.zeros_like(o.plan)                  # never made
    _zero_filled(b, DERR_PLAN)


@pytest.mark.parametrize("M", [10, 300])
@pytest.mark.parametrize("what", ["null", "misaligned", "rank_high", "rank_low"])
def test_bad_table_entry(M, what):
    b = Batch(np.arange(M) % 2, [8, 8], 256, 128)
    b.make_plan()
    if what == "null":
        b.ad.t_A[1] = 0
    elif what == "misaligned":
        b.ad.t_B[1] += 8
    else:
        b.ad.t_rank[1] = 9 if what == "rank_high" else -1
    _zero_filled(b, DERR_TABLE)


def test_entries_of_adapters_without_rows_are_not_read_forward():
    b = Batch([0, 2, 2], [8, 8, 8], 256, 128)
    b.ad.t_A[1] = 0
    b.ad.t_rank[1] = 500
    b.make_plan()
    b.forward()
    torch.cuda.synchronize()
    assert X.exl3_workspace_error(b.ws) == 0
    check(b, dx=False, grads=False)


@pytest.mark.parametrize("wide", ["in", "out"])
@pytest.mark.parametrize("rows", ["many"], indirect=True)
def test_offsets_beyond_32_bits(wide):
    M, width = 430_000, 5120                            # 2.2e9 elements
    fin, fout = (width, 128) if wide == "in" else (128, width)
    ids = np.full(M, -1, np.int32)
    ids[-5:] = [0, 1, 0, 1, 1]
    g = torch.Generator().manual_seed(0)
    x = torch.zeros(M, fin, dtype=torch.float16, device="cuda")
    dy = torch.zeros(M, fout, dtype=torch.float16, device="cuda")
    x[-5:] = torch.randn(5, fin, generator=g).half().cuda()
    dy[-5:] = torch.randn(5, fout, generator=g).half().cuda() * 0.1
    s = Batch(ids[-5:], [8, 16], fin, fout, "f16", seed=1, pad=0)
    s.x.copy_(x[-5:])
    s.dy.copy_(dy[-5:])
    plan = torch.empty(X.exl3_lora_plan_bytes(M, 2), dtype=torch.uint8, device="cuda")
    ws = torch.empty(X.exl3_lora_workspace_bytes(M, 2, fin, fout, 16), dtype=torch.uint8, device="cuda")
    h = torch.empty(M, s.ad.h_cols, dtype=torch.float16, device="cuda")
    y, dx = torch.empty_like(dy), torch.empty_like(x)
    X.exl3_lora_plan(torch.from_numpy(ids).cuda(), 2, plan)
    X.exl3_lora_forward(x, plan, s.ad, y, ws, base=dy, h=h)
    X.exl3_lora_backward(dy, x, h, plan, s.ad, s.grads, ws, dx=dx, dx_base=x)
    torch.cuda.synchronize()
    s.base, s.dx_base, s.y, s.dx = s.dy, s.x, y[-5:], dx[-5:]
    check(s)
    assert not y[:-5].any() and not dx[:-5].any()


def test_refuses_host_memory_and_short_buffers():
    b = Batch([0, 1], [8, 8], 256, 128)
    b.make_plan()
    s = torch.cuda.current_stream()
    for t in ("x", "y", "base"):
        kw = {"x": b.x, "y": b.y, "base": b.base}
        kw[t] = kw[t].cpu()
        with pytest.raises(Exl3Error) as e:
            X.exl3_lora_forward(kw["x"], b.plan, b.ad, kw["y"], b.ws, base=kw["base"], stream=s)
        assert e.value.code == -2
    with pytest.raises(Exl3Error) as e:
        X.exl3_lora_forward(b.x, b.plan, b.ad, b.y, b.ws[:256], base=b.base)
    assert e.value.code == -6
    with pytest.raises(Exl3Error) as e:
        X.exl3_lora_plan(b.ids, b.N, b.plan[:256])
    assert e.value.code == -6
    torch.cuda.synchronize()
    assert torch.isnan(b.y).all()


def test_an_overflowing_h_is_an_infinity():
    """f16, h beyond 65504: infinities of the product's sign, not NaN, and no other row is touched."""
    b = Batch([0, 0, 1], [16, 16], 256, 128, "f16")
    b.A[0].fill_(4.0)
    b.B[0].fill_(1.0)
    b.x[0].fill_(100.0)             # h = 102400 in every rank
    b.x[1].fill_(0.5)
    b.make_plan()
    b.forward()
    torch.cuda.synchronize()
    assert bool((b.y[0] == float("inf")).all())
    want = _f64(b.base[1]) + 2.0 * 16 * 512
    assert np.all(np.abs(_f64(b.y[1]) - want) <= 2.0 ** -11 * np.abs(want) * 1.01)
    assert bool(torch.isfinite(b.y[2:]).all())
