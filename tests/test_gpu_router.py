"""Router on the GPU against its definitions in float64.

Tolerances (set from the arithmetic).  p = exp(l - m) / s: the subtraction
rounds |l - m| <= 64 to 2^-24 relative (3.8e-6 of p), expf gives 2 ulp, a sum
of at most 1024 positive terms and the division a few 2^-24 more: 1e-5 in all.
Every output then rounds once to its own type.  A gradient element is a
difference of terms of size p (|G| + sum p |G|): each carries 2e-5 of that."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("needs a GPU", allow_module_level=True)

import trellis_quantized_moe_gb300 as X  # noqa: E402
from trellis_quantized_moe_gb300.binding import Exl3Error  # noqa: E402

_T = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
_HALF_ULP = {"f16": 2.0 ** -11, "bf16": 2.0 ** -8, "f32": 2.0 ** -24}
_TINY = {"f16": 2.0 ** -25, "bf16": 1e-38, "f32": 1e-38}
RTOL = 1e-5


def _f64(t):
    return t.double().cpu().numpy()


def oracle(z, k, renorm, valid=None, d_rw=None, d_loss=0.0):
    """ids, rw, stats, counts, loss, d_logits and the size of its terms, in float64."""
    M, E = z.shape
    key = np.where(np.isnan(z), -np.inf, z)
    ids = np.argsort(-key, axis=1, kind="stable")[:, :k]
    with np.errstate(invalid="ignore", divide="ignore"):
        m = np.max(z, axis=1, keepdims=True) if M else np.zeros((0, 1))
        ref = np.where(m == -np.inf, 0.0, m)
        ex = np.exp(z - ref)
        s = ex.sum(axis=1, keepdims=True)
        p = np.where(s == 0, 0.0, ex / np.where(s == 0, 1.0, s))
        stats = np.concatenate([ref, s], axis=1)
    t = np.arange(M)[:, None]
    w = p[t, ids]
    tot = w.sum(axis=1, keepdims=True)
    rw = np.where(tot == 0, 0.0, w / np.where(tot == 0, 1.0, tot)) if renorm else w
    v = np.ones(M, bool) if valid is None else valid.astype(bool)
    T = int(v.sum())
    c = np.bincount(ids[v].ravel(), minlength=E) if M else np.zeros(E, int)
    loss = E / (k * T) * float((c * p[v].mean(axis=0)).sum()) if T else 0.0
    G = np.zeros((M, E))
    if T:
        G += v[:, None] * (d_loss * E / (k * T * T) * c)
    dl = np.zeros((M, E))
    size = np.zeros((M, E))
    if d_rw is not None and not renorm:
        np.add.at(G, (np.broadcast_to(t, ids.shape), ids), d_rw)
    dl += p * (G - (p * G).sum(axis=1, keepdims=True))
    size += p * (np.abs(G) + (p * np.abs(G)).sum(axis=1, keepdims=True))
    if d_rw is not None and renorm:
        dl[t, ids] += rw * (d_rw - (rw * d_rw).sum(axis=1, keepdims=True))
        size[t, ids] += rw * (np.abs(d_rw) + (rw * np.abs(d_rw)).sum(axis=1, keepdims=True))
    return dict(ids=ids, rw=rw, stats=stats, counts=np.append(c, T), loss=loss, dl=dl, size=size)


class Call:
    """One forward (and backward) call on given logits."""

    def __init__(self, logits, k, rw="f32", renorm=False, valid=None, balance=True, d_rw=None, d_loss=None,
                 backward=False, stream=None, stats=True):
        M, E = logits.shape
        dev = logits.device
        self.ids = torch.full((M, k), -9, dtype=torch.int32, device=dev)
        self.rw = torch.full((M, k), float("nan"), dtype=_T[rw], device=dev)
        self.stats = torch.empty((M, 2), dtype=torch.float32, device=dev) if stats else None
        self.counts = torch.full((E + 1,), -9, dtype=torch.int32, device=dev) if balance else None
        self.loss = torch.full((1,), float("nan"), device=dev) if balance else None
        ws = torch.randint(0, 255, (X.exl3_router_workspace_bytes(M, E),), dtype=torch.uint8, device=dev)
        self.go = lambda: X.exl3_router_forward(
            logits, self.ids, self.rw, renorm=renorm, stats=self.stats, valid=valid, counts=self.counts,
            loss=self.loss, workspace=ws if balance else None, stream=stream)
        self.go()
        if backward:
            self.dl = torch.full_like(logits, float("nan"))
            b = d_loss is not None
            self.back = lambda: X.exl3_router_backward(
                logits, self.ids, self.stats, self.dl, renorm=renorm, d_rw=d_rw, valid=valid if b else None,
                counts=self.counts if b else None, d_loss=d_loss, stream=stream)
            self.back()
        torch.cuda.synchronize()


def _logits(M, E, dtype, seed, spread=2.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(M, E, generator=g) * spread - 1.2 * torch.log(1.0 + torch.arange(E))).to(_T[dtype]).cuda()


def _check(got, ref, rw, dtype, backward=True):
    assert np.array_equal(got.ids.cpu().numpy(), ref["ids"])
    g = _f64(got.rw)
    tol = (RTOL + _HALF_ULP[rw] * 1.01) * ref["rw"] + _TINY[rw]
    assert np.all(np.abs(g - ref["rw"]) <= tol)
    if got.stats is not None:
        stats, want = _f64(got.stats), ref["stats"]
        assert np.array_equal(stats[:, 0], want[:, 0])
        assert np.all(np.abs(stats[:, 1] - want[:, 1]) <= RTOL * want[:, 1])
    if got.counts is not None:
        assert np.array_equal(got.counts.cpu().numpy(), ref["counts"])
        assert abs(float(got.loss) - ref["loss"]) <= 2 * RTOL * ref["loss"]
    if backward:
        tol = 2 * RTOL * ref["size"] + 1.01 * _HALF_ULP[dtype] * np.abs(ref["dl"]) + _TINY[dtype]
        assert np.all(np.abs(_f64(got.dl) - ref["dl"]) <= tol)


SHAPES = [(1, 1, 1), (1, 192, 8), (2, 2, 2), (3, 7, 3), (5, 31, 31), (7, 33, 4), (16, 8, 2), (33, 64, 6),
          (257, 160, 8), (64, 257, 9), (9, 512, 8), (1000, 288, 8), (4, 1000, 32), (6, 1024, 10), (31, 96, 1)]


@pytest.mark.parametrize("M,E,k", SHAPES)
@pytest.mark.parametrize("dtype,rw", [("f32", "f32"), ("bf16", "f16"), ("f16", "bf16")])
@pytest.mark.parametrize("renorm", [False, True])
def test_forward_and_backward(M, E, k, dtype, rw, renorm):
    z = _logits(M, E, dtype, seed=M + E)
    valid = (torch.arange(M) % 5 != 2).to(torch.uint8).cuda()
    d_rw = torch.randn(M, k, generator=torch.Generator().manual_seed(k)).to(_T[rw]).cuda()
    d_loss = torch.tensor([0.37], device="cuda")
    got = Call(z, k, rw, renorm, valid, d_rw=d_rw, d_loss=d_loss, backward=True)
    ref = oracle(_f64(z), k, renorm, valid.cpu().numpy(), _f64(d_rw), float(d_loss))
    _check(got, ref, rw, dtype)


@pytest.mark.parametrize("rows", ["none", "no_valid", "all_valid_null"])
def test_valid_mask_extremes(rows):
    z = _logits(21, 24, "f32", 3)
    valid = None if rows == "all_valid_null" else torch.full((21,), 0 if rows == "no_valid" else 1,
                                                           dtype=torch.uint8, device="cuda")
    d_loss = torch.tensor([1.5], device="cuda")
    got = Call(z, 4, valid=valid, d_loss=d_loss, backward=True)
    ref = oracle(_f64(z), 4, False, None if valid is None else valid.cpu().numpy(), None, 1.5)
    _check(got, ref, "f32", "f32")
    if rows == "no_valid":
        assert float(got.loss) == 0.0 and not got.dl.any() and not got.counts.any()


def test_empty_batch():
    z = torch.empty(0, 16, device="cuda")
    got = Call(z, 4, d_loss=torch.ones(1, device="cuda"), backward=True)
    assert not got.counts.any() and float(got.loss) == 0.0


def test_any_nonzero_byte_is_valid():
    z = _logits(40, 16, "f32", 5)
    valid = torch.tensor([0, 1, 2, 255] * 10, dtype=torch.uint8, device="cuda")
    got = Call(z, 3, valid=valid)
    _check(got, oracle(_f64(z), 3, False, valid.cpu().numpy() != 0), "f32", "f32", backward=False)


@pytest.mark.parametrize("E,k", [(8, 8), (40, 7), (192, 8), (700, 16)])
def test_ties_go_to_the_lower_expert(E, k):
    g = torch.Generator().manual_seed(E)
    z = torch.randint(-2, 2, (50, E), generator=g).float()
    z[0] = 0.0
    z[1] = torch.where(torch.arange(E) % 2 == 0, -0.0, 0.0)      # -0 and +0 tie
    z = z.cuda()
    _check(Call(z, k), oracle(_f64(z), k, False), "f32", "f32", backward=False)


@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_switched_off_experts_and_empty_rows(renorm, dtype):
    E, k = 70, 6
    z = _logits(12, E, dtype, 8)
    z[0] = float("-inf")                                # nothing left
    z[1, :] = float("-inf")
    z[1, 65] = -3.0                                     # one expert left
    z[2, 5:] = float("-inf")                            # fewer than k left
    z[3, :5] = torch.finfo(_T[dtype]).min               # the type's lowest value
    z[4, :] = torch.finfo(_T[dtype]).min
    d_rw = torch.randn(12, k, generator=torch.Generator().manual_seed(1)).cuda()
    got = Call(z, k, renorm=renorm, d_rw=d_rw, d_loss=torch.tensor([2.0], device="cuda"), backward=True)
    ref = oracle(_f64(z), k, renorm, None, _f64(d_rw), 2.0)
    _check(got, ref, "f32", dtype)
    assert got.ids[0].tolist() == list(range(k)) and not got.rw[0].any() and not got.dl[0].any()


def test_large_logits_and_spreads():
    z = torch.tensor([[60000.0, 59990.0, -60000.0, 0.0], [-60000.0, -60001.0, -60000.5, -59999.0]],
                     device="cuda")
    _check(Call(z, 2), oracle(_f64(z), 2, False), "f32", "f32", backward=False)


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_nan_and_inf_stay_in_their_row(bad):
    z = _logits(9, 130, "f32", 4)
    clean = Call(z, 5, d_rw=torch.ones(9, 5, device="cuda"), balance=False, backward=True)
    z[4, 77] = bad
    got = Call(z, 5, d_rw=torch.ones(9, 5, device="cuda"), balance=False, backward=True)
    keep = [t for t in range(9) if t != 4]
    assert torch.isnan(got.rw[4]).all() and torch.isnan(got.dl[4]).all()
    ids = got.ids[4].tolist()
    assert len(set(ids)) == 5 and all(0 <= e < 130 for e in ids)
    assert (77 == ids[0]) if bad == float("inf") else (77 not in ids)
    for a, b in ((got.ids, clean.ids), (got.rw, clean.rw), (got.dl, clean.dl)):
        assert torch.equal(a[keep], b[keep])
    b = Call(z, 5)
    assert torch.isnan(b.loss).all()


def test_a_padding_row_of_nan_leaves_the_loss():
    z = _logits(9, 30, "bf16", 4)
    valid = torch.ones(9, dtype=torch.uint8, device="cuda")
    valid[4] = 0
    want = Call(z, 5, valid=valid)
    z[4] = float("nan")
    got = Call(z, 5, valid=valid)
    assert torch.equal(got.loss, want.loss) and torch.equal(got.counts, want.counts)


@pytest.mark.parametrize("renorm", [False, True])
def test_gradient_against_differences(renorm):
    """A central difference of the float64 objective along a random direction (choices fixed by wide gaps)."""
    M, E, k = 11, 14, 3
    rng = np.random.default_rng(5)
    z = np.stack([rng.permutation(E) * 0.35 for _ in range(M)])
    valid = (np.arange(M) % 4 != 1).astype(np.uint8)
    d_rw, d_loss = rng.normal(size=(M, k)).astype(np.float32), 0.8
    zt = torch.from_numpy(z.astype(np.float32)).cuda()
    got = Call(zt, k, renorm=renorm, valid=torch.from_numpy(valid).cuda(),
               d_rw=torch.from_numpy(d_rw).cuda(), d_loss=torch.tensor([d_loss], device="cuda"), backward=True)
    z = z.astype(np.float32).astype(np.float64)
    base = oracle(z, k, renorm, valid)

    def objective(zz):
        o = oracle(zz, k, renorm, valid)
        assert np.array_equal(o["ids"], base["ids"])
        return float((d_rw * o["rw"]).sum()) + np.float32(d_loss) * o["loss"]

    for seed in range(4):
        v = np.random.default_rng(seed).normal(size=z.shape)
        h = 1e-4
        num = (objective(z + h * v) - objective(z - h * v)) / (2 * h)
        # third-order remainder h^2 |v|^3 / 6 ~ 1e-8 * 150 * 3 and 2e-5 of the terms' sum
        assert abs(num - float((_f64(got.dl) * v).sum())) <= 1e-5 + 2e-5 * float((base["rw"].size))


def test_outputs_are_optional():
    z = _logits(30, 48, "bf16", 6)
    full = Call(z, 4)
    slim = Call(z, 4, balance=False, stats=False)
    nolse = Call(z, 4, stats=False)
    assert torch.equal(full.ids, slim.ids) and torch.equal(full.rw, slim.rw)
    assert torch.equal(full.loss, nolse.loss) and torch.equal(full.counts, nolse.counts)


def test_backward_in_place_and_bad_ids():
    z = _logits(30, 48, "f32", 6)
    d = torch.randn(30, 4, device="cuda")
    c = Call(z, 4, d_rw=d, balance=False, backward=True)
    zz = z.clone()
    X.exl3_router_backward(zz, c.ids, c.stats, zz, d_rw=d)
    torch.cuda.synchronize()
    assert torch.equal(zz, c.dl)
    ids, dz, d0 = c.ids.clone(), torch.empty_like(z), d.clone()
    ids[3, 1], ids[4, 2] = 48, -1
    d0[3, 1] = d0[4, 2] = 0.0
    X.exl3_router_backward(z, ids, c.stats, dz, d_rw=d)
    torch.cuda.synchronize()
    want = torch.empty_like(z)
    X.exl3_router_backward(z, c.ids, c.stats, want, d_rw=d0)
    torch.cuda.synchronize()
    assert torch.allclose(dz, want, rtol=1e-5, atol=1e-7)


def test_same_bits_every_time_and_on_another_stream():
    z = _logits(5000, 192, "bf16", 2)
    d = torch.randn(5000, 8, device="cuda")
    dl = torch.tensor([0.5], device="cuda")
    a = Call(z, 8, d_rw=d, d_loss=dl, backward=True)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for stream in (None, side):
        b = Call(z, 8, d_rw=d, d_loss=dl, backward=True, stream=stream)
        for n in ("ids", "rw", "stats", "counts", "loss", "dl"):
            assert torch.equal(getattr(a, n), getattr(b, n)), n


def test_graph_replay():
    z = _logits(700, 96, "bf16", 2)
    c = Call(z, 6, d_rw=torch.ones(700, 6, device="cuda"), d_loss=torch.ones(1, device="cuda"), backward=True)
    g = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(g, stream=side):
        c.go()
        c.back()
    z2 = _logits(700, 96, "bf16", 77)
    want = Call(z2, 6, d_rw=torch.ones(700, 6, device="cuda"), d_loss=torch.ones(1, device="cuda"), backward=True)
    z.copy_(z2)
    g.replay()
    torch.cuda.synchronize()
    for n in ("ids", "rw", "counts", "loss", "dl"):
        assert torch.equal(getattr(c, n), getattr(want, n)), n


def test_graph_of_copies_and_calls():
    """Captured right after a copy and between memsets, as the first and the last node of a graph."""
    z, src = _logits(90, 64, "f32", 2), _logits(90, 64, "f32", 3)
    c = Call(z, 6, d_rw=torch.ones(90, 6, device="cuda"), d_loss=torch.ones(1, device="cuda"), backward=True)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        z.copy_(src)
        c.go()
        c.dl.zero_()
        c.back()
    want = Call(src, 6, d_rw=torch.ones(90, 6, device="cuda"), d_loss=torch.ones(1, device="cuda"), backward=True)
    for _ in range(2):
        z.zero_()
        g.replay()
        torch.cuda.synchronize()
        for n in ("ids", "rw", "counts", "loss", "dl"):
            assert torch.equal(getattr(c, n), getattr(want, n)), n


def test_offsets_beyond_32_bits():
    M, E, k = 2_200_000, 1024, 2                       # 2.25e9 logits
    z = torch.zeros(M, E, dtype=torch.float16, device="cuda")
    tail = _logits(64, E, "f16", 9)
    z[-64:] = tail
    got = Call(z, k, rw="f16", balance=False, d_rw=torch.ones(M, k, dtype=torch.float16, device="cuda"), backward=True)
    ref = oracle(_f64(tail), k, False, None, np.ones((64, k)))
    assert got.ids[0].tolist() == [0, 1]
    got.ids, got.rw, got.stats, got.dl = got.ids[-64:], got.rw[-64:], got.stats[-64:], got.dl[-64:]
    _check(got, ref, "f16", "f16")


def test_refuses_host_memory():
    z = torch.zeros(4, 8)
    with pytest.raises(Exl3Error) as e:
        X.exl3_router_forward(z, torch.zeros(4, 2, dtype=torch.int32), torch.zeros(4, 2),
                              stream=torch.cuda.current_stream())
    assert e.value.code == -2


def test_refuses_a_short_workspace():
    z = _logits(4000, 16, "f32", 1)
    ids = torch.full((4000, 2), -5, dtype=torch.int32, device="cuda")
    rw = torch.full((4000, 2), -5.0, device="cuda")
    n = X.exl3_router_workspace_bytes(4000, 16)
    ws = torch.zeros(n, dtype=torch.uint8, device="cuda")[:n - 256]
    with pytest.raises(Exl3Error) as e:
        X.exl3_router_forward(z, ids, rw, counts=torch.zeros(17, dtype=torch.int32, device="cuda"),
                              loss=torch.zeros(1, device="cuda"), workspace=ws)
    torch.cuda.synchronize()
    assert e.value.code == -6 and (ids == -5).all() and (rw == -5).all()


def test_feeds_the_expert_layer():
    """Routed by exl3_router_forward, the layer gives the bytes it gives with the oracle's ids and weights."""
    from workloads import MoEWorkload, config
    w = MoEWorkload(config(0))
    s = w.spec
    ex = X.DeviceExperts.from_workload(w)
    x = torch.from_numpy(w.x).cuda()
    z = _logits(s.M, s.E, "f32", 12)
    r = Call(z, s.topk, rw="f16", balance=False)
    ws = torch.empty(X.exl3_moe_workspace_bytes(s.M, s.topk, s.E, s.hidden, s.inter, s.capacity),
                     dtype=torch.uint8, device="cuda")
    outs = []
    for ids, rw in ((r.ids, r.rw), (torch.from_numpy(oracle(_f64(z), s.topk, False)["ids"].astype(np.int32)).cuda(),
                                    r.rw)):
        out = torch.empty((s.M, s.hidden), dtype=torch.float16, device="cuda")
        X.exl3_moe_forward(x, ids, rw, ex, s.capacity, ws, out)
        torch.cuda.synchronize()
        assert X.exl3_workspace_error(ws) == 0
        outs.append(out)
    assert torch.equal(*outs) and torch.isfinite(outs[0]).all() and outs[0].abs().max() > 0


@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("E", [192, 40])
def test_small_probabilities_have_fp32s_precision(E, renorm):
    """Logits on a grid of 1/64, so that l - m is exact, and the chosen ones about ten apart: weights
    down to 1e-33.  What is left to round: exp (1 ulp = 2 * 2^-24), the sum s (V + 5 additions), a
    division (1), with renorm a second sum (5) and division (1): 24 * 2^-24 with V = 6 and exp's own
    error in s.  A gradient adds sums of products of the same kind and three roundings."""
    k, M, eps = 8, 400, 2.0 ** -24
    g = torch.Generator().manual_seed(E)
    z = torch.randint(-90 * 64, -85 * 64, (M, E), generator=g).float() / 64
    gaps = torch.randint(9 * 64, 11 * 64, (M, k), generator=g).float() / 64
    at = torch.argsort(torch.rand(M, E, generator=g), dim=1)[:, :k]
    z.scatter_(1, at, 3.0 - torch.cumsum(gaps, dim=1) + gaps[:, :1])
    d_rw = torch.randn(M, k, generator=g).cuda()
    z = z.cuda()
    got = Call(z, k, "f32", renorm, d_rw=d_rw, balance=False, backward=True)
    ref = oracle(_f64(z), k, renorm, None, _f64(d_rw))
    assert np.array_equal(got.ids.cpu().numpy(), ref["ids"])
    off = np.abs(_f64(got.rw) - ref["rw"])
    assert np.all(off <= 24 * eps * ref["rw"]), f"weights: {(off / ref['rw']).max() / eps:.1f} * 2^-24"
    off = np.abs(_f64(got.dl) - ref["dl"])
    assert np.all(off <= 48 * eps * ref["size"] + 1e-44), f"gradients: {(off / (ref['size'] + 1e-40)).max() / eps:.1f} * 2^-24"


def test_bool_mask_of_valid_rows():
    z = _logits(40, 16, "bf16", 5)
    valid = torch.arange(40, device="cuda") % 3 != 1
    d_loss = torch.ones(1, device="cuda")
    a, b = (Call(z, 3, valid=v, d_loss=d_loss, backward=True) for v in (valid, valid.to(torch.uint8)))
    for n in ("ids", "rw", "counts", "loss", "dl"):
        assert torch.equal(getattr(a, n), getattr(b, n)), n
    with pytest.raises(ValueError):
        Call(z, 3, valid=valid.to(torch.int32))
