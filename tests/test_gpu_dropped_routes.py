"""Routes of -1 in the fused layer, by itself and between dispatch and combine.

A dropped route adds nothing, whatever its weight; a token without routes is zero.
The workspace begins as NaN bytes and the output as NaN, so that a row that nobody
writes, or a staging row that nobody filled, shows."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("needs a GPU", allow_module_level=True)

import trellis_quantized_moe_gb300 as X  # noqa: E402
from workloads import CB_MCG, MoESpec, MoEWorkload  # noqa: E402
from gpu_common import assert_close_linear, moe_inputs, oracle_rows, out_tensor, to_f64  # noqa: E402

_REGIME = 8          # word of the workspace's header: 1 where the tcgen05 kernels ran


def workload(M, E, k, act="f16", ids="i32", rw="f32", residual=(), inter=256):
    return MoEWorkload(MoESpec("dropped", 512, inter, E, k, M, act, ids, rw, np.full(E, 4), np.full(E, CB_MCG),
                               seed=7, capacity=64, residual_K=list(residual)))


def drop(w, how, seed=0):
    """-1 into the workload's ids, NaN into their weights."""
    rng = np.random.default_rng(seed)
    M, k = w.ids.shape
    gone = np.zeros((M, k), bool)
    if how == "some":
        gone = rng.random((M, k)) < 0.3
        gone[rng.random(M) < 0.2] = True               # whole tokens
        gone[0], gone[-1] = True, True
        gone[M // 2] = False
    elif how == "one left":
        gone[:] = True
        gone[M // 2, k - 1] = False
    elif how == "last":
        gone.reshape(-1)[-max(1, M * k // 3):] = True
    else:
        gone[:] = True
    w.ids[gone] = -1
    return gone


def layer(w, gone, expect=0):
    s = w.spec
    ex = X.DeviceExperts.from_workload(w)
    x, ids, rw = moe_inputs(w)
    rw[torch.from_numpy(gone).cuda()] = float("nan")
    out = out_tensor(w).fill_(float("nan"))
    ws = torch.full((X.exl3_moe_workspace_bytes(s.M, s.topk, s.E, s.hidden, s.inter, s.capacity),), 0xFF,
                    dtype=torch.uint8, device="cuda")
    if s.residual_K:
        X.exl3_moe_additive(x, ids, rw, ex, X.DeviceStages(w.residual, w.alpha, s.residual_K, s.E), s.capacity, ws, out)
    else:
        X.exl3_moe_forward(x, ids, rw, ex, s.capacity, ws, out)
    torch.cuda.synchronize()
    assert X.exl3_workspace_error(ws) == expect
    return out, int(ws[:64].view(torch.int32)[_REGIME])


# one warp's plan; the rotate kernel and its ring (4096 rows), with the decode kernels below and above 128 tokens
# and the tcgen05 ones; residual stages
CASES = [(1, 8, 2, 0, {}), (16, 8, 2, 0, {}), (4, 16, 8, 0, dict(ids="i64", act="bf16")), (32, 8, 1, 0, {}),
         (17, 8, 2, 0, dict(ids="i64")), (64, 8, 2, 0, {}), (128, 64, 32, 0, dict(act="bf16")), (128, 8, 3, 0, {}),
         (136, 512, 2, 0, dict(ids="i64")), (2100, 1024, 2, 0, {}), (300, 8, 2, 1, dict(act="bf16")), (300, 8, 1, 1, {}),
         (2300, 8, 2, 1, dict(ids="i64")), (16, 8, 2, 0, dict(residual=(2,))), (50, 8, 2, 0, dict(residual=(3,))),
         (1100, 8, 2, 1, dict(residual=(2,)))]


@pytest.mark.parametrize("M,E,k,regime,kw", CASES)
@pytest.mark.parametrize("how", ["some", "last", "one left", "all"])
def test_layer_with_dropped_routes(M, E, k, regime, kw, how):
    w = workload(M, E, k, **kw)
    gone = drop(w, how, seed=M)
    out, took = layer(w, gone)
    if how in ("some", "last"):
        assert took == regime
    none = gone.all(axis=1)
    got = to_f64(out)
    assert np.all(got[none] == 0)
    live = np.flatnonzero(~none)
    if live.size:
        live = np.unique(np.concatenate([live[:40], live[-40:], live[len(live) // 2:][:1]]))
        assert_close_linear(got[live], oracle_rows(w, tokens=live), w.spec.act, f"dropped {how} M={M}")


@pytest.mark.parametrize("M,E,k,residual", [(16, 8, 2, ()), (100, 8, 2, ()), (128, 64, 32, ()), (50, 8, 2, (2,))])
def test_a_dropped_route_is_a_weight_of_zero(M, E, k, residual):
    """Up to 128 tokens bit for bit: fma(0, d, sum) is the sum."""
    w = workload(M, E, k, rw="f32", residual=residual)
    full = w.ids.copy()
    gone = drop(w, "some", seed=3)
    out, _ = layer(w, gone)
    w.ids[:] = full
    w.rw[gone] = 0.0
    want, _ = layer(w, np.zeros_like(gone))
    assert torch.equal(out, want)


@pytest.mark.parametrize("M", [8, 60, 400])
@pytest.mark.parametrize("bad", [-2, 8])
def test_other_ids_are_errors_still(M, bad):
    w = workload(M, 8, 2)
    gone = drop(w, "some")
    w.ids[M // 2, 1] = bad
    out, _ = layer(w, gone, expect=X.binding.DERR_ROUTE_ID)
    assert bool((out == 0).all())


def test_route_pack_by_itself_takes_no_dropped_routes():
    for M in (4, 400):
        ids = torch.zeros((M, 2), dtype=torch.int32, device="cuda")
        ids[1, 1] = -1
        new = lambda *n: torch.empty(n, dtype=torch.int32, device="cuda")
        info = new(4)
        X.exl3_route_pack(ids, 4, 8, new(5), new(2 * M), new(X.exl3_route_pack_max_tiles(M, 2, 4, 8), 3), info)
        torch.cuda.synchronize()
        assert int(info[0]) == X.binding.DERR_ROUTE_ID


def test_replays_with_changing_drops():
    """A captured call on new ids: with drops, without, and with others."""
    w = workload(64, 8, 2)
    s, full = w.spec, w.ids.copy()
    ex = X.DeviceExperts.from_workload(w)
    x, ids, rw = moe_inputs(w)
    out = out_tensor(w)
    ws = torch.empty(X.exl3_moe_workspace_bytes(s.M, s.topk, s.E, s.hidden, s.inter, s.capacity), dtype=torch.uint8,
                     device="cuda")
    go = lambda: X.exl3_moe_forward(x, ids, rw, ex, s.capacity, ws, out)
    go()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        go()
    for seed, how in enumerate(("some", None, "all", "one left", None)):
        w.ids[:] = full
        if how:
            drop(w, how, seed)
        ids.copy_(torch.from_numpy(w.ids))
        out.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        fresh = out.clone()
        ws.fill_(0xFF)
        out.fill_(float("nan"))
        go()
        torch.cuda.synchronize()
        assert torch.equal(out, fresh) and bool(out.isfinite().all())


def test_two_streams_at_once():
    """Batches with and without drops, each with buffers of its own, over the same experts."""
    ex, jobs = None, []
    for M, how in ((24, "some"), (100, None), (900, "last")):
        w = workload(M, 8, 2)
        ex = ex or X.DeviceExperts.from_workload(w)
        if how:
            drop(w, how, M)
        s = w.spec
        buffers = lambda: (out_tensor(w).fill_(float("nan")), torch.full(
            (X.exl3_moe_workspace_bytes(s.M, s.topk, s.E, s.hidden, s.inter, s.capacity),), 0xFF, dtype=torch.uint8,
            device="cuda"))
        jobs.append((moe_inputs(w), s.capacity, torch.cuda.Stream(), buffers(), buffers()))
    torch.cuda.synchronize()
    for (x, ids, rw), cap, _, (out, ws), _ in jobs:
        X.exl3_moe_forward(x, ids, rw, ex, cap, ws, out)
    torch.cuda.synchronize()
    for _ in range(20):
        for (x, ids, rw), cap, stream, _, (out, ws) in jobs:
            X.exl3_moe_forward(x, ids, rw, ex, cap, ws, out, stream=stream)
    torch.cuda.synchronize()
    for _, _, _, (alone, _), (out, _) in jobs:
        assert torch.equal(alone, out) and bool(out.isfinite().all())


@pytest.mark.parametrize("M,how", [(12, "some"), (200, "some"), (2300, "last"), (200, "one left"), (200, "all")])
def test_a_dropped_batch_through_its_experts(M, how):
    """Plan -> dispatch -> the layer on one route a row -> adapters -> combine, and the weights' gradient."""
    w = workload(M, 8, 2, rw="f32")
    gone = drop(w, how, seed=1)
    s, R = w.spec, M * 2
    ex = X.DeviceExperts.from_workload(w)
    x, ids, rw = moe_inputs(w)
    i32 = lambda *n: torch.empty(n, dtype=torch.int32, device="cuda")
    offsets, packed, slots, experts = i32(s.E + 1), i32(R), i32(M, 2), i32(R)
    ws = torch.empty(X.exl3_dispatch_workspace_bytes(M, 2, s.E), dtype=torch.uint8, device="cuda")
    X.exl3_dispatch_plan(ids, s.E, offsets, packed, slots, ws, experts=experts)
    nan = lambda n: torch.full((n, s.hidden), float("nan"), dtype=x.dtype, device="cuda")
    xp, frozen, y, out = nan(R), nan(R), nan(R), nan(M)
    X.exl3_dispatch(x, slots, xp)
    moe = torch.full((X.exl3_moe_workspace_bytes(R, 1, s.E, s.hidden, s.inter, s.capacity),), 0xFF, dtype=torch.uint8,
                     device="cuda")
    X.exl3_moe_forward(xp, experts.view(-1, 1), torch.ones((R, 1), device="cuda"), ex, s.capacity, moe, frozen)
    # adapters that add nothing (B = 0): their ids are the same, their rows the frozen ones
    zero = lambda: [torch.zeros(8, s.hidden, dtype=x.dtype, device="cuda") for _ in range(s.E)]
    ad = X.DeviceAdapters(zero(), zero(), [1.0] * s.E)
    plan = torch.empty(X.exl3_lora_plan_bytes(R, s.E), dtype=torch.uint8, device="cuda")
    lora = torch.empty(X.exl3_lora_workspace_bytes(R, s.E, s.hidden, s.hidden, 8), dtype=torch.uint8, device="cuda")
    X.exl3_lora_plan(experts, s.E, plan)
    xl = torch.where(xp.isnan(), 0.0, xp)              # an adapter plan's rows of -1 are read as base, not as x
    X.exl3_lora_forward(xl, plan, ad, y, lora, base=frozen)
    X.exl3_combine(y, slots, out, rw=rw)
    d_rw = torch.full_like(rw, float("nan"))
    X.exl3_combine_backward(x, y, slots, None, d_rw=d_rw)
    torch.cuda.synchronize()
    assert all(X.exl3_workspace_error(t) == 0 for t in (ws, moe, lora))
    live = int((~gone).sum())
    assert torch.equal(y[:live], frozen[:live]) and bool((frozen[live:] == 0).all())
    got = to_f64(out)
    assert np.all(got[gone.all(axis=1)] == 0)
    some = np.flatnonzero(~gone.all(axis=1))[:80]
    if some.size:
        assert_close_linear(got[some], oracle_rows(w, tokens=some), s.act, f"through the experts, {how}")
    at = slots.long().clamp(min=0)
    want = (x.double()[:, None] * y.double()[at]).sum(2).masked_fill(slots < 0, 0)
    size = (x.double()[:, None] * y.double()[at]).abs().sum(2)
    # at most 512 products one after the other in fp32, rounded once
    assert bool(((d_rw.double() - want).abs() <= (513 * 2.0 ** -24 * size).masked_fill(slots < 0, 0)).all())
