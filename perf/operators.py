"""The router with its balance loss and the low-rank adapters, as measured cases.

Two families of calls a user of the routed-expert layer makes around it:

* the router: logits -> top-k experts and route weights; in training also the
  per-expert counts, the balance loss and the gradient of the logits;
* low-rank adapters of many requests beside a shared projection: base output
  plus scale * (x A^T) B with every row's own adapter; in training also the
  gradients of x, A and B.

``own`` selects the framework's entry points; otherwise the same quantities are
computed by elementary torch operations in float32.
"""
import math
import random

import numpy as np
import torch

own = False

_DT = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
_SIZE = {"f16": 2, "bf16": 2, "f32": 4}


# --------------------------------------------------------------------------- cases
def _router(name, M, E, k, dtype, rw, train, renorm=False, pad=0.0, off=0):
    return {"name": name, "op": "router", "M": M, "E": E, "k": k, "dtype": dtype, "rw": rw,
            "train": train, "renorm": renorm, "pad": pad, "off": off}


def _lora(name, M, requests, adapters, idle, lo, hi, fin, fout, dtype, train):
    return {"name": name, "op": "lora", "M": M, "requests": requests, "adapters": adapters,
            "idle": idle, "rank_lo": lo, "rank_hi": hi, "in": fin, "out": fout, "dtype": dtype,
            "train": train}


def listed():
    return [
        # one decode token through the router of a 192-expert layer
        _router("route_token", 1, 192, 8, "f32", "f32", False),
        # a prompt chunk; weights renormalised over the chosen experts, three experts switched off
        _router("route_prompt", 2000, 192, 8, "bf16", "bf16", False, renorm=True, off=3),
        # the smallest training step: a small layer, a short batch
        _router("route_train_small", 16, 8, 2, "f16", "f16", True, renorm=True),
        # an ordinary training batch with padding tokens, float32 logits, 288 experts
        _router("route_train_padded", 4097, 288, 8, "f32", "f32", True, pad=0.1),
        # a large training batch
        _router("route_train_large", 65536, 192, 8, "bf16", "f32", True),
        # one decode token of one request
        _lora("adapter_token", 1, 1, 1, 0, 16, 16, 5120, 1536, "bf16", False),
        # a decode batch: 64 requests of one token, 40 adapters of mixed ranks, five without one
        _lora("adapter_decode", 64, 64, 40, 5, 8, 64, 5120, 1536, "bf16", False),
        # prompts and decode tokens in one batch, small ragged ranks, the down projection
        _lora("adapter_mixed", 1000, 23, 7, 2, 4, 32, 1536, 5120, "f16", False),
        # many prompts at once
        _lora("adapter_prompts", 16384, 40, 16, 0, 16, 16, 5120, 1536, "bf16", False),
        # a short fine-tuning batch of one adapter
        _lora("adapter_train_small", 300, 3, 1, 0, 8, 8, 4096, 1408, "f16", True),
        # an ordinary fine-tuning batch of two adapters
        _lora("adapter_train", 4096, 8, 2, 0, 32, 32, 1536, 5120, "bf16", True),
        # a large batch of high ranks
        _lora("adapter_train_large", 8192, 24, 2, 0, 64, 128, 5120, 1536, "bf16", True),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    top = {}
    for c in listed():
        w = work(c)
        for key in w:
            top[key] = max(top.get(key, 0), w[key])
    while True:
        if rng.random() < 0.4:
            E = _log_int(rng, 8, 512)
            c = _router("", _log_int(rng, 1, 65536), E, rng.randint(1, min(E, 10)),
                        rng.choice(["f16", "bf16", "f32"]), rng.choice(["f16", "bf16", "f32"]),
                        rng.random() < 0.6, rng.random() < 0.5, rng.choice([0.0, 0.0, 0.1, 0.5]),
                        rng.choice([0, 0, 1, E // 8]))
        else:
            M = _log_int(rng, 1, 16384)
            requests = M if rng.random() < 0.3 and M <= 512 else _log_int(rng, 1, min(M, 256))
            idle = rng.choice([0, 0, requests // 8])
            adapters = _log_int(rng, 1, min(requests - idle, 64))
            hi = _log_int(rng, 4, 128)
            lo = hi if rng.random() < 0.5 else rng.randint(1, hi)
            fin, fout = (128 * rng.choice([4, 5, 6, 8, 10, 11, 12, 16, 20, 28, 32, 40, 47])
                         for _ in range(2))
            c = _lora("", M, requests, adapters, idle, lo, hi, fin, fout,
                      rng.choice(["f16", "bf16"]), rng.random() < 0.5)
        w = work(c)
        if all(w[key] <= top[key] for key in w):
            del c["name"]
            return c


# --------------------------------------------------------------------------- what a batch looks like
def _ranks(c):
    n, lo, hi = c["adapters"], c["rank_lo"], c["rank_hi"]
    return [lo + (hi - lo) * i // max(n - 1, 1) for i in range(n)]


def _requests(c):
    """(rows, adapter or -1) of every request: ragged lengths that add up to M, every adapter used."""
    rng = random.Random("-".join(str(c[k]) for k in ("M", "requests", "adapters", "idle")))
    q = c["requests"]
    cuts = sorted(rng.sample(range(1, c["M"]), q - 1)) if q > 1 else []
    rows = [b - a for a, b in zip([0] + cuts, cuts + [c["M"]])]
    live = q - c["idle"]
    which = [i if i < c["adapters"] else rng.randrange(c["adapters"]) for i in range(live)]
    return list(zip(rows, which + [-1] * c["idle"]))


def work(c):
    M = c["M"]
    if c["op"] == "router":
        E, k, s, sr = c["E"], c["k"], _SIZE[c["dtype"]], _SIZE[c["rw"]]
        n = M * E * s + M * k * (4 + sr)
        f = 5 * M * E
        if c["train"]:
            n += M * E * s + M * k * sr + M + 4 * (E + 2)
            f += 6 * M * E
        return {"bytes": n, "flops": f}
    s, fin, fout, ranks = _SIZE[c["dtype"]], c["in"], c["out"], _ranks(c)
    reqs = _requests(c)
    live = sum(n for n, a in reqs if a >= 0)
    weights = sum(ranks) * (fin + fout) * s
    n = live * fin * s + 2 * M * fout * s + weights + 4 * M
    f = sum(2 * rows * ranks[a] * (fin + fout) for rows, a in reqs if a >= 0)
    if c["train"]:
        n += live * fout * s + 2 * M * fin * s + weights
        f *= 3
    return {"bytes": n, "flops": f}


# --------------------------------------------------------------------------- inputs
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _normal(g, shape, scale=1.0):
    return torch.randn(shape, generator=g, device="cuda") * scale


def _router_inputs(c, seed):
    g = _gen(seed)
    M, E, k = c["M"], c["E"], c["k"]
    # a trained router's preferences: N(0, 1) per token on a Zipf-shaped bias over the experts
    order = torch.randperm(E, generator=g, device="cuda")
    bias = -1.2 * torch.log(order.float() + 1.0)
    logits = (_normal(g, (M, E)) * 1.5 + bias).to(_DT[c["dtype"]])
    if c["off"]:
        logits[:, torch.randperm(E, generator=g, device="cuda")[:c["off"]]] = float("-inf")
    d = {"logits": logits}
    if c["train"]:
        d["valid"] = (torch.rand(M, generator=g, device="cuda") >= c["pad"]).to(torch.uint8)
        d["d_rw"] = _normal(g, (M, k)).to(_DT[c["rw"]])
        d["d_loss"] = torch.full((1,), 0.01, device="cuda") * (1 + torch.rand(1, generator=g, device="cuda"))
    return d


def _lora_inputs(c, seed):
    g = _gen(seed)
    M, fin, fout, dt = c["M"], c["in"], c["out"], _DT[c["dtype"]]
    reqs = _requests(c)
    random.Random(seed).shuffle(reqs)
    ids = np.concatenate([np.full(n, a, np.int32) for n, a in reqs])
    d = {
        "ids": torch.from_numpy(ids).cuda(),
        "rows": [torch.from_numpy(np.flatnonzero(ids == a)).cuda() for a in range(c["adapters"])],
        "x": _normal(g, (M, fin)).to(dt),
        "base": _normal(g, (M, fout)).to(dt),
        "A": [(_normal(g, (r, fin), 1 / math.sqrt(fin))).to(dt) for r in _ranks(c)],
        "B": [(_normal(g, (r, fout), 0.02)).to(dt) for r in _ranks(c)],
        "scale": [[2.0, 1.0, 0.5][i % 3] for i in range(c["adapters"])],
    }
    if c["train"]:
        d["dy"] = _normal(g, (M, fout), 0.02).to(dt)
        d["dx_base"] = _normal(g, (M, fin), 0.02).to(dt)
    return d


def prepare(case, seed):
    c = case
    st = _router_inputs(c, seed) if c["op"] == "router" else _lora_inputs(c, seed)
    st["case"] = c
    if not own:
        return st
    import trellis_quantized_moe_gb300 as X
    M, dev = c["M"], "cuda"
    if c["op"] == "router":
        E, k = c["E"], c["k"]
        st["ids"] = torch.empty((M, k), dtype=torch.int32, device=dev)
        st["rw"] = torch.empty((M, k), dtype=_DT[c["rw"]], device=dev)
        if c["train"]:
            st["stats"] = torch.empty((M, 2), dtype=torch.float32, device=dev)
            st["counts"] = torch.empty(E + 1, dtype=torch.int32, device=dev)
            st["loss"] = torch.empty(1, dtype=torch.float32, device=dev)
            st["d_logits"] = torch.empty_like(st["logits"])
            st["ws"] = torch.empty(X.exl3_router_workspace_bytes(M, E), dtype=torch.uint8, device=dev)
        return st
    ad = X.DeviceAdapters(st["A"], st["B"], st["scale"])
    st["adapters"] = ad
    st["plan"] = torch.empty(X.exl3_lora_plan_bytes(M, ad.N), dtype=torch.uint8, device=dev)
    # one plan serves every adapted projection that this batch passes through
    X.exl3_lora_plan(st["ids"], ad.N, st["plan"])
    st["y"] = torch.empty_like(st["base"])
    st["ws"] = torch.empty(X.exl3_lora_workspace_bytes(M, ad.N, ad.in_features, ad.out_features,
                                                        ad.max_rank), dtype=torch.uint8, device=dev)
    if c["train"]:
        st["h"] = torch.empty((M, ad.h_cols), dtype=_DT[c["dtype"]], device=dev)
        st["dx"] = torch.empty_like(st["x"])
        st["dA"] = [torch.empty_like(a) for a in st["A"]]
        st["dB"] = [torch.empty_like(b) for b in st["B"]]
        st["grads"] = X.DeviceAdapters(st["dA"], st["dB"], st["scale"])
    return st


# --------------------------------------------------------------------------- one pass
def run(state):
    c = state["case"]
    if c["op"] == "router":
        return _router_own(c, state) if own else _router_plain(c, state)
    return _lora_own(c, state) if own else _lora_plain(c, state)


def _router_own(c, s):
    import trellis_quantized_moe_gb300 as X
    if not c["train"]:
        X.exl3_router_forward(s["logits"], s["ids"], s["rw"], renorm=c["renorm"])
        return {"ids": s["ids"], "rw": s["rw"]}
    X.exl3_router_forward(s["logits"], s["ids"], s["rw"], renorm=c["renorm"], stats=s["stats"],
                          valid=s["valid"], counts=s["counts"], loss=s["loss"], workspace=s["ws"])
    X.exl3_router_backward(s["logits"], s["ids"], s["stats"], s["d_logits"], renorm=c["renorm"],
                           d_rw=s["d_rw"], valid=s["valid"], counts=s["counts"], d_loss=s["d_loss"])
    return {"ids": s["ids"], "rw": s["rw"], "counts": s["counts"], "loss": s["loss"],
            "d_logits": s["d_logits"]}


def _router_plain(c, s):
    logits, k, E = s["logits"], c["k"], c["E"]
    l = logits.float()
    m = l.max(dim=1, keepdim=True).values
    e = torch.exp(l - torch.where(torch.isinf(m), torch.zeros_like(m), m))
    p = e / e.sum(dim=1, keepdim=True)
    ids = torch.sort(l, dim=1, descending=True, stable=True).indices[:, :k]
    chosen = p.gather(1, ids)
    total = chosen.sum(dim=1, keepdim=True)
    w = chosen / total if c["renorm"] else chosen
    out = {"ids": ids.to(torch.int32), "rw": w.to(_DT[c["rw"]])}
    if not c["train"]:
        return out
    v = s["valid"].float()
    T = v.sum().clamp(min=1)
    hit = torch.zeros_like(p).scatter_(1, ids, 1.0) * v[:, None]
    cnt = hit.sum(dim=0)
    mean = (p * v[:, None]).sum(dim=0) / T
    out["counts"] = torch.cat([cnt, v.sum()[None]]).round().to(torch.int32)
    out["loss"] = (E / (k * T) * (cnt * mean).sum()).reshape(1)
    G = v[:, None] * (s["d_loss"] * E / (k * T * T) * cnt)
    d = s["d_rw"].float()
    if not c["renorm"]:
        G = G.scatter_add(1, ids, d)
    dl = p * (G - (p * G).sum(dim=1, keepdim=True))
    if c["renorm"]:
        dl = dl.scatter_add(1, ids, w * (d - (w * d).sum(dim=1, keepdim=True)))
    out["d_logits"] = dl.to(logits.dtype)
    return out


def _lora_own(c, s):
    import trellis_quantized_moe_gb300 as X
    X.exl3_lora_forward(s["x"], s["plan"], s["adapters"], s["y"], s["ws"], base=s["base"],
                        h=s.get("h"))
    if not c["train"]:
        return {"y": s["y"]}
    X.exl3_lora_backward(s["dy"], s["x"], s["h"], s["plan"], s["adapters"], s["grads"], s["ws"],
                         dx=s["dx"], dx_base=s["dx_base"])
    return {"y": s["y"], "dx": s["dx"], "dA": s["dA"], "dB": s["dB"]}


def _lora_plain(c, s):
    dt = _DT[c["dtype"]]
    y = s["base"].float()
    if c["train"]:
        dx, dA, dB = s["dx_base"].float(), [], []
    for rows, A, B, scale in zip(s["rows"], s["A"], s["B"], s["scale"]):
        A, B, x = A.float(), B.float(), s["x"][rows].float()
        h = x @ A.T
        y[rows] += scale * (h @ B)
        if c["train"]:
            dy = s["dy"][rows].float()
            dh = scale * (dy @ B.T)
            dx[rows] += dh @ A
            dA.append((dh.T @ x).to(dt))
            dB.append((scale * (h.T @ dy)).to(dt))
    if not c["train"]:
        return {"y": y.to(dt)}
    return {"y": y.to(dt), "dx": dx.to(dt), "dA": dA, "dB": dB}


# --------------------------------------------------------------------------- 64-bit values
def exact(case, seed):
    return _router_exact(case, seed) if case["op"] == "router" else _lora_exact(case, seed)


def _router_exact(c, seed):
    """The definitions in float64, a row's softmax and the two gradients written from dlog p."""
    d = _router_inputs(c, seed)
    z = d["logits"].double().cpu().numpy()
    M, E, k = c["M"], c["E"], c["k"]
    ids = np.argsort(-z, axis=1, kind="stable")[:, :k]
    t = np.arange(M)[:, None]
    p = np.exp(z - z.max(axis=1, keepdims=True))
    p /= p.sum(axis=1, keepdims=True)
    w = p[t, ids]
    norm = w.sum(axis=1, keepdims=True) if c["renorm"] else np.ones((M, 1))
    out = {"ids": ids.astype(np.int32), "rw": w / norm}
    if c["train"]:
        v = d["valid"].cpu().numpy().astype(bool)
        T = int(v.sum())
        counts = np.bincount(ids[v].ravel(), minlength=E)
        out["counts"] = np.append(counts, T).astype(np.int32)
        f = counts / (k * T) if T else np.zeros(E)
        out["loss"] = np.array([E * np.dot(f, p[v].mean(axis=0)) if T else 0.0])
        # dL/dp of the balance term, then through p = softmax(z)
        gl = float(d["d_loss"].double().item())
        dp = np.where(v[:, None], gl * E * f / max(T, 1), 0.0)
        dz = p * (dp - (dp * p).sum(axis=1, keepdims=True))
        # weights w_j = p_j / norm: d log w_j / dz_e = [e = S_j] - q_e, q the
        # softmax over what the weights are normalised by
        g = d["d_rw"].double().cpu().numpy() * (w / norm)
        if c["renorm"]:
            q = np.zeros((M, E))
            q[t, ids] = w / norm
        else:
            q = p
        dz -= q * g.sum(axis=1, keepdims=True)
        dz[t, ids] += g
        out["d_logits"] = dz
    return out


def _lora_exact(c, seed):
    """Per request, the definition's sums in float64 with the update matrix s A^T B formed from its factors."""
    d = _lora_inputs(c, seed)
    x, y = d["x"].double(), d["base"].double()
    if c["train"]:
        dy, dx, dA, dB = d["dy"].double(), d["dx_base"].double(), [], []
    ids = d["ids"].long()
    for a in range(c["adapters"]):
        At, Bt, s = d["A"][a].double(), d["B"][a].double(), d["scale"][a]
        on = torch.nonzero(ids == a).squeeze(1)
        xa = x.index_select(0, on)
        y.index_add_(0, on, torch.einsum("ti,ri,ro->to", xa, At, s * Bt))
        if c["train"]:
            ga = dy.index_select(0, on)
            dx.index_add_(0, on, torch.einsum("to,ro,ri->ti", ga, s * Bt, At))
            dA.append(torch.einsum("to,ro,ti->ri", ga, s * Bt, xa))
            dB.append(torch.einsum("ti,ri,to->ro", xa, s * At, ga))
    if not c["train"]:
        return {"y": y}
    return {"y": y, "dx": dx, "dA": dA, "dB": dB}
