"""The projection operators' workloads: plain forms, calls, inputs and the work of one pass.

Four operators around the hyper-connection read, whose 16-bit images (width 2560) are what they read:

    project         y[t] = W x[t] + scale[a] B[a] (A[a] x[t]),  a = adapter[t]  (a < 0: W x[t] alone)
    route           the top k of E experts per token, their weights, and the rows sorted by expert
    expert_project  y[i] = W[e] x[rows[i]] for offsets[e] <= i < offsets[e + 1], and its gated form
                    silu(W_gate x) * (W_up x)
    expert_combine  out[t] = sum over s of weights[t, s] * y[pos[t, s]]

Weights are [outputs, inputs] row-major, as the read's own.  `own` chooses between the plain forms (elementary
torch operations in 32 bits) and the library's calls; `exact` states the same results in 64 bits.
"""
import math

import numpy as np
import torch

own = False

_TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def listed():
    return [
        # one decoded token through a square projection of the read's width, its request's adapter beside it
        dict(name="project_token", op="project", T=1, K=2560, N=2560, type="bf16", out="bf16", rank=16,
             adapters=8, requests=1),
        # one verify window of every request in flight: 25 tokens, the read's short-window limit
        dict(name="project_windows", op="project", T=25, K=2560, N=10240, type="fp16", out="fp16", rank=32,
             adapters=6, requests=5),
        # a mixed batch: the end of a prompt and windows of other requests, the wide stream axis as input, fp32 out
        dict(name="project_mixed", op="project", T=333, K=10240, N=2560, type="bf16", out="fp32", rank=64,
             adapters=16, requests=24),
        # a prefill chunk of a few long prompts
        dict(name="project_prefill", op="project", T=8192, K=2560, N=10240, type="bf16", out="bf16", rank=16,
             adapters=4, requests=5),
        # one decoded token's eight experts of 64, gate and up products with the activation
        dict(name="experts_token", op="experts", T=1, k=8, E=64, K=2560, N=1024, gate=True, gather=True,
             type="bf16", out="bf16", skew=0.0),
        # a verify window of 8 tokens, the experts' product back to the read's width
        dict(name="experts_window", op="experts", T=8, k=8, E=64, K=1024, N=2560, gate=False, gather=False,
             type="fp16", out="fp16", skew=0.0),
        # a small batch over uneven experts, odd output width
        dict(name="experts_ragged", op="experts", T=301, k=6, E=32, K=2560, N=1023, gate=True, gather=True,
             type="bf16", out="bf16", skew=1.0),
        # a prefill chunk: 65536 rows over 64 uneven experts
        dict(name="experts_prefill", op="experts", T=8192, k=8, E=64, K=2560, N=1024, gate=True, gather=True,
             type="bf16", out="bf16", skew=0.5),
        # a verify window's routing, where launches are all that counts
        dict(name="route_window", op="route", T=8, E=64, k=8, renorm=True, type="fp32", masked=0.0),
        # the longest prefill call, some of its tokens padding
        dict(name="route_prefill", op="route", T=32768, E=128, k=8, renorm=False, type="fp32", masked=0.1),
        # joining one window's experts
        dict(name="combine_window", op="combine", T=8, k=8, C=2560, type="fp16", out="fp32", dropped=0.0),
        # joining a prefill chunk's experts, a few slots dropped
        dict(name="combine_prefill", op="combine", T=8192, k=8, C=2560, type="bf16", out="bf16", dropped=0.05),
    ]


def _spread(rng, low, high):
    """A whole number between low and high, even over its logarithm."""
    return max(low, min(high, round(math.exp(rng.uniform(math.log(low), math.log(high + 1))))))


def draw(rng):
    op = rng.choice(["project", "project", "experts", "experts", "route", "combine"])
    kind = rng.choice(["bf16", "fp16"])
    out = rng.choice([kind, kind, "fp32"])
    if op == "project":
        K, N = 8 * _spread(rng, 16, 1280), _spread(rng, 17, 10240)
        T = _spread(rng, 1, min(8192, max(1, 8192 * 2560 * 10240 // (K * N))))
        return dict(op=op, T=T, K=K, N=N, type=kind, out=out, rank=8 * _spread(rng, 1, 16), adapters=_spread(rng, 1, 32),
                    requests=min(T, _spread(rng, 1, 48)))
    if op == "experts":
        E, gate = _spread(rng, 1, 128), rng.random() < 0.5
        K = 8 * _spread(rng, 16, 320)
        N = _spread(rng, 17, max(17, min(2560, 64 * 2048 * 2560 // (E * K * (2 if gate else 1)))))
        k = rng.randint(1, min(E, 8))
        T = _spread(rng, 1, min(8192, 65536 * 2048 * 2560 // (k * K * N * (2 if gate else 1))))
        return dict(op=op, T=T, k=k, E=E, K=K, N=N, gate=gate, gather=rng.random() < 0.5, type=kind, out=out,
                    skew=rng.choice([0.0, 0.5, 1.0]))
    if op == "route":
        E = _spread(rng, 2, 256)
        return dict(op=op, T=_spread(rng, 1, 16384), E=E, k=rng.randint(1, min(E, 8)), renorm=rng.random() < 0.5,
                    type=rng.choice(["fp32", "bf16"]), masked=rng.choice([0.0, 0.1]))
    return dict(op=op, T=_spread(rng, 1, 8192), k=rng.randint(1, 8), C=8 * _spread(rng, 8, 320), type=kind, out=out,
                dropped=rng.choice([0.0, 0.05]))


def _normal(gen, shape, sigma, dtype):
    return torch.empty(shape, dtype=dtype, device="cuda").normal_(0.0, sigma, generator=gen)


def _pick(gen, T, E, k, skew):
    """k different experts for each of T tokens; `skew` makes some experts more popular than others."""
    score = torch.rand((T, E), generator=gen, device="cuda").clamp_(min=1e-9).log_().neg_().log_().neg_()
    score += skew * torch.randn((E,), generator=gen, device="cuda")
    return score.topk(k, dim=1).indices


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    host = np.random.default_rng(seed)
    T, s = case["T"], dict(case)
    kind, out = _TYPES[case["type"]], _TYPES.get(case.get("out"))
    if case["op"] == "project":
        K, N, r, n = case["K"], case["N"], case["rank"], case["adapters"]
        cuts = np.sort(host.choice(T - 1, case["requests"] - 1, replace=False) + 1) if case["requests"] > 1 else []
        lengths = np.diff(np.concatenate([[0], cuts, [T]]).astype(np.int64))
        # one request in eight has no adapter
        of_request = np.where(host.random(len(lengths)) < 0.125, -1, host.integers(0, n, len(lengths)))
        s.update(x=_normal(gen, (T, K), 1.0, kind), W=_normal(gen, (N, K), 0.02, kind),
                 A=_normal(gen, (n, r, K), 0.02, kind), B=_normal(gen, (n, N, r), 0.02, kind),
                 scale=torch.rand((n,), generator=gen, device="cuda") * 1.5 + 0.5,
                 adapter=torch.from_numpy(np.repeat(of_request, lengths).astype(np.int32)).cuda(),
                 y=torch.empty((T, N), dtype=out, device="cuda"))
    elif case["op"] == "experts":
        E, k, K, N = case["E"], case["k"], case["K"], case["N"]
        ids, order = _pick(gen, T, E, k, case["skew"]).reshape(-1).sort(stable=True)
        offsets = torch.searchsorted(ids, torch.arange(E + 1, device="cuda"))
        counts = offsets.diff()
        # the plain form's plan: the experts that have rows, each row's place in its expert, the longest expert
        active = counts.nonzero().flatten()
        s.update(x=_normal(gen, (T if case["gather"] else T * k, K), 1.0, kind),
                 W=_normal(gen, (E, 2 * N if case["gate"] else N, K), 0.02, kind), offsets=offsets.int(),
                 rows=(order // k).int() if case["gather"] else None, active=active,
                 group=torch.searchsorted(active, ids), place=torch.arange(T * k, device="cuda") - offsets[ids],
                 longest=int(counts.max()), y=torch.empty((T * k, N), dtype=out, device="cuda"))
    elif case["op"] == "route":
        logits = torch.randn((T, case["E"]), generator=gen, device="cuda")
        # padding tokens: every expert masked out
        logits[torch.rand((T,), generator=gen, device="cuda") < case["masked"]] = -math.inf
        s.update(logits=logits.to(kind))
    else:
        k = case["k"]
        pos = torch.randperm(T * k, generator=gen, device="cuda").reshape(T, k).int()
        pos[torch.rand((T, k), generator=gen, device="cuda") < case["dropped"]] = -1
        weights = torch.rand((T, k), generator=gen, device="cuda")
        s.update(y=_normal(gen, (T * k, case["C"]), 1.0, kind), pos=pos, weights=weights / weights.sum(1, keepdim=True),
                 to=torch.empty((T, case["C"]), dtype=out, device="cuda"))
    return s


def _own(s):
    from hyper_connection_residual_amd import projections as p
    if s["op"] == "project":
        return p.project(s["x"], s["W"], adapter=s["adapter"], A=s["A"], B=s["B"], scale=s["scale"], out=s["y"])
    if s["op"] == "experts":
        return p.expert_project(s["x"], s["W"], s["offsets"], rows=s["rows"], gate=s["gate"], out=s["y"])
    if s["op"] == "route":
        return p.route(s["logits"], s["k"], renorm=s["renorm"])
    return p.expert_combine(s["y"], s["pos"], s["weights"], out=s["to"])


def run(state):
    s = state
    if own:
        return _own(s)
    if s["op"] == "project":
        x, n = s["x"].float(), s["adapters"]
        # every adapter's A at once, the other adapters' columns then cleared, every adapter's B at once
        v = (x @ s["A"].float().flatten(0, 1).T).view(-1, n, s["rank"])
        mine = (s["adapter"][:, None] == torch.arange(n, device=x.device)) * s["scale"]
        beside = (v * mine[:, :, None]).flatten(1) @ s["B"].float().transpose(1, 2).flatten(0, 1)
        return (x @ s["W"].float().T + beside).to(s["y"].dtype)
    if s["op"] == "experts":
        x = s["x"].float()
        x = x[s["rows"].long()] if s["gather"] else x
        # the experts that have rows, each padded to the longest
        padded = x.new_zeros((s["active"].numel(), s["longest"], s["K"]))
        padded[s["group"], s["place"]] = x
        y = torch.bmm(padded, s["W"][s["active"]].float().transpose(1, 2))[s["group"], s["place"]]
        if s["gate"]:
            g, u = y[:, :s["N"]], y[:, s["N"]:]
            y = g / (1.0 + torch.exp(-g)) * u
        return y.to(s["y"].dtype)
    if s["op"] == "route":
        z, E, k = s["logits"].float(), s["E"], s["k"]
        T = z.shape[0]
        top, ids = (t[:, :k] for t in z.sort(dim=1, descending=True, stable=True))
        some = top > -math.inf
        peak = torch.where(some[:, :1], top[:, :1], 0.0)
        e = torch.exp(top - peak)
        total = e.sum(1, keepdim=True) if s["renorm"] else torch.exp(z - peak).sum(1, keepdim=True)
        weights = torch.where(some, e / total, 0.0)
        flat, order = torch.where(some, ids, E).flatten().sort(stable=True)
        offsets = torch.searchsorted(flat, torch.arange(E + 1, device=z.device))
        at = torch.empty_like(order)
        at[order] = torch.arange(T * k, device=z.device)
        return (torch.where(some, ids, -1).int(), weights, offsets.int(), torch.where(flat < E, order // k, -1).int(),
                torch.where(some, at.view(T, k), -1).int())
    pos = s["pos"].long()
    w = torch.where(pos >= 0, s["weights"], 0.0)
    return (s["y"].float()[pos.clamp(min=0)] * w[:, :, None]).sum(1).to(s["to"].dtype)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "project":
        x = s["x"].double()
        y = x @ s["W"].double().T
        for a in range(case["adapters"]):
            mine = s["adapter"] == a
            y[mine] += s["scale"][a].double() * ((x[mine] @ s["A"][a].double().T) @ s["B"][a].double().T)
        return y
    if case["op"] == "experts":
        y = torch.zeros((case["T"] * case["k"], case["N"]), dtype=torch.float64, device="cuda")
        at = s["offsets"].tolist()
        for e in range(case["E"]):
            if at[e] == at[e + 1]:
                continue
            mine = slice(at[e], at[e + 1])
            x = s["x"][s["rows"][mine].long()] if case["gather"] else s["x"][mine]
            h = x.double() @ s["W"][e].double().T
            if case["gate"]:
                g, u = h.chunk(2, dim=1)
                h = g * torch.sigmoid(g) * u
            y[mine] = h
        return y
    if case["op"] == "route":
        z = s["logits"].double()
        ids = z.sort(dim=1, descending=True, stable=True).indices[:, :case["k"]]
        top = z.gather(1, ids)
        some = top > -math.inf
        w = torch.softmax(top if case["renorm"] else z, dim=1)
        w = w if case["renorm"] else w.gather(1, ids)
        return None, torch.where(some, w, 0.0), None, None, None
    y = torch.zeros((case["T"], case["C"]), dtype=torch.float64, device="cuda")
    for j in range(case["k"]):
        have = s["pos"][:, j] >= 0
        y[have] += s["weights"][have, j, None].double() * s["y"][s["pos"][have, j].long()].double()
    return y


def _touched(of, tries, each=1):
    """How many of `of` things `tries` even choices of `each` different ones are expected to touch."""
    return of * (1.0 - (1.0 - min(1.0, each / of)) ** tries)


def work(case):
    c, T = case, case["T"]
    size = {"bf16": 2, "fp16": 2, "fp32": 4}
    wide, out = size[c["type"]], size.get(c.get("out"))
    if c["op"] == "project":
        K, N, r = c["K"], c["N"], c["rank"]
        used = _touched(c["adapters"], c["requests"])
        return {"bytes": wide * (T * K + N * K + used * r * (K + N)) + out * T * N + 4 * T,
                "flops": 2.0 * T * (N * K + r * (K + N))}
    if c["op"] == "experts":
        rows, K, N, wn = T * c["k"], c["K"], c["N"], c["N"] * (2 if c["gate"] else 1)
        read = wide * K * (T if c["gather"] else rows) + (4 * rows if c["gather"] else 0)
        return {"bytes": read + wide * _touched(c["E"], T, c["k"]) * wn * K + out * rows * N, "flops": 2.0 * rows * wn * K}
    if c["op"] == "route":
        # read the logits; write ids, weights, rows and pos of every slot
        return {"bytes": wide * T * c["E"] + 16 * T * c["k"] + 4 * (c["E"] + 1), "flops": 3.0 * T * c["E"]}
    return {"bytes": wide * T * c["k"] * c["C"] * (1.0 - c["dropped"]) + 8 * T * c["k"] + out * T * c["C"],
            "flops": 2.0 * T * c["k"] * c["C"]}
