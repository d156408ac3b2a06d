"""Cases of the router, the few-token layer and the adapted projection.

``run`` computes a case in its plain form (elementary torch operations in 32
bits, 64 where a selection border needs it), or with ``own`` set through the
package's entry points ``gate``, ``layer`` and ``project``; ``exact`` computes
it in 64 bits from the definition.

Activations and router weights lie on a grid (integers times a power of two)
whose products sum without rounding in FP32 in any order, so that the router's
selection is the same number for every order of summation and its expert ids
can be compared exactly.
"""

import math

import torch

own = False

_E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ----------------------------------------------------------------------------
# cases


def _gate(name, T, E, k, H, scoring, bias, renorm, wf32, shared=0):
    return dict(name=name, op="gate", T=T, E=E, k=k, H=H, scoring=scoring, bias=bias, renorm=renorm, wf32=wf32,
                shared=shared)


def _layer(name, T, E, k, H, I, gran, scoring, bias, renorm, shared):
    return dict(name=name, op="layer", T=T, E=E, k=k, H=H, I=I, gran=gran, scoring=scoring, bias=bias,
                renorm=renorm, wf32=False, shared=shared)


def _project(name, T, N, K, gran, L, R, mix):
    return dict(name=name, op="project", T=T, N=N, K=K, gran=gran, L=L, R=R, mix=mix)


def listed():
    return [
        # one token of a decode step through a 256-expert router (sigmoid scores, correction bias)
        _gate("gate_t1", 1, 256, 8, 6144, "sigmoid", True, True, False, shared=1),
        # a decode batch, softmax over all the experts without renormalisation
        _gate("gate_t64", 64, 256, 8, 6144, "softmax", False, False, False),
        # a prefill chunk, router weights kept in FP32
        _gate("gate_t8192", 8192, 256, 8, 6144, "sigmoid", True, True, True),
        # an odd number of tokens through a small router
        _gate("gate_odd", 333, 96, 6, 2048, "softmax", True, True, False),
        # the tiny layer: nothing but latency
        _layer("layer_tiny", 3, 8, 2, 512, 256, 16, "softmax", False, False, 0),
        # one token of a decode step through a whole layer, with its shared expert
        _layer("layer_t1", 1, 257, 8, 6144, 2048, 16, "sigmoid", True, True, 1),
        # a few tokens (a speculative decode step), group32 weights
        _layer("layer_t5", 5, 256, 8, 6144, 2048, 32, "softmax", False, True, 0),
        # the largest few-token batch
        _layer("layer_t16", 16, 256, 8, 6144, 2048, 16, "softmax", False, False, 0),
        # one token with its adapter through a fused gate/up projection
        _project("project_t1", 1, 4096, 6144, 16, 8, 16, "each"),
        # a decode batch in which every request has an adapter of its own or none
        _project("project_t37", 37, 6144, 2048, 32, 24, 32, "each"),
        # an odd batch, rows that are no multiple of a tile
        _project("project_odd", 203, 1968, 2048, 16, 5, 8, "runs"),
        # prefill chunks of a few requests, each a run of tokens
        _project("project_t8192", 8192, 4096, 6144, 32, 16, 64, "runs"),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    case = _draw(rng)
    del case["name"]
    return case


def _draw(rng):
    op = rng.choice(("gate", "layer", "project"))
    if op == "gate":
        E = _log_int(rng, 4, 384)
        return _gate("", _log_int(rng, 1, 6000), E, rng.randint(1, min(10, E)), 8 * _log_int(rng, 8, 896),
                     rng.choice(("softmax", "sigmoid")), rng.random() < 0.5, rng.random() < 0.5, rng.random() < 0.4,
                     rng.choice((0, 0, 1, 2)))
    if op == "layer":
        shared = rng.choice((0, 0, 1))
        E = _log_int(rng, 4, 200)
        return _layer("", _log_int(rng, 1, 16), E + shared, rng.randint(1, min(8, E)), 256 * _log_int(rng, 1, 22),
                      256 * _log_int(rng, 1, 8), rng.choice((16, 32)), rng.choice(("softmax", "sigmoid")),
                      rng.random() < 0.5, rng.random() < 0.5, shared)
    return _project("", _log_int(rng, 1, 6000), 16 * _log_int(rng, 16, 256), 256 * _log_int(rng, 1, 24),
                    rng.choice((16, 32)), _log_int(rng, 1, 48), 8 * rng.randint(1, 8), rng.choice(("each", "runs")))


# ----------------------------------------------------------------------------
# inputs


def _grid(g, shape, sigma, top, unit):
    """Integers round(N(0, sigma)) within [-top, top], times unit."""
    v = torch.randn(shape, generator=g, device="cuda").mul_(sigma).round_().clamp_(-top, top)
    return v.mul_(unit)


def _fp4(g, E, N, K, gran):
    """Uniform E2M1 codes; E4M3 scales log-uniform in [2^-10, 2^-3], or UE8M0 exponents uniform in [-10, -2]."""
    w = torch.randint(0, 256, (E, N, K // 2), generator=g, device="cuda", dtype=torch.uint8)
    if gran == 16:
        u = torch.rand((E, N, K // 16), generator=g, device="cuda")
        sf = u.mul_(7).sub_(10).exp2_().to(torch.float8_e4m3fn).view(torch.uint8)
    else:
        sf = torch.randint(117, 126, (E, N, K // 32), generator=g, device="cuda", dtype=torch.uint8)
    return w, sf


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 7919 + 13)
    s = {"case": dict(case)}
    if case["op"] == "project":
        T, N, K, L, R = (case[n] for n in ("T", "N", "K", "L", "R"))
        s["x"] = _grid(g, (T, K), 16.0, 127, 1 / 16).bfloat16()
        w, sf = _fp4(g, 1, N, K, case["gran"])
        s["w"], s["w_sf"] = w[0], sf[0]
        s["w_gs"] = 0.5 + 1.5 * torch.rand(1, generator=g, device="cuda") if case["gran"] == 16 else None
        s["a"] = (torch.randn((L, R, K), generator=g, device="cuda") / math.sqrt(K)).bfloat16()
        s["b"] = (torch.randn((L, N, R), generator=g, device="cuda") / math.sqrt(R)).bfloat16()
        if case["mix"] == "each":
            # every token a request of its own; one in L + 1 without an adapter
            s["id"] = torch.randint(-1, L, (T,), generator=g, device="cuda", dtype=torch.int32)
        else:
            # runs of tokens: one adapter (or none) for each of a few requests
            n = max(1, min(T, 2 * L))
            cut = torch.randint(0, T + 1, (n - 1,), generator=g, device="cuda").sort().values
            run_of = torch.bucketize(torch.arange(T, device="cuda"), cut, right=True)
            s["id"] = torch.randint(-1, L, (n,), generator=g, device="cuda", dtype=torch.int32)[run_of]
        s["scale"] = 0.5 + 1.5 * torch.rand(L, generator=g, device="cuda")
        return s
    T, E, H = case["T"], case["E"], case["H"]
    routed = E - case["shared"] if case["op"] == "layer" else E
    s["x"] = _grid(g, (T, H), 16.0, 127, 1 / 16).bfloat16()
    # logits of about unit variance; FP32 router weights hold 12 bits, bfloat16 ones 8
    unit = 2.0 ** -round(math.log2(math.sqrt(H)))
    if case["wf32"]:
        s["gate_w"] = _grid(g, (routed, H), 256.0, 2047, unit / 256)
    else:
        s["gate_w"] = _grid(g, (routed, H), 16.0, 127, unit / 16).bfloat16()
    s["bias"] = 0.05 * torch.randn(routed, generator=g, device="cuda") if case["bias"] else None
    if case["op"] == "layer":
        I, gran = case["I"], case["gran"]
        s["w13"], s["w13_sf"] = _fp4(g, E, 2 * I, H, gran)
        s["w2"], s["w2_sf"] = _fp4(g, E, H, I, gran)
        s["w13_gs"] = 0.5 + 1.5 * torch.rand(E, generator=g, device="cuda") if gran == 16 else None
        s["w2_gs"] = 0.5 + 1.5 * torch.rand(E, generator=g, device="cuda") if gran == 16 else None
    return s


# ----------------------------------------------------------------------------
# the plain forms


def _factor(case):
    """The factor on the routed weights (2.5 where they are renormalised, as such models have it)."""
    return 2.5 if case["renorm"] else 1.0


def _plain_gate(s):
    case = s["case"]
    x, k, shared = s["x"].float(), case["k"], case["shared"]
    logits = x @ s["gate_w"].float().t()
    # scores in 64 bits: the selection compares values next to a border
    z = logits.double()
    p = torch.softmax(z, -1) if case["scoring"] == "softmax" else torch.sigmoid(z)
    sel = p if s["bias"] is None else p + s["bias"].double()
    ids = torch.sort(sel, dim=-1, descending=True, stable=True).indices[:, :k]
    w = torch.gather(p, 1, ids)
    if case["renorm"]:
        w = w / w.sum(-1, keepdim=True)
    w = (w * _factor(case)).float()
    ids = ids.int()
    if shared:
        T, E = logits.shape
        ids = torch.cat([ids, (E + torch.arange(shared, device=ids.device, dtype=torch.int32)).expand(T, shared)], 1)
        w = torch.cat([w, torch.ones((T, shared), device=w.device)], 1)
    return ids, w


def _plain_weight(w, sf, gs, gran, dtype=torch.float32):
    """FP4 codes [..., N, K/2] and block scales [..., N, K/gran] -> values [..., N, K]."""
    m = torch.tensor(_E2M1, device=w.device, dtype=dtype)
    tab = torch.cat([m, -m])
    pair = torch.stack([tab.repeat(16), tab.repeat_interleave(16)], 1)  # byte -> (low nibble, high nibble)
    v = pair[w.long()].flatten(-2)
    if gran == 16:
        sc = sf.view(torch.float8_e4m3fn).to(dtype)
    else:
        sc = torch.exp2(sf.to(dtype) - 127)
    v = v.view(*v.shape[:-1], -1, gran).mul_(sc.unsqueeze(-1)).flatten(-2)
    return v if gs is None else v.mul_(gs.to(dtype).view(-1, *([1] * (v.dim() - 1))) if v.dim() > 2 else gs.to(dtype))


def _plain_layer(s):
    case = s["case"]
    ids, w = _plain_gate(s)
    T, ke = ids.shape
    I, gran = case["I"], case["gran"]
    flat = ids.flatten().long()
    xa = s["x"].float().repeat_interleave(ke, 0).unsqueeze(-1)  # one row per assignment
    w13 = _plain_weight(s["w13"][flat], s["w13_sf"][flat], None if s["w13_gs"] is None else s["w13_gs"][flat], gran)
    g = torch.bmm(w13, xa).squeeze(-1)
    del w13
    h = (g[:, :I] * torch.sigmoid(g[:, :I]) * g[:, I:]).unsqueeze(-1)
    w2 = _plain_weight(s["w2"][flat], s["w2_sf"][flat], None if s["w2_gs"] is None else s["w2_gs"][flat], gran)
    y = torch.bmm(w2, h).view(T, ke, -1)
    return (y * w.unsqueeze(-1)).sum(1).bfloat16()


def _plain_project(s):
    case = s["case"]
    L, R, N = case["L"], case["R"], case["N"]
    x = s["x"].float()
    y = x @ _plain_weight(s["w"], s["w_sf"], s["w_gs"], case["gran"]).t()
    # every adapter for every token, the others' masked away
    mine = torch.arange(L, device=x.device, dtype=torch.int32) == s["id"].unsqueeze(1)
    u = (x @ s["a"].float().view(L * R, -1).t()).view(-1, L, R)
    u = u * (mine * s["scale"]).unsqueeze(-1)
    y = y + u.flatten(1) @ s["b"].float().permute(0, 2, 1).reshape(L * R, N)
    return y.bfloat16()


def run(s):
    case = s["case"]
    if not own:
        if case["op"] == "gate":
            return _plain_gate(s)
        return _plain_layer(s) if case["op"] == "layer" else _plain_project(s)
    import block_scaled_fp4_topk_amd as moe
    if case["op"] == "gate":
        return moe.gate(s["x"], s["gate_w"], case["k"], bias=s["bias"], scoring=case["scoring"],
                        renormalize=case["renorm"], scale=_factor(case), shared=case["shared"])
    if case["op"] == "layer":
        return moe.layer(s["x"], s["gate_w"], case["k"], s["w13"], s["w13_sf"], s["w13_gs"], s["w2"], s["w2_sf"],
                         s["w2_gs"], case["gran"], bias=s["bias"], scoring=case["scoring"],
                         renormalize=case["renorm"], scale=_factor(case), shared=case["shared"])
    return moe.project(s["x"], s["w"], s["w_sf"], s["w_gs"], case["gran"], lora_a=s["a"], lora_b=s["b"],
                       lora_id=s["id"], lora_scale=s["scale"])


# ----------------------------------------------------------------------------
# the definition in 64 bits


def _exact_gate(case, s):
    logits = torch.matmul(s["x"].double(), s["gate_w"].double().T)
    if case["scoring"] == "softmax":
        e = torch.exp(logits - logits.amax(1, keepdim=True))
        p = e / e.sum(1, keepdim=True)
    else:
        p = 1.0 / (1.0 + torch.exp(-logits))
    left = p.clone() if s["bias"] is None else p + s["bias"].double()
    rows = torch.arange(p.shape[0], device=p.device)
    ids, ws = [], []
    for _ in range(case["k"]):
        best = left.amax(1, keepdim=True)
        i = (left == best).to(torch.uint8).argmax(1)  # the lowest index among equals
        ids.append(i)
        ws.append(p[rows, i])
        left[rows, i] = -math.inf
    ids, w = torch.stack(ids, 1), torch.stack(ws, 1)
    if case["renorm"]:
        w = w / w.sum(1, keepdim=True)
    w = w * _factor(case)
    for j in range(case["shared"]):
        ids = torch.cat([ids, torch.full_like(ids[:, :1], p.shape[1] + j)], 1)
        w = torch.cat([w, torch.ones_like(w[:, :1])], 1)
    return ids.int(), w


def _exact_fp4(codes, sf, gs, gran):
    """One matrix: codes [N, K/2], scales [N, K/gran], gs a number or None."""
    nib = torch.stack([codes & 15, codes >> 4], -1).flatten(1)
    mag, sign = (nib & 7).double(), 1.0 - 2.0 * (nib >> 3).double()
    ex = torch.clamp(torch.floor(mag / 2), min=1)  # E2M1: 2^(e-1) (1 + m/2), subnormal m/2 at e = 0
    v = torch.where(mag < 2, mag / 2, torch.exp2(ex - 1) * (1 + (mag - 2 * ex) / 2)) * sign
    b = sf.view(torch.float8_e4m3fn).double() if gran == 16 else torch.exp2(sf.double() - 127)
    v = v * b.repeat_interleave(gran, 1)
    return v if gs is None else v * gs.double()


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "gate":
        return _exact_gate(case, s)
    gran = case["gran"]
    if case["op"] == "project":
        x = s["x"].double()
        y = x @ _exact_fp4(s["w"], s["w_sf"], s["w_gs"], gran).T
        for l in range(case["L"]):
            at = (s["id"] == l).nonzero()[:, 0]
            if at.numel():
                u = x[at] @ s["a"][l].double().T
                y[at] += s["scale"][l].double() * (u @ s["b"][l].double().T)
        return y
    ids, w = _exact_gate(case, s)
    I = case["I"]
    y = torch.zeros((case["T"], case["H"]), dtype=torch.float64, device="cuda")
    for e in torch.unique(ids).tolist():
        t, j = (ids == e).nonzero(as_tuple=True)
        gs13 = None if s["w13_gs"] is None else s["w13_gs"][e]
        gs2 = None if s["w2_gs"] is None else s["w2_gs"][e]
        g = s["x"][t].double() @ _exact_fp4(s["w13"][e], s["w13_sf"][e], gs13, gran).T
        h = g[:, :I] / (1.0 + torch.exp(-g[:, :I])) * g[:, I:]
        y[t] += w[t, j].unsqueeze(1) * (h @ _exact_fp4(s["w2"][e], s["w2_sf"][e], gs2, gran).T)
    return y


# ----------------------------------------------------------------------------
# what a pass cannot do without


def work(case):
    T = case["T"]
    if case["op"] == "project":
        N, K, L, R, gran = (case[n] for n in ("N", "K", "L", "R", "gran"))
        tokens = T * L / (L + 1)  # with an adapter
        used = L * (1 - (1 - 1 / (L + 1)) ** (T if case["mix"] == "each" else min(T, 2 * L)))
        return {"bytes": 2 * T * (K + N) + N * K // 2 + N * K // gran + 2 * used * R * (K + N) + 4 * T,
                "flops": 2 * T * N * K + 2 * tokens * R * (K + N)}
    H, k, sh = case["H"], case["k"], case["shared"]
    routed = case["E"] - sh if case["op"] == "layer" else case["E"]
    b = 2 * T * H + (4 if case["wf32"] else 2) * routed * H + (4 * routed if case["bias"] else 0)
    f = 2 * T * routed * H
    if case["op"] == "gate":
        return {"bytes": b + 8 * T * (k + sh), "flops": f}
    active = routed * (1 - (1 - k / routed) ** T) + sh  # expected number of experts with a token
    per = 3 * H * case["I"]
    return {"bytes": b + active * per * (1 / 2 + 1 / case["gran"]) + 2 * T * H, "flops": f + 2 * T * (k + sh) * per}
