"""Cases of the products grouped by expert, their gradients, and the block norms.

``run`` computes a case in its plain form (elementary torch operations in 32
bits), or with ``own`` set through the package's entry points ``grouped``,
``grouped_dx``, ``grouped_dw``, ``block_norm`` and ``block_norm_grad``;
``exact`` computes it in 64 bits from the definition.
"""

import math

import torch

own = False

_E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
_EPS = 1e-6


# ----------------------------------------------------------------------------
# cases


def _prod(name, op, M, E, N, K, gran=0, f32=False):
    """gran: 0 for bfloat16 weights, 16 or 32 for FP4 ones; f32: a float32 output."""
    return dict(name=name, op=op, M=M, E=E, N=N, K=K, gran=gran, f32=f32)


def _norm(name, op, T, H, post, gate, sig, f32):
    """gate: "none", "channel" [H], "token" [T] or "full" [T, H]; f32: a float32 residual stream."""
    return dict(name=name, op=op, T=T, H=H, post=post, gate=gate, sig=sig, f32=f32)


def listed():
    return [
        # one token of a decode step: 8 of 64 bfloat16 experts, a row each
        _prod("grouped_t1", "grouped", 8, 64, 4096, 6144),
        # a small decode batch over FP4 experts of a checkpoint (16 tokens, 8 experts each)
        _prod("grouped_decode_fp4", "grouped", 128, 64, 4096, 6144, gran=16),
        # a prefill or training batch of 2048 tokens, 8 experts each
        _prod("grouped_batch", "grouped", 16384, 64, 4096, 6144),
        # sizes that are no multiple of a tile
        _prod("grouped_odd", "grouped", 1111, 40, 1000, 696, f32=True),
        # fine-tuning through frozen FP4 experts: the gradient towards the rows
        _prod("dx_batch_fp4", "dx", 8192, 32, 4096, 6144, gran=32),
        # the gradient through the low-rank factor of every expert
        _prod("dx_lowrank", "dx", 4000, 64, 32, 6144),
        # the weight gradients of a training batch, in float32 as an optimiser takes them
        _prod("dw_batch", "dw", 16384, 16, 4096, 6144, f32=True),
        # those of a low-rank factor
        _prod("dw_lowrank", "dw", 4000, 64, 32, 6144),
        # the norms between two layers for one token
        _norm("norm_t1", "norm", 1, 6144, True, "channel", False, False),
        # and for a prefill chunk, with a sigmoid gate per token as shared experts have it
        _norm("norm_t8192", "norm", 8192, 6144, True, "token", True, False),
        # their backward pass for a training batch, a float32 residual stream
        _norm("norm_grad_t8192", "norm_grad", 8192, 6144, True, "channel", False, True),
        # and an odd one with a gate per element
        _norm("norm_grad_odd", "norm_grad", 333, 2056, True, "full", True, False),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    case = _draw(rng)
    del case["name"]
    return case


def _draw(rng):
    op = rng.choice(("grouped", "grouped", "dx", "dw", "norm", "norm_grad"))
    if op in ("norm", "norm_grad"):
        return _norm("", op, _log_int(rng, 1, 6000), 8 * _log_int(rng, 8, 896), rng.random() < 0.7,
                     rng.choice(("none", "channel", "token", "full")), rng.random() < 0.5, rng.random() < 0.5)
    gran = 0 if op == "dw" else rng.choice((0, 0, 16, 32))
    step = 32 if gran else 8
    M, E = _log_int(rng, 1, 8192), _log_int(rng, 1, 64)
    N, K = 8 * _log_int(rng, 16, 512), step * _log_int(rng, 512 // step, 5632 // step)
    small = rng.choice((0, 0, 0, 1, 2))  # a low-rank factor's sizes
    if small == 1:
        N = 8 * _log_int(rng, 1, 16)
    elif small == 2 and not gran:
        K = 8 * _log_int(rng, 1, 16)
    return _prod("", op, M, E, N, K, gran, rng.random() < 0.4)


# ----------------------------------------------------------------------------
# inputs


def _fp4(g, E, N, K, gran):
    """Uniform E2M1 codes; E4M3 scales log-uniform in [2^-10, 2^-3], or UE8M0 exponents uniform in [-10, -2]."""
    w = torch.randint(0, 256, (E, N, K // 2), generator=g, device="cuda", dtype=torch.uint8)
    if gran == 16:
        u = torch.rand((E, N, K // 16), generator=g, device="cuda")
        return w, u.mul_(7).sub_(10).exp2_().to(torch.float8_e4m3fn).view(torch.uint8)
    return w, torch.randint(117, 126, (E, N, K // 32), generator=g, device="cuda", dtype=torch.uint8)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 7907 + 29)

    def randn(*shape, sigma=1.0, dtype=torch.bfloat16):
        return torch.randn(shape, generator=g, device="cuda", dtype=dtype).mul_(sigma)

    s = {"case": dict(case)}
    if case["op"] in ("norm", "norm_grad"):
        T, H = case["T"], case["H"]
        stream = torch.float32 if case["f32"] else torch.bfloat16
        s["h"] = randn(T, H, sigma=3.0, dtype=stream)
        s["y"] = randn(T, H, sigma=0.5)
        s["pre_w"] = 1 + randn(H, sigma=0.2)
        s["post_w"] = 1 + randn(H, sigma=0.2) if case["post"] else None
        shape = {"none": None, "channel": (H,), "token": (T,), "full": (T, H)}[case["gate"]]
        s["gate"] = None if shape is None else randn(*shape)
        if case["op"] == "norm_grad":
            s["dh"] = randn(T, H, sigma=0.01, dtype=stream)
            s["dn"] = randn(T, H, sigma=0.01)
        return s
    M, E, N, K, gran = (case[n] for n in ("M", "E", "N", "K", "gran"))
    # the experts' popularity within a factor of a few, as a trained router has it
    p = torch.exp(0.5 * torch.randn(E, generator=g, device="cuda"))
    expert = torch.multinomial(p, M, replacement=True, generator=g).sort().values
    s["offsets"] = torch.searchsorted(expert, torch.arange(E + 1, device="cuda")).int()
    rows = (s["offsets"][1:] - s["offsets"][:-1]).tolist()
    # what a program that has counted its rows knows: the experts with rows, and the most of one
    s["active"] = torch.tensor([e for e in range(E) if rows[e]], device="cuda")
    s["most"] = max(rows)
    if case["op"] != "grouped":
        s["dy"] = randn(M, N, sigma=0.1)
    if case["op"] != "dx":
        s["x"] = randn(M, K)
    s["w"] = s["w_sf"] = s["w_gs"] = None
    if case["op"] != "dw":
        if gran:
            s["w"], s["w_sf"] = _fp4(g, E, N, K, gran)
            s["w_gs"] = 0.5 + 1.5 * torch.rand(E, generator=g, device="cuda") if gran == 16 else None
        else:
            s["w"] = randn(E, N, K, sigma=1 / math.sqrt(K))
    return s


# ----------------------------------------------------------------------------
# the plain forms


def _plain_weight(s):
    """The active experts' weights in 32 bits."""
    at, gran = s["active"], s["case"]["gran"]
    if not gran:
        return s["w"][at].float()
    m = torch.tensor(_E2M1, device="cuda")
    tab = torch.cat([m, -m])
    pair = torch.stack([tab.repeat(16), tab.repeat_interleave(16)], 1)  # byte -> (low nibble, high nibble)
    v = pair[s["w"][at].int()].flatten(-2)
    sf = s["w_sf"][at]
    sc = sf.view(torch.float8_e4m3fn).float() if gran == 16 else torch.exp2(sf.float() - 127)
    v = v.view(*v.shape[:-1], -1, gran).mul_(sc.unsqueeze(-1)).flatten(-2)
    return v if s["w_gs"] is None else v.mul_(s["w_gs"][at].view(-1, 1, 1))


def _place(s):
    """Of each row: its expert's place among the active ones, and its own among the expert's."""
    r = torch.arange(s["case"]["M"], device="cuda", dtype=torch.int32)
    e = torch.bucketize(r, s["offsets"][1:], right=True)
    return torch.bucketize(e, s["active"]), (r - s["offsets"][e]).long()


def _padded(s, x, at):
    """Rows [M, C] as [active experts, most rows of one, C] in 32 bits, zeros behind an expert's last."""
    v = torch.zeros((s["active"].numel(), s["most"], x.shape[1]), device="cuda")
    v[at] = x.float()
    return v


def _plain_product(s):
    case, at = s["case"], _place(s)
    dtype = torch.float32 if case["f32"] else torch.bfloat16
    if case["op"] == "grouped":
        return torch.bmm(_padded(s, s["x"], at), _plain_weight(s).transpose(1, 2))[at].to(dtype)
    if case["op"] == "dx":
        return torch.bmm(_padded(s, s["dy"], at), _plain_weight(s))[at].to(dtype)
    dw = torch.zeros((case["E"], case["N"], case["K"]), device="cuda", dtype=dtype)
    dw[s["active"]] = torch.bmm(_padded(s, s["dy"], at).transpose(1, 2), _padded(s, s["x"], at)).to(dtype)
    return dw


_SCALE, _H_SCALE = 0.75, 1.25


def _gate_of(s, x):
    """The gate of every element, broadcast, in x's type."""
    if s["gate"] is None:
        return None
    g = s["gate"].to(x.dtype)
    return g.unsqueeze(1) if s["case"]["gate"] == "token" else g


def _plain_norm(s):
    y, h = s["y"].float(), s["h"].float()
    if s["post_w"] is not None:
        y = y * torch.rsqrt((y * y).mean(-1, keepdim=True) + _EPS) * s["post_w"].float()
    g = _gate_of(s, y)
    if g is not None:
        y = y * (torch.sigmoid(g) if s["case"]["sig"] else g)
    h = _H_SCALE * h + _SCALE * y
    n = h * torch.rsqrt((h * h).mean(-1, keepdim=True) + _EPS) * s["pre_w"].float()
    return h.to(s["h"].dtype), n.bfloat16()


def _plain_norm_grad(s):
    case = s["case"]
    h, y, dn = s["h"].float(), s["y"].float(), s["dn"].float()
    r = torch.rsqrt((h * h).mean(-1, keepdim=True) + _EPS)
    hh = h * r
    u = dn * s["pre_w"].float()
    d_pre = (dn * hh).sum(0)
    d = s["dh"].float() + r * (u - hh * (u * hh).mean(-1, keepdim=True))
    d_h = (_H_SCALE * d).to(s["h"].dtype)
    ry, yy, a = None, None, y
    if s["post_w"] is not None:
        ry = torch.rsqrt((y * y).mean(-1, keepdim=True) + _EPS)
        yy = y * ry
        a = yy * s["post_w"].float()
    g, d_gate = _gate_of(s, y), None
    da = _SCALE * d
    if g is not None:
        act = torch.sigmoid(g) if case["sig"] else g
        d_gate = da * a * (act * (1 - act)) if case["sig"] else da * a
        d_gate = (d_gate.sum(0) if case["gate"] == "channel" else d_gate.sum(1) if case["gate"] == "token" else
                  d_gate.to(s["gate"].dtype))
        da = da * act
    if s["post_w"] is None:
        return d_h, da.bfloat16(), None, d_gate, d_pre
    v = da * s["post_w"].float()
    dy = ry * (v - yy * (v * yy).mean(-1, keepdim=True))
    return d_h, dy.bfloat16(), (da * yy).sum(0), d_gate, d_pre


def run(s):
    case = s["case"]
    op = case["op"]
    if not own:
        return _plain_norm(s) if op == "norm" else _plain_norm_grad(s) if op == "norm_grad" else _plain_product(s)
    import block_scaled_fp4_topk_amd as moe
    act = "sigmoid" if case.get("sig") else None
    if op == "norm":
        return moe.block_norm(s["h"], s["y"], post_w=s["post_w"], gate=s["gate"], gate_act=act, scale=_SCALE,
                              h_scale=_H_SCALE, pre_w=s["pre_w"], eps=_EPS)
    if op == "norm_grad":
        return moe.block_norm_grad(s["dh"], s["dn"], s["h"], s["y"], post_w=s["post_w"], gate=s["gate"], gate_act=act,
                                   scale=_SCALE, h_scale=_H_SCALE, pre_w=s["pre_w"], eps=_EPS)
    dtype = torch.float32 if case["f32"] else torch.bfloat16
    if op == "dw":
        return moe.grouped_dw(s["dy"], s["x"], s["offsets"], out_dtype=dtype)
    if op == "dx":
        return moe.grouped_dx(s["dy"], s["w"], s["offsets"], w_sf=s["w_sf"], w_gs=s["w_gs"], gran_k=case["gran"] or None,
                              out_dtype=dtype)
    return moe.grouped(s["x"], s["w"], s["offsets"], w_sf=s["w_sf"], w_gs=s["w_gs"], gran_k=case["gran"] or None,
                       out_dtype=dtype)


# ----------------------------------------------------------------------------
# the definition in 64 bits


def _exact_weight(s, e):
    """One expert's matrix."""
    if not s["case"]["gran"]:
        return s["w"][e].double()
    codes, sf, gran = s["w"][e], s["w_sf"][e], s["case"]["gran"]
    nib = torch.stack([codes & 15, codes >> 4], -1).flatten(1)
    mag, sign = (nib & 7).double(), 1.0 - 2.0 * (nib >> 3).double()
    ex = torch.clamp(torch.floor(mag / 2), min=1)  # E2M1: 2^(e-1) (1 + m/2), subnormal m/2 at e = 0
    v = torch.where(mag < 2, mag / 2, torch.exp2(ex - 1) * (1 + (mag - 2 * ex) / 2)) * sign
    b = sf.view(torch.float8_e4m3fn).double() if gran == 16 else torch.exp2(sf.double() - 127)
    v = v * b.repeat_interleave(gran, 1)
    return v if s["w_gs"] is None else v * s["w_gs"][e].double()


def _exact_product(case, s):
    M, E, N, K, op = (case[n] for n in ("M", "E", "N", "K", "op"))
    off = s["offsets"].tolist()
    out = torch.zeros({"grouped": (M, N), "dx": (M, K), "dw": (E, N, K)}[op], dtype=torch.float64, device="cuda")
    for e in range(E):
        a, b = off[e], off[e + 1]
        if a == b:
            continue
        if op == "grouped":
            out[a:b] = s["x"][a:b].double() @ _exact_weight(s, e).T
        elif op == "dx":
            out[a:b] = s["dy"][a:b].double() @ _exact_weight(s, e)
        else:
            out[e] = s["dy"][a:b].double().T @ s["x"][a:b].double()
    return out


def _exact_rms(x, w):
    return x / torch.sqrt(torch.mean(x ** 2, dim=1, keepdim=True) + _EPS) * w


def _exact_branch(case, y, post_w, gate):
    a = y if post_w is None else _exact_rms(y, post_w)
    if gate is not None:
        f = 1 / (1 + torch.exp(-gate)) if case["sig"] else gate
        a = a * (f[:, None] if case["gate"] == "token" else f)
    return _SCALE * a


def _exact_norm(case, s):
    d = {n: None if s.get(n) is None else s[n].double() for n in ("h", "y", "pre_w", "post_w", "gate", "dh", "dn")}
    if case["op"] == "norm":
        h = _H_SCALE * d["h"] + _exact_branch(case, d["y"], d["post_w"], d["gate"])
        return h, _exact_rms(h, d["pre_w"])
    # the gradient by differentiating the definition: first the norm behind the sum, then the branch
    for n in ("h", "y", "pre_w", "post_w", "gate"):
        if d[n] is not None:
            d[n].requires_grad_()
    _exact_rms(d["h"], d["pre_w"]).backward(d["dn"])
    total = d["h"].grad + d["dh"]
    _exact_branch(case, d["y"], d["post_w"], d["gate"]).backward(total)
    grad = [None if d[n] is None else d[n].grad for n in ("y", "post_w", "gate", "pre_w")]
    return (_H_SCALE * total, *grad)


def exact(case, seed):
    s = prepare(case, seed)
    return _exact_norm(case, s) if case["op"] in ("norm", "norm_grad") else _exact_product(case, s)


# ----------------------------------------------------------------------------
# what a pass cannot do without


def work(case):
    f = 4 if case["f32"] else 2
    if case["op"] in ("norm", "norm_grad"):
        T, H = case["T"], case["H"]
        gate = {"none": 0, "channel": H, "token": T, "full": T * H}[case["gate"]]
        weights = H * (2 if case["post"] else 1)
        if case["op"] == "norm":
            return {"bytes": T * H * (2 * f + 4) + 2 * gate + 2 * weights, "flops": 12 * T * H}
        d_gate = gate * (2 if case["gate"] == "full" else 4)
        return {"bytes": T * H * (3 * f + 6) + 2 * gate + d_gate + 6 * weights, "flops": 25 * T * H}
    M, E, N, K, gran = (case[n] for n in ("M", "E", "N", "K", "gran"))
    flops = 2 * M * N * K
    if case["op"] == "dw":
        return {"bytes": 2 * M * (N + K) + E * N * K * f + 4 * (E + 1), "flops": flops}
    # the expected number of experts with a row, were they equally popular
    active = E * (1 - (1 - 1 / E) ** M)
    per = N * K * 2 if not gran else N * K // 2 + N * K // gran
    rows = M * (2 * K + f * N) if case["op"] == "grouped" else M * (2 * N + f * K)
    return {"bytes": rows + active * per + 4 * (E + 1), "flops": flops}
