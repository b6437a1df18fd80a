"""The operators around the Sparse-BitLinear products in a training step and in serving, as cases that can be timed
and compared: the root-mean-square norm that takes in the residual and feeds the quantised products (and its backward
pass), the AdamW step over many master weights at once (states in 32 or 8 bits), and the linear softmax cross entropy
at the end of the network (and its backward pass).

`own` False: plain torch, in 32 bits (64 where a rounding border is near).  `own` True: the framework's entry points.
"""
import math

import torch

own = False

NORM_EPS = 1e-5
LR, BETA1, BETA2, ADAM_EPS, DECAY, STEP = 1e-3, 0.9, 0.95, 1e-8, 0.1, 7
IGNORE = -100
BLOCK = 256  # elements that share a scale in the 8-bit states
FLUSH = 2.0 ** -100  # a block whose largest magnitude is below this holds zeros


def listed():
    return [
        # serving, one new token: a linear's fp32 output joins the bf16 residual stream and leaves as int8 codes
        {"name": "norm_t1_k2560", "op": "norm", "t": 1, "k": 2560, "x": "f32", "stream": "bf16", "residual": True,
         "gain": True, "quant": True},
        # training, attention input of the 2560-wide network: both branches' sum, codes for the products, dW's operand
        {"name": "norm_t4096_k2560", "op": "norm", "t": 4096, "k": 2560, "x": "f32", "stream": "bf16", "residual": True,
         "gain": True, "quant": True},
        # training, the norm before the FFN's down projection: no residual, the widest rows
        {"name": "norm_t8192_k6912", "op": "norm", "t": 8192, "k": 6912, "x": "bf16", "stream": "bf16",
         "residual": False, "gain": True, "quant": True},
        # training, three products (q, k, v) share the normalised input, so three gradients arrive
        {"name": "norm_bwd_t4096_k2560_3dy", "op": "norm_bwd", "t": 4096, "k": 2560, "stream": "bf16", "dy": "bf16",
         "dys": 3, "residual": True, "gain": True},
        # the same on a fp32 residual stream, an odd number of rows, gradients in fp32
        {"name": "norm_bwd_t8191_k2560_f32", "op": "norm_bwd", "t": 8191, "k": 2560, "stream": "f32", "dy": "f32",
         "dys": 1, "residual": True, "gain": True},
        # the small tensors of a network: gains and other vectors of odd lengths
        {"name": "adamw32_small", "op": "adamw", "sizes": "2560*8,6912*4,1001,77,1,640*64", "nodecay": 15, "bits": 32,
         "grad": "f32", "master": True},
        # one transformer block of the 30-layer training step: q, k, v, o, gate, up, down and its norms' gains
        {"name": "adamw32_block", "op": "adamw", "sizes": "2560x2560*4,6912x2560*3,2560*2,6912", "nodecay": 3,
         "bits": 32, "grad": "bf16", "master": True},
        {"name": "adamw8_block", "op": "adamw", "sizes": "2560x2560*4,6912x2560*3,2560*2,6912", "nodecay": 3,
         "bits": 8, "grad": "bf16", "master": True},
        # a short batch over a small odd vocabulary
        {"name": "ce_t63_v4099_d512", "op": "ce", "t": 63, "v": 4099, "d": 512},
        # the training step's 8192 tokens over a large vocabulary
        {"name": "ce_t8192_v32768_d2560", "op": "ce", "t": 8192, "v": 32768, "d": 2560},
        {"name": "ce_bwd_t63_v4099_d512", "op": "ce_bwd", "t": 63, "v": 4099, "d": 512},
        {"name": "ce_bwd_t4096_v32768_d2560", "op": "ce_bwd", "t": 4096, "v": 32768, "d": 2560},
    ]


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["norm", "norm_bwd", "adamw", "ce", "ce_bwd"])
    if op == "norm":
        stream = rng.choice(["bf16", "f32"])
        return {"op": op, "t": _log(rng, 1, 8191), "k": 64 * _log(rng, 1, 108), "x": rng.choice(["bf16", "f32"]),
                "stream": stream, "residual": rng.random() < 0.7, "gain": rng.random() < 0.8,
                "quant": rng.random() < 0.7}
    if op == "norm_bwd":
        return {"op": op, "t": _log(rng, 1, 8191), "k": 8 * _log(rng, 8, 320), "stream": rng.choice(["bf16", "f32"]),
                "dy": rng.choice(["bf16", "f32"]), "dys": rng.randint(1, 3), "residual": rng.random() < 0.7,
                "gain": rng.random() < 0.8}
    if op == "adamw":
        sizes = ["%dx%d" % (_log(rng, 8, 6912), _log(rng, 64, 2560)) for _ in range(rng.randint(1, 4))]
        vectors = ["%d" % _log(rng, 1, 6912) for _ in range(rng.randint(0, 6))]
        return {"op": op, "sizes": ",".join(sizes + vectors), "nodecay": len(vectors), "bits": rng.choice([8, 32]),
                "grad": rng.choice(["bf16", "f32"]), "master": rng.random() < 0.6}
    return {"op": op, "t": _log(rng, 1, 4096), "v": _log(rng, 17, 32768), "d": 8 * _log(rng, 8, 320)}


def _numels(sizes):
    got = []
    for part in sizes.split(","):
        shape, _, times = part.partition("*")
        got += [math.prod(int(x) for x in shape.split("x"))] * int(times or 1)
    return got


def _offsets(numels):
    """Where each tensor starts in the flat buffers: at whole blocks, so that no block of a state spans two tensors."""
    at = [0]
    for n in numels:
        at.append(at[-1] + -(-n // BLOCK) * BLOCK)
    return at


def _type(name):
    return {"bf16": torch.bfloat16, "f32": torch.float32}[name]


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, std=1.0, mean=0.0, dtype=torch.float32):
        v = torch.randn(*shape, generator=gen, device="cuda", dtype=torch.float32)
        return v.mul_(std).add_(mean).to(dtype)

    def empty(*shape, dtype=torch.float32):
        return torch.empty(*shape, device="cuda", dtype=dtype)

    s = dict(case)
    op = case["op"]
    if op in ("norm", "norm_bwd"):
        t, k, stream = case["t"], case["k"], _type(case["stream"])
        s["gain_w"] = normal(k, std=0.1, mean=1.0, dtype=torch.bfloat16) if case["gain"] else None
        if op == "norm":
            s["x_in"] = normal(t, k, dtype=_type(case["x"]))
            s["res_in"] = normal(t, k, std=2.0, dtype=stream) if case["residual"] else None
            if t > 8:  # padding: rows of zeros behind the last sequence
                s["x_in"][-(t // 64 + 1):] = 0
                if case["residual"]:
                    s["res_in"][-(t // 64 + 1):] = 0
            s["h"] = empty(t, k, dtype=stream) if case["residual"] else None
            s["rstd"] = empty(t)
            s["out"] = empty(t, k, dtype=torch.bfloat16)
            s["xq"] = empty(t, k, dtype=torch.int8) if case["quant"] else None
            s["xscale"] = empty(t) if case["quant"] else None
        else:
            s["h"] = normal(t, k, std=2.0, dtype=stream)
            h64 = s["h"].double()
            s["rstd"] = (h64.square().mean(1) + NORM_EPS).rsqrt().float()
            del h64
            s["dys_in"] = [normal(t, k, std=0.01, dtype=_type(case["dy"])) for _ in range(case["dys"])]
            s["dres"] = normal(t, k, std=0.01, dtype=stream) if case["residual"] else None
            s["dh"] = empty(t, k, dtype=stream)
            s["dx"] = empty(t, k, dtype=torch.bfloat16) if case["stream"] == "f32" else None
            s["dgain"] = empty(k) if case["gain"] else None
            if own:
                from sparse_linear_layers_bitlinear_b200 import sbl
                s["ws"] = empty(max(sbl.rmsnorm_backward_workspace_bytes(t, k), 1), dtype=torch.uint8)
        return s
    if op == "adamw":
        numels = _numels(case["sizes"])
        at = _offsets(numels)
        n = at[-1]
        live = torch.zeros(n, device="cuda", dtype=torch.bool)
        for a, m in zip(at, numels):
            live[a:a + m] = True
        master = normal(n, std=0.02).mul_(live)
        row = torch.rand(n // BLOCK, 1, generator=gen, device="cuda").mul_(6).sub_(3).exp_()  # gradients differ by rows
        scale = (1e-3 * row).expand(-1, BLOCK).reshape(-1)
        s["w"] = master.to(torch.bfloat16)
        s["grad_in"] = normal(n).mul_(scale).mul_(live).to(_type(case["grad"]))
        m = normal(n, std=0.4).mul_(scale).mul_(live)
        v = normal(n, std=0.5).abs_().add_(0.2).mul_(scale.square()).mul_(live)
        s["w_master"] = master if case["master"] else None
        if case["bits"] == 8:
            s["m"], s["m_scale"] = _store8(m)
            s["v"], s["v_scale"] = _store8(v.sqrt(), True)
        else:
            s["m"], s["v"], s["m_scale"], s["v_scale"] = m, v, None, None
        s["decayed"] = at[len(numels) - case["nodecay"]]
        if own:
            from sparse_linear_layers_bitlinear_b200 import sbl

            def part(flat, i, per=1):
                return None if flat is None else flat[at[i] // per:at[i] // per + -(-numels[i] // per)]

            s["plan"] = sbl.AdamWTensors([
                sbl.AdamWTensor(w=part(s["w"], i), grad=part(s["grad_in"], i), m=part(s["m"], i), v=part(s["v"], i),
                                m_scale=part(s["m_scale"], i, BLOCK), v_scale=part(s["v_scale"], i, BLOCK),
                                master=part(s["w_master"], i), decay=i < len(numels) - case["nodecay"])
                for i in range(len(numels))])
        return s
    t, v, d = case["t"], case["v"], case["d"]
    s["h_in"] = normal(t, d, dtype=torch.bfloat16)
    s["w_in"] = normal(v, d, std=0.02, dtype=torch.bfloat16)
    s["targets"] = torch.randint(0, v, (t,), generator=gen, device="cuda")
    if t > 8:  # prompts and padding carry no loss
        s["targets"][torch.rand(t, generator=gen, device="cuda") < 0.1] = IGNORE
    if op == "ce":
        s["loss"], s["lse"] = empty(t), empty(t)
    else:
        s["lse"] = torch.cat([torch.logsumexp(a.double() @ s["w_in"].double().T, 1) for a in s["h_in"].split(2048)]).float()
        s["dloss"] = normal(t, std=0.2, mean=1.0) / t
        s["dh"], s["dw"] = empty(t, d, dtype=torch.bfloat16), empty(v, d, dtype=torch.bfloat16)
    if own:
        from sparse_linear_layers_bitlinear_b200 import sbl
        s["ws"] = empty(sbl.linear_ce_workspace_bytes(t, v, d, backward=op == "ce_bwd"), dtype=torch.uint8)
    return s


def _store8(x, positive=False):
    """Blocks of 256 values as e4m3 with a scale each: the block's largest magnitude stands at 448.  `positive`: no
    value but zero becomes zero (a second moment of zero would let the step grow without bound)."""
    x = x.reshape(-1, BLOCK)
    top = x.abs().amax(1, keepdim=True)
    used = top >= FLUSH
    q = torch.where(used, x * (448 / torch.where(used, top, 1.0)), 0.0)
    if positive:
        q = torch.where(q > 0, q.clamp_min(2.0 ** -9), q)
    return q.to(torch.float8_e4m3fn).reshape(-1), torch.where(used, top / 448, 0.0).reshape(-1)


def _load8(q, scale):
    return (q.float().reshape(-1, BLOCK) * scale[:, None]).reshape(-1)


def _plain_norm(s):
    stream = _type(s["stream"])
    if s["residual"]:
        h = (s["x_in"].float() + s["res_in"].float()).to(stream)
    else:
        h = s["x_in"]
    hf = h.float()
    # 64 bits: the codes below are at a rounding border where the last bit of rstd counts
    rstd = (1 / (hf.double().square().mean(1) + NORM_EPS).sqrt()).float()
    xn = hf * rstd[:, None]
    if s["gain"]:
        xn = xn * s["gain_w"].float()
    xn = xn.to(torch.bfloat16)
    out = {"rstd": rstd}
    if s["residual"]:
        out["h"] = h
    if not s["quant"]:
        return out | {"xn": xn}
    xf = xn.float()
    top = xf.abs().amax(1).clamp_min(1e-5)
    # quotients in 64 bits: whole codes come of a rounding, ties among them
    code = ((127 * xf).double() / top.double()[:, None]).round()
    return out | {"xhat": (code * top.double()[:, None] / 127).to(torch.bfloat16), "xscale": top}


def _plain_norm_bwd(s):
    stream = _type(s["stream"])
    g = s["dys_in"][0].float()
    if s["dys"] > 1:
        g = g + s["dys_in"][1].float()
    if s["dys"] > 2:
        g = g + s["dys_in"][2].float()
    hat = s["h"].float() * s["rstd"][:, None]
    wg = g * s["gain_w"].float() if s["gain"] else g
    dh = s["rstd"][:, None] * (wg - hat * (wg * hat).mean(1, keepdim=True))
    if s["residual"]:
        dh = dh + s["dres"].float()
    out = {"dh": dh.to(stream)}
    if s["stream"] == "f32":
        out["dx"] = dh.to(torch.bfloat16)
    if s["gain"]:
        out["dgain"] = (g * hat).sum(0)
    return out


def _plain_adamw(s):
    g = s["grad_in"].float()
    eight = s["bits"] == 8
    m = _load8(s["m"], s["m_scale"]) if eight else s["m"]
    v = _load8(s["v"], s["v_scale"]).square() if eight else s["v"]
    m = BETA1 * m + (1 - BETA1) * g
    v = BETA2 * v + (1 - BETA2) * g * g
    w = s["w_master"] if s["master"] else s["w"].float()
    step = (m / (1 - BETA1 ** STEP)) / ((v / (1 - BETA2 ** STEP)).sqrt() + ADAM_EPS)
    n = s["decayed"]
    w = torch.cat([w[:n] * (1 - LR * DECAY), w[n:]]) - LR * step
    s["w"].copy_(w)
    if s["master"]:
        s["w_master"].copy_(w)
    if eight:
        for name, q in (("m", _store8(m)), ("v", _store8(v.sqrt(), True))):
            s[name].copy_(q[0])
            s[name + "_scale"].copy_(q[1])
    else:
        s["m"].copy_(m)
        s["v"].copy_(v)
    return _adamw_outputs(s)


def _adamw_outputs(s):
    return {name: s[name] for name in ("w", "w_master", "m", "v", "m_scale", "v_scale") if s[name] is not None}


def _plain_ce(s):
    z = s["h_in"].float() @ s["w_in"].float().T
    top = z.amax(1, keepdim=True)
    lse = top[:, 0] + (z - top).exp().sum(1).log()
    live = s["targets"] != IGNORE
    at = torch.where(live, s["targets"], 0)
    return {"loss": torch.where(live, lse - z.gather(1, at[:, None])[:, 0], 0.0), "lse": lse}


def _plain_ce_bwd(s):
    h, w = s["h_in"].float(), s["w_in"].float()
    live = s["targets"] != IGNORE
    at = torch.where(live, s["targets"], 0)
    dz = (h @ w.T - s["lse"][:, None]).exp()
    dz.scatter_add_(1, at[:, None], torch.full_like(dz[:, :1], -1.0))
    dz *= torch.where(live, s["dloss"], 0.0)[:, None]
    return {"dh": (dz @ w).to(torch.bfloat16), "dw": (dz.T @ h).to(torch.bfloat16)}


def run(state):
    s, op = state, state["op"]
    if not own:
        return {"norm": _plain_norm, "norm_bwd": _plain_norm_bwd, "adamw": _plain_adamw, "ce": _plain_ce,
                "ce_bwd": _plain_ce_bwd}[op](s)
    from sparse_linear_layers_bitlinear_b200 import sbl
    if op == "norm":
        name = "xhat" if s["quant"] else "xn"
        sbl.rmsnorm_forward(s["x_in"], s["t"], s["k"], NORM_EPS, residual=s["res_in"], weight=s["gain_w"],
                            h_out=s["h"], rstd_out=s["rstd"], xq_out=s["xq"], xscale_out=s["xscale"],
                            **{name + "_out": s["out"]})
        out = {"rstd": s["rstd"], name: s["out"]}
        if s["residual"]:
            out["h"] = s["h"]
        if s["quant"]:
            out["xscale"] = s["xscale"]
        return out
    if op == "norm_bwd":
        sbl.rmsnorm_backward(s["h"], s["rstd"], s["dys_in"], s["t"], s["k"], s["dh"], weight=s["gain_w"],
                             dres=s["dres"], dx=s["dx"], dw=s["dgain"], workspace=s["ws"])
        out = {"dh": s["dh"]}
        if s["stream"] == "f32":
            out["dx"] = s["dx"]
        if s["gain"]:
            out["dgain"] = s["dgain"]
        return out
    if op == "adamw":
        sbl.adamw_step(s["plan"], STEP, lr=LR, beta1=BETA1, beta2=BETA2, eps=ADAM_EPS, weight_decay=DECAY)
        return _adamw_outputs(s)
    if op == "ce":
        sbl.linear_ce_forward(s["h_in"], s["w_in"], s["targets"], s["t"], s["v"], s["d"], s["loss"], s["lse"], s["ws"],
                              ignore_index=IGNORE)
        return {"loss": s["loss"], "lse": s["lse"]}
    sbl.linear_ce_backward(s["h_in"], s["w_in"], s["targets"], s["lse"], s["dloss"], s["t"], s["v"], s["d"], s["dh"],
                           s["dw"], s["ws"], ignore_index=IGNORE)
    return {"dh": s["dh"], "dw": s["dw"]}


def work(case):
    op = case["op"]
    if op in ("norm", "norm_bwd"):
        t, k = case["t"], case["k"]
        size = {"bf16": 2, "f32": 4}
        stream = size[case["stream"]]
        gain = 2 * k if case["gain"] else 0
        if op == "norm":
            read = size[case["x"]] + (stream if case["residual"] else 0)
            wrote = (stream if case["residual"] else 0) + 2 + (1 if case["quant"] else 0)
            return {"bytes": t * k * (read + wrote) + gain + t * (8 if case["quant"] else 4), "flops": 8 * t * k}
        read = stream + case["dys"] * size[case["dy"]] + (stream if case["residual"] else 0)
        wrote = stream + (2 if case["stream"] == "f32" else 0)
        return {"bytes": t * k * (read + wrote) + 3 * gain + 4 * t, "flops": 12 * t * k}
    if op == "adamw":
        numels = _numels(case["sizes"])
        n, blocks = sum(numels), sum(-(-m // BLOCK) for m in numels)
        grad = {"bf16": 2, "f32": 4}[case["grad"]]
        weight = 4 + 4 + 2 if case["master"] else 2 + 2
        states = (4 * n + 16 * blocks) if case["bits"] == 8 else 16 * n
        return {"bytes": n * (grad + weight) + states, "flops": 16 * n}
    t, v, d = case["t"], case["v"], case["d"]
    if op == "ce":
        return {"bytes": 2 * (t + v) * d + 16 * t, "flops": 2 * t * v * d}
    return {"bytes": 4 * (t + v) * d + 16 * t, "flops": 6 * t * v * d}


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "norm":
        # the stored stream and the normalised rows are bf16 (or fp32) by definition: the quantiser takes them so
        h = s["x_in"].double()
        out = {}
        if case["residual"]:
            h = (h + s["res_in"].double()).to(_type(case["stream"])).double()
            out["h"] = h
        out["rstd"] = (h.pow(2).sum(1) / case["k"] + NORM_EPS).pow(-0.5)
        y = h * out["rstd"].unsqueeze(1)
        if case["gain"]:
            y = y * s["gain_w"].double()
        if not case["quant"]:
            return out | {"xn": y}
        y = y.to(torch.bfloat16).double()
        top = y.abs().max(1, keepdim=True).values.clamp(min=1e-5)
        # a scale is the largest bf16 value of its row: of two neighbours at a border either is right
        return out | {"xhat": torch.round(127 * y / top) * top / 127, "xscale": None}
    if op == "norm_bwd":
        h, r = s["h"].double(), s["rstd"].double().unsqueeze(1)
        g = sum(x.double() for x in s["dys_in"])
        u = g * s["gain_w"].double() if case["gain"] else g
        dh = u * r - h * r.pow(3) * ((u * h).sum(1, keepdim=True) / case["k"])
        if case["residual"]:
            dh = dh + s["dres"].double()
        out = {"dh": dh}
        if case["stream"] == "f32":
            out["dx"] = dh
        if case["gain"]:
            out["dgain"] = torch.einsum("tk,tk,t->k", g, h, r[:, 0])
        return out
    if op == "adamw":
        g = s["grad_in"].double()
        m, v = s["m"].double(), s["v"].double()
        if case["bits"] == 8:
            m = m * s["m_scale"].double().repeat_interleave(BLOCK)
            v = (v * s["v_scale"].double().repeat_interleave(BLOCK)) ** 2
        m = m + (1 - BETA1) * (g - m)
        v = v + (1 - BETA2) * (g.pow(2) - v)
        w = (s["w_master"] if case["master"] else s["w"]).double()
        rate = torch.zeros_like(w)
        rate[:s["decayed"]] = LR * DECAY
        hat = math.sqrt(1 - BETA2 ** STEP) / (1 - BETA1 ** STEP)
        w = w - rate * w - LR * hat * m / (v.sqrt() + ADAM_EPS * math.sqrt(1 - BETA2 ** STEP))
        out = {"w": w}
        if case["master"]:
            out["w_master"] = w
        if case["bits"] == 32:
            return out | {"m": m, "v": v}
        for name, x in (("m", m), ("v", v.sqrt())):  # the 8-bit values before their rounding
            top = x.view(-1, BLOCK).abs().max(1).values
            out[name + "_scale"] = top / 448
            unit = torch.where(top > 0, 448 / top, 0.0)
            out[name] = x * unit.repeat_interleave(BLOCK)
        return out
    h, w = s["h_in"].double(), s["w_in"].double()
    live = (s["targets"] != IGNORE).double()
    at = s["targets"].clamp(min=0)
    if op == "ce":
        lse, hit = [], []
        for a, i in zip(h.split(1024), at.split(1024)):
            z = a @ w.T
            lse.append(torch.logsumexp(z, 1))
            hit.append((a * w[i]).sum(1))
        lse = torch.cat(lse)
        return {"loss": (lse - torch.cat(hit)) * live, "lse": lse}
    dh, dw = [], torch.zeros_like(w)
    rows = s["dloss"].double() * live
    for a, i, r, e in zip(h.split(1024), at.split(1024), rows.split(1024), s["lse"].double().split(1024)):
        dz = torch.exp(a @ w.T - e[:, None])
        dz[torch.arange(len(i), device=i.device), i] -= 1
        dz *= r[:, None]
        dh.append(dz @ w)
        dw += dz.T @ a
    return {"dh": torch.cat(dh), "dw": dw}
