"""Cases of the selective scan, its short convolution, the layer norm and gradient clipping: what is timed, in plain form
and through the library.

The short convolution of each channel c, over the last W rows of its sequence, with an optional SiLU:

    y_t = act(bias + sum_j w[j] x_{t - W + 1 + j})

The selective scan keeps for every sequence and channel a state h [N] and per token does

    dt = softplus(delta + bias),   h <- exp(dt A) h + dt x B,   y = (C . h + D x) silu(z)

(A [channels, N]; B, C [N] of a token are shared by the channels of a group).  The layer norm does

    s = x + residual (rounded to the stored type),   y = (s - mean(s)) / sqrt(var(s) + eps) * w + b

and clipping scales a list of gradients by min(1, most / (norm + 1e-6)), norm being that of all of them together.

Ops:  convstep   new tokens of decoding sequences against a pool of their last inputs, updated in place
      conv       whole prompts: outputs and the inputs to carry on from
      convtrain  forward and backward over whole sequences
      step       the scan's new tokens against a pool of states, updated in place
      prefill    the scan over whole prompts: outputs and the state after each sequence
      train      the scan forward and backward over whole sequences
      norm       residual layer norm, forward     normtrain  forward and backward
      clip       the global norm of many gradients, and the clipped gradients
"""
import math

import torch

own = False
DEVICE = "cuda"
EPS = 1e-5
MOST = 1.0              # the norm that gradients are clipped to
PLAIN_VALUES = 1 << 26  # channels x states x rows that the plain form of the scan takes together


def listed():
    return [
        # a server's batch, one token each, in front of the scan
        dict(name="convstep_64x4096_bf16", op="convstep", n=64, t=1, d=4096, w=4, pool=70, math="bf16"),
        # pre-training batch, both directions
        dict(name="convtrain_8x2048x4096_bf16", op="convtrain", lens="8x2048", d=4096, w=4, start=0, math="bf16"),
        # one user's next token: latency
        dict(name="step_1x2048_bf16", op="step", n=1, t=1, d=2048, g=1, s=16, pool=4, math="bf16"),
        # a server's batch: the states' bandwidth
        dict(name="step_192x4096_bf16", op="step", n=192, t=1, d=4096, g=1, s=16, pool=200, math="bf16"),
        # one long document: few channels, the serial axis is the bound
        dict(name="prefill_1x16384x2048_bf16", op="prefill", lens="16384", d=2048, g=1, s=16, start=0, math="bf16"),
        # a serving batch of prompts of all lengths, an empty and a one-token one among them, states carried in, two groups
        dict(name="prefill_ragged_bf16", op="prefill", lens="0,1,64,63,65,511,1025,2048,4100,333,1,2999,700,128,1777,96",
             d=2560, g=2, s=16, start=1, math="bf16"),
        # pre-training batch, both directions
        dict(name="train_8x2048x4096_bf16", op="train", lens="8x2048", d=4096, g=1, s=16, start=0, math="bf16"),
        # the trunk width and window of this repository's smoke workload, fp32
        dict(name="train_32x64x128_fp32", op="train", lens="32x64", d=128, g=1, s=16, start=0, math="fp32"),
        # the norm of one decoding batch, odd width, fp32: latency
        dict(name="norm_37x1001_fp32", op="norm", rows=37, d=1001, math="fp32"),
        # a training batch's rows, odd count, both directions
        dict(name="normtrain_16383x2560_bf16", op="normtrain", rows=16383, d=2560, math="bf16"),
        # the parameters of a small trunk and cell: 26 tensors of 3 to 24,576 values, fp32: latency
        dict(name="clip_small_fp32", op="clip", sizes="24576,49152,384,128,10240,8192,128,4,10240,8192,128,4,128,128,3,5,"
             "2048,2048,512,512,128,128,4096,4096,64,1001", kind="fp32"),
        # a large trunk's: matrices in bf16, their norms and gates in fp32
        dict(name="clip_large_mixed", op="clip", sizes=",".join(["41943040,20971520,10485760,2560,4096,65537"] * 8),
             kind="mixed"),
    ]


def draw(rng):
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    most = max(_cost(c) for c in listed())
    while True:
        op = rng.choice(("convstep", "conv", "convtrain", "step", "prefill", "train", "norm", "normtrain", "clip"))
        bits = rng.choice(("bf16", "bf16", "fp32"))
        c = dict(op=op, math=bits)
        if op == "clip":
            c = dict(op=op, kind=rng.choice(("bf16", "fp32", "mixed")),
                     sizes=",".join(str(log(1, 1 << 24)) for _ in range(log(1, 100))))
        elif op in ("norm", "normtrain"):
            c.update(rows=log(1, 65536), d=8 * log(1, 1024) if rng.random() < 0.7 else log(2, 8192))
        else:
            if "conv" in op:
                c.update(d=8 * log(4, 1024), w=rng.choice((2, 3, 4, 4, 4, 8)))
            else:
                g = rng.choice((1, 1, 1, 2, 4))
                c.update(d=8 * g * max(1, log(4, 1024) // g), g=g, s=rng.choice((4, 8, 16, 16, 16, 24, 32, 64)))
            if "step" in op:
                n = log(1, 256)
                c.update(n=n, t=rng.choice((1, 1, 2, 5)), pool=n + rng.randrange(1, 9))
            else:
                if rng.random() < 0.5:
                    lens = "%dx%d" % (log(1, 64), log(1, 8192))
                else:
                    lens = ",".join(str(rng.choice((0, 1, log(2, 4096), log(2, 4096)))) for _ in range(rng.randrange(2, 17)))
                c.update(lens=lens, start=0 if "train" in op else rng.randrange(2))
                if not 1 <= sum(_lens(c)) <= 32768 or max(_lens(c)) > 16384:
                    continue
        if _cost(c) <= most:
            return c


def _lens(case):
    """Sequence lengths: "8x2048" is eight of 2048, "1,64,0" a packed batch."""
    text = case["lens"]
    if "x" in text:
        n, t = text.split("x")
        return [int(t)] * int(n)
    return [int(t) for t in text.split(",")]


def _types(case):
    """The stored type; of a list of gradients, each one's."""
    if case["op"] != "clip":
        return torch.bfloat16 if case["math"] == "bf16" else torch.float32
    sizes = [int(n) for n in case["sizes"].split(",")]
    half = {"bf16": lambda n: True, "fp32": lambda n: False, "mixed": lambda n: n >= 8192}[case["kind"]]
    return [(n, torch.bfloat16 if half(n) else torch.float32) for n in sizes]


def _cost(case):
    w = work(case)
    return max(w["bytes"], w["flops"] / 10)


def work(case):
    if case["op"] == "clip":
        pairs = _types(case)
        return {"bytes": 2.0 * sum(n * t.itemsize for n, t in pairs) + 4, "flops": 3.0 * sum(n for n, _ in pairs)}
    size = _types(case).itemsize
    if case["op"] == "norm":
        n = case["rows"] * case["d"]
        return {"bytes": 4.0 * n * size + 8 * case["d"], "flops": 8.0 * n}
    if case["op"] == "normtrain":
        n = case["rows"] * case["d"]
        return {"bytes": 8.0 * n * size + 16 * case["d"], "flops": 20.0 * n}
    d = case["d"]
    if "step" in case["op"]:
        seqs, rows = case["n"], case["n"] * case["t"]
    else:
        seqs, rows = len(_lens(case)), sum(_lens(case))
    if "conv" in case["op"]:
        w = case["w"]
        states = 2 * seqs if case["op"] == "convstep" else seqs * (1 + case["start"]) if case["op"] == "conv" else 0
        bytes_ = 2.0 * rows * d * size + states * (w - 1) * d * size + 4 * d * (w + 1)
        flops = (2.0 * w + 4) * rows * d
        if case["op"] == "convtrain":       # x and grad_y, grad_x; the weights' gradients
            bytes_ += 3.0 * rows * d * size + 8 * d * (w + 1)
            flops += (6.0 * w + 8) * rows * d
        return {"bytes": bytes_, "flops": flops}
    g, s = case["g"], case["s"]
    states = 2 * seqs if case["op"] == "step" else seqs * (1 + case["start"]) if case["op"] == "prefill" else 0
    bytes_ = rows * (4.0 * d + 2 * g * s) * size + 4.0 * states * d * s + 4.0 * d * (s + 2)
    flops = rows * d * (7.0 * s + 10)       # dt A, exp, dt x B, the state's update, C . h
    if case["op"] == "train":               # x, delta, z, B, C and grad_y; their gradients; A's, D's and the bias's
        bytes_ += rows * (7.0 * d + 4 * g * s) * size + 8.0 * d * (s + 2)
        flops += rows * d * (21.0 * s + 20)
    return {"bytes": bytes_, "flops": flops}


def prepare(case, seed):
    gen = torch.Generator(device=DEVICE).manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, device=DEVICE, generator=gen)

    def uniform(*shape):
        return torch.rand(*shape, device=DEVICE, generator=gen)

    state = dict(case=dict(case))
    if case["op"] == "clip":
        # gradients of very different sizes from tensor to tensor
        state["grads"] = [(normal(n) * 10.0 ** (float(uniform(1)) * 3 - 4)).to(t) for n, t in _types(case)]
        return state
    dtype = _types(case)
    if "norm" in case["op"]:
        rows, d = case["rows"], case["d"]
        state["x"] = normal(rows, d).to(dtype)
        state["residual"] = (2 * normal(rows, d) + 0.5 * normal(d)).to(dtype)
        state["weight"], state["bias"] = 1 + 0.2 * normal(d), 0.2 * normal(d)
        if case["op"] == "normtrain":
            state["grad_y"], state["grad_s"] = normal(rows, d).to(dtype), normal(rows, d).to(dtype)
        return state
    d = case["d"]
    if "step" in case["op"]:
        lead = (case["n"], case["t"])
        order = torch.randperm(case["pool"], device=DEVICE, generator=gen)
        state["slots"] = order[: case["n"]].to(torch.int32)
    else:
        lens = _lens(case)
        lead = (len(lens), lens[0]) if "x" in case["lens"] else (sum(lens),)
        ends = torch.tensor([0] + lens, device=DEVICE).cumsum(0)
        state["offsets"] = ends.to(torch.int32) if len(lead) == 1 else None
    if "conv" in case["op"]:
        w = case["w"]
        state["x"] = normal(*lead, 2 * d).to(dtype)[..., :d]        # beside its gate in one projection's output
        state["weight"] = (2 * uniform(d, w) - 1) * w ** -0.5
        state["bias"] = 0.1 * normal(d)
        if case["op"] == "convstep":
            state["pool"] = normal(case["pool"], w - 1, d).to(dtype)
        elif case["op"] == "conv":
            state["start"] = normal(len(lens), w - 1, d).to(dtype) if case["start"] else None
        else:
            state["grad_y"] = normal(*lead, d).to(dtype)
        return state
    g, s = case["g"], case["s"]
    v = normal(*lead, d)
    state["x"] = (v * torch.sigmoid(v)).to(dtype)                   # behind the convolution's SiLU
    state["z"] = normal(*lead, 2 * d).to(dtype)[..., d:]
    # time steps log-uniform in [0.001, 0.1] at the bias, moved by the token
    dt = torch.exp(uniform(d) * math.log(100.0) + math.log(0.001))
    state["bias"] = dt + torch.log(-torch.expm1(-dt))
    state["delta"] = (0.5 * normal(*lead, d)).to(dtype)
    state["A"] = -(torch.arange(1, s + 1, device=DEVICE) * (0.5 + uniform(d, s)))
    state["D"] = 1 + 0.2 * normal(d)
    # B and C behind the step's low-rank part in one projection's output
    proj = normal(*lead, 40 + 2 * g * s).to(dtype)
    state["B"] = proj[..., 40:40 + g * s].unflatten(-1, (g, s))
    state["C"] = proj[..., 40 + g * s:].unflatten(-1, (g, s))
    if case["op"] == "step":
        state["pool"] = 0.3 * normal(case["pool"], d, s)
    elif case["op"] == "prefill":
        state["start"] = 0.3 * normal(len(lens), d, s) if case["start"] else None
    else:
        state["grad_y"] = normal(*lead, d).to(dtype)
    return state


def run(state):
    op = state["case"]["op"]
    if own:
        return _OWN[op](state)
    return _PLAIN[op](state)


# ------------------------------------------------------------------ the library's calls

def _lib(case):
    import recurrent_cell_gb300 as cfc

    return cfc, cfc.MATH_BF16 if case["math"] == "bf16" else cfc.MATH_FP32


def _empty(t):
    return torch.empty(t.shape, dtype=t.dtype, device=t.device)


def _workspace(size):
    return torch.empty(size, dtype=torch.uint8, device=DEVICE)


def _own_convstep(s):
    cfc, mode = _lib(s["case"])
    y = _empty(s["x"])
    cfc.cfc_conv_step(s["x"], s["weight"], s["pool"], y, bias=s["bias"], slots=s["slots"], math=mode)
    return {"y": y, "pool": s["pool"]}


def _own_conv(s):
    cfc, mode = _lib(s["case"])
    case = s["case"]
    y = _empty(s["x"])
    final = torch.empty(len(_lens(case)), case["w"] - 1, case["d"], dtype=y.dtype, device=DEVICE)
    cfc.cfc_conv_forward(s["x"], s["weight"], y, bias=s["bias"], seq_offsets=s["offsets"], initial_state=s["start"],
                         final_state=final, math=mode)
    return {"y": y, "state": final}


def _own_convtrain(s):
    cfc, mode = _lib(s["case"])
    x, weight, bias, off = s["x"], s["weight"], s["bias"], s["offsets"]
    y = _empty(x)
    cfc.cfc_conv_forward(x, weight, y, bias=bias, seq_offsets=off, math=mode)
    gx, gw, gb = _empty(x), _empty(weight), _empty(bias)
    ws = _workspace(cfc.cfc_conv_workspace_bytes(x[..., 0].numel(), *weight.shape, math=mode))
    cfc.cfc_conv_backward(x, weight, s["grad_y"], gx, gw, ws, bias=bias, grad_bias=gb, seq_offsets=off, math=mode)
    return {"y": y, "grad_x": gx, "grad_w": gw, "grad_bias": gb}


def _own_step(s):
    cfc, mode = _lib(s["case"])
    y = _empty(s["x"])
    cfc.cfc_ssm_step(s["x"], s["delta"], s["A"], s["B"], s["C"], s["pool"], y, D=s["D"], z=s["z"], delta_bias=s["bias"],
                     slots=s["slots"], math=mode)
    return {"y": y, "pool": s["pool"]}


def _scan_workspace(cfc, mode, case, save):
    lens = _lens(case)
    return _workspace(cfc.cfc_ssm_workspace_bytes(sum(lens), len(lens), case["d"], case["g"], case["s"], mode, save=save))


def _own_prefill(s):
    cfc, mode = _lib(s["case"])
    case = s["case"]
    y = _empty(s["x"])
    final = torch.empty(len(_lens(case)), case["d"], case["s"], device=DEVICE)
    cfc.cfc_ssm_forward(s["x"], s["delta"], s["A"], s["B"], s["C"], y, _scan_workspace(cfc, mode, case, False), D=s["D"],
                        z=s["z"], delta_bias=s["bias"], seq_offsets=s["offsets"], initial_state=s["start"],
                        final_state=final, math=mode)
    return {"y": y, "state": final}


def _own_train(s):
    cfc, mode = _lib(s["case"])
    names = ("x", "delta", "A", "B", "C", "D", "z", "bias")
    x, delta, A, B, C, D, z, bias = (s[n] for n in names)
    y, ws = _empty(x), _scan_workspace(cfc, mode, s["case"], True)
    cfc.cfc_ssm_forward(x, delta, A, B, C, y, ws, D=D, z=z, delta_bias=bias, seq_offsets=s["offsets"], save=True, math=mode)
    gx, gdelta, gA, gB, gC, gD, gz, gbias = grads = [_empty(s[n]) for n in names]
    cfc.cfc_ssm_backward(x, delta, A, B, C, s["grad_y"], gx, gdelta, gA, gB, gC, ws, D=D, z=z, delta_bias=bias, grad_D=gD,
                         grad_z=gz, grad_delta_bias=gbias, seq_offsets=s["offsets"], math=mode)
    return dict(zip(["y"] + ["grad_" + n for n in names], [y] + grads))


def _own_norm(s):
    cfc, mode = _lib(s["case"])
    y, stream = _empty(s["x"]), _empty(s["x"])
    cfc.cfc_layernorm_forward(s["x"], s["weight"], y, bias=s["bias"], residual=s["residual"], residual_out=stream, eps=EPS,
                              math=mode)
    return {"y": y, "s": stream}


def _own_normtrain(s):
    cfc, mode = _lib(s["case"])
    x, weight, bias = s["x"], s["weight"], s["bias"]
    y, stream, gx = _empty(x), _empty(x), _empty(x)
    mean, rstd = torch.empty(x.shape[0], device=DEVICE), torch.empty(x.shape[0], device=DEVICE)
    cfc.cfc_layernorm_forward(x, weight, y, bias=bias, residual=s["residual"], residual_out=stream, mean=mean, rstd=rstd,
                              eps=EPS, math=mode)
    gw, gb = _empty(weight), _empty(bias)
    ws = _workspace(cfc.cfc_layernorm_workspace_bytes(*x.shape))
    cfc.cfc_layernorm_backward(stream, weight, mean, rstd, s["grad_y"], gx, gw, ws, grad_bias=gb,
                               grad_residual_out=s["grad_s"], math=mode)
    return {"y": y, "s": stream, "grad_x": gx, "grad_w": gw, "grad_bias": gb}


def _own_clip(s):
    import recurrent_cell_gb300 as cfc

    grads = s["grads"]
    out, norm = [_empty(g) for g in grads], torch.empty(1, device=DEVICE)
    ws = _workspace(cfc.cfc_grad_clip_workspace_bytes(len(grads)))
    cfc.cfc_grad_clip(grads, MOST, norm, ws, out=out)
    return {"norm": norm, "grads": out}


_OWN = dict(convstep=_own_convstep, conv=_own_conv, convtrain=_own_convtrain, step=_own_step, prefill=_own_prefill,
            train=_own_train, norm=_own_norm, normtrain=_own_normtrain, clip=_own_clip)


# ------------------------------------------------------------------ the plain forms

def _row_plan(case):
    """For the rows of all sequences one after another: each row's place in its sequence and its sequence."""
    lens = torch.tensor(_lens(case), device=DEVICE)
    seq = torch.repeat_interleave(torch.arange(len(lens), device=DEVICE), lens)
    first = lens.cumsum(0) - lens
    return torch.arange(len(seq), device=DEVICE) - first[seq], seq, first, lens


def _silu(v):
    return v / (1 + torch.exp(-v))


def _window(x, start, case):
    """The W inputs that row r of [rows, d] sees, [W, rows, d]; before the sequence: its start [sequences, W - 1, d] or 0."""
    w = case["w"]
    place, seq, _, _ = _row_plan(case)
    rows, out = torch.arange(len(place), device=DEVICE), []
    for back in range(w - 1, -1, -1):
        inside = (place >= back)[:, None]
        early = 0.0 if start is None else start[seq, (place - back + w - 1).clamp(max=w - 2)] if back else 0.0
        out.append(torch.where(inside, x[(rows - back).clamp(min=0)], early))
    return torch.stack(out)


def _conv(window, weight, bias):
    return _silu((window * weight.T[:, None]).sum(0) + bias)


def _plain_convstep(s):
    case, slots = s["case"], s["slots"].long()
    x, w = s["x"].float(), case["w"]
    seen = torch.cat([s["pool"][slots].float(), x], 1)
    window = torch.stack([seen[:, j:j + case["t"]] for j in range(w)])
    y = _silu((window * s["weight"].T[:, None, None]).sum(0) + s["bias"])
    s["pool"][slots] = seen[:, case["t"]:].to(s["pool"].dtype)
    return {"y": y.to(s["x"].dtype), "pool": s["pool"]}


def _plain_conv(s):
    case, w = s["case"], s["case"]["w"]
    x = s["x"].reshape(-1, case["d"]).float()
    start = None if s["start"] is None else s["start"].float()
    y = _conv(_window(x, start, case), s["weight"], s["bias"])
    _, _, first, lens = _row_plan(case)
    place = lens[:, None] - (w - 1) + torch.arange(w - 1, device=DEVICE)        # of the kept inputs
    early = torch.zeros((), device=DEVICE)
    if start is not None:
        early = torch.gather(start, 1, (place + w - 1).clamp(max=w - 2)[..., None].expand(-1, -1, case["d"]))
    final = torch.where((place >= 0)[..., None], x[(first[:, None] + place).clamp(0, len(x) - 1)], early)
    return {"y": y.to(s["x"].dtype).reshape(s["x"].shape), "state": final.to(s["x"].dtype)}


def _plain_convtrain(s):
    case, dtype, d = s["case"], s["x"].dtype, s["case"]["d"]
    leaves = [t.requires_grad_() for t in (s["x"].reshape(-1, d).float(), s["weight"].detach().clone(),
                                           s["bias"].detach().clone())]
    with torch.enable_grad():
        y = _conv(_window(leaves[0], None, case), leaves[1], leaves[2])
        gx, gw, gb = torch.autograd.grad(y, leaves, s["grad_y"].reshape(-1, d).float())
    shape = s["x"].shape
    return {"y": y.detach().to(dtype).reshape(shape), "grad_x": gx.to(dtype).reshape(shape), "grad_w": gw, "grad_bias": gb}


def _softplus(v):
    return torch.logaddexp(v, torch.zeros_like(v))


def _plain_step(s):
    x, delta, z, B, C = (s[n].float() for n in ("x", "delta", "z", "B", "C"))
    slots, per, out = s["slots"].long(), s["case"]["d"] // s["case"]["g"], []
    h = s["pool"][slots]
    for t in range(x.shape[1]):
        dt = _softplus(delta[:, t] + s["bias"])
        b, c = (m[:, t].repeat_interleave(per, 1) for m in (B, C))
        h = torch.exp(dt[..., None] * s["A"]) * h + (dt * x[:, t])[..., None] * b
        out.append(((h * c).sum(-1) + s["D"] * x[:, t]) * _silu(z[:, t]))
    s["pool"][slots] = h
    return {"y": torch.stack(out, 1).to(s["x"].dtype), "pool": s["pool"]}


def _scan(x, delta, A, B, C, D, z, bias, start, plan, longest):
    """The scan over [rows, channels] in 32 bits, B and C [rows, channels, N]: spans of 1, 2, 4, ... rows joined
    in pairs, (a, b) then (a', b') being (a a', a' b + b')."""
    place, seq, _, _ = plan
    dt = _softplus(delta + bias)
    a = torch.exp(dt[..., None] * A)
    b = (dt * x)[..., None] * B
    begin = (place == 0)[:, None, None]
    if start is not None:
        b = b + torch.where(begin, a * start[seq], 0.0)
    a = torch.where(begin, 0.0, a)
    span = 1
    while span < longest:
        b = torch.cat([b[:span], b[span:] + a[span:] * b[:-span]])
        a = torch.cat([a[:span], a[span:] * a[:-span]])
        span *= 2
    return ((b * C).sum(-1) + D * x) * _silu(z), b


def _blocks(case):
    """Ranges of channels that the plain form takes together, each within a group."""
    per = case["d"] // case["g"]
    most = max(1, min(per, PLAIN_VALUES // (sum(_lens(case)) * case["s"])))
    return [(g, g * per + c, min(g * per + c + most, (g + 1) * per)) for g in range(case["g"]) for c in range(0, per, most)]


def _plain_prefill(s):
    case, d = s["case"], s["case"]["d"]
    x, delta, z = (s[n].reshape(-1, d).float() for n in ("x", "delta", "z"))
    B, C = (s[n].reshape(-1, case["g"], case["s"]).float() for n in ("B", "C"))
    plan, lens = _row_plan(case), _lens(case)
    y = torch.empty(s["x"].shape, dtype=s["x"].dtype, device=DEVICE).view(-1, d)
    final = torch.zeros(len(lens), d, case["s"], device=DEVICE) if s["start"] is None else s["start"].clone()
    some = plan[3] > 0
    last = (plan[2] + plan[3] - 1)[some]
    for g, i, j in _blocks(case):
        start = None if s["start"] is None else s["start"][:, i:j]
        out, h = _scan(x[:, i:j], delta[:, i:j], s["A"][i:j], B[:, g:g + 1], C[:, g:g + 1], s["D"][i:j], z[:, i:j],
                       s["bias"][i:j], start, plan, max(lens))
        y[:, i:j] = out.to(y.dtype)
        final[some, i:j] = h[last]
    return {"y": y.view(s["x"].shape), "state": final}


def _plain_train(s):
    case, d, dtype = s["case"], s["case"]["d"], s["x"].dtype
    x, delta, z, gy = (s[n].reshape(-1, d).float() for n in ("x", "delta", "z", "grad_y"))
    B, C = (s[n].reshape(-1, case["g"], case["s"]).float() for n in ("B", "C"))
    plan, longest = _row_plan(case), max(_lens(case))
    y, gx, gdelta, gz = (torch.empty(x.shape, dtype=dtype, device=DEVICE) for _ in range(4))
    gA, gD, gbias = (torch.empty_like(s[n]) for n in ("A", "D", "bias"))
    gB, gC = torch.zeros_like(B), torch.zeros_like(C)
    for g, i, j in _blocks(case):
        parts = (x[:, i:j], delta[:, i:j], s["A"][i:j], B[:, g:g + 1], C[:, g:g + 1], s["D"][i:j], z[:, i:j], s["bias"][i:j])
        leaves = [t.detach().clone().requires_grad_() for t in parts]
        with torch.enable_grad():
            out, _ = _scan(*leaves, None, plan, longest)
            grads = torch.autograd.grad(out, leaves, gy[:, i:j])
        y[:, i:j] = out.detach().to(dtype)
        for to, n in ((gx, 0), (gdelta, 1), (gz, 6)):
            to[:, i:j] = grads[n].to(dtype)
        gA[i:j], gD[i:j], gbias[i:j] = grads[2], grads[5], grads[7]
        gB[:, g:g + 1] += grads[3]
        gC[:, g:g + 1] += grads[4]
    like = s["x"].shape
    return {"y": y.view(like), "grad_x": gx.view(like), "grad_delta": gdelta.view(like), "grad_A": gA,
            "grad_B": gB.to(dtype).view(s["B"].shape), "grad_C": gC.to(dtype).view(s["C"].shape), "grad_D": gD,
            "grad_z": gz.view(like), "grad_bias": gbias}


def _plain_norm(s):
    dtype = s["x"].dtype
    stream = (s["x"].float() + s["residual"].float()).to(dtype)
    z = stream.float()
    z = z - z.mean(-1, keepdim=True)
    n = z * (z.square().mean(-1, keepdim=True) + EPS).rsqrt()
    return {"y": (n * s["weight"] + s["bias"]).to(dtype), "s": stream}


def _plain_normtrain(s):
    dtype, weight = s["x"].dtype, s["weight"]
    stream = (s["x"].float() + s["residual"].float()).to(dtype)
    z = stream.float()
    z = z - z.mean(-1, keepdim=True)
    rstd = (z.square().mean(-1, keepdim=True) + EPS).rsqrt()
    n = z * rstd
    dy = s["grad_y"].float()
    dn = dy * weight
    dx = s["grad_s"].float() + rstd * (dn - dn.mean(-1, keepdim=True) - n * (dn * n).mean(-1, keepdim=True))
    return {"y": (n * weight + s["bias"]).to(dtype), "s": stream, "grad_x": dx.to(dtype), "grad_w": (dy * n).sum(0),
            "grad_bias": dy.sum(0)}


def _plain_clip(s):
    total = torch.stack([g.float().square().sum() for g in s["grads"]]).sum()
    norm = total.sqrt().reshape(1)
    factor = (MOST / (norm + 1e-6)).clamp(max=1.0)
    return {"norm": norm, "grads": [(g.float() * factor).to(g.dtype) for g in s["grads"]]}


_PLAIN = dict(convstep=_plain_convstep, conv=_plain_conv, convtrain=_plain_convtrain, step=_plain_step,
              prefill=_plain_prefill, train=_plain_train, norm=_plain_norm, normtrain=_plain_normtrain, clip=_plain_clip)


# ------------------------------------------------------------------ 64 bits

def exact(case, seed):
    """The definitions in 64 bits, the scan token by token."""
    state = prepare(case, seed)
    op = case["op"]
    if op == "clip":
        grads = [g.double() for g in state["grads"]]
        norm = math.sqrt(sum(float((g * g).sum()) for g in grads))
        factor = min(1.0, MOST / (norm + 1e-6))
        return {"norm": torch.tensor([norm], dtype=torch.float64, device=DEVICE), "grads": [g * factor for g in grads]}
    if "norm" in op:
        return _exact_norm(state)
    if "conv" in op:
        return _exact_conv(case, state)
    return _exact_scan(case, state)


def _exact_norm(s):
    stream = (s["x"].double() + s["residual"].double()).to(s["x"].dtype).double()
    var, mean = torch.var_mean(stream, -1, correction=0, keepdim=True)
    w, sd = s["weight"].double(), torch.sqrt(var + EPS)
    n = (stream - mean) / sd
    got = {"y": n * w + s["bias"].double(), "s": stream}
    if s["case"]["op"] == "normtrain":
        dy = s["grad_y"].double()
        g = dy * w
        inner = (g * (stream - mean)).mean(-1, keepdim=True)
        got["grad_x"] = s["grad_s"].double() + (g - g.mean(-1, keepdim=True)) / sd - (stream - mean) * inner / sd ** 3
        got["grad_w"], got["grad_bias"] = (dy * n).sum(0), dy.sum(0)
    return got


def _exact_conv(case, s):
    """Sequence by sequence."""
    d, w = case["d"], case["w"]
    weight, bias = s["weight"].double(), s["bias"].double()
    x = s["x"].double().reshape(-1, d)
    step = case["op"] == "convstep"
    lens = [case["t"]] * case["n"] if step else _lens(case)
    y, gx = torch.zeros_like(x), torch.zeros_like(x)
    gw, gb, kept, at = torch.zeros_like(weight), torch.zeros_like(bias), [], 0
    for i, n in enumerate(lens):
        early = torch.zeros(w - 1, d, dtype=torch.float64, device=DEVICE)
        if step:
            early = s["pool"][int(s["slots"][i])].double()
        elif s.get("start") is not None:
            early = s["start"][i].double()
        seen = torch.cat([early, x[at:at + n]])
        kept.append(seen[n:])
        pre = sum(weight[:, j] * seen[j:j + n] for j in range(w)) + bias
        gate = torch.sigmoid(pre)
        y[at:at + n] = pre * gate
        if case["op"] == "convtrain":
            p = s["grad_y"].double().reshape(-1, d)[at:at + n] * gate * (1 + pre * (1 - gate))
            into = torch.zeros_like(seen)
            for j in range(w):
                into[j:j + n] += weight[:, j] * p
                gw[:, j] += (p * seen[j:j + n]).sum(0)
            gb += p.sum(0)
            gx[at:at + n] = into[w - 1:]
        at += n
    y = y.reshape(s["x"].shape)
    if case["op"] == "convtrain":
        return {"y": y, "grad_x": gx.reshape(s["x"].shape), "grad_w": gw, "grad_bias": gb}
    if step:
        pool = s["pool"].double()
        pool[s["slots"].long()] = torch.stack(kept)
        return {"y": y, "pool": pool}
    return {"y": y, "state": torch.stack(kept)}


def _exact_scan(case, s):
    d, n, per = case["d"], case["s"], case["d"] // case["g"]
    train = case["op"] == "train"
    lens = [case["t"]] * case["n"] if case["op"] == "step" else _lens(case)
    if sum(lens) * d * n > (1.2e9 if train else 5e9):
        return None
    x, z, delta = (s[m].double().reshape(-1, d) for m in ("x", "z", "delta"))
    B, C = (s[m].double().reshape(-1, case["g"], n) for m in ("B", "C"))
    A, D = s["A"].double(), s["D"].double()
    pre = delta + s["bias"].double()
    dt = torch.clamp(pre, min=0) + torch.log1p(torch.exp(-pre.abs()))
    begin = torch.tensor([0] + lens).cumsum(0)[:-1].tolist()
    # sequences by falling length: those that still run at token i come first
    order = sorted(range(len(lens)), key=lambda i: -lens[i])
    place = torch.tensor([begin[i] for i in order], device=DEVICE)
    running = [sum(1 for m in lens if m > i) for i in range(max(lens))]
    h = torch.zeros(len(lens), d, n, dtype=torch.float64, device=DEVICE)
    if case["op"] == "step":
        h = s["pool"].double()[s["slots"].long()][order]
    elif s.get("start") is not None:
        h = s["start"].double()[order]
    inner, before = torch.zeros_like(x), []
    for i, m in enumerate(running):
        r = place[:m] + i
        if train:
            before.append(h[:m].clone())
        b = B[r].repeat_interleave(per, 1)
        h[:m] = torch.exp(dt[r][..., None] * A) * h[:m] + (dt[r] * x[r])[..., None] * b
        inner[r] = torch.einsum("ngcs,ngs->ngc", h[:m].unflatten(1, (-1, per)), C[r]).flatten(1)
    inner = inner + D * x
    gate = torch.sigmoid(z)
    y = (inner * z * gate).reshape(s["x"].shape)
    final = torch.empty_like(h)
    final[order] = h
    if case["op"] == "step":
        pool = s["pool"].double()
        pool[s["slots"].long()] = final
        return {"y": y, "pool": pool}
    if not train:
        return {"y": y, "state": final}
    gy = s["grad_y"].double().reshape(-1, d)
    gz = gy * inner * gate * (1 + z * (1 - gate))
    g = gy * z * gate
    gx, gdt = D * g, torch.zeros_like(dt)
    gA, gB, gC = torch.zeros_like(A), torch.zeros_like(B), torch.zeros_like(C)
    dh = torch.zeros_like(h)
    for i in reversed(range(len(running))):
        m = running[i]
        r = place[:m] + i
        b, c = (t[r].repeat_interleave(per, 1) for t in (B, C))
        a = torch.exp(dt[r][..., None] * A)
        after = a * before[i] + (dt[r] * x[r])[..., None] * b
        gC[r] = (g[r][..., None] * after).unflatten(1, (-1, per)).sum(2)
        dh[:m] += g[r][..., None] * c
        da = dh[:m] * a * before[i]
        gA += (da * dt[r][..., None]).sum(0)
        inflow = (dh[:m] * b).sum(-1)
        gdt[r] = (da * A).sum(-1) + inflow * x[r]
        gx[r] += inflow * dt[r]
        gB[r] = (dh[:m] * (dt[r] * x[r])[..., None]).unflatten(1, (-1, per)).sum(2)
        dh[:m] *= a
        before[i] = None
    gdelta = gdt * torch.sigmoid(pre)
    like = s["x"].shape
    return {"y": y, "grad_x": gx.reshape(like), "grad_delta": gdelta.reshape(like), "grad_A": gA,
            "grad_B": gB.reshape(s["B"].shape), "grad_C": gC.reshape(s["C"].shape), "grad_D": (g * x).sum(0),
            "grad_z": gz.reshape(like), "grad_bias": gdelta.sum(0)}
