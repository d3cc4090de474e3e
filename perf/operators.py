"""Cases of the gated delta rule and of the residual RMS norm: what is timed, in plain form and through the library.

The gated delta rule keeps, for every sequence and value head, a matrix state S [d_k, d_v] and per token does

    S <- exp(g) S,   u = beta (v - S^T k),   S <- S + k u^T,   o = scale S^T q

(q and k of a value head come from the query/key head that its group shares).  The residual norm does

    s = x + residual (rounded to the stored type),   y = s / sqrt(mean(s^2) + eps) * w

and writes y in the stored type or in 8 bits with one scale a group of columns.

Ops:  step      new tokens of decoding sequences against a pool of states, updated in place
      prefill   whole prompts: outputs and the state after each sequence
      train     forward and backward over whole sequences
      norm      residual norm, forward        norm8   the same with an output in 8 bits
      normtrain residual norm, forward and backward
"""
import math

import torch

own = False
DEVICE = "cuda"
EPS = 1e-6
CHUNK = 64      # tokens that the plain form of the rule takes together


def listed():
    return [
        # one user's next token, 16 heads of the usual size: latency
        dict(name="step_1x16_bf16", op="step", n=1, t=1, hk=16, hv=16, dk=128, dv=128, pool=4, math="bf16"),
        # a server's batch, grouped heads, one token each: the states' bandwidth
        dict(name="step_192x32_bf16", op="step", n=192, t=1, hk=16, hv=32, dk=128, dv=128, pool=200, math="bf16"),
        # four drafted tokens a sequence in fp32, odd count, heads of 64 x 96
        dict(name="step_37x6_t4_fp32", op="step", n=37, t=4, hk=6, hv=6, dk=64, dv=96, pool=40, math="fp32"),
        # one long document: few heads, the serial axis is the bound
        dict(name="prefill_1x16384_bf16", op="prefill", lens="16384", hk=16, hv=16, dk=128, dv=128, start=0, math="bf16"),
        # a serving batch of prompts of all lengths, an empty and a one-token one among them, states carried in
        dict(name="prefill_ragged_bf16", op="prefill", lens="0,1,64,63,65,511,1025,2048,4100,333,1,2999,700,128,1777,96",
             hk=8, hv=16, dk=128, dv=128, start=1, math="bf16"),
        # pre-training batch: 128 heads in all
        dict(name="train_8x2048_bf16", op="train", lens="8x2048", hk=16, hv=16, dk=128, dv=128, start=0, math="bf16"),
        # the trunk width and window of this repository's smoke workload, two heads of 64, fp32
        dict(name="train_32x64_fp32", op="train", lens="32x64", hk=2, hv=2, dk=64, dv=64, start=0, math="fp32"),
        # packed documents of odd lengths, three value heads to a key head
        dict(name="train_ragged_bf16", op="train", lens="1000,1,777,64,130,2049,0,511", hk=2, hv=6, dk=64, dv=96, start=0, math="bf16"),
        # the norm of one decoding batch: latency
        dict(name="norm_33x2048_bf16", op="norm", rows=33, d=2048, math="bf16"),
        # the trunk rows of the mid workload (1024 x 64 positions of 128), fp32, both directions
        dict(name="normtrain_65536x128_fp32", op="normtrain", rows=65536, d=128, math="fp32"),
        # a long prompt's rows in front of an 8-bit product, one scale a row
        dict(name="norm8_16384x4096_bf16", op="norm8", rows=16384, d=4096, group=4096, math="bf16"),
        # a training batch's rows, odd count, both directions
        dict(name="normtrain_16383x2560_bf16", op="normtrain", rows=16383, d=2560, math="bf16"),
    ]


def draw(rng):
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    most = max(_cost(c) for c in listed())
    while True:
        op = rng.choice(("step", "prefill", "train", "norm", "norm8", "normtrain"))
        bits = rng.choice(("bf16", "bf16", "fp32"))
        if op in ("step", "prefill", "train"):
            hk = rng.choice((1, 2, 3, 4, 8, 16))
            c = dict(op=op, hk=hk, hv=hk * rng.choice((1, 1, 2, 3)), dk=rng.choice((32, 64, 80, 128, 128)),
                     dv=rng.choice((32, 64, 96, 128, 128)), math=bits)
            if op == "step":
                n = log(1, 256)
                c.update(n=n, t=rng.choice((1, 1, 2, 5)), pool=n + rng.randrange(1, 9))
            else:
                if rng.random() < 0.5:
                    lens = "%dx%d" % (log(1, 64), log(1, 8192))
                else:
                    lens = ",".join(str(rng.choice((0, 1, log(2, 4096), log(2, 4096)))) for _ in range(rng.randrange(2, 17)))
                c.update(lens=lens, start=rng.randrange(2) if op == "prefill" else 0)
                total = sum(_lens(c))
                if not 1 <= total <= 32768 or max(_lens(c)) > 16384:
                    continue
        else:
            d = 16 * log(4, 512) if op == "norm8" or rng.random() < 0.7 else log(64, 8192)
            c = dict(op=op, rows=log(1, 65536), d=d, math=bits)
            if op == "norm8":
                c["group"] = rng.choice([d] + [n for n in (64, 128) if d % n == 0])
        if _cost(c) <= most:
            return c


def _lens(case):
    """Sequence lengths: "8x2048" is eight of 2048, "1,64,0" a packed batch."""
    text = case["lens"]
    if "x" in text:
        n, t = text.split("x")
        return [int(t)] * int(n)
    return [int(t) for t in text.split(",")]


def _type(case):
    return torch.bfloat16 if case["math"] == "bf16" else torch.float32


def _cost(case):
    w = work(case)
    return max(w["bytes"], w["flops"] / 50)


def work(case):
    size = 2 if case["math"] == "bf16" else 4
    if case["op"] in ("step", "prefill", "train"):
        hk, hv, dk, dv = (case[n] for n in ("hk", "hv", "dk", "dv"))
        if case["op"] == "step":
            tokens, states = case["n"] * case["t"], 2 * case["n"]
        else:
            tokens = sum(_lens(case))
            states = len(_lens(case)) * (1 + case["start"]) if case["op"] == "prefill" else 0
        inputs = tokens * ((2 * hk * dk + hv * dv) * size + 2 * hv * 4)
        outputs = tokens * hv * dv * size
        flops = 7.0 * tokens * hv * dk * dv          # decay, S^T k, k u^T, S^T q
        if case["op"] == "train":                    # inputs and grad_o again, the five gradients
            inputs += inputs + outputs
            outputs += tokens * (2 * hk * dk + hv * dv + 2 * hv) * size
            flops += 15.0 * tokens * hv * dk * dv    # seven outer or matrix-vector products and the decay
        return {"bytes": inputs + outputs + states * hv * dk * dv * 4.0, "flops": flops}
    rows, d = case["rows"], case["d"]
    n = rows * d
    if case["op"] == "norm":
        return {"bytes": 4.0 * n * size + 4 * d, "flops": 5.0 * n}
    if case["op"] == "norm8":
        return {"bytes": 3.0 * n * size + n + 4 * d + 4.0 * n / case["group"], "flops": 7.0 * n}
    return {"bytes": 4.0 * n * size + 4 * d + 4.0 * n * size + 8 * d, "flops": 15.0 * n}


def prepare(case, seed):
    gen = torch.Generator(device=DEVICE).manual_seed(seed)
    dtype = _type(case)

    def normal(*shape):
        return torch.randn(*shape, device=DEVICE, generator=gen)

    def uniform(*shape):
        return torch.rand(*shape, device=DEVICE, generator=gen)

    state = dict(case=dict(case))
    if case["op"] in ("step", "prefill", "train"):
        hk, hv, dk, dv = (case[n] for n in ("hk", "hv", "dk", "dv"))
        if case["op"] == "step":
            lead = (case["n"], case["t"])
        else:
            lens = _lens(case)
            lead = (len(lens), lens[0]) if "x" in case["lens"] else (sum(lens),)
        # projections of one stream of rows: queries and keys of unit length, keys with a shared direction
        q = normal(*lead, hk, dk)
        k = normal(*lead, hk, dk) + 0.5 * normal(hk, dk)
        state["q"] = (q / q.norm(dim=-1, keepdim=True)).to(dtype)
        state["k"] = (k / k.norm(dim=-1, keepdim=True)).to(dtype)
        state["v"] = normal(*lead, hv, dv).to(dtype)
        # log-decays -a softplus(x + b): a in [1, 16], softplus(b) log-uniform in [0.001, 0.1] a head
        step = torch.exp(uniform(hv) * math.log(100.0) + math.log(0.001))
        bias = step + torch.log(-torch.expm1(-step))
        state["g"] = -(1 + 15 * uniform(hv)) * torch.nn.functional.softplus(0.5 * normal(*lead, hv) + bias)
        state["beta"] = torch.sigmoid(normal(*lead, hv))
        state["scale"] = dk ** -0.5
        state["offsets"] = None
        if len(lead) == 1:
            ends = torch.tensor([0] + lens, device=DEVICE).cumsum(0)
            state["offsets"] = ends.to(torch.int32)
        if case["op"] == "step":
            state["pool"] = 0.3 * normal(case["pool"], hv, dk, dv)
            order = torch.randperm(case["pool"], device=DEVICE, generator=gen)
            state["slots"] = order[: case["n"]].to(torch.int32)
        if case["op"] == "prefill":
            state["start"] = 0.3 * normal(len(lens), hv, dk, dv) if case["start"] else None
        if case["op"] == "train":
            state["grad_o"] = normal(*lead, hv, dv).to(dtype)
    else:
        rows, d = case["rows"], case["d"]
        state["x"] = normal(rows, d).to(dtype)
        state["residual"] = (2 * normal(rows, d)).to(dtype)
        state["weight"] = 1 + 0.2 * normal(d)
        if case["op"] == "normtrain":
            state["grad_y"] = normal(rows, d).to(dtype)
            state["grad_s"] = normal(rows, d).to(dtype)
    return state


def run(state):
    op = state["case"]["op"]
    if own:
        return _OWN[op](state)
    return _PLAIN[op](state)


# ------------------------------------------------------------------ the library's calls

def _math(cfc, case):
    return cfc.MATH_BF16 if case["math"] == "bf16" else cfc.MATH_FP32


def _workspace(cfc, case):
    n, total = len(_lens(case)), sum(_lens(case))
    size = cfc.cfc_gdr_workspace_bytes(total, n, case["hk"], case["hv"], case["dk"], case["dv"], _math(cfc, case),
                                       save=case["op"] == "train")
    return torch.empty(size, dtype=torch.uint8, device=DEVICE)


def _own_step(s):
    import recurrent_cell_gb300 as cfc

    o = torch.empty_like(s["v"])
    cfc.cfc_gdr_step(s["q"], s["k"], s["v"], s["g"], s["beta"], s["pool"], o, slots=s["slots"], scale=s["scale"],
                     math=_math(cfc, s["case"]))
    return {"o": o, "pool": s["pool"]}


def _own_prefill(s):
    import recurrent_cell_gb300 as cfc

    case = s["case"]
    o, workspace = torch.empty_like(s["v"]), _workspace(cfc, case)
    final = torch.empty(len(_lens(case)), case["hv"], case["dk"], case["dv"], device=DEVICE)
    cfc.cfc_gdr_forward(s["q"], s["k"], s["v"], s["g"], s["beta"], o, workspace, seq_offsets=s["offsets"],
                        initial_state=s["start"], final_state=final, scale=s["scale"], math=_math(cfc, case))
    return {"o": o, "state": final}


def _own_train(s):
    import recurrent_cell_gb300 as cfc

    q, k, v, g, beta = (s[n] for n in ("q", "k", "v", "g", "beta"))
    o, workspace, mode = torch.empty_like(v), _workspace(cfc, s["case"]), _math(cfc, s["case"])
    cfc.cfc_gdr_forward(q, k, v, g, beta, o, workspace, seq_offsets=s["offsets"], save=True, scale=s["scale"],
                        math=mode)
    grads = [torch.empty_like(q), torch.empty_like(k), torch.empty_like(v),
             torch.empty_like(g, dtype=q.dtype), torch.empty_like(beta, dtype=q.dtype)]
    cfc.cfc_gdr_backward(q, k, v, g, beta, s["grad_o"], *grads, workspace, seq_offsets=s["offsets"],
                         scale=s["scale"], math=mode)
    return dict(zip(("o", "grad_q", "grad_k", "grad_v", "grad_g", "grad_beta"), [o] + grads))


def _own_norm(s):
    import recurrent_cell_gb300 as cfc

    y, stream = torch.empty_like(s["x"]), torch.empty_like(s["x"])
    cfc.cfc_rmsnorm_forward(s["x"], s["weight"], y=y, residual=s["residual"], residual_out=stream, eps=EPS,
                            math=_math(cfc, s["case"]))
    return {"y": y, "s": stream}


def _own_norm8(s):
    import recurrent_cell_gb300 as cfc

    rows, d, group = (s["case"][n] for n in ("rows", "d", "group"))
    stream = torch.empty_like(s["x"])
    y8 = torch.empty(rows, d, dtype=torch.float8_e4m3fn, device=DEVICE)
    scales = torch.empty(rows, d // group, device=DEVICE)
    cfc.cfc_rmsnorm_forward(s["x"], s["weight"], residual=s["residual"], residual_out=stream, y8=y8, y8_scale=scales,
                            eps=EPS, math=_math(cfc, s["case"]))
    return {"y8": y8, "scale": scales, "s": stream}


def _own_normtrain(s):
    import recurrent_cell_gb300 as cfc

    x, weight, mode = s["x"], s["weight"], _math(cfc, s["case"])
    y, stream, grad_x = torch.empty_like(x), torch.empty_like(x), torch.empty_like(x)
    rstd, grad_w = torch.empty(x.shape[0], device=DEVICE), torch.empty_like(weight)
    cfc.cfc_rmsnorm_forward(x, weight, y=y, residual=s["residual"], residual_out=stream, rstd=rstd, eps=EPS,
                            math=mode)
    size = cfc.cfc_rmsnorm_workspace_bytes(*x.shape)
    workspace = torch.empty(size, dtype=torch.uint8, device=DEVICE)
    cfc.cfc_rmsnorm_backward(stream, weight, rstd, s["grad_y"], grad_x, grad_w, workspace,
                             grad_residual_out=s["grad_s"], math=mode)
    return {"y": y, "s": stream, "grad_x": grad_x, "grad_w": grad_w}


_OWN = dict(step=_own_step, prefill=_own_prefill, train=_own_train, norm=_own_norm, norm8=_own_norm8,
            normtrain=_own_normtrain)


# ------------------------------------------------------------------ the plain forms

def _padded(x, offsets):
    """[rows, ...] packed -> [sequences, longest, ...], zero past each end; uniform batches as they are."""
    if offsets is None:
        return x.float()
    starts, lens = offsets[:-1].long(), (offsets[1:] - offsets[:-1]).long()
    at = torch.arange(int(lens.max()), device=x.device)
    inside = at[None] < lens[:, None]
    rows = torch.where(inside, starts[:, None] + at[None], 0)
    return x.float()[rows] * inside.reshape(inside.shape + (1,) * (x.dim() - 1))


def _packed(x, offsets):
    if offsets is None:
        return x
    lens = offsets[1:] - offsets[:-1]
    return x[torch.arange(x.shape[1], device=x.device)[None] < lens[:, None]]


def _rule(q, k, v, g, beta, scale, start):
    """The rule over [sequences, tokens, heads, d] in 32 bits, CHUNK tokens at a time: inside a chunk the corrections
    u solve (I + A) u = beta (v - exp(G) S^T k) with A_ij = beta_i exp(G_i - G_j) k_i.k_j, j < i."""
    n, t, hv, dv = v.shape
    dk, more = k.shape[-1], -t % CHUNK
    q, k = (x.repeat_interleave(hv // x.shape[2], dim=2) for x in (q, k))

    def chunks(x):
        x = torch.nn.functional.pad(x, (0, 0) * (x.dim() - 2) + (0, more))
        x = x.reshape(n, (t + more) // CHUNK, CHUNK, *x.shape[2:])
        return x.movedim(3, 1)                          # [sequences, heads, chunks, CHUNK, ...]

    q, k, v, g, beta = (chunks(x) for x in (q, k, v, g, beta))
    total = g.cumsum(-1)
    low = torch.ones(CHUNK, CHUNK, dtype=torch.bool, device=v.device).tril()
    decay = torch.where(low, total[..., :, None] - total[..., None, :], 0.0).exp() * low
    a = beta[..., None] * (k @ k.mT) * decay * low.tril(-1)
    # the inverse of I + A, blocks of 1, 2, 4, ... joined in pairs
    inverse = torch.eye(CHUNK, device=v.device).expand_as(a)
    at = torch.arange(CHUNK, device=v.device)
    for size in (1, 2, 4, 8, 16, 32):
        block = at // size
        join = (block[:, None] % 2 == 1) & (block[None] == block[:, None] - 1)
        inverse = inverse - inverse @ (a * join) @ inverse
    w = inverse @ (beta[..., None] * total[..., None].exp() * k)
    u0 = inverse @ (beta[..., None] * v)
    p = (q @ k.mT) * decay
    q_in = q * total[..., None].exp()
    k_out = k * (total[..., -1:] - total)[..., None].exp()
    keep = total[..., -1].exp()
    s = torch.zeros(n, hv, dk, dv, device=v.device) if start is None else start.float()
    out = []
    for c in range(v.shape[2]):
        u = u0[:, :, c] - w[:, :, c] @ s
        out.append(q_in[:, :, c] @ s + p[:, :, c] @ u)
        s = keep[:, :, c, None, None] * s + k_out[:, :, c].mT @ u
    o = scale * torch.cat(out, 2).movedim(1, 2)[:, :t] if out else v.new_zeros(n, 0, hv, dv)
    return o, s


def _plain_step(s):
    q, k, v, g, beta = (s[n].float() for n in ("q", "k", "v", "g", "beta"))
    hv = v.shape[2]
    q, k = (x.repeat_interleave(hv // x.shape[2], dim=2) for x in (q, k))
    slots, out = s["slots"].long(), []
    state = s["pool"][slots]
    for i in range(v.shape[1]):
        state = state * g[:, i].exp()[..., None, None]
        u = beta[:, i, :, None] * (v[:, i] - (state * k[:, i, :, :, None]).sum(-2))
        state = state + k[:, i, :, :, None] * u[..., None, :]
        out.append(s["scale"] * (state * q[:, i, :, :, None]).sum(-2))
    s["pool"][slots] = state
    return {"o": torch.stack(out, 1).to(s["v"].dtype), "pool": s["pool"]}


def _plain_prefill(s):
    off = s["offsets"]
    o, final = _rule(*(_padded(s[n], off) for n in ("q", "k", "v", "g", "beta")), s["scale"], s["start"])
    return {"o": _packed(o, off).to(s["v"].dtype), "state": final}


def _plain_train(s):
    off, names = s["offsets"], ("q", "k", "v", "g", "beta")
    leaves = [_padded(s[n], off).requires_grad_() for n in names]
    with torch.enable_grad():
        o, _ = _rule(*leaves, s["scale"], None)
        grads = torch.autograd.grad(o, leaves, _padded(s["grad_o"], off))
    dtype = s["v"].dtype
    got = {"o": _packed(o.detach(), off).to(dtype)}
    got.update(("grad_" + n, _packed(x, off).to(dtype)) for n, x in zip(names, grads))
    return got


def _plain_norm(s):
    stream = (s["x"].float() + s["residual"].float()).to(s["x"].dtype)
    y = stream.float()
    y = y * (y.square().mean(-1, keepdim=True) + EPS).rsqrt() * s["weight"]
    return {"y": y.to(s["x"].dtype), "s": stream}


def _plain_norm8(s):
    stream = (s["x"].float() + s["residual"].float()).to(s["x"].dtype)
    y = stream.float()
    y = y * (y.square().mean(-1, keepdim=True) + EPS).rsqrt() * s["weight"]
    y = y.reshape(y.shape[0], -1, s["case"]["group"])
    most = y.abs().amax(-1, keepdim=True)
    scale = torch.where(most > 0, most / 448.0, 1.0)
    y8 = (y / scale).clamp(-448.0, 448.0).to(torch.float8_e4m3fn)
    return {"y8": y8.reshape(stream.shape), "scale": scale[..., 0], "s": stream}


def _plain_normtrain(s):
    dtype, weight = s["x"].dtype, s["weight"]
    stream = (s["x"].float() + s["residual"].float()).to(dtype)
    z = stream.float()
    rstd = (z.square().mean(-1, keepdim=True) + EPS).rsqrt()
    n = z * rstd
    dy = s["grad_y"].float()
    dn = dy * weight
    dx = s["grad_s"].float() + rstd * (dn - n * (dn * n).mean(-1, keepdim=True))
    return {"y": (n * weight).to(dtype), "s": stream, "grad_x": dx.to(dtype), "grad_w": (dy * n).sum(0)}


_PLAIN = dict(step=_plain_step, prefill=_plain_prefill, train=_plain_train, norm=_plain_norm, norm8=_plain_norm8,
              normtrain=_plain_normtrain)


# ------------------------------------------------------------------ 64 bits

def exact(case, seed):
    """The definitions token by token, in 64 bits."""
    kept, state = {}, prepare(case, seed)
    if case["op"] in ("norm", "norm8", "normtrain"):
        return _exact_norm(case, state)
    q, k, v, g, beta = (state[n].double() for n in ("q", "k", "v", "g", "beta"))
    hv = v.shape[-2]
    q, k = (x.repeat_interleave(hv // x.shape[-2], dim=-2) for x in (q, k))
    scale = state["scale"]
    if case["op"] == "step":
        lens, first = [case["t"]] * case["n"], state["pool"].double()[state["slots"].long()]
    else:
        lens = _lens(case)
        first = torch.zeros(len(lens), hv, case["dk"], case["dv"], dtype=torch.float64, device=DEVICE)
        if state.get("start") is not None:
            first = state["start"].double()
    if sum(lens) * hv * case["dk"] * case["dv"] * (8 if case["op"] == "train" else 1) > 2e11 or max(lens) > 16384:
        return None
    q, k, v = (x.reshape(-1, *x.shape[-2:]) for x in (q, k, v))
    g, beta = (x.reshape(-1, hv) for x in (g, beta))
    begin = torch.tensor([0] + lens).cumsum(0)[:-1].tolist()
    # sequences by falling length: those that still run at token i come first
    order = sorted(range(len(lens)), key=lambda i: -lens[i])
    s = first[order].clone()
    o = torch.zeros_like(v)
    running = [sum(1 for n in lens if n > i) for i in range(max(lens))]
    place = torch.tensor([begin[i] for i in order], device=DEVICE)

    def one(s, i, m):
        """Token i of the first m sequences: the decayed state, the correction, its error."""
        r = place[:m] + i
        sd = s * g[r].exp()[..., None, None]
        e = v[r] - torch.einsum("nhkv,nhk->nhv", sd, k[r])
        u = beta[r][..., None] * e
        return r, sd, e, u

    for i, m in enumerate(running):
        if case["op"] == "train" and i % 64 == 0:
            kept[i] = s[:m].clone()
        r, sd, e, u = one(s[:m], i, m)
        s[:m] = sd + k[r][..., None] * u[..., None, :]
        o[r] = scale * torch.einsum("nhkv,nhk->nhv", s[:m], q[r])
    final = torch.empty_like(s)
    final[order] = s
    if case["op"] == "step":
        pool = state["pool"].double()
        pool[state["slots"].long()] = final
        return {"o": o.reshape(state["v"].shape), "pool": pool}
    if case["op"] == "prefill":
        return {"o": o.reshape(state["v"].shape), "state": final}
    do = state["grad_o"].double().reshape(o.shape)
    dq, dk, dv, dg, db = (torch.zeros_like(x) for x in (q, k, v, g, beta))
    ds = torch.zeros_like(s)
    for block in sorted(kept, reverse=True):
        inside, before = kept[block], []
        for i in range(block, min(block + 64, len(running))):
            before.append(inside[: running[i]])
            r, sd, e, u = one(before[-1], i, running[i])
            inside = sd + k[r][..., None] * u[..., None, :]
        for i in reversed(range(block, min(block + 64, len(running)))):
            m = running[i]
            r, sd, e, u = one(before[i - block], i, m)
            after = sd + k[r][..., None] * u[..., None, :]
            d = ds[:m] + scale * q[r][..., None] * do[r][..., None, :]
            dq[r] = scale * torch.einsum("nhkv,nhv->nhk", after, do[r])
            du = torch.einsum("nhkv,nhk->nhv", d, k[r])
            de = beta[r][..., None] * du
            db[r] = (du * e).sum(-1)
            dv[r] = de
            dsd = d - k[r][..., None] * de[..., None, :]
            dk[r] = torch.einsum("nhkv,nhv->nhk", d, u) - torch.einsum("nhkv,nhv->nhk", sd, de)
            dg[r] = (dsd * sd).sum((-1, -2))
            ds[:m] = dsd * g[r].exp()[..., None, None]
    hk = case["hk"]
    dq, dk = (x.reshape(x.shape[0], hk, hv // hk, -1).sum(2) for x in (dq, dk))
    shapes = [state[n].shape for n in ("v", "q", "k", "v", "g", "beta")]
    return dict(zip(("o", "grad_q", "grad_k", "grad_v", "grad_g", "grad_beta"),
                    (x.reshape(n) for x, n in zip((o, dq, dk, dv, dg, db), shapes))))


def _exact_norm(case, state):
    dtype = state["x"].dtype
    stream = state["x"].double() + state["residual"].double()
    s = stream.to(dtype).double()
    weight = state["weight"].double()
    rms = torch.sqrt((s * s).sum(-1, keepdim=True) / case["d"] + EPS)
    y = s / rms * weight
    if case["op"] == "norm":
        return {"y": y, "s": s}
    if case["op"] == "norm8":
        parts = y.reshape(case["rows"], -1, case["group"])
        scale = parts.abs().amax(-1, keepdim=True) / 448.0
        return {"y8": (parts / scale).reshape(y.shape), "scale": scale[..., 0], "s": s}
    dy = state["grad_y"].double()
    inner = (dy * weight * s).sum(-1, keepdim=True) / case["d"]
    dx = state["grad_s"].double() + dy * weight / rms - s * inner / rms ** 3
    return {"y": y, "s": s, "grad_x": dx, "grad_w": (dy * s / rms).sum(0)}
