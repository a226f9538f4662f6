"""Operator cases of the gated delta rule and of layer norm: their inputs, plain forms and 64-bit values.

The gated delta rule of one head (state S [d_v, d_k]; queries and keys brought to unit length):

    g_t = -exp(a_log) softplus(a_raw_t + dt_bias)      beta_t = sigmoid(b_raw_t)
    u_t = beta_t (v_t - exp(g_t) S_{t-1} k_t)          S_t = exp(g_t) S_{t-1} + u_t k_t^T
    y_t = scale S_t q_t

``prefill`` takes a state in and gives y and the state behind the last token, ``train`` is a forward and a
backward pass, ``step`` one token for each sequence of a batch, its state updated in place.  Value head h reads
query and key head h / (heads / groups).

Layer norm of a row x: y = (x - mean) / sqrt(var + eps) w + b (``norm``); ``norm_grad`` is its backward pass, with
the residual path's gradient added to the row's and the sums over rows for w and b.

``own`` chooses between the plain forms (elementary torch operations in 32 bits) and this package's kernels.
"""
import math

import torch

own = False

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
EPS_UNIT = 1e-6    # added to the sum of squares of a query or key before its root
EPS_NORM = 1e-5
CHUNK = 64


def listed():
    def gd(name, op, act, batch, seqlen, heads, groups, d_k, d_v):
        return dict(name=name, op=op, act=act, batch=batch, seqlen=seqlen, heads=heads, groups=groups, d_k=d_k, d_v=d_v)

    def ln(name, op, x, y, rows, dim):
        return dict(name=name, op=op, x=x, y=y, rows=rows, dim=dim)

    return [
        # one user's next token: a call that is all latency
        gd("step_one", "step", "bf16", 1, 1, 16, 16, 128, 128),
        # a serving batch's next token: the states of all sequences read and written once
        gd("step_batch", "step", "bf16", 256, 1, 32, 16, 128, 128),
        # a short prompt at the Mamba-3 core's head layout (24 heads of 64 over one shared group of 128)
        gd("prefill_short", "prefill", "f16", 1, 577, 24, 1, 128, 64),
        # a long prompt of one sequence: few heads, many steps
        gd("prefill_long", "prefill", "bf16", 1, 16384, 32, 16, 128, 128),
        # a small model in full precision, as one checks a training run with, at an odd length
        gd("train_f32", "train", "f32", 2, 150, 8, 4, 64, 64),
        # the 130M width (24 heads of 64) at its training length
        gd("train_130m", "train", "bf16", 4, 2048, 24, 24, 64, 64),
        # the 2.8B width (5120 = 40 heads of 128) at the long training length
        gd("train_2p8b", "train", "bf16", 2, 8192, 40, 40, 128, 128),
        # the norm before one token's block
        ln("norm_token", "norm", "f32", "bf16", 1, 2560),
        # the norm before a block in training: residual stream in f32, what the block reads in bf16
        ln("norm_train", "norm", "f32", "bf16", 16384, 5120),
        # an odd width and an odd number of rows
        ln("norm_grad_odd", "norm_grad", "bf16", "bf16", 1001, 1537),
        # the backward pass of norm_train
        ln("norm_grad_train", "norm_grad", "f32", "bf16", 16384, 5120),
        # every head's output normed by itself: many short rows
        ln("norm_grad_heads", "norm_grad", "f16", "f16", 196608, 64),
    ]


def _spread(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["step", "prefill", "train", "norm", "norm_grad"])
    if op in ("norm", "norm_grad"):
        dim = _spread(rng, 2, 16384)
        return dict(op=op, x=rng.choice(["f32", "bf16", "f16"]), y=rng.choice(["f32", "bf16", "f16"]),
                    rows=_spread(rng, 1, min(400000, 80000000 // dim)), dim=dim)
    groups = rng.choice([1, 2, 3, 4, 8, 16])
    heads = groups * rng.choice([1, 1, 2, 3])
    d_k, d_v = 8 * rng.randint(2, 16), 8 * rng.randint(2, 32)
    act = rng.choice(["f32", "bf16", "bf16", "f16"])
    if op == "step":
        batch, seqlen = _spread(rng, 1, min(512, 100000000 // (heads * d_k * d_v))), 1
    else:
        seqlen = _spread(rng, 1, 12000)
        batch = _spread(rng, 1, max(1, min(16, 16384 // seqlen, 400000000 // (seqlen * heads * (d_k + d_v)))))
    return dict(op=op, act=act, batch=batch, seqlen=seqlen, heads=heads, groups=groups, d_k=d_k, d_v=d_v)


def prepare(case, seed):
    c, dev = case, "cuda"
    gen = torch.Generator(device=dev)
    gen.manual_seed(int(seed))

    def normal(*shape, to=torch.float32):
        return torch.randn(*shape, generator=gen, device=dev).to(to)

    def uniform(low, high, *shape):
        return low + (high - low) * torch.rand(*shape, generator=gen, device=dev)

    s = dict(case=dict(c))
    if c["op"] in ("norm", "norm_grad"):
        xt, yt, n, d = TYPES[c["x"]], TYPES[c["y"]], c["rows"], c["dim"]
        # a residual stream: rows of unequal size, away from zero
        s["x"] = (normal(n, d) * uniform(0.5, 4.0, n, 1) + normal(n, 1)).to(xt)
        s["w"], s["b"] = 1.0 + 0.1 * normal(d), 0.1 * normal(d)
        if c["op"] == "norm_grad":
            s["dy"], s["d_add"] = normal(n, d, to=yt), normal(n, d, to=xt)
            x = s["x"].double()    # what the forward pass keeps
            s["mean"] = x.mean(1).float()
            s["rstd"] = (x.var(1, unbiased=False) + EPS_NORM).rsqrt().float()
        if own:
            import state_space_sequence_selective_amd as mscan
            s["norm"] = mscan.LayerNorm(mscan.NormDims.make(n, d, x=c["x"], y=c["y"], eps=EPS_NORM), device=dev)
        return s
    at, B, T, H, G, K, V = TYPES[c["act"]], c["batch"], c["seqlen"], c["heads"], c["groups"], c["d_k"], c["d_v"]
    s["q"], s["k"], s["v"] = normal(B, T, G, K, to=at), normal(B, T, G, K, to=at), normal(B, T, H, V, to=at)
    s["a_raw"], s["b_raw"] = normal(B, T, H), normal(B, T, H)
    # decay rates of 1 to 16 and steps of 0.001 to 0.1, as a model starts with
    s["a_log"] = uniform(1.0, 16.0, H).log()
    dt = uniform(math.log(1e-3), math.log(1e-1), H).exp()
    s["dt_bias"] = dt + torch.log(-torch.expm1(-dt))
    if c["op"] == "train":
        s["dy"] = normal(B, T, H, V, to=at)
    else:
        s["state"] = 0.3 * normal(B, H, V, K)
    if own:
        import state_space_sequence_selective_amd as mscan
        dims = mscan.GDeltaDims.make(batch=B, seqlen=T, heads=H, groups=G, d_k=K, d_v=V, act=c["act"])
        s["core"] = mscan.GatedDeltaCore(dims, device=dev, train=c["op"] == "train")
    return s


def run(s):
    if own:
        return _run_own(s)
    op = s["case"]["op"]
    if op == "norm":
        return dict(zip(("y", "mean", "rstd"), _norm(s["x"], s["w"], s["b"], TYPES[s["case"]["y"]])))
    if op == "norm_grad":
        return _norm_grad(s)
    if op == "step":
        return _step(s)
    if op == "prefill":
        y, state = _chunked(*(s[n] for n in GD_INPUTS), s["state"])
        return dict(y=y.to(s["v"].dtype), state=state)
    return _train(s)


def _run_own(s):
    op = s["case"]["op"]
    if op == "norm":
        n = s["norm"]
        y = n.forward(s["x"], s["w"], s["b"])
        return dict(y=y, mean=n.mean, rstd=n.rstd)
    if op == "norm_grad":
        n = s["norm"]
        n.zero_grads()
        dx = n.backward(s["x"], s["w"], s["dy"], d_add=s["d_add"], mean=s["mean"], rstd=s["rstd"])
        return dict(dx=dx, dw=n.dw, db=n.db)
    core = s["core"]
    if op == "step":
        y = core.step(s, s["state"])
        return dict(y=y, state=s["state"])
    if op == "prefill":
        y = core.forward(s, h0=s["state"])
        return dict(y=y, state=core.h_last)
    core.zero_grads()
    y = core.forward(s)
    g = core.backward(s, s["dy"])
    return dict(g, y=y)


# ---------------------------------------------------------------- plain forms

GD_INPUTS = ("q", "k", "v", "a_raw", "b_raw", "a_log", "dt_bias")


def _norm(x, w, b, to):
    x = x.float()
    mean = x.mean(1, keepdim=True)
    c = x - mean
    rstd = torch.rsqrt((c * c).mean(1, keepdim=True) + EPS_NORM)
    return (c * rstd * w + b).to(to), mean[:, 0], rstd[:, 0]


def _norm_grad(s):
    dy, rstd = s["dy"].float(), s["rstd"][:, None]
    n = (s["x"].float() - s["mean"][:, None]) * rstd
    dn = dy * s["w"]
    dx = rstd * (dn - dn.mean(1, keepdim=True) - n * (dn * n).mean(1, keepdim=True)) + s["d_add"].float()
    return dict(dx=dx.to(s["x"].dtype), dw=(dy * n).sum(0), db=dy.sum(0))


def _softplus(x):
    return x.clamp_min(0.0) + torch.log1p(torch.exp(-x.abs()))


def _unit(x):
    return x * torch.rsqrt((x * x).sum(-1, keepdim=True) + EPS_UNIT)


def _step(s):
    q, k, v = (s[n][:, 0].float() for n in ("q", "k", "v"))
    state, share = s["state"], v.shape[1] // k.shape[1]
    q = _unit(q).repeat_interleave(share, 1) / math.sqrt(q.shape[-1])
    k = _unit(k).repeat_interleave(share, 1)
    decay = torch.exp(-torch.exp(s["a_log"]) * _softplus(s["a_raw"][:, 0] + s["dt_bias"]))
    beta = torch.sigmoid(s["b_raw"][:, 0])
    state *= decay[:, :, None, None]
    u = beta[:, :, None] * (v - (state * k[:, :, None, :]).sum(-1))
    state += u[:, :, :, None] * k[:, :, None, :]
    y = (state * q[:, :, None, :]).sum(-1)
    return dict(y=y[:, None].to(s["v"].dtype), state=state)


def _chunked(q, k, v, a_raw, b_raw, a_log, dt_bias, state):
    """y [B, T, H, d_v] and the last state, both f32: chunks of 64 tokens, each one's u from one unit lower triangular
    system (its inverse by repeated squaring), the state carried from chunk to chunk."""
    B, T, H, V = v.shape
    share, K, C = H // k.shape[2], k.shape[3], CHUNK
    n = -(-T // C)

    def chunks(x):    # [B, T, H, d] -> [B, H, n, C, d], zeros behind the last token
        x = torch.cat([x, x.new_zeros(B, n * C - T, *x.shape[2:])], 1)
        return x.view(B, n, C, *x.shape[2:]).permute(0, 3, 1, 2, 4)

    q = chunks(_unit(q.float()).repeat_interleave(share, 2)) / math.sqrt(K)
    k = chunks(_unit(k.float()).repeat_interleave(share, 2))
    v = chunks(v.float())
    g = chunks((-torch.exp(a_log) * _softplus(a_raw + dt_bias))[..., None])
    beta = chunks(torch.sigmoid(b_raw)[..., None])
    G = g[..., 0].double().cumsum(-1)
    diff = G[..., :, None] - G[..., None, :]
    lower = torch.ones(C, C, dtype=torch.bool, device=v.device).tril()
    D = torch.where(lower, diff, -math.inf).float().exp()
    e = G.float().exp()[..., None]
    kt = k.transpose(-1, -2).contiguous()
    N = -(beta * torch.matmul(k, kt) * D).tril(-1)
    inv = torch.eye(C, device=v.device) + N
    for _ in range(5):    # (I - N)^-1 = (I + N)(I + N^2)(I + N^4) ...: N^64 = 0
        N = torch.matmul(N, N)
        inv = inv + torch.matmul(inv, N)
    W, U0 = torch.matmul(inv, beta * e * k), torch.matmul(inv, beta * v)
    P, eq = torch.matmul(q, kt) * D, e * q
    last = G[..., -1:]
    kd = (k * (last - G).float().exp()[..., None]).transpose(-1, -2).contiguous()
    el = last.float().exp()[..., None]
    S = v.new_zeros(B, H, K, V) if state is None else state.transpose(-1, -2).contiguous()
    ys = []
    for i in range(n):
        u = U0[:, :, i] - torch.matmul(W[:, :, i], S)
        ys.append(torch.matmul(eq[:, :, i], S) + torch.matmul(P[:, :, i], u))
        S = el[:, :, i] * S + torch.matmul(kd[:, :, i], u)
    y = torch.stack(ys, 2).reshape(B, H, n * C, V)[:, :, :T].transpose(1, 2)
    return y, S.transpose(-1, -2)


def _train(s):
    leaves = [s[n].detach().requires_grad_() for n in GD_INPUTS]
    y, _ = _chunked(*leaves, None)
    grads = torch.autograd.grad(y, leaves, s["dy"].float())
    return dict(zip(GD_INPUTS, grads), y=y.detach().to(s["v"].dtype))


# ------------------------------------------------------------------- bytes and operations


def work(case):
    c = case
    size = {"f32": 4, "bf16": 2, "f16": 2}
    if c["op"] in ("norm", "norm_grad"):
        n, d, x, y = c["rows"], c["dim"], size[c["x"]], size[c["y"]]
        if c["op"] == "norm":
            return dict(bytes=n * d * (x + y) + 8 * d + 8 * n, flops=8 * n * d)
        return dict(bytes=n * d * (3 * x + y) + 12 * d + 8 * n, flops=14 * n * d)
    B, T, H, G, K, V, a = c["batch"], c["seqlen"], c["heads"], c["groups"], c["d_k"], c["d_v"], size[c["act"]]
    qkv, y, gates, state = B * T * (2 * G * K + H * V) * a, B * T * H * V * a, B * T * H * 8, B * H * K * V * 4
    flops = 7 * B * T * H * K * V    # decay, S k, the update, S q
    if c["op"] == "train":
        return dict(bytes=2 * qkv + 2 * y + 2 * gates + 16 * H, flops=3 * flops)
    return dict(bytes=qkv + y + gates + 2 * state + 8 * H, flops=flops)


# ------------------------------------------------------------------- values in 64 bits


def exact(case, seed):
    s = prepare(case, seed)
    s = {n: x.double() if isinstance(x, torch.Tensor) else x for n, x in s.items()}
    op = case["op"]
    if op in ("norm", "norm_grad"):
        return _exact_norm(s, op)
    if case["seqlen"] > 20000:
        return None
    return _exact_delta(s, op)


def _exact_norm(s, op):
    x, w, d = s["x"], s["w"], s["x"].shape[1]
    if op == "norm":
        mean = x.sum(1) / d
        rstd = 1.0 / ((x - mean[:, None]).square().sum(1) / d + EPS_NORM).sqrt()
        return dict(y=(x - mean[:, None]) * rstd[:, None] * w + s["b"], mean=mean, rstd=rstd)
    mean, rstd, dy = s["mean"], s["rstd"], s["dy"]
    xhat = (x - mean[:, None]) * rstd[:, None]
    a = (dy * w).sum(1) / d
    b = (dy * w * xhat).sum(1) / d
    return dict(dx=s["d_add"] + (dy * w - a[:, None] - xhat * b[:, None]) * rstd[:, None],
                dw=(dy * xhat).sum(0), db=dy.sum(0))


def _exact_delta(s, op):
    """Token by token, states [B, H, d_v, d_k]; the backward pass goes through each chunk's states from the last token
    to the first, after computing them again from the chunk's first."""
    q, k, v = s["q"], s["k"], s["v"]
    B, T, H, V = v.shape
    G, K = k.shape[2], k.shape[3]
    head = torch.arange(H, device=v.device) // (H // G)
    scale = K ** -0.5
    rq = ((q * q).sum(3, keepdim=True) + EPS_UNIT).pow(-0.5)
    rk = ((k * k).sum(3, keepdim=True) + EPS_UNIT).pow(-0.5)
    qn, kn = (q * rq)[:, :, head], (k * rk)[:, :, head]
    z = s["a_raw"] + s["dt_bias"]
    sp = torch.logaddexp(z, torch.zeros_like(z))
    rate = s["a_log"].exp()
    alpha = torch.exp(-rate * sp)
    beta = 1.0 / (1.0 + torch.exp(-s["b_raw"]))

    def forward(S, t):
        aS = alpha[:, t, :, None, None] * S
        miss = v[:, t] - torch.matmul(aS, kn[:, t, :, :, None])[..., 0]
        u = beta[:, t, :, None] * miss
        return torch.baddbmm(aS.view(B * H, V, K), u.reshape(B * H, V, 1), kn[:, t].reshape(B * H, 1, K)).view(B, H, V, K), miss, u

    S = torch.zeros(B, H, V, K, dtype=torch.float64, device=v.device) if op == "train" else s["state"]
    y, kept, C = torch.empty_like(v), [], 128
    for t in range(T):
        if op == "train" and t % C == 0:
            kept.append(S)
        S, _, _ = forward(S, t)
        y[:, t] = scale * torch.matmul(S, qn[:, t, :, :, None])[..., 0]
    if op != "train":
        return dict(y=y, state=S)

    dy = s["dy"]
    dqn, dkn, dv = torch.empty_like(qn), torch.empty_like(kn), torch.empty_like(v)
    dalpha, dbeta = torch.empty_like(alpha), torch.empty_like(beta)
    dS = torch.zeros_like(S)
    for first in reversed(range(0, T, C)):
        states, S = [], kept.pop()
        for t in range(first, min(first + C, T)):
            new, miss, u = forward(S, t)
            states.append((S, new, miss, u))
            S = new
        for t in reversed(range(first, min(first + C, T))):
            old, new, miss, u = states.pop()
            kt, bt, at, d = kn[:, t], beta[:, t, :, None], alpha[:, t, :, None, None], scale * dy[:, t]
            dqn[:, t] = torch.matmul(d[:, :, None, :], new)[:, :, 0]
            dS = dS + d[..., None] * qn[:, t, :, None, :]
            du = torch.matmul(dS, kt[..., None])[..., 0]
            dbeta[:, t] = (du * miss).sum(2)
            dv[:, t] = bt * du
            dkn[:, t] = torch.matmul(u[:, :, None, :], dS)[:, :, 0] - torch.matmul((bt * du)[:, :, None, :], at * old)[:, :, 0]
            back = dS - (bt * du)[..., None] * kt[:, :, None, :]    # the gradient of exp(g) S
            dalpha[:, t] = (back * old).sum((2, 3))
            dS = at * back

    def to_raw(d, n, r):    # the sum over the heads that share a row, then the unit length's adjoint
        d = d.view(B, T, G, H // G, K).sum(3)
        return r * (d - n * (d * n).sum(3, keepdim=True))

    dg = dalpha * alpha
    dz = -rate * dg / (1.0 + torch.exp(-z))
    return dict(q=to_raw(dqn, q * rq, rq), k=to_raw(dkn, k * rk, rk), v=dv, a_raw=dz, b_raw=dbeta * beta * (1.0 - beta),
                a_log=(-rate * sp * dg).sum((0, 1)), dt_bias=dz.sum((0, 1)), y=y)
