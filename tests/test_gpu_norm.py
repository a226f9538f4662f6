"""GPU parity of layer norm (include/mamba_norm.h) against the float64 oracle.

Tolerances, on |gpu - oracle| / |oracle| in the 2-norm.  f32 outputs: sums of
n terms with partial sums of at most 2^9 in a row round by 2^-24 sqrt(2^9) =
1.4e-6 of the terms' size; x - mean cancels |mean| / deviation <= 4 of it, and
three such steps follow one another: 1.7e-5, taken as 2e-5.  A 16-bit output
adds half a step of its type, eps / 2.
"""
import numpy as np
import pytest
import torch

from oracle import gdelta as og

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


@pytest.fixture(scope="module")
def mscan():
    import state_space_sequence_selective_amd as m
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    m.load()
    return m


def check(name, gpu, want):
    g = gpu.detach().double().cpu().numpy()
    assert g.shape == want.shape and np.isfinite(g).all(), name
    norm, off = np.linalg.norm(want), np.linalg.norm(g - want)
    bound = 2e-5 + (0.0 if gpu.dtype == torch.float32 else torch.finfo(gpu.dtype).eps / 2)
    assert off <= bound * norm, "%s: %.2e > %.2e" % (name, off / norm, bound)


def make(rows, dim, x, y, seed=0):
    g = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=g)
    t = dict(x=(n(rows, dim) * (0.5 + 3 * torch.rand(rows, 1, generator=g)) + n(rows, 1)).to(TYPES[x]), w=1 + 0.1 * n(dim),
             b=0.1 * n(dim), dy=n(rows, dim).to(TYPES[y]), d_add=n(rows, dim).to(TYPES[x]))
    return {k: v.cuda() for k, v in t.items()}, {k: v.double().numpy() for k, v in t.items()}


# one element, one vector, each team's first and last width, odd ones
DIMS = [1, 2, 7, 8, 64, 127, 128, 129, 256, 257, 512, 513, 1023, 1025, 2048, 2049, 4096, 4097, 8192, 8193, 16384]


@pytest.mark.parametrize("dim", DIMS)
@pytest.mark.parametrize("x,y", [("f32", "bf16"), ("bf16", "bf16"), ("f16", "f32"), ("f32", "f32")])
def test_widths(mscan, dim, x, y):
    t, r = make(37, dim, x, y, seed=dim)
    ln = mscan.LayerNorm(mscan.NormDims.make(37, dim, x, y, eps=1e-2))
    ln.forward(t["x"], t["w"], t["b"])
    out, mean, rstd = og.layernorm_forward(r["x"], r["w"], r["b"], eps=1e-2)
    for n, a, w in (("y", ln.y, out), ("mean", ln.mean, mean), ("rstd", ln.rstd, rstd)):
        check(n, a, w)
    ln.zero_grads()
    ln.backward(t["x"], t["w"], t["dy"], d_add=t["d_add"])
    # with the statistics that the backward reads, as f32
    want = og.layernorm_backward(r["dy"], r["x"], r["w"], r["d_add"], ln.mean.double().cpu().numpy(), ln.rstd.double().cpu().numpy())
    for n, a, w in zip(("dx", "dw", "db"), (ln.dx, ln.dw, ln.db), want):
        if dim == 1 and n == "dw":   # the row is its own mean: dw is rounding of zero
            assert float(a.abs().max()) <= 37 * 100 * 2 ** -22
            continue
        check(n, a, w)


@pytest.mark.parametrize("x", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("y", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("rows", [1, 3, 5000])
def test_types_and_rows(mscan, x, y, rows):
    t, r = make(rows, 96, x, y, seed=rows)
    ln = mscan.LayerNorm(mscan.NormDims.make(rows, 96, x, y))
    ln.forward(t["x"], t["w"], t["b"])
    out, mean, rstd = og.layernorm_forward(r["x"], r["w"], r["b"])
    check("y", ln.y, out)
    ln.zero_grads()
    ln.backward(t["x"], t["w"], t["dy"], d_add=t["d_add"])
    for n, a, w in zip(("dx", "dw", "db"), (ln.dx, ln.dw, ln.db), og.layernorm_backward(r["dy"], r["x"], r["w"], r["d_add"])):
        check(n, a, w)


def test_without_weights_statistics_or_sums(mscan):
    t, r = make(9, 200, "bf16", "f32", seed=1)
    d = mscan.NormDims.make(9, 200, "bf16", "f32")
    y = torch.empty(9, 200, device="cuda")
    mscan.layernorm_fwd(d, t["x"], y=y)
    out, mean, rstd = og.layernorm_forward(r["x"])
    check("y", y, out)
    m, s = (torch.from_numpy(a).float().cuda() for a in (mean, rstd))
    dx = torch.empty_like(t["x"])
    mscan.layernorm_bwd(d, t["x"], None, m, s, t["dy"], dx=dx)
    check("dx", dx, og.layernorm_backward(r["dy"], r["x"])[0])


def test_sums_accumulate_and_dx_may_be_d_add(mscan):
    t, r = make(300, 130, "f32", "bf16", seed=2)
    ln = mscan.LayerNorm(mscan.NormDims.make(300, 130, "f32", "bf16"))
    ln.forward(t["x"], t["w"], t["b"])
    ln.zero_grads()
    ln.backward(t["x"], t["w"], t["dy"], d_add=t["d_add"])
    dw, db, dx = ln.dw.clone(), ln.db.clone(), ln.dx.clone()
    ln.dx.copy_(t["d_add"])
    ln.backward(t["x"], t["w"], t["dy"], d_add=ln.dx)
    assert torch.equal(ln.dx, dx) and torch.equal(ln.dw, 2 * dw) and torch.equal(ln.db, 2 * db)


def test_far_mean(mscan):
    """A mean 1000 times the deviation: the variance comes from the centred row."""
    t, _ = make(8, 1000, "f32", "f32", seed=3)
    x = t["x"] / 4 + 1000.0
    ln = mscan.LayerNorm(mscan.NormDims.make(8, 1000, "f32", "f32"))
    ln.forward(x, t["w"], t["b"])
    _, mean, rstd = og.layernorm_forward(x.double().cpu().numpy())
    check("mean", ln.mean, mean)
    # the mean's own rounding, 2^-24 * 1000 * a few, is 1e-4 of a deviation and enters the variance by its square
    check("rstd", ln.rstd, rstd)


def test_rows_do_not_touch_one_another(mscan):
    t, _ = make(40, 129, "bf16", "bf16", seed=4)
    ln = mscan.LayerNorm(mscan.NormDims.make(40, 129, "bf16", "bf16"))
    clean = ln.forward(t["x"], t["w"], t["b"]).clone()
    t["x"][7] = float("nan")
    t["x"][11, 3] = float("inf")
    y = ln.forward(t["x"], t["w"], t["b"])
    keep = [i for i in range(40) if i not in (7, 11)]
    assert torch.equal(y[keep], clean[keep]) and bool(torch.isnan(y[7]).all())


def test_graph_replay(mscan):
    xs = [make(70, 300, "f32", "bf16", seed=s)[0] for s in (1, 2, 3)]
    live = {n: t.clone() for n, t in xs[0].items()}
    d = mscan.NormDims.make(70, 300, "f32", "bf16")
    eager, ln = mscan.LayerNorm(d), mscan.LayerNorm(d)
    step = lambda o, t: (o.zero_grads(), o.forward(t["x"], t["w"], t["b"]), o.backward(t["x"], t["w"], t["dy"], t["d_add"]))
    step(ln, live)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(ln, live)
    for t in xs + xs[:1]:
        for n in live:
            live[n].copy_(t[n])
        graph.replay()
        torch.cuda.synchronize()
        step(eager, t)
        torch.cuda.synchronize()
        for n in ("y", "mean", "rstd", "dx", "dw", "db"):
            assert torch.equal(getattr(ln, n), getattr(eager, n)), n


def test_block_of_norm_core_and_head_norm(mscan):
    """As a block uses them: norm of the f32 residual, the gated delta rule, each head's output normed; and back."""
    B, T, H, K = 1, 100, 2, 32
    D = H * K
    g = torch.Generator().manual_seed(8)
    n = lambda *s: torch.randn(*s, generator=g)
    resid, gates = n(B * T, D).cuda(), {k: n(B, T, H).cuda() for k in ("a_raw", "b_raw")}
    par = dict(a_log=torch.rand(H, generator=g).cuda(), dt_bias=(-3 + n(H)).cuda())
    w = [(1 + 0.1 * n(d)).cuda() for d in (D, K)]
    b = [(0.1 * n(d)).cuda() for d in (D, K)]
    dz = n(B * T * H, K).cuda()
    pre = mscan.LayerNorm(mscan.NormDims.make(B * T, D, "f32", "f32"))
    post = mscan.LayerNorm(mscan.NormDims.make(B * T * H, K, "f32", "f32"))
    core = mscan.GatedDeltaCore(mscan.GDeltaDims.make(B, T, H, K, K, act="f32"))
    for o in (pre, post, core):
        o.zero_grads()
    x = pre.forward(resid, w[0], b[0]).view(B, T, H, K)     # q, k and v are all the normed row here
    inp = dict(q=x, k=x, v=x, **gates, **par)
    y = core.forward(inp)
    post.forward(y.view(-1, K), w[1], b[1])
    dy = post.backward(y.view(-1, K), w[1], dz).view(y.shape)
    gr = core.backward(inp, dy)
    dx = pre.backward(resid, w[0], (gr["q"] + gr["k"] + gr["v"]).view(B * T, D).contiguous(), d_add=resid)
    f = lambda t: t.double().cpu().numpy()
    xo = og.layernorm_forward(f(resid), f(w[0]), f(b[0]))[0].reshape(B, T, H, K)
    args = dict(q=xo, k=xo, v=xo, **{k: f(v) for k, v in dict(gates, **par).items()})
    yo, _ = og.forward(**args)
    zo = og.layernorm_forward(yo.reshape(-1, K), f(w[1]), f(b[1]))[0]
    dyo, dw1, db1 = og.layernorm_backward(f(dz), yo.reshape(-1, K), f(w[1]))
    go = og.backward(dyo.reshape(yo.shape), **args)
    dxo, dw0, db0 = og.layernorm_backward((go["q"] + go["k"] + go["v"]).reshape(B * T, D), f(resid), f(w[0]), f(resid))
    # three operators one after the other, and a head norm that divides by deviations down to a tenth of a typical one:
    # ten times the single operator's bound
    for name, a, want in (("z", post.y, zo), ("dx", dx, dxo), ("dw0", pre.dw, dw0), ("dw1", post.dw, dw1),
                          ("a_log", gr["a_log"], go["a_log"])):
        off = np.linalg.norm(f(a) - want) / np.linalg.norm(want)
        assert off <= 2e-4, (name, off)
