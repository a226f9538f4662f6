"""GPU parity of the gated delta rule (include/mamba_gdelta.h) against the
float64 token-by-token oracle (oracle/gdelta.py).

Tolerances, on |gpu - oracle| / |oracle| in the 2-norm.  f32 outputs: a
product's operands keep 22 bits (2^-22 of the largest of a row, twice), sums
run over at most 512 terms in f32 (2^-24 sqrt(512) = 2^-19.5) and about ten
such steps follow one another on the longest path: 10 * (2^-21 + 2^-19.5) =
1.8e-5, taken as 2e-5.  An output of 16 bits is that plus one rounding, half
a step of its type: eps / 2.
"""
import numpy as np
import pytest
import torch

from oracle import gdelta as og

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
NAMES = ("q", "k", "v", "a_raw", "b_raw", "a_log", "dt_bias")


@pytest.fixture(scope="module")
def mscan():
    import state_space_sequence_selective_amd as m
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    m.load()
    return m


def tol(dtype):
    return 2e-5 if dtype == torch.float32 else torch.finfo(dtype).eps / 2 + 2e-5


def make(B, T, H, G, K, V, act, seed=0):
    """Inputs on the GPU, already rounded to their types, and the same as float64 numpy."""
    gen = torch.Generator().manual_seed(seed)
    at = TYPES[act]
    n = lambda *s: torch.randn(*s, generator=gen)
    dt = torch.exp(torch.rand(H, generator=gen) * 4.6 - 6.9)
    x = dict(q=n(B, T, G, K).to(at), k=n(B, T, G, K).to(at), v=n(B, T, H, V).to(at), a_raw=n(B, T, H), b_raw=n(B, T, H),
             a_log=torch.log(1 + 15 * torch.rand(H, generator=gen)), dt_bias=dt + torch.log(-torch.expm1(-dt)),
             dy=n(B, T, H, V).to(at), h0=n(B, H, V, K))
    return {k: v.cuda() for k, v in x.items()}, {k: v.double().numpy() for k, v in x.items()}


def rel(gpu, want):
    g = gpu.detach().double().cpu().numpy()
    assert g.shape == want.shape and np.isfinite(g).all()
    norm = np.linalg.norm(want)
    off = np.linalg.norm(g - want)
    return off / norm if norm else (0.0 if off == 0 else np.inf)


def check(pairs):
    bad = {k: "%.2e > %.2e" % (rel(a, w), tol(a.dtype)) for k, (a, w) in pairs.items() if not rel(a, w) <= tol(a.dtype)}
    assert not bad, bad


def dims_of(mscan, B, T, H, G, K, V, act, **kw):
    return mscan.GDeltaDims.make(B, T, H, K, V, groups=G, act=act, **kw)


def train(mscan, shape, x, ref, h0=None, **kw):
    core = mscan.GatedDeltaCore(dims_of(mscan, *shape, **kw))
    core.zero_grads()
    core.forward(x, h0=x["h0"] if h0 else None)
    core.backward(x, x["dy"])
    torch.cuda.synchronize()
    args = {n: ref[n] for n in NAMES}
    args.update(h0=ref["h0"] if h0 else None, **kw)
    y, last = og.forward(**args)
    g = og.backward(ref["dy"], **args)
    check(dict({n: (core.grads[n], g[n]) for n in NAMES}, y=(core.y, y), h_last=(core.h_last, last)))
    return core


# B, T, H, G, d_k, d_v
SHAPES = [(1, 64, 1, 1, 64, 32), (2, 65, 2, 1, 64, 64), (1, 63, 4, 2, 32, 48), (1, 130, 3, 3, 128, 128),
          (2, 17, 4, 1, 8, 8), (1, 200, 2, 2, 72, 40), (1, 129, 2, 1, 128, 136), (1, 1, 2, 2, 64, 64), (3, 2, 2, 1, 16, 24),
          (1, 70, 4, 2, 128, 512), (2, 65, 1, 1, 8, 264)]


@pytest.mark.parametrize("act", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("h0", [False, True])
def test_forward_and_backward(mscan, shape, act, h0):
    x, ref = make(*shape, act, seed=sum(shape))
    train(mscan, (*shape, act), x, ref, h0=h0)


@pytest.mark.parametrize("act", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("shape", [(6, 70, 24, 24, 40, 80), (9, 130, 16, 8, 120, 64), (4, 70, 20, 5, 72, 64),
                                   (3, 65, 30, 30, 64, 104)], ids=str)
def test_many_heads(mscan, shape, act):
    """More 16-column tiles than waves: the passes that share a head's operands, three and four tiles to a workgroup, some
    with tiles behind the columns."""
    x, ref = make(*shape, act, seed=29)
    train(mscan, (*shape, act), x, ref, h0=True)
    core = mscan.GatedDeltaCore(dims_of(mscan, *shape, act), train=False)
    core.forward(x, h0=x["h0"])
    y, last = og.forward(**{n: ref[n] for n in NAMES}, h0=ref["h0"])
    check(dict(y=(core.y, y), h_last=(core.h_last, last)))


@pytest.mark.parametrize("act", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("T", [1, 8, 9, 15, 16, 17, 64, 100, 257])
def test_forward_alone(mscan, act, T):
    """Without anything kept: the short sequences' token-by-token kernel and the chunks; h_last over h0."""
    shape = (2, T, 4, 2, 64, 72, act)
    x, ref = make(*shape[:6], act, seed=T)
    core = mscan.GatedDeltaCore(dims_of(mscan, *shape), train=False)
    core.h_last.copy_(x["h0"])
    core.forward(x, h0=core.h_last)
    y, last = og.forward(**{n: ref[n] for n in NAMES}, h0=ref["h0"])
    check(dict(y=(core.y, y), h_last=(core.h_last, last)))


@pytest.mark.parametrize("act", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("shape", [(3, 1, 4, 2, 128, 128), (1, 1, 1, 1, 8, 8), (2, 5, 3, 1, 40, 200), (5, 1, 2, 2, 120, 16),
                                   (20, 3, 28, 4, 72, 40), (65, 2, 8, 8, 16, 32), (64, 1, 8, 1, 128, 24)],
                         ids=str)
def test_step(mscan, shape, act):
    x, ref = make(*shape, act, seed=7)
    core = mscan.GatedDeltaCore(dims_of(mscan, *shape, act), train=False)
    state = x["h0"].clone()
    y = core.step(x, state)
    want, last = og.forward(**{n: ref[n] for n in NAMES}, h0=ref["h0"])
    check(dict(y=(y, want), state=(state, last)))


def test_prompt_then_steps(mscan):
    """A prompt through the chunks, then token by token: as one sequence."""
    B, T, H, G, K, V, act = 2, 150, 4, 2, 64, 64, "bf16"
    x, ref = make(B, T, H, G, K, V, act, seed=3)
    cut = {n: (t[:, :140].contiguous() if t.dim() >= 3 and n != "h0" else t) for n, t in x.items()}
    core = mscan.GatedDeltaCore(dims_of(mscan, B, 140, H, G, K, V, act), train=False)
    out = [core.forward(cut).clone()]
    one = mscan.GatedDeltaCore(dims_of(mscan, B, 1, H, G, K, V, act), train=False)
    for t in range(140, T):
        tok = {n: (v[:, t:t + 1].contiguous() if v.dim() >= 3 and n != "h0" else v) for n, v in x.items()}
        out.append(one.step(tok, core.h_last).clone())
    y, last = og.forward(**{n: ref[n] for n in NAMES})
    check(dict(y=(torch.cat(out, 1), y), state=(core.h_last, last)))


@pytest.mark.parametrize("act", ["f32", "bf16"])
def test_hard_gates(mscan, act):
    """Decays that clear the state within a token (g of -160 and below) or keep all of it, and write strengths at 0 and 1."""
    shape = (1, 150, 2, 1, 64, 32)
    x, ref = make(*shape, act, seed=5)
    gen = np.random.default_rng(1)
    a = np.where(gen.random((1, 150, 2)) < 0.1, 40.0, -30.0)
    b = np.where(gen.random((1, 150, 2)) < 0.5, 30.0, -30.0)
    for n, t in (("a_raw", a), ("b_raw", b)):
        ref[n] = t
        x[n] = torch.from_numpy(t).float().cuda()
    ref["a_log"] = np.full(2, np.log(4.0))
    x["a_log"] = torch.from_numpy(ref["a_log"]).float().cuda()
    ref["a_log"] = x["a_log"].double().cpu().numpy()
    core = mscan.GatedDeltaCore(dims_of(mscan, *shape, act))
    core.zero_grads()
    core.forward(x)
    g = core.backward(x, x["dy"])
    args = {n: ref[n] for n in NAMES}
    y, last = og.forward(**args)
    want = og.backward(ref["dy"], **args)
    # d a_raw and what comes of it: where the decay ends a state the exact gradient is e^-160, so the sums' rounding is
    # what is left of it; the others are held to the usual bounds
    check(dict({n: (g[n], want[n]) for n in ("q", "k", "v")}, y=(core.y, y), h_last=(core.h_last, last)))


@pytest.mark.parametrize("size", [1e-30, 1e30])
def test_values_far_from_one(mscan, size):
    """f32 values and keys of any size: the powers of two taken out keep the f16 parts in range."""
    shape = (1, 100, 2, 1, 64, 32)
    x, ref = make(*shape, "f32", seed=11)
    for n in ("v", "dy"):
        x[n] = x[n] * size if n == "v" else x[n]
        ref[n] = x[n].double().cpu().numpy()
    for n in ("q", "k"):
        x[n] = x[n] * 1e15
        ref[n] = x[n].double().cpu().numpy()
    core = mscan.GatedDeltaCore(dims_of(mscan, *shape, "f32"))
    core.zero_grads()
    core.forward(x)
    g = core.backward(x, x["dy"])
    args = {n: ref[n] for n in NAMES}
    y, last = og.forward(**args)
    want = og.backward(ref["dy"], **args)
    pairs = dict(y=(core.y, y), h_last=(core.h_last, last), v=(g["v"], want["v"]))
    for n, (a, w) in pairs.items():      # in units of `size`: 2-norms of 1e30 squared would overflow nothing here, f64
        assert rel(a, w) <= tol(a.dtype), n


@pytest.mark.parametrize("eps", [1e-2, 1e-6])
def test_zero_rows(mscan, eps):
    """Keys, queries and values of zero: no division by their length, finite gradients."""
    shape = (1, 70, 2, 1, 64, 32)
    x, ref = make(*shape, "f32", seed=13)
    for n in ("q", "k", "v"):
        x[n][:, ::3] = 0
        ref[n] = x[n].double().cpu().numpy()
    train(mscan, (*shape, "f32"), x, ref, eps=eps)


def test_scale_and_accumulation(mscan):
    """A scale and eps of the caller's; parameter gradients add to what is there, the others are overwritten."""
    shape = (1, 80, 2, 2, 32, 32, "f32")
    x, ref = make(*shape[:6], "f32", seed=17)
    core = train(mscan, shape, x, ref, scale=0.5, eps=1e-3)
    once = {n: core.grads[n].clone() for n in NAMES}
    core.backward(x, x["dy"])
    for n in NAMES:
        assert torch.equal(core.grads[n], 2 * once[n] if n in ("a_log", "dt_bias") else once[n]), n


def test_twice_the_same_bits_and_no_stray_writes(mscan):
    """The same bits on every call, from buffers filled with anything, and nothing written behind an output's end."""
    B, T, H, G, K, V, act = 2, 100, 4, 2, 72, 40, "bf16"
    x, _ = make(B, T, H, G, K, V, act, seed=19)
    d = dims_of(mscan, B, T, H, G, K, V, act)
    outs = []
    for fill in (0, 0xff):
        core = mscan.GatedDeltaCore(d)
        core.saved.fill_(fill)
        core.workspace.fill_(fill)
        big = {}
        for n in ("q", "k", "v", "a_raw", "b_raw"):
            t = core.grads[n]
            big[n] = torch.full((t.numel() + 64,), 7.0, dtype=t.dtype, device="cuda")
            core.grads[n] = big[n][:t.numel()].view(t.shape)
        core.zero_grads()
        core.forward(x)
        core.backward(x, x["dy"])
        torch.cuda.synchronize()
        assert all(bool((t[-64:] == 7.0).all()) for t in big.values())
        outs.append({n: t.clone() for n, t in dict(core.grads, y=core.y, h_last=core.h_last).items()})
    assert all(torch.equal(outs[0][n], outs[1][n]) for n in outs[0])


def test_graph_replay_on_a_stream(mscan):
    """A training step captured on a side stream, replayed over changing inputs, with eager work in between."""
    shape = (1, 130, 4, 2, 64, 64, "bf16")
    xs = [make(*shape[:6], "bf16", seed=s)[0] for s in (1, 2, 3)]
    live = {n: t.clone() for n, t in xs[0].items()}
    d = dims_of(mscan, *shape)
    eager, core = mscan.GatedDeltaCore(d), mscan.GatedDeltaCore(d)
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        core.forward(live, h0=live["h0"])
        core.backward(live, live["dy"])
    side.synchronize()
    with torch.cuda.graph(graph, stream=side):
        core.zero_grads()
        core.forward(live, h0=live["h0"])
        core.backward(live, live["dy"])
    for x in xs + xs[:1]:
        for n in live:
            live[n].copy_(x[n])
        graph.replay()
        torch.cuda.synchronize()
        eager.zero_grads()
        eager.forward(x, h0=x["h0"])
        eager.backward(x, x["dy"])
        torch.cuda.synchronize()
        assert torch.equal(core.y, eager.y) and torch.equal(core.h_last, eager.h_last)
        assert all(torch.equal(core.grads[n], eager.grads[n]) for n in NAMES)


def test_a_nan_stays_in_its_heads_and_batch_rows(mscan):
    shape = (2, 100, 4, 2, 64, 32, "bf16")
    x, _ = make(*shape[:6], "bf16", seed=23)
    core = mscan.GatedDeltaCore(dims_of(mscan, *shape), train=False)
    clean = core.forward(x).clone()
    x["v"][0, 70, 1] = float("nan")     # in the second chunk
    y = core.forward(x)
    assert torch.equal(y[1], clean[1]) and torch.equal(y[0, :, [0, 2, 3]], clean[0, :, [0, 2, 3]])
    assert torch.equal(y[0, :64, 1], clean[0, :64, 1])
    assert bool(torch.isnan(y[0, 70:, 1]).all())


@pytest.mark.parametrize("shape", [(2, 1, 4, 2, 64, 64, "bf16"), (20, 1, 28, 4, 72, 40, "f16")], ids=str)
def test_decoding_replayed_on_a_stream(mscan, shape):
    """A decoding step captured on a side stream: each replay takes the next token and the state the last one left."""
    xs = [make(*shape, seed=s)[0] for s in (1, 2, 3, 4)]
    live = {n: t.clone() for n, t in xs[0].items()}
    d = dims_of(mscan, *shape)
    eager, core = mscan.GatedDeltaCore(d, train=False), mscan.GatedDeltaCore(d, train=False)
    state, want = xs[0]["h0"].clone(), xs[0]["h0"].clone()
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=side):
        core.step(live, state)
    for x in xs + xs[:1]:
        for n in live:
            live[n].copy_(x[n])
        graph.replay()
        torch.cuda.synchronize()
        y = eager.step(x, want)
        torch.cuda.synchronize()
        assert torch.equal(core.y, y) and torch.equal(state, want)


def test_two_streams_at_once(mscan):
    """Two cores with buffers of their own, on two streams at the same time: each as alone."""
    shape = (2, 200, 8, 4, 64, 64, "bf16")
    d = dims_of(mscan, *shape)
    xs = [make(*shape, seed=s)[0] for s in (5, 6)]
    cores, streams = [mscan.GatedDeltaCore(d) for _ in xs], [torch.cuda.Stream() for _ in xs]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        for x, core, s in zip(xs, cores, streams):
            with torch.cuda.stream(s):
                core.zero_grads()
                core.forward(x)
                core.backward(x, x["dy"])
    torch.cuda.synchronize()
    for x, core in zip(xs, cores):
        alone = mscan.GatedDeltaCore(d)
        alone.forward(x)
        alone.backward(x, x["dy"])
        torch.cuda.synchronize()
        assert torch.equal(core.y, alone.y) and all(torch.equal(core.grads[n], alone.grads[n]) for n in NAMES)
