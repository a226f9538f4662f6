"""Refusals of the gated delta rule's and layer norm's entry points: each is
made before any launch, so they are checked without a GPU."""
import ctypes
import os
import re

import pytest


@pytest.fixture(scope="module")
def pkg():
    import state_space_sequence_selective_amd as m
    if not os.path.exists(m.LIB_PATH):
        pytest.skip("libmamba_scan.so not built")
    m.load()
    return m


def gd(pkg, **kw):
    return pkg.GDeltaDims.make(**dict(dict(batch=2, seqlen=100, heads=4, groups=2, d_k=64, d_v=32, act="bf16"), **kw))


def ln(pkg, **kw):
    return pkg.NormDims.make(**dict(dict(rows=10, dim=100), **kw))


@pytest.mark.parametrize("kw,status,msg", [
    (dict(batch=0), 1, "batch"), (dict(seqlen=0), 1, "seqlen"), (dict(heads=0), 1, "heads"),
    (dict(groups=0), 1, "groups"), (dict(heads=5), 1, "multiple of groups"), (dict(act=3), 1, "act"),
    (dict(act=-1), 1, "act"), (dict(d_k=0), 1, "d_k"), (dict(d_v=-8), 1, "d_v"), (dict(d_k=12), 2, "d_k"),
    (dict(d_k=136), 2, "d_k"), (dict(d_v=12), 2, "d_v"), (dict(d_v=520), 2, "d_v"),
    (dict(scale=float("nan")), 1, "scale"), (dict(scale=float("inf")), 1, "scale"),
    (dict(scale=1e-7), 1, "scale"), (dict(scale=-2e6), 1, "scale"), (dict(eps=0.0), 1, "eps"),
    (dict(eps=float("nan")), 1, "eps"), (dict(seqlen=(1 << 24) + 1), 3, "seqlen"),
    (dict(batch=1 << 25), 3, "batch"),
    (dict(heads=1 << 15, d_v=512), 3, "heads"), (dict(batch=1 << 19, heads=16), 3, "2^23"),
])
def test_gdelta_dims(pkg, kw, status, msg):
    for f in (pkg.gdelta_saved_bytes, pkg.gdelta_workspace_bytes):
        with pytest.raises(pkg.MambaScanError, match="mamba_gdelta_.*" + msg.replace("^", r"\^")) as e:
            f(gd(pkg, **kw))
        assert e.value.status == status


@pytest.mark.parametrize("kw,status,msg", [
    (dict(rows=0), 1, "rows"), (dict(dim=0), 1, "dim"), (dict(dim=16385), 2, "dim"), (dict(x=7), 1, "x is"),
    (dict(y=-1), 1, "y is"), (dict(eps=0.0), 1, "eps"), (dict(rows=1 << 40), 3, "rows"),
])
def test_norm_dims(pkg, kw, status, msg):
    with pytest.raises(pkg.MambaScanError, match="mamba_layernorm_.*" + msg) as e:
        pkg.layernorm_workspace_bytes(ln(pkg, **kw))
    assert e.value.status == status


P, BIG = ctypes.c_void_p, ctypes.c_size_t(1 << 40)


def calls(pkg):
    """Every entry point's pointer arguments by name, the needed ones, and the call; addresses are never dereferenced."""
    lib = pkg.load()
    d, n = gd(pkg), ln(pkg)
    seven = ["q", "k", "v", "a_raw", "b_raw", "a_log", "dt_bias"]

    def fwd(a, saved=BIG, ws=BIG):
        return lib.mamba_gdelta_fwd(ctypes.byref(d), *(a[x] for x in seven), a["h0"], a["y"], a["h_last"], a["saved"], saved,
                                    a["workspace"], ws, None)

    def bwd(a, saved=BIG, ws=BIG):
        return lib.mamba_gdelta_bwd(ctypes.byref(d), *(a[x] for x in seven), 0, a["saved"], saved, a["dy"], a["d_q"],
                                    a["d_k"], a["d_v"], a["d_a_raw"], a["d_b_raw"], a["d_a_log"], a["d_dt_bias"],
                                    a["workspace"], ws, None)

    def step(a):
        return lib.mamba_gdelta_step(ctypes.byref(d), *(a[x] for x in seven), a["state"], a["y"], None)

    def nfwd(a):
        return lib.mamba_layernorm_fwd(ctypes.byref(n), a["x"], a["w"], a["b"], a["y"], a["mean"], a["rstd"], None)

    def nbwd(a, ws=BIG):
        return lib.mamba_layernorm_bwd(ctypes.byref(n), a["x"], a["w"], a["mean"], a["rstd"], a["dy"], a["d_add"], a["dx"],
                                       a["d_w"], a["d_b"], a["workspace"], ws, None)

    grads = ["d_q", "d_k", "d_v", "d_a_raw", "d_b_raw", "d_a_log", "d_dt_bias"]
    return {
        "mamba_gdelta_fwd": (fwd, seven + ["y"], ["h0", "h_last", "saved", "workspace"]),
        "mamba_gdelta_bwd": (bwd, seven + ["saved", "dy", "workspace"] + grads, []),
        "mamba_gdelta_step": (step, seven + ["state", "y"], []),
        "mamba_layernorm_fwd": (nfwd, ["x", "y", "mean", "rstd"], ["w", "b"]),
        "mamba_layernorm_bwd": (nbwd, ["x", "mean", "rstd", "dy", "dx", "workspace"], ["w", "d_add", "d_w", "d_b"]),
    }


@pytest.mark.parametrize("name", ["mamba_gdelta_fwd", "mamba_gdelta_bwd", "mamba_gdelta_step", "mamba_layernorm_fwd",
                                  "mamba_layernorm_bwd"])
def test_pointers(pkg, name):
    call, needed, optional = calls(pkg)[name]
    good = {n: P(0x10000) for n in needed + optional}
    for n in needed:
        assert call(dict(good, **{n: None})) == 1
        assert name in pkg.last_error() and n in pkg.last_error() and "NULL" in pkg.last_error()
    for n in needed + optional:
        assert call(dict(good, **{n: P(0x10002)})) == 1, n
        assert name in pkg.last_error() and n + " is not" in pkg.last_error()


def test_sizes(pkg):
    table = calls(pkg)
    for name, kw in (("mamba_gdelta_fwd", "saved"), ("mamba_gdelta_bwd", "saved"), ("mamba_gdelta_bwd", "ws"),
                     ("mamba_layernorm_bwd", "ws")):
        call, needed, optional = table[name]
        good = {n: P(0x10000) for n in needed + optional}
        assert call(good, **{kw: ctypes.c_size_t(100)}) == 3
        assert name in pkg.last_error() and "needed" in pkg.last_error()
    call, needed, optional = table["mamba_gdelta_fwd"]
    good = dict({n: P(0x10000) for n in needed}, h0=None, h_last=None, saved=None, workspace=None)
    assert call(good) == 1 and "workspace is NULL" in pkg.last_error()      # 100 tokens, nothing saved
    assert call(dict(good, workspace=P(0x10000)), ws=ctypes.c_size_t(100)) == 3
    call, needed, _ = table["mamba_layernorm_fwd"]
    good = dict({n: P(0x10000) for n in needed}, w=None, b=None)
    assert call(dict(good, mean=None)) == 1 and call(dict(good, rstd=None)) == 1   # both or neither


def test_layout(pkg):
    """16 chunk-heads and 8 chunk-groups (2 batch rows, 4 heads of 2 groups, 2 chunks of 64 tokens), piece by piece."""
    al = lambda b: (b + 255) // 256 * 256
    heads, groups, tri = 16, 8, 16 * 6 * 1024
    for act, planes in (("bf16", 1), ("f32", 2)):
        family = al(groups * planes * 8 * 1024)      # d_k 64: 8 fragments of 1 KB a plane
        fwd = (al(groups * 4 * 64 * 4) + 3 * family + al(heads * 5 * 64 * 4) + al(heads * 64 * 8) + al(planes * tri) + al(2 * tri)
               + al(heads * 4) + al(8 * 4))
        saved = fwd + family + 2 * al(2 * tri) + 2 * al(heads * 64 * 32 * 4)
        bwd = al(heads * 4) + al(8 * 4) + al(heads * 8) + 2 * al(heads * 64 * 32 * 4)
        assert pkg.gdelta_saved_bytes(gd(pkg, act=act)) == saved
        assert pkg.gdelta_workspace_bytes(gd(pkg, act=act)) == max(fwd, bwd)
    assert pkg.layernorm_workspace_bytes(ln(pkg, rows=5000, dim=5120)) == 512 * 2 * 5120 * 4
    assert pkg.layernorm_workspace_bytes(ln(pkg, rows=100000, dim=64)) == 1024 * 2 * 64 * 4
    assert pkg.layernorm_workspace_bytes(ln(pkg, rows=100, dim=5120)) == 100 * 2 * 5120 * 4


def test_binding_checks(pkg):
    import torch
    d = gd(pkg, seqlen=1)
    s = d.shapes()
    cpu = {n: torch.zeros(sh) for n, sh in dict(q=s["qk"], k=s["qk"], v=s["v"], a_raw=s["gate"], b_raw=s["gate"],
                                                a_log=s["h"], dt_bias=s["h"]).items()}
    with pytest.raises(ValueError, match="device tensor"):
        pkg.gdelta_step(d, *cpu.values(), torch.zeros(s["state"]), y=torch.zeros(s["v"]))
    with pytest.raises(TypeError, match="torch.Tensor"):
        pkg.layernorm_fwd(ln(pkg), [1.0], y=torch.zeros(10, 100))


def test_step_tokens_is_the_headers(pkg):
    text = open(os.path.join(os.path.dirname(__file__), "..", "include", "mamba_gdelta.h")).read()
    assert int(re.search(r"define MAMBA_GDELTA_STEP_TOKENS (\d+)", text).group(1)) == pkg._lib.GDELTA_STEP_TOKENS
    train = pkg.gdelta_workspace_bytes(gd(pkg, seqlen=9))
    for seqlen, size in ((8, 0), (9, train)):
        core = pkg.GatedDeltaCore(gd(pkg, seqlen=seqlen), device="cpu", train=False)
        assert core.workspace.numel() == size
