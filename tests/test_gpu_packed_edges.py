"""The packed calls away from their defaults: other eps, values of very different sizes along the
tokens, values that are not finite, and what a call may be given."""
import pytest

import _packed_ref as R

pytestmark = pytest.mark.gpu

ENTRIES = ["step", "generic", "mfma"]


def run(x, entry, **kw):
    """An entry point on the case (``kw``: further arguments); returns (out, pool)."""
    import torch
    import chunked_gated_delta_gdr_amd as G
    d = {n: t.cuda() if isinstance(t, torch.Tensor) else t for n, t in x.items()}
    out = torch.full(x["v"].shape, 7.0, dtype=x["v"].dtype, device="cuda")
    kw = dict(dict(beta=d["beta"], log_alpha=d["log_alpha"], state_index=d["index"], has_state=d["has"], qk_norm=x["qk_norm"],
                   norm_weight=d["norm_weight"], norm_gate=d["norm_gate"], out=out, scale=x["scale"]), **kw)
    print(f"[case] {entry} lens {x['lens'][:8]} q {tuple(x['q'].shape)} v {tuple(x['v'].shape)} {x['q'].dtype}", flush=True)
    if entry == "step":
        G.gdr_packed_step(d["q"], d["k"], d["v"], d["pool"], cu_seqlens=d["cu"], **kw)
    else:
        G.gdr_packed_fwd(d["q"], d["k"], d["v"], d["cu"], state=d["pool"], impl=entry, **kw)
    torch.cuda.synchronize()
    return out.cpu(), d["pool"].cpu()


def io_tol(x, entry):
    """One rounding to the type; bf16 outputs of the chunked kernel take one fp16 part each of P, E and S."""
    import torch
    io = x["v"].dtype
    return R.half_step(io) + (2.0 ** -11 if entry == "mfma" and io == torch.bfloat16 else 0.0)


def normalised(x, eps):
    """The case with q and k over their L2 norms in 64 bits."""
    q, k = x["q"].double(), x["k"].double()
    return dict(x, q=q / (q.square().sum(-1, keepdim=True) + eps).sqrt(), k=k / (k.square().sum(-1, keepdim=True) + eps).sqrt(),
                qk_norm=False)


@pytest.mark.parametrize("entry", ENTRIES)
@pytest.mark.parametrize("io", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("eps", [0.0, 1e-3, 2.0])
@pytest.mark.parametrize("lens", [[1], [63], [64], [65], [130, 5, 0, 64]], ids=str)
def test_key_norm_eps(entry, io, eps, lens):
    """eps = 0 too: rows past a sequence's end are no keys of size 0."""
    import torch
    x = R.make(lens, Hk=2, Hv=4, Dk=64, Dv=32, io=io, qk_norm=True, seed=81 + len(lens))
    out, pool = run(x, entry, qk_eps=eps)
    ref_o, ref_p = R.delta(normalised(x, eps), torch.zeros(x["v"].shape))
    tol = R.state_tol(max(lens))
    assert R.rel(pool, ref_p) <= tol
    assert R.rel(out, ref_o) <= io_tol(x, entry) + tol


def test_output_norm_of_the_most_rows():
    """n_tokens * Hv at its limit, 2^26: the norm's launch has its rows too."""
    import torch
    import chunked_gated_delta_gdr_amd as G
    x = R.make([70], Hk=1, Hv=32, Dk=8, Dv=8, norm=True, seed=85)
    want_o, want_p = run(x, "mfma")
    N = 2 ** 26 // 32
    at = {n: torch.zeros((N,) + x[n].shape[1:], dtype=x[n].dtype, device="cuda") for n in ("q", "k", "v", "beta", "log_alpha")}
    for n, t in at.items():
        t[N - 70:] = x[n].cuda()
    out = torch.full((N, 32, 8), 7.0, dtype=torch.bfloat16, device="cuda")
    pool = x["pool"].cuda()
    cu = torch.tensor([N - 70, N], dtype=torch.int32, device="cuda")
    G.gdr_packed_fwd(at["q"], at["k"], at["v"], cu, beta=at["beta"], log_alpha=at["log_alpha"], state=pool, scale=x["scale"],
                     norm_weight=x["norm_weight"].cuda(), out=out, impl="mfma")
    torch.cuda.synchronize()
    assert torch.equal(out[N - 70:].cpu(), want_o) and torch.equal(pool.cpu(), want_p)
    assert bool((out[:N - 70] == 7.0).all())


@pytest.mark.parametrize("entry", ["fwd", "step"])
def test_every_tensor_by_name(entry):
    import torch
    import chunked_gated_delta_gdr_amd as G
    x = R.make([3, 2], seed=86)
    d = {n: x[n].cuda() for n in ("q", "k", "v", "beta", "log_alpha")}
    d.update(cu_seqlens=x["cu"].cuda(), scale=x["scale"])
    want = run(x, "step" if entry == "step" else "mfma")
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for stream in (None, side):
        pool = x["pool"].cuda()
        torch.cuda.synchronize()
        got = getattr(G, f"gdr_packed_{entry}")(state=pool, stream=stream, **d)
        torch.cuda.synchronize()
        assert torch.equal(got.cpu(), want[0]) and torch.equal(pool.cpu(), want[1])


@pytest.mark.parametrize("entry", ENTRIES)
def test_scale_and_eps_may_be_tensors_that_change(entry):
    """Their values at the call count, not those that an earlier call met."""
    import torch
    x = R.make([3, 2], qk_norm=True, norm=True, seed=84)
    t = {n: torch.tensor(0.0) for n in ("scale", "qk_eps", "norm_eps")}
    for values in (dict(scale=0.5, qk_eps=1e-6, norm_eps=1e-2), dict(scale=3.0, qk_eps=2.0, norm_eps=5.0)):
        for n, v in values.items():
            t[n].fill_(v)
        got, want = run(x, entry, **t), run(x, entry, **values)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("entry", ENTRIES)
def test_a_pool_without_slots_is_refused(entry):
    """It is no missing pool, with which sequences start from zeros."""
    import torch
    import chunked_gated_delta_gdr_amd as G
    x = R.make([3, 2], slots=2, index=[0, 1], seed=83)
    with pytest.raises((ValueError, G.GdrError)):
        run(dict(x, pool=x["pool"][:0]), entry)


@pytest.mark.parametrize("entry", ENTRIES)
@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("size", [1e-12, 1e-20, 1e-24, 1e-30])
def test_tiny_keys_under_the_norm(entry, io, size):
    """Keys and queries far below eps's root: k / sqrt(eps), as small as it is."""
    import torch
    x = R.make([70, 2], Dk=64, Dv=32, io=io, qk_norm=True, has=[False, False], seed=82)
    for n in "qk":
        x[n] = (x[n].double() * size).to(x[n].dtype)
    x["scale"] = 1.0 / (1e3 * size)   # (outputs of v's size times k's)
    out, pool = run(x, entry)
    ref_o, ref_p = R.delta(normalised(x, 1e-6), torch.zeros(x["v"].shape))
    assert R.rel(pool, ref_p) <= R.state_tol(70)
    if size >= 1e-12:   # (beyond, the output's own products leave fp32's range or io's)
        assert R.rel(out, ref_o) <= io_tol(x, entry) + R.state_tol(70)


@pytest.mark.parametrize("entry", ENTRIES)
@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("name", ["q", "k", "v", "beta", "log_alpha", "pool"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("at", [0, 20, 63, 64, 69])
def test_what_is_not_finite_reaches_no_earlier_token(entry, io, name, bad, at):
    """The tokens in front keep their values, and of a bad value or state row the other value channels."""
    import torch
    if name == "log_alpha" and bad > 0:
        pytest.skip("log_alpha <= 0")
    x = R.make([70, 5], Hk=2, Hv=4, Dk=64, Dv=64, io=io, seed=94)
    ref_o, ref_p = R.delta(x, torch.zeros(x["v"].shape))
    y = dict(x, **{name: x[name].clone()})
    if name == "pool":
        y["pool"][0, 1, 3, 5] = bad
    elif name == "v":
        y["v"][at, 1, 3] = bad
    else:
        y[name][at, 0] = bad
    out, pool = run(y, entry)
    tol = io_tol(x, entry) + R.state_tol(70)
    if name != "pool" and at > 0:
        assert R.rel(out[:at], ref_o[:at]) <= tol
    assert R.rel(out[70:], ref_o[70:]) <= tol and R.rel(out[:, 2:], ref_o[:, 2:]) <= tol
    assert R.rel(pool[1], ref_p[1]) <= R.state_tol(70) and R.rel(pool[:, 2:], ref_p[:, 2:]) <= R.state_tol(70)
    if name in ("v", "pool"):
        rest = [c for c in range(64) if c != 3]
        assert R.rel(out[:, :, rest], ref_o[:, :, rest]) <= tol
        assert R.rel(pool[:, :, rest], ref_p[:, :, rest]) <= R.state_tol(70)
        assert not torch.isfinite(out[at if name == "v" else 0:70, 1, 3].float()).any()
    elif name == "q":
        rest = [i for i in range(75) if i != at]
        assert R.rel(out[rest], ref_o[rest]) <= tol and R.rel(pool, ref_p) <= R.state_tol(70)
    else:
        assert not torch.isfinite(out[at:70, 0].float()).all() and not torch.isfinite(pool[0, 0]).all()


def decays(x):
    """How far the decays of a sequence may be off: e^x takes x with a rounding of 2^-24 of itself."""
    la = x["log_alpha"].double()
    return 2.0 ** -24 * float((-la).clamp(max=100).sum(0).max())


def row_sizes(x):
    """Of every token and head, the size that its output S q has where q is as far from S's large directions as
    a random one: |S| scale / sqrt(Dv), in 64 bits."""
    import math
    import torch
    k, v = x["k"].double(), x["v"].double()
    k = k.repeat_interleave(v.shape[1] // k.shape[1], 1)
    sizes, t = torch.zeros(v.shape[:2], dtype=torch.float64), 0
    for s, n in enumerate(x["lens"]):
        S = x["pool"][s].double() * (1.0 if x["has"] is None else float(x["has"][s]))
        for i in range(t, t + n):
            S = S * x["log_alpha"][i].double().exp()[:, None, None]
            d = x["beta"][i].double()[:, None] * (v[i] - torch.matmul(S, k[i][:, :, None])[..., 0])
            S = S + d[:, :, None] * k[i][:, None, :]
            sizes[i] = S.square().sum((1, 2)).sqrt() * x["scale"] / math.sqrt(v.shape[2])
        t += n
    return sizes


def check_rows(x, entry, rows, out, ref):
    """Every row and head by itself.  A row is S q with a unit q: a relative error e of the products' factors leaves
    e |S| |q| at most (Cauchy-Schwarz), which is row_sizes, however small the row is by q's direction.  e: a
    rounding of 2^-12 for each of the three one-part factors of a bf16 output (2^-11, adding like their root);
    four state tolerances, one for S and three for the products; each decay's own rounding."""
    import torch
    err = (out.double() - ref).square().mean(-1).sqrt()[rows]
    part = 2.0 ** -11 if entry == "mfma" and x["v"].dtype == torch.bfloat16 else 0.0
    tol = R.half_step(x["v"].dtype) * ref.square().mean(-1).sqrt() + (part + 4 * R.state_tol(max(x["lens"])) + decays(x)) * row_sizes(x)
    assert (err <= tol[rows]).all(), float((err / tol[rows]).max())


@pytest.mark.parametrize("entry", ENTRIES)
@pytest.mark.parametrize("io", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("big", [1e4, 1e6, 1e8, 1e12, 1e20])
@pytest.mark.parametrize("what", ["state", "value"])
@pytest.mark.parametrize("how", ["reset", "decays"])
@pytest.mark.parametrize("dims", [(64, 64), (128, 40)], ids=str)
def test_what_decays_leaves_no_trace(entry, io, big, what, how, dims):
    """A state or a value far larger than the rest, gone again within its chunk: what follows is
    as exact as it is without."""
    if io == "f16" and what == "value" and big > 1e4:
        pytest.skip("beyond fp16")
    x = R.make([70, 2, 64], Dk=dims[0], Dv=dims[1], io=io, seed=91)
    if what == "state":
        x["pool"] = x["pool"] * big
    else:
        x["v"][[7, 79]] = (x["v"][[7, 79]].double() * big).to(x["v"].dtype)
    import math
    for start in (0, 72):
        if how == "reset":
            x["log_alpha"][start + 20] = float("-inf")
        else:
            x["log_alpha"][start + 10:start + 26] = -1.25 * math.log(big) / 16
    import torch
    out, pool = run(x, entry)
    ref_o, ref_p = R.delta(x, torch.zeros(x["v"].shape))
    for s in (0, 2):
        assert R.rel(pool[s], ref_p[s]) <= R.state_tol(70) + decays(x)
    rows = torch.ones(136, dtype=torch.bool)
    if io == "f16":   # (rows that fp16 does not hold)
        rows = (ref_o.abs().amax((1, 2)) < 6e4)
    check_rows(x, entry, rows, out, ref_o)


@pytest.mark.parametrize("entry", ENTRIES)
@pytest.mark.parametrize("io", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("big", [1e4, 1e6, 1e9, 1e15])
@pytest.mark.parametrize("has", [False, True])
def test_what_comes_later_leaves_no_trace(entry, io, big, has):
    """A large value costs the tokens before it nothing."""
    import torch
    if io == "f16" and big > 1e4:
        pytest.skip("beyond fp16")
    x = R.make([70, 2, 64], Dk=64, Dv=64, io=io, has=[has] * 3, seed=92)
    x["v"][[40, 100]] = (x["v"][[40, 100]].double() * big).to(x["v"].dtype)
    out, pool = run(x, entry)
    ref_o, ref_p = R.delta(x, torch.zeros(x["v"].shape))
    assert R.rel(pool, ref_p) <= R.state_tol(70)
    check_rows(x, entry, [i for i in range(136) if i < 40 or 70 <= i < 100], out, ref_o)


@pytest.mark.parametrize("entry", ENTRIES)
@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("step", [-0.05, -0.3, -1.0, -3.0, -20.0])
def test_decays_of_every_size(entry, io, step):
    """Values alike in size under weak to strong decays, some heads with each."""
    import torch
    x = R.make([200, 64, 1, 65], Hk=2, Hv=4, Dk=64, Dv=64, io=io, seed=93)
    x["log_alpha"] = (x["log_alpha"] * 0 + step) * torch.rand(x["log_alpha"].shape, generator=torch.Generator().manual_seed(5)) * 2
    x["log_alpha"][:, 1] = 0.0
    out, pool = run(x, entry)
    ref_o, ref_p = R.delta(x, torch.zeros(x["v"].shape))
    # (each token's decay is a rounding of 2^-24 of its exponent; what is older than a few tokens is gone under a strong one)
    tol = R.state_tol(200) + 2.0 ** -24 * min(80.0, -step * 200)
    assert R.rel(pool, ref_p) <= tol
    assert R.rel(out, ref_o) <= io_tol(x, entry) + tol


@pytest.mark.parametrize("entry", ENTRIES)
@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("size", [1e3, 1e8, 1e15, 1e25])
def test_keys_that_grow_out_of_the_chunk(entry, io, size):
    """Keys far from units, with which a chunk's inverse leaves fp32: the tokens in front know nothing of it."""
    import torch
    x = R.make([70, 3], Dk=64, Dv=64, io=io, seed=95)
    ref_o, _ = R.delta(x, torch.zeros(x["v"].shape))
    x["k"][30:64] = (x["k"][30:64].double() * size).to(x["k"].dtype)
    out, _ = run(x, entry)
    tol = io_tol(x, entry) + R.state_tol(70)
    assert R.rel(out[:30], ref_o[:30]) <= tol and R.rel(out[70:], ref_o[70:]) <= tol


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("size", [1e10, 1e25, 1e31, 1e37])
def test_huge_keys_under_the_norm(io, size):
    """Chunked, each row on its own scale: up to the type's largest (sums of squares would end at 1e19)."""
    import torch
    x = R.make([70, 2], Dk=64, Dv=32, io=io, qk_norm=True, seed=87)
    for n in "qk":
        x[n] = (x[n].double() / x[n].double().abs().amax(-1, keepdim=True) * size).to(x[n].dtype)
    out, pool = run(x, "mfma")
    ref_o, ref_p = R.delta(normalised(x, 1e-6), torch.zeros(x["v"].shape))
    assert R.rel(pool, ref_p) <= R.state_tol(70) and R.rel(out, ref_o) <= io_tol(x, "mfma") + R.state_tol(70)


@pytest.mark.parametrize("entry", ENTRIES)
@pytest.mark.parametrize("io", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("heads,dims,shift", [((2, 6), (72, 24), 3), ((20, 40), (128, 64), 1), ((40, 40), (64, 48), 0), ((1, 2), (8, 8), 1)],
                         ids=str)
def test_some_columns_token_by_token(entry, io, heads, dims, shift):
    """States of 1e8 in some value channels, reset in the first and in the third chunk, over views of a wider
    projection, pooled slots and more workgroups than CUs: each channel to its own size, and the rows."""
    import torch
    from test_gpu_packed import call
    x = R.make([200, 70, 1, 0, 66], Hk=heads[0], Hv=heads[1], Dk=dims[0], Dv=dims[1], io=io, slots=7, index=[6, 0, 3, 2, 1],
               qk_norm=True, seed=96)
    x["pool"][:, :, 3::16] *= 1e8
    for start in (0, 128, 200, 271):
        x["log_alpha"][start + 30] = float("-inf")
    out, pool = (t.cpu() for t in call(x, entry, wide=True, shift=shift))
    ref_o, ref_p = R.delta(x, torch.full(x["v"].shape, 7.0))
    for c in range(dims[1]):
        assert R.rel(pool[[6, 0, 1], :, c], ref_p[[6, 0, 1], :, c]) <= 2 * R.state_tol(200), c
    assert torch.equal(pool[[2, 4, 5]], x["pool"][[2, 4, 5]])
    after = [i for i in range(337) if 30 <= i < 200 or 230 <= i < 270 or i >= 301]
    assert R.rel(out[after], ref_o[after]) <= io_tol(x, entry) + 2 * R.state_tol(200)
