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
