"""The norms away from their defaults: eps = 0, infinite values under 8-bit outputs, far gates."""
import pytest

import _packed_ref as R
from test_gpu_norm import GATE, STAT, dev, make

pytestmark = pytest.mark.gpu


# widths of every number of lanes a row up to 64, which share a workgroup with other rows, and one wider
@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("loads", [1, 8, 16, 31, 33, 48, 64, 65, 96, 128, 129, 192, 193, 256])
@pytest.mark.parametrize("rows", [1, 5, 33])
@pytest.mark.parametrize("gate", [False, True])
def test_gradient_without_eps(io, loads, rows, gate):
    """Lanes without a row add nothing to the weight's gradient, whatever 1 / sqrt(0) is."""
    import torch
    import chunked_gated_delta_gdr_amd as G
    D = loads * (4 if io == "f32" else 8) - loads % 2
    x = make(rows, D, io, gate=gate, seed=rows + D)
    dy = torch.randn(rows, D, generator=torch.Generator().manual_seed(3), dtype=torch.float64).to(R.IO[io])
    leaves = [x[n].double().requires_grad_() for n in ("x", "weight", "gate") if x[n] is not None]
    y, _ = R.norm(leaves[0], weight=leaves[1], gate=leaves[2] if gate else None, eps=0.0)
    grads = torch.autograd.grad((y * dy.double()).sum(), leaves)
    d = dev(x)
    got = G.gdr_rms_norm_bwd(d["x"], dy.cuda(), weight=d["weight"], gate=d["gate"], eps=0.0)
    out = G.gdr_rms_norm(d["x"], weight=d["weight"], gate=d["gate"], eps=0.0)[0]
    half = R.half_step(R.IO[io])
    assert R.rel(out.cpu(), y.detach()) <= half + STAT + GATE
    n = leaves[0].detach() / leaves[0].detach().square().mean(-1, keepdim=True).sqrt()
    act = 1.0 if not gate else (x["gate"].double() * torch.sigmoid(x["gate"].double())).abs()
    size = (dy.double().abs() * act * n.abs()).sum(0)
    assert ((got["dweight"].cpu().double() - grads[1]).abs() <= 2 * (STAT + GATE) * size + 1e-30).all()
    u = dy.double().abs() * x["weight"].double().abs() * act
    r = 1 / leaves[0].detach().square().mean(-1, keepdim=True).sqrt()
    terms = r * (u + n.abs() * (u * n.abs()).mean(-1, keepdim=True))
    err = (got["dx"].cpu().double() - grads[0]).abs()
    assert (err <= half * grads[0].abs() + 2 * (STAT + GATE) * terms + 2.0 ** -24).all()
    if gate:
        assert torch.isfinite(got["dgate"].float()).all()


def test_eps_may_be_a_tensor_that_changes():
    """Its value at the call counts, not the one that an earlier call met."""
    import torch
    import chunked_gated_delta_gdr_amd as G
    d = dev(make(3, 40, "f32", seed=2))
    eps = torch.tensor(0.0)
    for value in (1e-6, 3.0, 100.0):
        eps.fill_(value)
        assert torch.equal(G.gdr_rms_norm(d["x"], eps=eps)[0], G.gdr_rms_norm(d["x"], eps=value)[0])
        assert torch.equal(G.gdr_rms_norm_bwd(d["x"], d["x"], eps=eps)["dx"], G.gdr_rms_norm_bwd(d["x"], d["x"], eps=value)["dx"])


@pytest.mark.parametrize("codes", ["int8", "float8_e4m3fn"])
@pytest.mark.parametrize("bad", [float("inf"), float("-inf")])
def test_eight_bit_codes_beside_an_infinity(codes, bad):
    """An infinite value makes its row's scale infinite and the finite ones' codes 0, and nothing else of it."""
    import torch
    import chunked_gated_delta_gdr_amd as G
    for D in (7, 300, 2048):
        x = make(4, D, "f32", gate=True, weight=False, seed=D)
        x["gate"] = x["gate"].abs() + 0.1
        want = [t.cpu() for t in G.gdr_rms_norm(out_dtype=getattr(torch, codes), **dev(x))[:2]]
        x["x"][2, 5] = x["x"][2, 5].abs() + 0.1
        x["gate"][2, 5] = abs(bad)   # silu(inf) = inf
        x["x"][2, 5] *= 1.0 if bad > 0 else -1.0
        out, scales = (t.cpu() for t in G.gdr_rms_norm(out_dtype=getattr(torch, codes), **dev(x))[:2])
        assert scales[2] == float("inf")
        rest = [i for i in range(D) if i != 5]
        assert (out[2, rest].float() == 0).all()
        keep = [0, 1, 3]
        assert torch.equal(out[keep].view(torch.uint8), want[0][keep].view(torch.uint8)) and torch.equal(scales[keep], want[1][keep])


@pytest.mark.parametrize("D", [64, 1000, 4096])
def test_far_gates_in_fp32(D):
    """silu and its slope keep fp32's relative precision out to where the exponential leaves the type."""
    import torch
    import chunked_gated_delta_gdr_amd as G
    x = make(9, D, "f32", gate=True, seed=D)
    x["gate"] = (torch.arange(9 * D, dtype=torch.float64).reshape(9, D) / (9 * D) * 160 - 80).float()
    d = dev(x)
    y, _ = R.norm(**x)
    # one rounding, the row's statistic, and 8 roundings of exp, the sum, the reciprocal and the products
    tol = R.half_step(torch.float32) * (1 + 8) + STAT
    err = (G.gdr_rms_norm(**d)[0].cpu().double() - y).abs()
    assert (err <= tol * y.abs()).all(), float((err / y.abs()).max() * 2.0 ** 24)
    # the slope sg (1 + z (1 - sg)): where z < -2 its two terms differ in size by z, no cancellation
    z = x["gate"].double()
    dy = torch.ones_like(x["x"])
    got = G.gdr_rms_norm_bwd(d["x"], dy.cuda(), weight=d["weight"], gate=d["gate"])["dgate"].cpu().double()
    h = x["x"].double()
    sg = torch.sigmoid(z)
    ref = h / (h.square().mean(-1, keepdim=True) + 1e-6).sqrt() * x["weight"].double() * sg * (1 + z * (1 - sg))
    far = z < -4
    assert ((got - ref).abs()[far] <= 2 * tol * ref.abs()[far]).all()
