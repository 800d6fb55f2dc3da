"""The gradient of the gated recurrence's rates at full size and on long rows.
Bounds as in test_gpu_causal.py."""
import math

import pytest
import torch

import model_ref as ref
from gpu_util import say
from test_gpu_causal import close
from test_gpu_gated import doubles, make
from test_gpu_model_use import FULL

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("shape", FULL, ids=lambda s: "b%d-d%d-L%d" % s[:3])
def test_dlam_full_size(shape, dtype):
    """dlam of sampled channels against float64, over every row of the batch."""
    import vision_mamba_selective_amd as vms
    batch, dim, L, short = shape
    lengths = None if short == L else [L - (L - short) * i // max(1, batch - 1) for i in range(batch)]
    t = make(91, dtype, batch, dim, L, lengths, True, False)
    say("case gated dlam full size %s %s" % (shape, dtype))
    args, kw = (t["x"], t["r"], t["i"], t["lam"]), dict(z=t["z"], h0=t["h0"], lengths=t["lengths"])
    _, _, saved = vms.gated_scan_saved(*args, **kw)
    got = vms.gated_scan_grad(*args, saved, t["dy"], dh=t["dh"], **kw)["dlam"]
    chans = sorted({0, dim // 2 + 1, dim - 1})
    d = doubles({k: t[k][:, chans] for k in ("x", "r", "i", "z", "h0", "dy", "dh")} | {"lam": t["lam"][chans]})
    y, h = ref.gated(d["x"], d["r"], d["i"], d["lam"], d["z"], d["h0"], lengths)
    close(got[chans], ref.gradients([y, h], [d["dy"].detach(), d["dh"].detach()], [d["lam"]])[0], "dlam")


@pytest.mark.parametrize("shape", [(1, 1, 1 << 24), (1, 600, 1 << 18), (3, 700, 1 << 17)], ids=str)
def test_dlam_of_long_rows_of_equal_terms(shape):
    """Equal tokens, so that the state settles and every term of dlam is the same:
    32,768 of them one after another in fp32 are off by 3e-4 of their sum. In
    blocks and 64 bits each term's own few roundings are left. The reference is
    the closed form: h_t = v (1 - a^(t+1)) / (1 - a), and the adjoint alike."""
    import vision_mamba_selective_amd as vms
    batch, dim, L = shape
    say("case gated dlam long rows %s" % (shape,))
    lam = torch.full((dim,), -3.0, device="cuda")
    x, zero = torch.ones(shape, device="cuda"), torch.zeros(shape, device="cuda")
    _, _, saved = vms.gated_scan_saved(x, zero, zero, lam)
    got = vms.gated_scan_grad(x, zero, zero, lam, saved, x)["dlam"]
    k = 8 * math.log1p(math.exp(-3.0))
    s, gate = k / 2, 0.5
    a, m = math.exp(-s), math.sqrt(-math.expm1(-2 * s))
    t = torch.arange(L, dtype=torch.float64)
    back = -torch.expm1(-s * (L - t)) / (1 - a)
    before = -torch.expm1(-s * t) / (1 - a) * m * gate
    terms = s * back * (a * a * gate / m - a * before)
    want = batch * float(terms.sum()) / (1 + math.exp(3.0)) / math.log1p(math.exp(-3.0))
    close(got, torch.full((dim,), want, dtype=torch.float64), "dlam")
