"""A sublayer's training step through the library: read with pre-norm, gated residual, their backwards, clipping.

The sublayer between the pre-norm and its output is an elementwise square, so that its gradient is elementary. fp32
storage throughout; the whole chain is compared with autograd in fp64 (bound: the library's fp32 tolerance for
a read and its backward, 1e-5 of the largest gradient, as the read's own tests, twice for the chain of two).
"""
import pytest
import torch

from depth_wise_attention_attnres_gb300 import binding as ar
from depth_wise_attention_attnres_gb300 import inputs
from tests import _residual as ref
from tests._gpu import TOL, dev, rel_err

pytestmark = pytest.mark.gpu
EPS = 1e-5


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()


@pytest.mark.parametrize("T,d,n", [(100, 256, 4), (37, 640, 6), (20, 100, 3)])
def test_training_step(T, d, n):
    g = inputs.generator(T, dev())
    V = inputs.history(n, T, d, "f32", g, dev())
    w, gamma = inputs.queries(1, d, 0.05, g, dev())[0].contiguous(), 1 + 0.3 * inputs.queries(1, d, 1.0, g, dev())[0]
    gpre, gpost = (1 + 0.3 * inputs.queries(1, d, 1.0, g, dev())[0] for _ in range(2))
    gnext = 1 + 0.3 * inputs.queries(1, d, 1.0, g, dev())[0]
    gate = inputs.randn((1, d), "f32", g, dev())
    target_n, target_x = inputs.randn((T, d), "f32", g, dev()), inputs.randn((T, d), "f32", g, dev())

    # Forward: z and its pre-norm, f = a^2, the stream z + 0.5 sigmoid(gate) RMSNorm(f), the next pre-norm.
    z, a, f = (torch.empty(T, d, device=dev()) for _ in range(3))
    ar.attnres_full_fwd_prenorm(V, n, w, gamma, EPS, gpre, EPS, z, a)
    torch.mul(a, a, out=f)
    xo, nxt = torch.empty_like(z), torch.empty_like(z)
    ar.attnres_gated_residual(f, z, gpost, EPS, gate, T, ar.GATE_SIGMOID, 0.5, xo, gnext, EPS, nxt)
    # Backward of L = <target_x, xo> + <target_n, nxt>.
    df, dz, dgate = torch.empty_like(f), torch.empty_like(z), torch.empty_like(gate)
    grads = {k: torch.zeros(d, device=dev()) for k in ("gpost", "gnext", "gpre", "w", "gamma")}
    dV = torch.zeros(n, T, d, device=dev())
    ar.attnres_gated_residual_bwd(f, gpost, EPS, gate, T, ar.GATE_SIGMOID, 0.5, xo, gnext, EPS, target_x, target_n, df, dz,
                                  dgate, grads["gpost"], grads["gnext"])
    ar.attnres_rmsnorm_bwd(z, gpre, EPS, df * 2 * a, dz, dz, grads["gpre"])
    ar.attnres_full_bwd(V, n, w, gamma, EPS, dz, dV, grads["w"], grads["gamma"])

    # The same in fp64 by autograd.
    leaf = {k: v.double().requires_grad_() for k, v in dict(V=V, w=w, gamma=gamma, gpre=gpre, gpost=gpost, gnext=gnext,
                                                            gate=gate).items()}

    def rms(x, gain):
        return gain * x / torch.sqrt((x * x).mean(-1, keepdim=True) + EPS)
    alpha = (rms(leaf["V"], leaf["gamma"]) * leaf["w"]).sum(-1).softmax(0)
    z64 = (alpha[..., None] * leaf["V"]).sum(0)
    f64 = rms(z64, leaf["gpre"]) ** 2
    x64 = z64 + 0.5 * torch.sigmoid(leaf["gate"]) * rms(f64, leaf["gpost"])
    n64 = rms(x64, leaf["gnext"])
    (x64 * target_x.double()).sum().add((n64 * target_n.double()).sum()).backward()
    tol = 2 * TOL["f32"]
    assert rel_err(xo, x64.detach().cpu()) <= tol and rel_err(nxt, n64.detach().cpu()) <= tol
    got = dict(grads, V=dV, gate=dgate)
    for k, t in got.items():
        assert rel_err(t, leaf[k].grad.cpu()) <= tol, k

    # The parameters' gradients clipped to half their norm, in place.
    params = [got[k] for k in ("gpost", "gnext", "gpre", "w", "gamma", "gate")]
    want = ref.norm_of(params)
    norm = torch.empty(1, device=dev())
    ar.attnres_grad_clip(params, want / 2, norm)
    assert abs(float(norm) - want) <= 1e-5 * want
    assert abs(ref.norm_of(params) - want / 2) <= 1e-5 * want
    assert ar.attnres_device_status() == 0
