"""GPU edges of the block operators: the activations at infinities, NaN and in their tails, and
single rows.  Bounds: see ops_reference.py, or beside the test."""
import pytest
import torch

import ops_reference as R
from ring_all_gather_amd import binding as B

from gpu_common import DEV, ctx
from test_gpu_ops import BF16, F32, empty, gen, normal

pytestmark = pytest.mark.gpu
INF, NAN = float("inf"), float("nan")


def values(*v):
    return torch.tensor(v, device=DEV).to(BF16)


def forward(z, name):
    """act(z) of a bf16 vector by fused_linear: no products, the bias alone."""
    M = z.numel()
    X, W = torch.zeros(1, 64, dtype=BF16, device=DEV), torch.zeros(M, 64, dtype=BF16, device=DEV)
    Y, Z = empty(1, M), empty(1, M)
    B.fused_linear(ctx(), X, W, Y, bias=z, act=name, Z=Z)
    assert torch.equal(torch.nan_to_num(Z[0]), torch.nan_to_num(z))
    return Y[0]


def backward(z, name):
    """(act(z), act'(z)) of a bf16 vector by gated_ffn_backward with dH = U = X = 1, T = 1: its dU
    and dG, each rounded to bf16."""
    F = z.numel()
    one = torch.ones(1, F, dtype=BF16, device=DEV)
    X, W = torch.ones(1, 64, dtype=BF16, device=DEV), torch.zeros(F, 64, dtype=BF16, device=DEV)
    dWg, dWu = empty(F, 64), empty(F, 64)
    B.gated_ffn_backward(ctx(), one, X, W, W, z[None], one, dWg=dWg, dWu=dWu, act=name)
    return dWu[:, 0], dWg[:, 0]


@pytest.mark.parametrize("name", R.ACTS)
def test_activations_at_the_ends_of_the_range(name):
    """Where z is infinite or huge, the value is the formula's in the forward and the backward
    pass alike (NaN where it is -inf * 0); the slope at infinity is its limit."""
    z = values(-INF, INF, -3e38, 3e38, -1e30, 1e30, -200.0, 200.0, 0.0, 1.0)
    want = R.act(z.double(), name)
    bound = R.BF * want.abs() + R.ACT_ERR[0] * want.abs() + R.ACT_ERR[1]
    value, slope = backward(z, name)
    R.check(forward(z, name), want, bound, "forward")
    R.check(value, want, bound, "value in the backward pass")
    ends = torch.ones(8, dtype=torch.float64, device=DEV)
    if name != "none":
        ends[::2] = 0.0
    assert torch.equal(slope[:8].double(), ends)


@pytest.mark.parametrize("name", R.ACTS)
def test_nan_stays_nan(name):
    """A NaN pre-activation gives NaN, in the value and in every gradient that passes through it."""
    z = values(NAN, 1.0, -1.0)
    assert forward(z, name).isnan().tolist() == [True, False, False]
    value, slope = backward(z, name)
    assert value.isnan().tolist() == [True, False, False]
    if name == "none":
        return   # its slope does not read z
    assert slope.isnan().tolist() == [True, False, False]
    X, W = torch.ones(1, 64, dtype=BF16, device=DEV), torch.ones(3, 64, dtype=BF16, device=DEV)
    dY, dW, db = torch.ones(1, 3, dtype=BF16, device=DEV), empty(3, 64), empty(3, dtype=F32)
    B.fused_linear_backward(ctx(), dY, X, W, dW=dW, dbias=db, act=name, Z=z[None])
    assert db.isnan().tolist() == [True, False, False]
    assert dW.isnan().all(1).tolist() == [True, False, False]


@pytest.mark.parametrize("name", ["gelu", "gelu_tanh", "silu"])
def test_tails_of_the_activations(name):
    """Values far below zero are good to their own size: bf16's rounding, and relative errors of
    2^-19 of the approximations and of 8 roundings of an exponent, which grow with it."""
    z = torch.linspace(-12.0, 0.0, 4001, device=DEV).to(BF16).unique()
    d = z.double()
    want = {"gelu": 0.5 * d * torch.erfc(-d / 2 ** 0.5),
            "gelu_tanh": d * torch.sigmoid(2 * (2 / torch.pi) ** 0.5 * (d + 0.044715 * d ** 3)),
            "silu": d * torch.sigmoid(d)}[name]
    power = {"gelu": d * d / 2, "gelu_tanh": 1.6 * (d.abs() + 0.0448 * d.abs() ** 3),
             "silu": d.abs()}[name]
    bound = want.abs() * (R.BF + 1.01 * (2.0 ** -19 + 8 * R.U32 * (power + 1)))
    normal_range = want.abs() > 2.0 ** -120   # smaller factors may be flushed to zero
    for got in (forward(z, name), backward(z, name)[0]):
        R.check(got[normal_range], want[normal_range], bound[normal_range], name)


# ------------------------------------------------------------------------------- single rows

def far(t, stride):
    """The one-row matrix t with another row stride, which no access may take into account."""
    assert t.shape[0] == 1
    return t.as_strided(t.shape, (stride, 1))


@pytest.mark.parametrize("stride", [131, 1 << 24, 1 << 33])
def test_one_row_of_any_stride(stride):
    """A single row has no second one, so its stride is not looked at: the last token of a long
    sequence, or a row of a matrix whose stride is no multiple of 16 bytes."""
    g = gen(51)
    K, N = 128, 70
    X, W, V = normal(g, 1, K), normal(g, N, K, std=0.1), normal(g, N, K, std=0.1)
    r, dY = normal(g, 1, N), normal(g, 1, N)
    w, b = normal(g, K), normal(g, K)

    def run(change):
        Y, Z, H, G, U = (empty(1, N) for _ in range(5))
        B.fused_linear(ctx(), change(X), W, Y, act="silu", residual=change(r), Z=Z)
        B.gated_ffn(ctx(), change(X), W, V, H, G=G, U=U)
        out = [Y, Z, H, G, U]
        for act in ("none", "silu"):
            dX, dW, dV, db = empty(1, K), empty(N, K), empty(N, K), empty(N, dtype=F32)
            B.fused_linear_backward(ctx(), change(dY), change(X), W, dX=dX, dW=dW, dbias=db,
                                    act=act, Z=None if act == "none" else Z)
            out += [dX.clone(), dW.clone(), db]
            B.gated_ffn_backward(ctx(), change(dY), change(X), W, V, G, U, dX=dX, dWg=dW, dWu=dV,
                                 act=act)
            out += [dX, dW, dV]
        y, mean, rstd = empty(1, K), empty(1, dtype=F32), empty(1, dtype=F32)
        B.layer_norm(ctx(), change(X), w, b, y, mean=mean, rstd=rstd)
        dx, dw, dn = empty(1, K), empty(K, dtype=F32), empty(K, dtype=F32)
        B.layer_norm_backward(ctx(), change(y), change(X), w, mean, rstd, dx, dw, dn)
        return out + [y, mean, rstd, dx, dw, dn]

    for got, want in zip(run(lambda t: far(t, stride)), run(lambda t: t)):
        assert not want.isnan().any() and torch.equal(got, want)


def test_one_row_residual_in_place():
    g = gen(52)
    X, W, r = normal(g, 1, 128), normal(g, 70, 128, std=0.1), normal(g, 1, 70)
    want, Y = empty(1, 70), r.clone()
    B.fused_linear(ctx(), X, W, want, act="silu", residual=r)
    B.fused_linear(ctx(), X, W, Y, act="silu", residual=far(Y, 73))
    assert torch.equal(Y, want)
