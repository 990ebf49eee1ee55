"""GPU parity of the block operators' products on every kernel that the planner gives them: tiles of
each size, whole and half, with K split and not, and the forms for few rows, at ragged rows and
columns of every alignment.  Beside each size stands the kernel with its workgroups (whole tiles /
half tiles / splits of K) on 256 compute units, so that a change of the planner's constants cannot
take a kernel out of the tests unseen.

Inputs are small integers (times powers of two where a scale is allowed), whose sums are exact in
fp32 in any order, so every output has to equal the rounded 64-bit result bit by bit."""
import ctypes

import pytest
import torch

from ring_all_gather_amd import binding as B

from gpu_common import DEV, ctx, say
from test_gpu_ops import BF16, F32, empty, gen, ints, strided

pytestmark = pytest.mark.gpu
BF, FP8 = "bf16", "fp8"
E4M3 = torch.float8_e4m3fn

FUSED_LINEAR = [
    (4200, 4360, 256, BF, "t256 256/100/1"),
    (4200, 4364, 256, BF, "t256 256/100/1"),
    (4200, 4358, 256, BF, "t256 256/100/1"),
    (4200, 4357, 256, BF, "t256 256/100/1"),
    (4200, 4360, 256, FP8, "t256 256/100/1"),
    (4200, 4364, 256, FP8, "t256 256/100/1"),
    (4200, 4358, 256, FP8, "t256 256/100/1"),
    (4200, 4357, 256, FP8, "t256 256/100/1"),
    (541, 7205, 128, BF, "t256 0/174/1"),
    (3653, 1070, 128, FP8, "t256 0/150/1"),
    (2050, 4358, 1024, BF, "t256 162/0/1"),
    (4568, 1801, 128, FP8, "t256 144/0/1"),
    (100, 50001, 128, BF, "t128 391/0/1"),
    (100, 50002, 128, BF, "t128 391/0/1"),
    (100, 50001, 128, FP8, "t128 391/0/1"),
    (100, 50004, 128, FP8, "t128 391/0/1"),
    (100, 333, 8192, BF, "t128d 96/0/32"),
    (100, 130, 8192, BF, "t128d 64/0/32"),
    (77, 132, 4096, BF, "t128d 64/0/32"),
    (77, 136, 4096, BF, "t128d 64/0/32"),
    (100, 333, 8192, FP8, "t128d 48/0/16"),
    (100, 130, 8192, FP8, "t128d 64/0/32"),
    (77, 517, 2048, FP8, "t128d 40/0/8"),
    (9, 8230, 128, BF, "few16x2"),
    (9, 8230, 128, FP8, "few16x2"),
    (17, 130, 256, BF, "few32"),
    (17, 130, 256, FP8, "few32"),
]

GATED_FFN = [
    (4200, 4360, 256, BF, "t256 512/166/1"),
    (4200, 4364, 256, BF, "t256 512/166/1"),
    (4200, 4358, 256, BF, "t256 512/166/1"),
    (4200, 4357, 256, BF, "t256 512/166/1"),
    (4200, 4360, 256, FP8, "t256 512/166/1"),
    (4200, 4364, 256, FP8, "t256 512/166/1"),
    (4200, 4358, 256, FP8, "t256 512/166/1"),
    (4200, 4357, 256, FP8, "t256 512/166/1"),
    (1411, 2307, 512, BF, "t256 0/228/1"),
    (2981, 889, 128, FP8, "t256 0/168/1"),
    (3968, 1043, 128, BF, "t256 144/0/1"),
    (1269, 3307, 128, FP8, "t256 130/0/1"),
    (100, 50001, 128, BF, "t128 782/0/1"),
    (100, 50002, 128, BF, "t128 782/0/1"),
    (100, 50001, 128, FP8, "t128 782/0/1"),
    (100, 333, 8192, BF, "t128d 96/0/16"),
    (100, 130, 8192, BF, "t128d 96/0/32"),
    (100, 333, 8192, FP8, "t128d 96/0/16"),
    (100, 130, 8192, FP8, "t128d 96/0/32"),
    (9, 8230, 128, BF, "few16x2"),
    (9, 8230, 128, FP8, "few16x2"),
    (17, 130, 256, BF, "few32"),
    (17, 130, 256, FP8, "few32"),
]

FUSED_LINEAR_BACKWARD = [
    (5973, 71, 512, "t128 dx 188/0/1 dw 128/0/32"),
    (1411, 2310, 2048, "t128 dx 192/0/1 dw 304/0/1"),
    (33, 1003, 6656, "t256 dx 104/0/4 dw 104/0/1"),
    (100, 3148, 768, "t128d dx 96/0/16 dw 150/0/1"),
    (5371, 1753, 128, "t128 dx 168/0/4 dw 112/0/8"),
    (796, 668, 5376, "t256 dx 0/168/1 dw 63/0/1"),
    (3699, 273, 1280, "t256 dx 0/150/1 dw 80/0/8"),
    (705, 569, 8064, "t256 dx 96/0/1 dw 96/0/1"),
    (798, 1651, 6912, "t256 dx 108/0/1 dw 148/82/1"),
    (5327, 73, 1280, "t256 dx 105/0/1 dw 80/0/16"),
    (2367, 1141, 4992, "t256 dx 156/88/1 dw 100/0/1"),
    (7174, 71, 2944, "t256 dx 320/56/1 dw 96/0/8"),
    (202, 3077, 1792, "t256 dx 56/0/8 dw 0/182/1"),
    (100, 1598, 2816, "t128 dx 88/0/4 dw 286/0/1"),
    (65, 5639, 1280, "t256 dx 80/0/16 dw 115/0/1"),
    (4352, 4608, 1024, "t256 dx 68/0/1 dw 0/144/1"),
    (1, 5639, 1280, "t256 dx 160/0/32 dw 96/38/1"),
]

GATED_FFN_BACKWARD = [
    (1818, 75, 1152, "t128 dx 135/0/1 dw 144/0/8"),
    (1411, 2310, 2048, "t128 dx 192/0/1 dw 608/0/1"),
    (100, 981, 896, "t128d dx 56/0/8 dw 112/0/1"),
    (1831, 1306, 256, "t128 dx 120/0/4 dw 176/0/4"),
    (557, 141, 7424, "t256 dx 0/174/1 dw 58/0/1"),
    (2149, 7876, 256, "t256 dx 0/144/8 dw 62/0/1"),
    (638, 324, 6528, "t256 dx 78/0/1 dw 104/0/1"),
    (1207, 857, 5888, "t256 dx 115/0/1 dw 141/86/1"),
    (6531, 245, 896, "t256 dx 104/0/1 dw 64/0/8"),
    (3182, 940, 3456, "t256 dx 144/76/1 dw 112/0/1"),
    (4408, 73, 2048, "t256 dx 128/32/1 dw 128/0/8"),
    (7241, 7258, 1152, "t256 dx 478/204/4 dw 290/0/1"),
    (492, 3525, 768, "t256 dx 48/0/8 dw 0/168/1"),
    (65, 833, 2432, "t128 dx 152/0/8 dw 266/0/1"),
    (65, 3005, 1792, "t256 dx 112/0/16 dw 144/48/1"),
    (1, 3005, 1792, "t256 dx 224/0/32 dw 64/208/1"),
]


def power(v):
    """A scale: 2^v."""
    return torch.tensor([2.0 ** v], device=DEV)


def test_the_tables_name_every_kernel():
    """Every tile and form of each forward product, and each kind of tile of both backward ones."""
    for table in (FUSED_LINEAR, GATED_FFN):
        have = {(t[3], t[4].split()[0]) for t in table}
        assert have >= {(d, k) for d in (BF, FP8)
                        for k in ("t256", "t128", "t128d", "few16x2", "few32")}
        for d in (BF, FP8):
            work = [t[4].split()[1].split("/") for t in table if t[3] == d and "/" in t[4]]
            assert any(int(w[0]) and int(w[1]) for w in work)        # whole and half tiles
            assert any(int(w[2]) > 1 for w in work)                  # K split
    for table in (FUSED_LINEAR_BACKWARD, GATED_FFN_BACKWARD):
        assert {t[3].split()[0] for t in table} == {"t256", "t128", "t128d"}
        for i in (2, 4):
            work = [t[3].split()[i].split("/") for t in table if t[3].startswith("t256")]
            assert any(int(w[1]) for w in work) and any(int(w[2]) > 1 for w in work)


@pytest.mark.parametrize("T,M,K,dtype,plan", FUSED_LINEAR)
def test_fused_linear(T, M, K, dtype, plan):
    say(f"case fused_linear T={T} M={M} K={K} {dtype} {plan}")
    fp8 = dtype == FP8
    assert ctx().ops_kernel_name("fused_linear", T, M, K, fp8) == f"rag_lin_{dtype}_{plan}"
    g = gen(T + M + K)
    X, W = ints(g, T, K), ints(g, M, K)
    b, r = ints(g, M, top=50), ints(g, T, M, top=50)
    z = X.double() @ W.double().t()
    s = {}
    if fp8:
        X, W, s = X.to(E4M3), W.to(E4M3), dict(scale_X=power(-1), scale_W=power(-2))
        z = z / 8
    z = z + b.double()
    want = (z.clamp(min=0) + r.double()).to(BF16)
    Y, Z = empty(T, M), empty(T, M)
    B.fused_linear(ctx(), X if fp8 else strided(X, 8), W, Y, bias=b, act="relu",
                   residual=strided(r, 3), Z=Z, **s)
    assert torch.equal(Z, z.to(BF16))
    assert torch.equal(Y, want)
    Y.copy_(r)   # the residual updated in place, its rows as aligned as the width lets them be
    B.fused_linear(ctx(), X, W, Y, bias=b, act="relu", residual=Y, **s)
    assert torch.equal(Y, want)
    B.fused_linear(ctx(), X, W, Y, **s)
    assert torch.equal(Y, (z - b.double()).to(BF16))


@pytest.mark.parametrize("T,F,K,dtype,plan", GATED_FFN)
def test_gated_ffn(T, F, K, dtype, plan):
    say(f"case gated_ffn T={T} F={F} K={K} {dtype} {plan}")
    fp8 = dtype == FP8
    assert ctx().ops_kernel_name("gated_ffn", T, F, K, fp8) == f"rag_ffn_{dtype}_{plan}"
    g = gen(T + F + K)
    X, Wg, Wu = ints(g, T, K), ints(g, F, K), ints(g, F, K, top=1)
    G64, U64 = X.double() @ Wg.double().t(), X.double() @ Wu.double().t()
    s = {}
    if fp8:
        X, Wg, Wu = X.to(E4M3), Wg.to(E4M3), Wu.to(E4M3)
        s = dict(scale_X=power(-1), scale_Wg=power(-2), scale_Wu=power(1))
        G64 = G64 / 8
    want = (G64.clamp(min=0) * U64).to(BF16)
    H, G, U = empty(T, F), empty(T, F), empty(T, F)
    B.gated_ffn(ctx(), X if fp8 else strided(X, 8), Wg, Wu, H, act="relu", G=G, U=U, **s)
    assert torch.equal(G, G64.to(BF16)) and torch.equal(U, U64.to(BF16))
    assert torch.equal(H, want)
    H.fill_(float("nan"))
    B.gated_ffn(ctx(), X, Wg, Wu, H, act="relu", **s)
    assert torch.equal(H, want)


@pytest.mark.parametrize("dw", [BF16, F32])
@pytest.mark.parametrize("T,M,K,plan", FUSED_LINEAR_BACKWARD)
def test_fused_linear_backward(T, M, K, plan, dw):
    say(f"case fused_linear_backward T={T} M={M} K={K} {dw} {plan}")
    assert ctx().ops_kernel_name("fused_linear_backward", T, M, K) == f"rag_backward_{plan}"
    g = gen(T + M + K)
    X, W, Z, dY = ints(g, T, K), ints(g, M, K), ints(g, T, M), ints(g, T, M, top=2)
    dZ = dY.double() * (Z > 0)
    dX, dW, db = empty(T, K), empty(M, K, dtype=dw), empty(M, dtype=F32)
    B.fused_linear_backward(ctx(), strided(dY, 3), strided(X, 8), W, dX=dX, dW=dW, dbias=db,
                            act="relu", Z=Z)
    assert torch.equal(dX, (dZ @ W.double()).to(BF16))
    assert torch.equal(dW, (dZ.t() @ X.double()).to(dw))
    assert torch.equal(db.double(), dZ.sum(0))


@pytest.mark.parametrize("dw", [BF16, F32])
@pytest.mark.parametrize("T,F,K,plan", GATED_FFN_BACKWARD)
def test_gated_ffn_backward(T, F, K, plan, dw):
    say(f"case gated_ffn_backward T={T} F={F} K={K} {dw} {plan}")
    assert ctx().ops_kernel_name("gated_ffn_backward", T, F, K) == f"rag_backward_{plan}"
    g = gen(T + F + K)
    X, Wg, Wu = ints(g, T, K), ints(g, F, K), ints(g, F, K)
    dH, G, U = ints(g, T, F, top=2), ints(g, T, F), ints(g, T, F)
    dG, dU = dH.double() * U.double() * (G > 0), dH.double() * G.double().clamp(min=0)
    dX, dWg, dWu = empty(T, K), empty(F, K, dtype=dw), empty(F, K, dtype=dw)
    B.gated_ffn_backward(ctx(), strided(dH, 3), strided(X, 8), Wg, Wu, G, U, dX=dX, dWg=dWg,
                         dWu=dWu, act="relu")
    assert torch.equal(dX, (dG @ Wg.double() + dU @ Wu.double()).to(BF16))
    assert torch.equal(dWg, (dG.t() @ X.double()).to(dw))
    assert torch.equal(dWu, (dU.t() @ X.double()).to(dw))


def test_kernel_names_are_checked():
    with pytest.raises(ValueError, match="unknown operator"):
        ctx().ops_kernel_name("layer_norm", 1, 8, 64)
    with pytest.raises(B.RagError, match="multiple of 128"):
        ctx().ops_kernel_name("fused_linear", 100, 64, 64, fp8=True)
    for args in ((4, 1, 8, 64, 0), (0, 0, 8, 64, 0), (2, 1, 8, 128, 1), (0, 1, 8, 64, B.RAG_F32)):
        buf = ctypes.create_string_buffer(128)
        assert B.lib().rag_ops_kernel_name(ctx().h, *args, buf, 128) == B.RAG_EINVAL
