"""GPU parity of layer norm on every kernel: each combination of x, y and weight types with each
number of vectors per thread, for even rows, odd ones and rows larger together than the caches,
forward and backward.  Bounds: see ops_reference.py."""
import pytest
import torch

import ops_reference as R
from ring_all_gather_amd import binding as B

from gpu_common import DEV, ctx, say
from test_gpu_ops import BF16, F32, empty, gen, normal, strided

pytestmark = pytest.mark.gpu

# x, y, weight: b bf16, f fp32
TYPES = ["bbb", "bbf", "ffb", "fff", "fbb", "fbf"]
# Vectors of 8 columns per thread, forward / backward: bf16 x; fp32 x
SIZES = [(520, 1000),     # 1 / 1; 1 / 1
         (520, 4088),     # 2 / 1; 2 / 1
         (520, 4104),     # 4 / 2; 2 / 1
         (520, 8200),     # 4 / 4; 2 / 2
         (3, 16384),      # 2 / 4; 2 / 2
         (3, 16392)]      # any width: rows read again
# (T, H) by bytes of x and y per element, more than 256 MiB together forward; vectors per thread as
# above: 1 / 1, 2 / 1, 4 / 2 and 4 / 4 with bf16 x, 1 / 1, 2 / 1, 2 / 1 and 2 / 2 with fp32 x
STREAMED = {4: [(33600, 2048), (17000, 4096), (8400, 8192), (8400, 8200)],
            6: [(22500, 2048), (11200, 4104), (5600, 8192), (5600, 8200)],
            8: [(17000, 2048), (8400, 4104), (4200, 8192), (4200, 8200)]}


def check_norm(T, H, types, pad=0):
    xt, yt, wt = (BF16 if c == "b" else F32 for c in types)
    g = gen(T * 3 + H)
    x = strided(normal(g, T, H, std=2.0, dtype=xt) + normal(g, T, 1, dtype=xt), pad)
    w, b = 1 + normal(g, H, std=0.3, dtype=wt), normal(g, H, dtype=wt)
    y, mean, rstd = empty(T, H, dtype=yt), empty(T, dtype=F32), empty(T, dtype=F32)
    B.layer_norm(ctx(), x, w, b, y, mean=mean, rstd=rstd, eps=1e-5)
    ry, rm, rr, ey, em, er = R.layer_norm(x.double(), w.double(), b.double(), 1e-5)
    R.check(y, ry, ey + (R.BF * ry.abs() if yt == BF16 else 0), "y")
    R.check(mean, rm, em, "mean")
    R.check(rstd, rr, er, "rstd")
    del ry, ey
    dy = strided(normal(g, T, H, dtype=yt), pad)
    dx, dw, db = empty(T, H, dtype=xt), empty(H, dtype=F32), empty(H, dtype=F32)
    B.layer_norm_backward(ctx(), dy, x, w, mean, rstd, dx, dw, db)
    rx, rw, rb, ex, ew, eb = R.layer_norm_backward(dy.double(), x.double(), w.double(),
                                                   mean.double(), rstd.double())
    R.check(dx, rx, ex + (R.BF * rx.abs() if xt == BF16 else 0), "dx")
    R.check(dw, rw, ew, "dweight")
    R.check(db, rb, eb, "dbias")


@pytest.mark.parametrize("types", TYPES)
@pytest.mark.parametrize("T,H", SIZES)
def test_layer_norm_even_rows(T, H, types):
    say(f"case layer_norm T={T} H={H} {types}")
    check_norm(T, H, types, pad=8)


@pytest.mark.parametrize("types", TYPES)
@pytest.mark.parametrize("T,H", SIZES)
def test_layer_norm_odd_rows(T, H, types):
    """One column fewer, and row strides that put every other row at an odd element."""
    H -= 1
    say(f"case layer_norm T={T} H={H} {types}")
    check_norm(T, H, types, pad=2)


@pytest.mark.parametrize("types", TYPES)
@pytest.mark.parametrize("i", range(4))
def test_layer_norm_streamed(i, types):
    T, H = STREAMED[sum(2 if c == "b" else 4 for c in types[:2])][i]
    say(f"case layer_norm streamed T={T} H={H} {types}")
    check_norm(T, H, types)


def test_layer_norm_sums_take_in_every_row_past_32_bits():
    """dbias and dweight over 525000 rows of more than 2^31 elements together, to the
    last row: with dy and xh +-1 both are whole numbers, which fp32 sums give exactly."""
    T, H = 525_000, 4104
    say(f"case layer_norm sums T={T} H={H}")
    sign = torch.ones(H, dtype=BF16, device=DEV)
    sign[::2] = -1.0
    x = (2.0 * sign).expand(T, H).contiguous()
    dy = sign.expand(T, H).contiguous()
    w = torch.ones(H, device=DEV)
    mean, rstd = torch.zeros(T, device=DEV), torch.full((T,), 0.5, device=DEV)
    dx, dw, db = torch.empty_like(x), empty(H, dtype=F32), empty(H, dtype=F32)
    B.layer_norm_backward(ctx(), dy, x, w, mean, rstd, dx, dw, db)
    assert torch.equal(db, T * sign.float())
    assert torch.equal(dw, torch.full_like(dw, float(T)))
    # dx = 0.5 (sign - mean(sign) - sign mean(1)) = 0
    assert dx.eq(0).all()
