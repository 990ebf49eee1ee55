"""Checks of the block operators' binding that need no GPU."""
import pytest
import torch

from ring_all_gather_amd import binding as B


class NoContext:
    h, device = None, 0


@pytest.mark.parametrize("rows", [2 ** 31, 2 ** 32, 2 ** 32 + 5])
def test_sizes_that_do_not_fit_an_int_are_refused(rows):
    """The C entry points take 32-bit sizes: 2^32 rows must not arrive as none."""
    x, w = torch.zeros(1, 64, dtype=torch.bfloat16), torch.zeros(8, 64, dtype=torch.bfloat16)
    many, out = x.expand(rows, 64), x[:, :8].expand(rows, 8)
    for call in (lambda: B.layer_norm(NoContext, many, w[0], None, many),
                 lambda: B.fused_linear(NoContext, many, w, out),
                 lambda: B.fused_linear(NoContext, x, w[:1].expand(rows, 64), out),
                 lambda: B.gated_ffn_backward(NoContext, out, many, w, w, out, out, dX=many)):
        with pytest.raises(ValueError, match="2\\^31"):
            call()


def test_fingerprints_of_both_code_objects():
    """Each code object of the library has its own SHA-256, by which profiles name their build."""
    ring, ops = B.kernels_fingerprint(), B.ops_fingerprint()
    assert ring != ops
    for digest in (ring, ops):
        assert len(digest) == 64 and int(digest, 16) >= 0
