"""Which operands of sgemv_rotary share bytes: views of one projection's output
that lie between each other head by head do not (addresses are never followed:
what is accepted ends at the launch, without a GPU, or is stopped by an
alignment that is checked before the overlaps)."""
import pytest

from activation_sparse_bit_amd import sgemv

torch = pytest.importorskip("torch")

A, DIM, H, T = 1 << 40, 64, 4, 5


def status(q, q_out, k, k_out, q_strides, k_strides, tokens=T, heads=H, qo_strides=None, ko_strides=None):
    args = sgemv._ROTARY.pack(q, q_out, k, k_out, 0, 9 * A, 10 * A, 0, *q_strides, *(qo_strides or q_strides), *k_strides,
                              *(ko_strides or k_strides), 0, 0, tokens, tokens, 0, heads if q else 0, heads, DIM, 32, 1, 32, 0, 0, 0, 0, 1.0)
    return sgemv.lib().sgemv_rotary(args, None, 0)


needs_no_gpu = pytest.mark.skipif(torch.cuda.is_available(), reason="addresses are made up: for machines without a GPU")


@needs_no_gpu
@pytest.mark.parametrize("tokens", [1, 5])
def test_heads_between_each_other(tokens):
    step = 3 * DIM                              # [tokens][heads][3][dim]
    strides = (H * step, step)
    for second in (DIM, 2 * DIM):
        k = A + 2 * second
        assert status(A, A, k, k, strides, strides, tokens) != sgemv.SGEMV_EINVAL
        assert status(k, k, A, A, strides, strides, tokens) != sgemv.SGEMV_EINVAL
    outside = (step, T * step)                  # [heads][tokens][3][dim]
    assert status(A, A, A + 2 * DIM, A + 2 * DIM, outside, outside, tokens) != sgemv.SGEMV_EINVAL


@needs_no_gpu
def test_heads_that_share_bytes():
    step = 3 * DIM
    strides = (H * step, step)
    for off in (0, 2, DIM, 2 * DIM - 2, 2 * step, 2 * step - DIM, 14 * step + 2):   # bytes: the same, a part, another head
        assert status(A, A, A + off, A + off, strides, strides) == sgemv.SGEMV_EINVAL, off
    # rows that are no whole number of heads' strides, other strides of heads: taken as one range
    assert status(A, A, A + 2 * DIM, A + 2 * DIM, (H * step + 8, step), (H * step + 8, step)) == sgemv.SGEMV_EINVAL
    assert status(A, A, A + 2 * DIM, A + 2 * DIM, (H * step, step), (H * step, 2 * DIM)) == sgemv.SGEMV_EINVAL
    # q's places with another stride for its output
    assert status(A, A, A + 2 * DIM, 7 * A, strides, strides, qo_strides=(H * step, 2 * DIM)) == sgemv.SGEMV_EINVAL
