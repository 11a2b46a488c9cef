"""Arguments of the products with an epilogue and the routed slots that must be
refused before anything is launched, without a GPU: the C ABI by status, the
tensor layer with tensors that are never read."""
import pytest
import torch


@pytest.fixture(scope="module")
def q():
    import quantized_weight_decode_amd as q
    try:
        q.lib()
    except ImportError as e:
        pytest.skip(str(e))
    return q


def meta(*shape, dtype=torch.uint8):
    return torch.empty(shape, dtype=dtype, device="meta")


@pytest.mark.parametrize("gs", [(1 << 32) + 64, (1 << 24) + 2, 1 << 31])
def test_group_size_that_a_c_int_would_wrap(q, gs):
    """2^32 + 64 columns per group is one scale per row; as a C int it would be
    64 and the kernel would read scales behind the buffer."""
    with pytest.raises(q.QgemvError) as e:
        q.i4g_linear(meta(8, 512), meta(8, 1, dtype=torch.float32),
                     meta(3, 1024, dtype=torch.float32), gs)
    assert e.value.status == 3
    with pytest.raises(q.QgemvError):
        q.i4g_grouped(meta(2, 8, 512), meta(2, 8, 1, dtype=torch.float32),
                      meta(3, 1024, dtype=torch.float32), meta(3, dtype=torch.int32), gs)
    with pytest.raises(q.QgemvError):
        q.i4g(meta(8, 512), meta(8, 1, dtype=torch.float32),
              meta(3, 1024, dtype=torch.float32), gs)
