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


BIG = (1 << 32) + 3          # 3 as a C int


def test_sizes_that_a_c_int_would_wrap(q):
    """Refused by name; a call with the wrapped sizes would fill three rows of
    the output, or sort by other experts."""
    f32, i32 = {"dtype": torch.float32}, {"dtype": torch.int32}

    def refused(f, *a, **k):
        with pytest.raises(q.QgemvError) as e:
            f(*a, **k)
        assert e.value.status == 2
    refused(q.i4g_linear, meta(8, 32), meta(8, 2, **f32), meta(BIG, 64, **f32), 32)
    refused(q.fp8b128_linear, meta(8, 64), meta(1, 1, **f32), meta(BIG, 64, **f32))
    refused(q.i4g_linear, meta(BIG, 32), meta(BIG, 2, **f32), meta(3, 64, **f32), 32)
    refused(q.i4g_grouped, meta(2, 8, 32), meta(2, 8, 2, **f32), meta(BIG, 64, **f32),
            meta(3, **i32), 32)
    refused(q.i4g_grouped, meta(2, 8, 32), meta(2, 8, 2, **f32), meta(3, 64, **f32),
            meta(3, **i32), 32, rows=meta(BIG, **i32))
    refused(q.moe_group, meta(4, 2, **i32), BIG)
    refused(q.moe_group, meta(4, 2, **i32), 3 - (1 << 32))
    refused(q.moe_group, meta(BIG, 2, **i32), 8)
    refused(q.moe_combine, meta(BIG, 8, **f32), meta(4, 2, **i32), meta(4, 2, **f32))
    refused(q.moe_combine, meta(4, 8, **f32), meta(BIG, 2, **i32), meta(BIG, 2, **f32))
    refused(q.moe_combine, meta(4, BIG, **f32), meta(4, 2, **i32), meta(4, 2, **f32))


def test_arguments_that_ask_for_a_gradient(q):
    """There is no backward pass: refused in grad mode, not detached silently;
    without it the call goes on (to the refusal of a tensor not on a GPU)."""
    w, s, x = meta(8, 32), meta(8, 2, dtype=torch.float32), meta(3, 64, dtype=torch.float32)
    sc, xs = meta(1, 1, dtype=torch.float32), {"dtype": torch.float32}
    i32 = {"dtype": torch.int32}
    h, pos, gates = meta(4, 8, **xs), meta(4, 2, **i32), meta(4, 2, **xs)

    def asks(t):
        return t.clone().requires_grad_()
    calls = [lambda g: q.i4g_linear(w, s, g(x), 32),
             lambda g: q.i4g_linear(w, g(s), x, 32),
             lambda g: q.i4g_linear(w, s, x, 32, bias=g(meta(8, **xs))),
             lambda g: q.i4g_linear(w, s, x, 32, residual=g(meta(3, 8, **xs))),
             lambda g: q.i4g_linear(w, s, x, 32, out=g(meta(3, 8, **xs))),
             lambda g: q.fp8b128_linear(meta(8, 64), sc, g(x)),
             lambda g: q.i4g_grouped(meta(2, 8, 32), meta(2, 8, 2, **xs), g(x), meta(3, **i32),
                                     32),
             lambda g: q.moe_combine(g(h), pos, gates),
             lambda g: q.moe_combine(h, pos, g(gates))]
    for f in calls:
        with pytest.raises(ValueError, match="gradient"):
            f(asks)
        with torch.no_grad(), pytest.raises(TypeError, match="CUDA"):
            f(asks)
        with pytest.raises(TypeError, match="CUDA"):
            f(lambda t: t)


@pytest.mark.parametrize("I,gs,dtype", [(32, 32, 0), (32, 32, 1), (30, 2, 0), (31, 6, 1)])
@pytest.mark.parametrize("E,R", [(1024, 2048), (1024, 1 << 15), (1, 1 << 15)])
def test_grouped_sizes_beyond_a_launch(q, E, R, I, gs, dtype):
    """A launch holds fewer than 2^32 work items: refused before anything runs."""
    a, O = 1 << 46, 1 << 24
    st = q.qgemv_i4g_grouped(a, 2 * a, O * 16, O * 16, E, 3 * a, None, 4 * a, 32, R, 5 * a, O, R,
                             I, O, gs, dtype, None, 6 * a, 1 << 45, 0)
    assert st == 2


def test_no_scratch_for_planes_that_no_kernel_packs(q):
    """Packed activations of 4 GB and more are never made: dense rows are cut
    into slices, grouped ones take the general kernel."""
    for dtype in (0, 1):
        T, I, E = 1 << 20, 7168, 64
        assert q.qgemv_grouped_workspace(T, T, E, I, 64, dtype) < 1 << 24
        assert q.qgemv_grouped_workspace(1 << 18, T, E, I, 64, dtype) > 1 << 31
        assert 1 << 31 < q.qgemv_linear_workspace(T, I, 64, dtype) < 9 << 30
        assert q.qgemv_linear_workspace(128, 1 << 24, 64, dtype) == 0
