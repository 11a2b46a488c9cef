"""float8 codes of the 8-bit products, without a GPU: those that ask for a
gradient are refused like every other argument that does."""
import pytest
import torch

F8 = torch.float8_e4m3fn


@pytest.fixture(scope="module")
def q():
    import quantized_weight_decode_amd as q
    try:
        q.lib()
    except ImportError as e:
        pytest.skip(str(e))
    return q


def f32(*shape):
    return torch.empty(shape, device="meta")


def f8(*shape):
    return f32(*shape).to(F8)


def asks(*shape):
    """Codes cast from a tensor that asks for a gradient, as autograd gives them."""
    t = f32(*shape).requires_grad_().to(F8)
    assert t.requires_grad
    return t


def leaf(*shape):
    return f8(*shape).requires_grad_()


CALLS = [
    ("w", lambda q, g: q.fp8b128_matmul(g(8, 200), f32(1, 2), f8(3, 200), f32(3, 2))),
    ("x", lambda q, g: q.fp8b128_matmul(f8(8, 200), f32(1, 2), g(3, 200), f32(3, 2))),
    ("one x", lambda q, g: q.fp8b128_matmul(f8(8, 200), f32(1, 2), g(200), f32(2))),
    ("grouped w", lambda q, g: q.fp8b128_matmul_grouped(
        g(2, 8, 200), f32(2, 1, 2), f8(3, 200), f32(3, 2), torch.empty(3, dtype=torch.int32))),
    ("grouped x", lambda q, g: q.fp8b128_matmul_grouped(
        f8(2, 8, 200), f32(2, 1, 2), g(3, 200), f32(3, 2), torch.empty(3, dtype=torch.int32))),
    ("out", lambda q, g: q.fp8_quantize(f32(3, 200), out=g(3, 200))),
    ("one out", lambda q, g: q.fp8_quantize(f32(200), out=g(200))),
]


@pytest.mark.parametrize("make", [asks, leaf])
@pytest.mark.parametrize("name,call", CALLS, ids=[n for n, _ in CALLS])
def test_codes_that_ask_for_a_gradient(q, name, call, make):
    with pytest.raises(ValueError, match="gradient"):
        call(q, make)


@pytest.mark.parametrize("name,call", CALLS, ids=[n for n, _ in CALLS])
def test_codes_that_ask_for_none(q, name, call):
    """The same calls get past that check: detached codes, and under no_grad."""
    with pytest.raises((TypeError, ValueError), match="CUDA|devices"):
        call(q, f8)
    def made(*shape):
        with torch.enable_grad():
            return asks(*shape)
    with torch.no_grad(), pytest.raises((TypeError, ValueError), match="CUDA|devices"):
        call(q, made)


def test_scratch_sizes(q):
    """Sizes that a C int would wrap are refused, and a product's scratch is asked for
    with its device current, by whose CUs it goes."""
    for f in (lambda n: q.matmul_workspace(n, 7168, 7168, torch.bfloat16, "cpu"),
              lambda n: q.matmul_workspace(300, n, 7168, torch.bfloat16, "cpu"),
              lambda n: q.matmul_workspace(300, 7168, n, torch.bfloat16, "cpu"),
              lambda n: q.matmul_grouped_workspace(n, 8, "cpu"),
              lambda n: q.matmul_grouped_workspace(300, n, "cpu")):
        for n in ((1 << 32) + 300, -1):
            with pytest.raises(q.QgemvError) as e:
                f(n)
            assert e.value.status == 2
    ws = q.matmul_workspace(300, 7168, 7168, torch.bfloat16, "cpu")
    assert ws.numel() == q.qgemv_matmul_workspace(300, 7168, 7168, 1, 0)


def test_scratch_goes_by_its_device(q, monkeypatch):
    current, asked = [0], []

    class Guard:
        def __init__(self, device):
            self.index = device.index

        def __enter__(self):
            self.before, current[0] = current[0], self.index

        def __exit__(self, *_):
            current[0] = self.before
    monkeypatch.setattr(q, "_on", Guard)
    monkeypatch.setattr(q, "qgemv_matmul_workspace",
                        lambda *_: asked.append(current[0]) or 4096)
    q.matmul_workspace(300, 7168, 7168, torch.bfloat16, torch.device("meta", 3))
    assert asked == [3] and current == [0]
