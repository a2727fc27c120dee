"""The 8-bit operators as torch code sees them: tensors without elements, and what
autograd is told of a tensor that a call writes to."""
import pytest
import torch

import sequence_re_layout_gb300 as basp                     # noqa: F401
from sequence_re_layout_gb300 import autograd, fp8
from test_gpu_fp8 import _built                             # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("quantized", [False, True])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_norm_of_no_columns(quantized, dtype):
    """rstd = (0 / 0 + eps)^-1/2, whatever the memory held before."""
    used = torch.full((4096,), 5.0, device="cuda")
    del used
    x, w = torch.empty(4096, 0, dtype=dtype, device="cuda"), torch.empty(0, dtype=dtype, device="cuda")
    y, h, rstd = fp8.rmsnorm(x, w, quantized=quantized)
    assert y.shape == h.shape == (4096, 0) and rstd.shape == (4096,)
    assert bool(torch.isnan(rstd).all())
    y, _, rstd = fp8.rmsnorm(x[:0], w, quantized=quantized)
    assert y.shape == (0, 0) and rstd.shape == (0,)


def norm_into(t):
    x, w = torch.ones(t.shape, dtype=t.dtype, device="cuda"), torch.ones(t.shape[1], dtype=t.dtype, device="cuda")
    return fp8.rmsnorm(x, w, residual=t.detach(), h=t)[1]


def product_into(t, accumulate=False):
    a, b = (fp8.quantize(torch.ones(n, 128, device="cuda")) for n in t.shape)
    return fp8.matmul(a, b, out=t, accumulate=accumulate)


WRITES = {"norm": norm_into, "product": product_into, "accumulate": lambda t: product_into(t, True)}


@pytest.mark.parametrize("write", sorted(WRITES))
def test_a_saved_tensor_that_was_overwritten_is_noticed(write):
    a = torch.zeros(4, 256, dtype=torch.bfloat16, device="cuda", requires_grad=True)
    y = torch.exp(a)                                         # saves its result
    WRITES[write](y.detach())
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.sum().backward()
    y = torch.exp(a)
    y.sum().backward()
    assert bool((a.grad == 1).all())


@pytest.mark.parametrize("write", sorted(WRITES))
def test_a_write_raises_the_version(write):
    t = torch.zeros(4, 256, dtype=torch.bfloat16, device="cuda")
    part = t[1:3, 16:144]
    assert WRITES[write](part) is part and t._version == part._version == 1
    with torch.inference_mode():                             # has no versions
        i = torch.zeros(4, 256, dtype=torch.bfloat16, device="cuda")
        assert WRITES[write](i) is i and bool((i != 0).all())


@pytest.mark.parametrize("write", sorted(WRITES))
def test_a_tensor_whose_gradient_is_followed_is_not_written_to(write):
    leaf = torch.zeros(4, 256, dtype=torch.bfloat16, device="cuda", requires_grad=True)
    for t in (leaf, leaf * 2, leaf[:, :128]):
        with pytest.raises(ValueError, match="must not require a gradient"):
            WRITES[write](t)
    assert leaf._version == 0 and bool((leaf == 0).all())
    with torch.no_grad():
        WRITES[write](leaf)
    assert leaf._version == 1 and bool((leaf != 0).all())


@pytest.mark.parametrize("shapes", [((6, 256), (2, 3, 256)), ((2, 3, 256), (6, 256)), ((256,), (1, 256))])
@pytest.mark.parametrize("through", ["y", "h", "both"])
@pytest.mark.parametrize("projected", [False, True])
def test_a_residual_under_other_leading_dimensions(shapes, through, projected):
    """The rows are the same, so are the results; the gradient has the residual's shape."""
    def run(residual_shape):
        g = torch.Generator().manual_seed(1)
        x, r = (torch.randn(s, generator=g).bfloat16().cuda().requires_grad_() for s in shapes)
        w = torch.randn(256, generator=g).bfloat16().cuda().requires_grad_()
        p = torch.randn(48, 256, generator=g).cuda().requires_grad_()
        leaf, r = r, r.view(residual_shape)
        y, h = autograd.rmsnorm_linear_fp8(x, w, p, residual=r) if projected else autograd.rmsnorm(x, w, r)
        dy, dh = torch.randn(y.shape, generator=g).bfloat16().cuda(), torch.randn(h.shape, generator=g).bfloat16().cuda()
        outs = {"y": [(y, dy)], "h": [(h, dh)], "both": [(y, dy), (h, dh)]}[through]
        torch.autograd.backward([o for o, _ in outs], [d for _, d in outs])
        assert h.shape == x.shape and leaf.grad.shape == leaf.shape
        return y, h, x.grad, leaf.grad

    for a, b in zip(run(shapes[1]), run(shapes[0])):
        assert torch.equal(a, b)
