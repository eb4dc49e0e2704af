"""The operators of a block together, as a program uses them.

Serving: sampling core -> projection with the adapters of many requests (one
image each) -> residual + norm with 8-bit output, each step against its
definition in 64 bits on the values it was given, then the whole block captured
and replayed on new inputs.  Training: core and norm under autograd, the
gradients of all leaves clipped together, against the 64-bit oracle.
"""
import numpy as np
import pytest
import torch

import deformable_convolution_sampling_dcn_b200 as d
import oracle
import synthetic_inputs as si
from parity import assert_close_bwd, assert_close_fwd
from test_norm_gpu import check_quant, definition as norm_definition
from test_proj_adapters_gpu import definition as adapters_definition

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("B,H,W", [(3, 9, 10), (2, 5, 6)])  # 270 rows, and 60: both routes of the projection
def test_serving_block(B, H, W, cuda_dev):
    shape = si.CoreShape(B=B, H=H, W=W, G=4, C=32, dtype="f16")
    gen = torch.Generator().manual_seed(1)
    gc, cout, rank = 128, 128, 16
    par = dict(weight=(torch.randn(cout, gc, generator=gen) * gc ** -0.5).half(), bias=torch.randn(cout, generator=gen).half(),
               a=(torch.randn(2, rank, gc, generator=gen) * gc ** -0.5).half(),
               b=(torch.randn(2, cout, rank, generator=gen) * 0.25).half(), scale=torch.tensor([0.5, 2.0]),
               start=(torch.arange(B + 1) * H * W).int(), which=torch.tensor([1, -1, 0][:B], dtype=torch.int32))
    norm_w = (1 + 0.1 * torch.randn(cout, generator=gen)).half()
    dev = {k: v.cuda() for k, v in par.items()}
    dev_w = norm_w.cuda()

    def block(x, offset, mask):
        core = d.dcn_core_forward(x, offset, mask, group=4)
        y = d.dcn_proj_adapters_forward(core, dev["weight"], dev["bias"], dev["a"], dev["b"], dev["start"], dev["which"],
                                        scale=dev["scale"])
        return core, y, d.dcn_add_rms_norm_forward(y, x, dev_w, quant="e4m3", group=128)

    def check(inp, core, y, o):
        assert_close_fwd(core, oracle.dcn_forward(inp["x"], inp["offset"], inp["mask"], G=4), "core")
        want, tol = adapters_definition(dict(par, x=core.cpu().view(-1, gc)))
        assert ((y.double().cpu().view(-1, cout) - want).abs() <= tol).all()
        h, yn, _ = norm_definition(y.cpu().view(-1, cout), inp["x"].view(-1, cout), norm_w, 1e-6)
        assert torch.equal(o.residual_out.cpu().view(-1, cout), h)
        check_quant(d.AddRmsNorm(None, None, o.out8.view(-1, cout), o.scale.view(-1, 1), None), yn, "e4m3", 128)

    inp = si.core_inputs(shape, 5)
    keys = ("x", "offset", "mask")
    bufs = [inp[k].cuda() for k in keys]
    core, y, o = block(*bufs)
    torch.cuda.synchronize()
    assert d._binding.take_device_error() == 0
    assert y.shape == (B, H, W, cout) and o.out8.shape == (B, H, W, cout)
    check(inp, core, y, o)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        core, y, o = block(*bufs)
    new = si.core_inputs(shape, 6)
    for k, b in zip(keys, bufs):
        b.copy_(new[k])
    g.replay()
    torch.cuda.synchronize()
    check(new, core, y, o)
    assert d._binding.take_device_error() == 0


def test_training_step(cuda_dev):
    shape = si.CoreShape(B=2, H=8, W=9, G=4, C=8, dtype="f32")
    inp = si.core_inputs(shape, 7)
    gen = torch.Generator().manual_seed(3)
    res, w = torch.randn(2, 8, 9, 32, generator=gen), 1 + 0.1 * torch.randn(32, generator=gen)
    gy, gh = torch.randn(2, 8, 9, 32, generator=gen), 0.3 * torch.randn(2, 8, 9, 32, generator=gen)
    leaves = [t.cuda().requires_grad_() for t in (inp["x"], inp["offset"], inp["mask"], res, w)]
    x, offset, mask, r, wt = leaves
    y, h = d.AddRmsNormFunction.apply(d.DCNCoreFunction.apply(x, offset, mask, 4), r, wt, 1e-6)
    torch.autograd.backward([y, h], [gy.cuda(), gh.cuda()])
    raw = [t.grad.clone() for t in leaves]
    norm = d.dcn_clip_grads([t.grad for t in leaves], 1.0)
    torch.cuda.synchronize()

    # 64 bits: the norm by autograd, the core by the oracle
    core = torch.from_numpy(oracle.dcn_forward(inp["x"], inp["offset"], inp["mask"], G=4))
    c64, r64, w64 = (t.double().requires_grad_() for t in (core, res, w))
    hd = c64 + r64
    yd = hd / torch.sqrt((hd * hd).mean(-1, keepdim=True) + 1e-6) * w64
    torch.autograd.backward([yd, hd], [gy.double(), gh.double()])
    rb = oracle.dcn_backward(inp["x"], inp["offset"], inp["mask"], c64.grad.numpy(), G=4)
    want = [rb["grad_x"], rb["grad_offset"], rb["grad_mask"], r64.grad.numpy(), w64.grad.numpy()]
    n = np.sqrt(sum(float((g ** 2).sum()) for g in want))
    assert abs(float(norm) - n) <= 1e-4 * n
    for name, leaf, before, ref in zip(("x", "offset", "mask", "residual", "weight"), leaves, raw, want):
        assert_close_bwd(before, ref, name, atomic=name == "x")
        assert_close_bwd(leaf.grad, ref / (n + 1e-6), name + " clipped", atomic=name == "x")
