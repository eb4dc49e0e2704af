"""Residual addition + root-mean-square norm on the GPU, its 8-bit outputs and
its gradients, against the definition in 64 bits.

Tolerances (u = 2^-24, half a step of fp32; uT = finfo(T).eps / 2).  The sum of
squares has at most 32 terms per thread and 10 tree levels, all terms positive:
relative error below 43u, so rstd is within 43u/2 and 2.5u of its own
operations, y within 26u, plus uT where it is stored in 16 bits: |y|(32u + uT).
"""
import numpy as np
import pytest
import torch

import deformable_convolution_sampling_dcn_b200 as d

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
EPS = 1e-6


def half_step(dt):
    return 0.0 if dt == torch.float32 else torch.finfo(dt).eps / 2


def tiny(dt):
    """Half of the smallest subnormal of a 16-bit type (fp16 outputs may be subnormal)."""
    return torch.finfo(dt).smallest_normal * torch.finfo(dt).eps / 2


def inputs(rows, cols, dt, seed, residual=True, weight=True, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    x = (torch.randn(rows, cols, generator=g) * scale).to(dt)
    r = (torch.randn(rows, cols, generator=g) * 2 * scale).to(dt) if residual else None
    w = (1 + 0.3 * torch.randn(cols, generator=g)).to(dt) if weight else None
    return x, r, w


def definition(x, r, w, eps=EPS):
    """(h in its type, y in 64 bits, rstd in 64 bits)."""
    h = x if r is None else (x.double() + r.double()).to(x.dtype)
    hd = h.double()
    rstd = 1.0 / torch.sqrt((hd * hd).mean(-1) + np.float32(eps).astype(np.float64))
    y = hd * rstd[:, None]
    return h, (y if w is None else y * w.double()), rstd


def gpu(*ts):
    return [None if t is None else t.cuda() for t in ts]


# widths: one column, below and above the 8-lane, warp and CTA teams, odd, ragged groups, the largest
COLS = [1, 2, 7, 8, 31, 32, 64, 100, 127, 128, 129, 136, 250, 256, 257, 512, 513, 520, 1000, 1024, 1032, 2049, 4096,
        5000, 16384]


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("cols", COLS)
def test_forward(cols, dtype, cuda_dev):
    dt = DT[dtype]
    for rows, residual, weight in ((1, True, True), (5, False, True), (37, True, False)):
        x, r, w = inputs(rows, cols, dt, cols + rows, residual, weight)
        o = d.dcn_add_rms_norm_forward(*gpu(x, r, w), eps=EPS, save_rstd=True)
        h, y, rstd = definition(x, r, w)
        assert o.out8 is None and o.scale is None and (o.residual_out is None) == (r is None)
        if r is not None:
            assert torch.equal(o.residual_out.cpu(), h)
        err = (o.out.double().cpu() - y).abs()
        assert (err <= y.abs() * (32 * U + half_step(dt)) + tiny(dt)).all(), float((err / y.abs()).max())
        assert ((o.rstd.double().cpu() - rstd).abs() <= rstd * 26 * U).all()


def check_quant(o, y, quant, group):
    rows, cols = y.shape
    top, ng = (448.0 if quant == "e4m3" else 127.0), (-(-cols // 128) if group else 1)
    assert o.scale.shape == (rows, ng) and o.out8.shape == (rows, cols)
    w = group or cols
    amax = torch.stack([p.abs().amax(-1) for p in y.split(w, dim=1)], 1)
    want = (amax / top).clamp(min=2.0 ** -126)
    s = o.scale.double().cpu()
    assert ((s - want).abs() <= want * 28 * U).all()  # y, the division and no more
    sc = s.repeat_interleave(w, 1)[:, :cols]
    q = o.out8.float().double().cpu()
    err = (q * sc - y).abs()
    slack = y.abs() * 32 * U + sc * 2 * U * top  # fp32 y, 1 / scale and their product
    if quant == "e4m3":  # half a step: 2^-4 of the value, 2^-10 below the smallest normal 2^-6
        assert (err <= torch.maximum(y.abs() * 2.0 ** -4, sc * 2.0 ** -10) + slack).all()
    else:
        assert q.abs().max() <= 127
        assert (err <= 0.5 * sc + slack).all()


@pytest.mark.parametrize("group", [0, 128])
@pytest.mark.parametrize("quant", ["e4m3", "int8"])
@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("cols", [1, 8, 24, 64, 100, 128, 136, 200, 256, 300, 512, 1000, 1024, 1160, 2047, 4096, 8200])
def test_forward_8bit(cols, dtype, quant, group, cuda_dev):
    for rows, keep in ((1, False), (19, True)):
        x, r, w = inputs(rows, cols, DT[dtype], 3 * cols + rows)
        o = d.dcn_add_rms_norm_forward(*gpu(x, r, w), eps=EPS, quant=quant, group=group, keep_out=keep)
        h, y, _ = definition(x, r, w)
        assert torch.equal(o.residual_out.cpu(), h)
        assert (o.out is not None) == keep
        if keep:
            err = (o.out.double().cpu() - y).abs()
            assert (err <= y.abs() * (32 * U + half_step(DT[dtype])) + tiny(DT[dtype])).all()
        check_quant(o, y, quant, group)


def test_many_rows_and_rows_past_a_grid(cuda_dev):
    """More rows than the persistent grid has teams, a ragged last round."""
    for rows, cols, dtype in ((148 * 8 * 8 * 2 + 3, 40, "bf16"), (30011, 256, "f16"), (2501, 2048, "f32")):
        x, r, w = inputs(rows, cols, DT[dtype], 5)
        o = d.dcn_add_rms_norm_forward(*gpu(x, r, w), eps=EPS, quant="int8")
        h, y, _ = definition(x, r, w)
        assert torch.equal(o.residual_out.cpu(), h)
        check_quant(o, y, "int8", 0)


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("cols", [8, 33, 256, 1000, 1032])
def test_special_values(cols, dtype, cuda_dev):
    """Zero rows give zeros, a NaN or an infinity stays in its own row."""
    x, _, w = inputs(7, cols, DT[dtype], 9)
    x[1] = 0
    x[3, cols // 2] = float("nan")
    x[5, 0] = float("inf")
    o = d.dcn_add_rms_norm_forward(x.cuda(), None, w.cuda(), eps=EPS, quant="e4m3", group=128, keep_out=True)
    q = d.dcn_add_rms_norm_forward(x.cuda(), None, w.cuda(), eps=EPS, quant="int8")
    _, y, _ = definition(x, None, w)
    out = o.out.double().cpu()
    ok = [0, 1, 2, 4, 6]
    assert (out[1] == 0).all() and (o.out8[1].float() == 0).all() and (q.out8[1] == 0).all()
    assert (o.scale[1] == 2.0 ** -126).all()
    assert ((out[ok] - y[ok]).abs() <= y[ok].abs() * (32 * U + half_step(DT[dtype])) + tiny(DT[dtype])).all()
    assert out[3].isnan().all() and o.out8[3].float().isnan().all() and o.scale[3].isnan().all()
    assert q.scale[3].isnan().all() and q.scale[5].isnan().all()
    assert out[5, 0].isnan() and (out[5, 1:] == 0).all()  # rstd 0: inf * 0, finite * 0
    assert not q.scale[[0, 1, 2, 4, 6]].isnan().any()


def test_large_values_and_tiny_values(cuda_dev):
    """fp16's largest values and rows far below eps keep their fp32 statistics."""
    x = torch.full((2, 512), 65504.0, dtype=torch.float16)
    x[1] = 6e-8
    o = d.dcn_add_rms_norm_forward(x.cuda(), eps=EPS)
    _, y, _ = definition(x, None, None)
    assert ((o.out.double().cpu() - y).abs() <= y.abs() * (32 * U + half_step(torch.float16)) + tiny(torch.float16)).all()


def off(t):
    """The tensor at an address that is a multiple of its element only."""
    return torch.empty(t.numel() + 3, dtype=t.dtype, device="cuda")[1:1 + t.numel()].view(t.shape).copy_(t)


@pytest.mark.parametrize("cols", [8, 120, 264, 512, 1032, 8192, 8200])
def test_unaligned_views(cols, cuda_dev):
    """Tensors that start off 16-byte boundaries, at widths that are aligned otherwise: the accesses go by
    elements and the order of the sums is another one, within the same tolerances."""
    for dtype, quant, group in (("bf16", None, 0), ("f32", "e4m3", 0), ("f16", "int8", 128), ("bf16", "e4m3", 128)):
        x, r, w = inputs(11, cols, DT[dtype], 21)
        o = d.dcn_add_rms_norm_forward(off(x), off(r), off(w), eps=EPS, quant=quant, group=group, keep_out=True)
        h, y, _ = definition(x, r, w)
        assert torch.equal(o.residual_out.cpu(), h)
        err = (o.out.double().cpu() - y).abs()
        assert (err <= y.abs() * (32 * U + half_step(DT[dtype])) + tiny(DT[dtype])).all()
        if quant:
            check_quant(o, y, quant, group)
        check_backward(11, cols, dtype, 22, place=off)


def step_off(t, k, fill):
    """(tensor k elements into a larger buffer, the buffer): the start is off 16 bytes by the same number of elements
    for all types, 8-bit ones included, with `fill` around it."""
    b = torch.full((t.numel() + 32,), fill, dtype=torch.float32).to(t.dtype).cuda()
    v = b[16 + k:16 + k + t.numel()].view(t.shape)
    v.copy_(t)
    return v, b


@pytest.mark.parametrize("quant,group", [(None, 0), ("e4m3", 0), ("int8", 128)])
@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("cols", [1, 3, 13, 57, 64, 67, 121, 127, 131, 250, 257, 300, 505, 515, 1000, 1017, 1023, 1025,
                                  2047, 4383, 9001, 16377, 16383])
def test_rows_in_step(cols, dtype, quant, group, cuda_dev):
    """Rows at every offset to 16 bytes, the same in all tensors; infinities around the inputs never count, the bytes
    around the outputs stay, in place too."""
    dt = DT[dtype]
    dt8 = {"e4m3": torch.float8_e4m3fn, "int8": torch.int8, None: None}[quant]
    for rows, k in ((1, 3), (9, 0), (4, 1), (37, 7 if dtype != "f32" else 2)):
        x, r, w = inputs(rows, cols, dt, cols + k, residual=k != 1)
        h, y, rstd = definition(x, r, w)
        xv, xb = step_off(x, k, float("inf"))
        rv, rb = (None, None) if r is None else step_off(r, k, float("inf"))
        ov, ob = step_off(torch.zeros_like(x), k, 5.0)
        qv, qb = (None, None) if quant is None else step_off(torch.zeros(rows, cols).to(dt8), k, 5.0)
        o = d.dcn_add_rms_norm_forward(xv, rv, w.cuda(), eps=EPS, quant=quant, group=group, out=ov, out8=qv,
                                       residual_out=None if r is None else xv, save_rstd=True)
        if r is not None:
            assert torch.equal(xv.cpu(), h)
        assert ((ov.double().cpu() - y).abs() <= y.abs() * (32 * U + half_step(dt)) + tiny(dt)).all()
        assert ((o.rstd.double().cpu() - rstd).abs() <= rstd * 26 * U).all()
        if quant:
            check_quant(o, y, quant, group)
        for b, fill in ((xb, float("inf")), (rb, float("inf")), (ob, 5.0), (qb, 5.0)):
            if b is not None:
                f = b.float()
                assert (f[:16 + k] == fill).all() and (f[16 + k + rows * cols:] == fill).all()


def test_many_rows_in_step(cuda_dev):
    """More rows than the persistent grids have teams."""
    for rows, cols, dtype, quant, group in ((9013, 61, "bf16", "int8", 0), (12001, 505, "f16", "e4m3", 128),
                                            (5734, 4383, "f16", "int8", 128), (2411, 2051, "f32", None, 0)):
        x, r, w = inputs(rows, cols, DT[dtype], 24)
        o = d.dcn_add_rms_norm_forward(*gpu(x, r, w), eps=EPS, quant=quant, group=group, keep_out=True)
        h, y, _ = definition(x, r, w)
        assert torch.equal(o.residual_out.cpu(), h)
        assert ((o.out.double().cpu() - y).abs() <= y.abs() * (32 * U + half_step(DT[dtype])) + tiny(DT[dtype])).all()
        if quant:
            check_quant(o, y, quant, group)


def test_outputs_end_with_the_row(cuda_dev):
    """Unaligned outputs inside larger buffers: nothing around them is written."""
    for rows, cols in ((5, 13), (3, 300), (2, 1001)):
        x, r, w = gpu(*inputs(rows, cols, torch.bfloat16, 23))
        bufs = [torch.full((rows * cols + 9,), 5, dtype=dt, device="cuda")
                for dt in (torch.bfloat16, torch.bfloat16, torch.int8)]
        views = [b[3:3 + rows * cols].view(rows, cols) for b in bufs]
        d.dcn_add_rms_norm_forward(x, r, w, out=views[0], residual_out=views[1], out8=views[2], quant="int8")
        d.dcn_add_rms_norm_backward(x, r, torch.ones(rows, device="cuda"), w, grad_x=views[0])
        for b in bufs:
            assert (b[:3] == 5).all() and (b[3 + rows * cols:] == 5).all()


def test_in_place_and_given_buffers(cuda_dev):
    x, r, w = inputs(13, 256, torch.bfloat16, 31)
    want = d.dcn_add_rms_norm_forward(*gpu(x, r, w))
    xg, rg, wg = gpu(x, r, w)
    o = d.dcn_add_rms_norm_forward(xg, rg, wg, residual_out=rg, out=xg)  # both over their inputs
    assert o.out is xg and o.residual_out is rg
    assert torch.equal(xg, want.out) and torch.equal(rg, want.residual_out)
    xg, rg, _ = gpu(x, r, w)
    d.dcn_add_rms_norm_forward(xg, rg, wg, residual_out=xg, out=rg)
    assert torch.equal(rg, want.out) and torch.equal(xg, want.residual_out)


def test_rows_beyond_32_bit_offsets(cuda_dev):
    """Element offsets past 2^32: the last rows of a 4.3 G element bf16 tensor."""
    rows, cols = 262145, 16384
    x = torch.empty(rows, cols, dtype=torch.bfloat16, device="cuda")
    g = torch.Generator().manual_seed(3)
    last = torch.randn(3, cols, generator=g).to(torch.bfloat16)
    x[:2].fill_(1.0)
    x[2:-3].zero_()
    x[-3:] = last.cuda()
    o = d.dcn_add_rms_norm_forward(x, eps=EPS, out=x)
    _, y, _ = definition(last, None, None)
    got = o.out[-3:].double().cpu()
    assert ((got - y).abs() <= y.abs() * (32 * U + half_step(torch.bfloat16))).all()
    assert (o.out[2:-3:50000] == 0).all()


# ------------------------------------------------------------------ backward

def backward_definition(gy, h, rstd, w, gh):
    gy, hd, rs = gy.double(), h.double(), rstd.double()[:, None]
    xh = hd * rs
    g = gy if w is None else gy * w.double()
    dot = (g * xh).mean(-1, keepdim=True)
    gx = rs * (g - xh * dot)
    # fp32 error of each part: 4 roundings of g and of the outer operations; the dot's sum has at most
    # 16 terms per thread, 10 tree levels and 4 roundings per term
    bound = rs * (6 * g.abs() + xh.abs() * (32 * (g * xh).abs().mean(-1, keepdim=True) + 8 * dot.abs())) * U
    if gh is not None:
        gx = gx + gh.double()
        bound = bound + U * gx.abs()
    gw = None if w is None else (gy * xh).sum(0)
    gw_abs = None if w is None else (gy * xh).abs().sum(0)
    return gx, bound, gw, gw_abs


def rows_in_a_chain(rows):
    """fp32 additions that one partial sum of the weight gradient can see: its rows (at least 148 CTAs share
    many rows, one CTA takes few), 2 shuffles and 16 warps of a CTA, 1184 / 128 rows of partial sums per
    thread and 7 tree levels, 4 roundings per term."""
    return -(-rows // 148) + 64 + 2 + 16 + 10 + 7 + 4


def check_backward(rows, cols, dtype, seed, weight=True, residual=True, place=torch.Tensor.cuda):
    dt = DT[dtype]
    h, gh, w = inputs(rows, cols, dt, seed, residual, weight)
    gy = torch.randn(rows, cols, generator=torch.Generator().manual_seed(seed + 1)).to(dt)
    rstd = definition(h, None, None)[2].float()
    gx, gw = d.dcn_add_rms_norm_backward(place(gy), place(h), rstd.cuda(), None if w is None else place(w),
                                         grad_residual_out=None if gh is None else place(gh))
    want, bound, want_w, abs_w = backward_definition(gy, h, rstd, w, gh)
    err = (gx.double().cpu() - want).abs()
    assert (err <= bound + want.abs() * (half_step(dt) + 2 * U) + tiny(dt)).all(), float(err.max())
    assert (gw is None) == (w is None)
    if w is not None:
        err = (gw.double().cpu() - want_w).abs()
        assert (err <= abs_w * rows_in_a_chain(rows) * U + want_w.abs() * half_step(dt) + tiny(dt)).all()


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("cols", COLS)
def test_backward(cols, dtype, cuda_dev):
    check_backward(1, cols, dtype, cols)
    check_backward(23, cols, dtype, cols + 1, residual=False)
    check_backward(41, cols, dtype, cols + 2, weight=False)


@pytest.mark.parametrize("rows,cols,dtype", [(20011, 256, "bf16"), (6001, 512, "f32"), (5003, 513, "f16"),
                                             (3001, 2048, "f32"), (40000, 40, "f32"), (1201, 16384, "bf16")])
def test_backward_many_rows(rows, cols, dtype, cuda_dev):
    check_backward(rows, cols, dtype, 7)


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("cols", [5, 61, 131, 505, 515, 1001, 1025, 1031, 2047, 4383, 8185, 8187, 8191, 12001])
def test_backward_in_step(cols, dtype, cuda_dev):
    """Rows off 16-byte boundaries by the same in all tensors, infinities around them, more rows than CTAs."""
    for rows, k in ((1, 3), (9, 0), (4, 1), (37, 7 if dtype != "f32" else 2), (1201, 0)):
        check_backward(rows, cols, dtype, cols + k, residual=k != 1, place=lambda t: step_off(t, k, float("inf"))[0])


@pytest.mark.parametrize("dtype", list(DT))
def test_backward_in_step_in_place(dtype, cuda_dev):
    h, gh, w = inputs(300, 1029, DT[dtype], 61)
    gy = torch.randn(300, 1029).to(DT[dtype])
    rstd = definition(h, None, None)[2].float().cuda()
    want = d.dcn_add_rms_norm_backward(*gpu(gy, h), rstd, w.cuda(), grad_residual_out=gh.cuda())
    for which in range(2):
        t = [step_off(v, 0, 5.0) for v in (gy, h, gh)]
        got = d.dcn_add_rms_norm_backward(t[0][0], t[1][0], rstd, w.cuda(), grad_residual_out=t[2][0],
                                          grad_x=t[2 * which][0])
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        b = t[2 * which][1].float()
        assert (b[:16] == 5).all() and (b[16 + 300 * 1029:] == 5).all()


def test_backward_repeats_bit_for_bit(cuda_dev):
    h, gh, w = gpu(*inputs(9001, 256, torch.float32, 4))
    gy = torch.randn_like(h)
    rstd = torch.rsqrt(h.square().mean(-1) + EPS)
    a = d.dcn_add_rms_norm_backward(gy, h, rstd, w, grad_residual_out=gh)
    for _ in range(3):
        b = d.dcn_add_rms_norm_backward(gy, h, rstd, w, grad_residual_out=gh)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_backward_in_place(cuda_dev):
    h, gh, w = inputs(17, 264, torch.bfloat16, 6)
    gy = torch.randn(17, 264).to(torch.bfloat16)
    rstd = definition(h, None, None)[2].float().cuda()
    want = d.dcn_add_rms_norm_backward(*gpu(gy, h), rstd, w.cuda(), grad_residual_out=gh.cuda())
    for which in ("grad_out", "grad_residual_out"):
        gyg, hg, wg, ghg = gpu(gy, h, w, gh)
        got = d.dcn_add_rms_norm_backward(gyg, hg, rstd, wg, grad_residual_out=ghg,
                                          grad_x=gyg if which == "grad_out" else ghg)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_gradients_against_differences(cuda_dev):
    """Central differences of the 64-bit definition along random directions, fp32 storage."""
    x, r, w = inputs(6, 96, torch.float32, 8)
    gy, gh = torch.randn(6, 96), torch.randn(6, 96)
    xg, rg, wg = (t.cuda().requires_grad_() for t in (x, r, w))
    y, h = d.AddRmsNormFunction.apply(xg, rg, wg, EPS)
    torch.autograd.backward([y, h], [gy.cuda(), gh.cuda()])

    def loss(x, r, w):
        hd = x + r
        yd = hd / torch.sqrt((hd * hd).mean(-1, keepdim=True) + EPS) * w
        return float((yd * gy.double()).sum() + (hd * gh.double()).sum())

    base = [t.double() for t in (x, r, w)]
    for i, leaf in enumerate((xg, rg, wg)):
        for s in range(3):
            v = torch.randn(base[i].shape, generator=torch.Generator().manual_seed(s)).double()
            step = 1e-5
            up, dn = list(base), list(base)
            up[i], dn[i] = base[i] + step * v, base[i] - step * v
            diff = (loss(*up) - loss(*dn)) / (2 * step)
            got = float((leaf.grad.double().cpu() * v).sum())
            # 576 terms of fp32 gradients, each within 1e-6 of its size, and the difference's own 1e-8
            assert abs(got - diff) <= 1e-6 * float((leaf.grad.double().cpu() * v).abs().sum()) + 1e-6


def test_autograd_forms(cuda_dev):
    """No residual, no weight, an unused output, a non-contiguous incoming gradient, leaves used twice."""
    x = torch.randn(9, 64, device="cuda", requires_grad=True)
    y, h = d.AddRmsNormFunction.apply(x, None, None, EPS)
    (y.t().contiguous().t() * 2).sum().backward()
    xd = x.detach().double().requires_grad_()
    (xd / torch.sqrt((xd * xd).mean(-1, keepdim=True) + EPS) * 2).sum().backward()
    assert torch.allclose(x.grad.double(), xd.grad, rtol=1e-4, atol=1e-6)
    x.grad = None
    y, h = d.AddRmsNormFunction.apply(x, x, None, EPS)  # the same leaf twice
    h.sum().backward()
    assert torch.equal(x.grad, torch.full_like(x, 2.0))
    w = torch.ones(64, device="cuda", requires_grad=True)
    x.grad = None
    y, h = d.AddRmsNormFunction.apply(x, None, w, EPS)
    y.sum().backward()
    assert x.grad is not None and w.grad is not None


def test_autograd_captured(cuda_dev):
    x, r, w = gpu(*inputs(200, 256, torch.bfloat16, 21))
    gy, gh = torch.randn_like(x), torch.randn_like(x)
    leaves = [t.clone().requires_grad_() for t in (x, r, w)]

    def step():
        return torch.autograd.grad(d.AddRmsNormFunction.apply(*leaves, EPS), leaves, (gy, gh))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        want = [t.clone() for t in step()]
    torch.cuda.current_stream().wait_stream(s)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = step()
    for t in got:
        t.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_empty_and_streams_and_graph(cuda_dev):
    w = torch.ones(64, device="cuda")
    o = d.dcn_add_rms_norm_forward(torch.empty(0, 64, device="cuda"), weight=w, quant="int8", save_rstd=True)
    assert o.out8.shape == (0, 64) and o.scale.shape == (0, 1) and o.rstd.shape == (0,)
    gw = torch.full((64,), 7.0, device="cuda")
    d.dcn_add_rms_norm_backward(torch.empty(0, 64, device="cuda"), torch.empty(0, 64, device="cuda"),
                                torch.empty(0, device="cuda"), w, grad_weight=gw)
    assert (gw == 0).all()

    x, r, w = gpu(*inputs(300, 512, torch.bfloat16, 12))
    gy = torch.randn_like(x)
    want = d.dcn_add_rms_norm_forward(x, r, w, save_rstd=True)
    wb = d.dcn_add_rms_norm_backward(gy, want.residual_out, want.rstd, w)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = d.dcn_add_rms_norm_forward(x, r, w)
    s.synchronize()
    assert torch.equal(got.out, want.out)
    # two graphs of the same calls, replayed in turn on new inputs: nothing is shared between them
    graphs = []
    for _ in range(2):
        xs = x.clone()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            o = d.dcn_add_rms_norm_forward(xs, r, w, save_rstd=True)
            b = d.dcn_add_rms_norm_backward(gy, o.residual_out, o.rstd, w)
        graphs.append((g, xs, o, b))
    graphs[1][1].copy_(x * 2)
    for g, *_ in graphs:
        g.replay()
    torch.cuda.synchronize()
    assert torch.equal(graphs[0][2].out, want.out)
    assert torch.equal(graphs[0][3][0], wb[0]) and torch.equal(graphs[0][3][1], wb[1])
    other = d.dcn_add_rms_norm_forward(x * 2, r, w)
    assert torch.equal(graphs[1][2].out, other.out)


@pytest.mark.parametrize("cols", [64, 512, 4096, 4099])
def test_more_than_32_bit_elements(cols, cuda_dev):
    """Offsets are 64-bit: the last rows of more than 2^32 elements give what they give by themselves.  Equal bits
    need equal orders of the sums, which rows off 16-byte boundaries have at equal offsets from one: 40 rows and a
    multiple of 8 rows before them."""
    rows = ((1 << 32) // cols + 70) // 8 * 8
    x = torch.zeros(rows, cols, dtype=torch.bfloat16, device="cuda")
    tail = torch.randn(40, cols, dtype=torch.bfloat16, device="cuda")
    x[-40:] = tail
    w = torch.rand(cols, dtype=torch.bfloat16, device="cuda")
    o = d.dcn_add_rms_norm_forward(x, None, w, quant="int8", keep_out=True, save_rstd=True)
    want = d.dcn_add_rms_norm_forward(tail, None, w, quant="int8", keep_out=True, save_rstd=True)
    for a, b in zip(o, want):
        assert (a is None and b is None) or torch.equal(a[-40:], b)
    assert not o.out[:-40].any() and not o.out8[:-40].any()
    del o
    gx, gw = d.dcn_add_rms_norm_backward(x, x, torch.cat([torch.ones(rows - 40, device="cuda"), want.rstd]), w)
    gx40, gw40 = d.dcn_add_rms_norm_backward(tail, tail, want.rstd, w)
    assert torch.equal(gx[-40:], gx40) and not gx[:-40].any()
    # the weight gradient adds 40 rows' products and zeros, in another order
    mag = (tail.double() ** 2 * want.rstd.double()[:, None]).abs().sum(0)
    assert ((gw.double() - gw40.double()).abs() <= mag * 2 * 50 * U + gw40.double().abs() * 2 * half_step(w.dtype)).all()


def test_binding_refusals(cuda_dev):
    x = torch.randn(4, 64, device="cuda")
    with pytest.raises(ValueError, match="contiguous"):
        d.dcn_add_rms_norm_forward(torch.randn(64, 4, device="cuda").t())
    with pytest.raises(TypeError):
        d.dcn_add_rms_norm_forward(x.double())
    with pytest.raises(TypeError):
        d.dcn_add_rms_norm_forward(x, x.half())
    with pytest.raises(ValueError, match="shape"):
        d.dcn_add_rms_norm_forward(x, x[:3])
    with pytest.raises(ValueError, match="shape"):
        d.dcn_add_rms_norm_forward(x, None, torch.ones(63, device="cuda"))
    with pytest.raises(ValueError, match="quant"):
        d.dcn_add_rms_norm_forward(x, quant="e5m2")
    with pytest.raises(ValueError, match="group"):
        d.dcn_add_rms_norm_forward(x, quant="int8", group=64)
    with pytest.raises(ValueError, match="same buffer"):
        d.dcn_add_rms_norm_forward(x, x, out=x, residual_out=x)
    with pytest.raises(ValueError):
        d.dcn_add_rms_norm_forward(x, keep_out=False)
    with pytest.raises(d.DcnError):
        d.dcn_add_rms_norm_forward(x, eps=0.0)
    with pytest.raises(d.DcnError):
        d.dcn_add_rms_norm_forward(torch.zeros(1, 16385, device="cuda"))
    with pytest.raises(ValueError):
        d.dcn_add_rms_norm_backward(x, x, torch.ones(4, device="cuda"), grad_weight=torch.ones(64, device="cuda"))
    with pytest.raises(d.DcnError):
        d.dcn_add_rms_norm_backward(x, x, torch.ones(4, device="cuda"), torch.ones(64, device="cuda"),
                                    workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))


@pytest.mark.parametrize("group", [0, 128])
@pytest.mark.parametrize("quant", ["e4m3", "int8"])
@pytest.mark.parametrize("cols,k", [(32, 0), (61, 0), (128, 0), (256, 0), (250, 1), (300, 3), (512, 0), (1000, 2),
                                    (1001, 0), (4096, 0), (4383, 1), (9001, 0)])
def test_codes_are_the_rounded_quotients(cols, k, quant, group, cuda_dev):
    """In fp32 `out` is the value that the codes are made of: they are out / scale, divided and rounded once each, with
    no step between (a product with 1 / scale puts some values on the other side of a border)."""
    x, r, w = inputs(4001, cols, torch.float32, cols + 5)
    place = gpu if k == 0 else lambda *ts: [step_off(t, k, 0.0)[0] for t in ts]
    o = d.dcn_add_rms_norm_forward(*place(x, r, w), eps=EPS, quant=quant, group=group, keep_out=True)
    s = o.scale.cpu().repeat_interleave(group or cols, 1)[:, :cols]
    v = o.out.cpu() / s
    if quant == "e4m3":
        assert torch.equal(o.out8.cpu().view(torch.uint8), v.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8))
    else:
        assert torch.equal(o.out8.cpu(), v.round().to(torch.int8))


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("cols", [40, 61, 256, 512, 1000, 1029, 4096, 12001])
def test_backward_of_a_frozen_weight(cols, dtype, cuda_dev):
    """grad_x without the weight's gradient: the same bits, no other launch, no workspace."""
    h, gh, w = gpu(*inputs(203, cols, DT[dtype], 71))
    gy = torch.randn(203, cols).to(DT[dtype]).cuda()
    rstd = definition(h.cpu(), None, None)[2].float().cuda()
    want, _ = d.dcn_add_rms_norm_backward(gy, h, rstd, w, grad_residual_out=gh)
    got, gw = d.dcn_add_rms_norm_backward(gy, h, rstd, w, grad_residual_out=gh, need_grad_weight=False)
    assert gw is None and torch.equal(got, want)
    got, gw = d.dcn_add_rms_norm_backward(gy, h, rstd, w, grad_residual_out=gh, grad_x=gh, need_grad_weight=False)
    assert gw is None and got is gh and torch.equal(got, want)
    with pytest.raises(ValueError):
        d.dcn_add_rms_norm_backward(gy, h, rstd, w, grad_weight=torch.empty_like(w), need_grad_weight=False)
    with pytest.raises(ValueError):
        d.dcn_add_rms_norm_backward(gy, h, rstd, w[1:], need_grad_weight=False)
    e, _ = d.dcn_add_rms_norm_backward(gy[:0], h[:0], rstd[:0], w, need_grad_weight=False)
    assert e.shape == (0, cols)


def test_autograd_asks_for_no_more_than_it_needs(cuda_dev, monkeypatch):
    """A frozen weight's gradient is not formed; a trained one beside frozen inputs is."""
    asked = []
    real = d.dcn_add_rms_norm_backward
    monkeypatch.setattr(d, "dcn_add_rms_norm_backward",
                        lambda *a, **k: asked.append(k.get("need_grad_weight", True)) or real(*a, **k))
    x, r, w = gpu(*inputs(9, 96, torch.float32, 72))
    gy = torch.randn_like(x)
    x.requires_grad_()
    y, _ = d.AddRmsNormFunction.apply(x, r, w, EPS)
    y.backward(gy)
    frozen = x.grad.clone()
    x.grad = None
    w.requires_grad_()
    y, h = d.AddRmsNormFunction.apply(x, r, w, EPS)
    y.backward(gy)
    assert asked == [False, True]
    assert torch.equal(x.grad, frozen) and w.grad is not None
    y, h = d.AddRmsNormFunction.apply(x.detach(), r, w, EPS)
    w.grad = None
    y.backward(gy)
    assert w.grad is not None and asked[-1]
    y, h = d.AddRmsNormFunction.apply(x, r, w.detach(), EPS)
    h.sum().backward()  # the norm's output is not used
