"""Global gradient norm and clipping on the GPU against 64 bits.

Tolerances (u = 2^-24): 4 fp32 squares, fused into their sum, are added in fp32
(at most 4u of the sum), or 8 exact squares of 16 bits (7u); everything above is
fp64 and the root is rounded once: at most 3.5u + u on the norm.  The factor
adds 3 roundings, the product one, a 16-bit output half a step.
"""
import math

import pytest
import torch

import deformable_convolution_sampling_dcn_b200 as d

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def tensors(sizes, dt, seed, scale=0.05):
    g = torch.Generator().manual_seed(seed)
    return [(torch.randn(s, generator=g) * scale).to(dt) for s in sizes]


def norm64(ts, kind=2.0):
    if not any(t.numel() for t in ts):
        return 0.0
    if kind == 2.0:
        return math.sqrt(sum(float(t.double().square().sum()) for t in ts))
    return max(float(t.double().abs().max()) for t in ts if t.numel())


def norm_tol(dt):
    return 5 * U


def check_clip(ts, got, norm, max_norm, eps, out_dt, tol_n):
    n = norm64(ts)
    assert abs(float(norm) - n) <= n * tol_n
    c = min(1.0, max_norm / (n + eps))
    for t, o in zip(ts, got):
        want = t.double() * c
        step = 0.0 if out_dt == torch.float32 else torch.finfo(out_dt).eps / 2
        small = torch.finfo(out_dt).smallest_normal * torch.finfo(out_dt).eps
        assert o.dtype == out_dt
        assert ((o.double().cpu() - want).abs() <= want.abs() * (tol_n + 5 * U + step) + small).all()


SIZES = [(1,), (3, 5), (0,), (512, 512), (512,), (17, 1023), (16384,), (16385,), (16383,), (2, 0, 3), (40000,), ()]


@pytest.mark.parametrize("out_dtype", [None, "f32", "f16", "bf16"])
@pytest.mark.parametrize("dtype", list(DT))
def test_clip(dtype, out_dtype, cuda_dev):
    dt = DT[dtype]
    for max_norm in (0.5, 1e6):
        ts = tensors(SIZES, dt, 3)
        gs = [t.cuda() for t in ts]
        outs = None if out_dtype is None else [torch.full(t.shape, 9.0, dtype=DT[out_dtype], device="cuda") for t in ts]
        norm = d.dcn_clip_grads(gs, max_norm, out=outs)
        check_clip(ts, outs or gs, norm, max_norm, 1e-6, DT[out_dtype or dtype], norm_tol(dt))
        if outs:
            assert all(torch.equal(g.cpu(), t) for g, t in zip(gs, ts))
        elif max_norm > 1:
            assert all(torch.equal(g.cpu(), t) for g, t in zip(gs, ts))  # a factor of one writes nothing


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("offset", [0, 1, 3, 7])
def test_views_of_one_buffer(offset, dtype, cuda_dev):
    """Tensors that start anywhere in a bucket, output buckets with another phase; neighbours stay untouched."""
    dt = DT[dtype]
    sizes = [5, 1, 16390, 8, 2047, 33, 50000, 2]
    total = sum(sizes)
    for out_dt, out_off in ((dt, 2), (torch.float32, offset), (torch.bfloat16, 5)):
        bucket = torch.randn(total + 16, generator=torch.Generator().manual_seed(offset)).to(dt)
        b = bucket.cuda()
        gs = list(b[offset:offset + total].split(sizes))
        out = torch.full((total + 16,), 3.0, dtype=out_dt, device="cuda")
        norm = d.dcn_clip_grads(gs, 1.0, out=list(out[out_off:out_off + total].split(sizes)))
        ts = list(bucket[offset:offset + total].split(sizes))
        check_clip(ts, out[out_off:out_off + total].split(sizes), norm, 1.0, 1e-6, out_dt, norm_tol(dt))
        assert (out[:out_off] == 3).all() and (out[out_off + total:] == 3).all()
        assert torch.equal(b.cpu(), bucket)
        d.dcn_clip_grads(gs, 0.25)  # in place
        check_clip(ts, gs, norm, 0.25, 1e-6, dt, norm_tol(dt))
        assert torch.equal(b[:offset].cpu(), bucket[:offset])
        assert torch.equal(b[offset + total:].cpu(), bucket[offset + total:])


@pytest.mark.parametrize("n", [1, 63, 64, 65, 959, 960, 961, 2000])
def test_table_sizes(n, cuda_dev):
    """Up to several tables of tensors, one of them with a single tensor."""
    sizes = [1 + (i * 37) % 300 for i in range(n)]
    ts = tensors(sizes, torch.float32, n)
    gs = [t.cuda() for t in ts]
    lst = d.GradList(gs)
    assert abs(float(d.dcn_grad_norm(lst)) - norm64(ts)) <= 5 * U * norm64(ts)
    norm = d.dcn_clip_grads(lst, 0.1)
    check_clip(ts, gs, norm, 0.1, 1e-6, torch.float32, 5 * U)


@pytest.mark.parametrize("n", [64, 960, 1920])
def test_empty_tensors_behind_a_full_table(n, cuda_dev):
    ts = tensors([(j % 7 + 1,) for j in range(n)] + [(0,)] * 5, torch.float32, 13)
    for max_norm in (0.1, 1e6):
        gs = [t.cuda() for t in ts]
        norm = torch.full((), -1.0, device="cuda")
        d.dcn_clip_grads(gs, max_norm, norm=norm)
        check_clip(ts, gs, norm, max_norm, 1e-6, torch.float32, norm_tol(torch.float32))
    assert abs(float(d.dcn_grad_norm([t.cuda() for t in ts])) - norm64(ts)) <= norm64(ts) * norm_tol(torch.float32)


def test_mixed_types(cuda_dev):
    ts = [torch.randn(1000).to(dt) for dt in (torch.float32, torch.bfloat16, torch.float16) for _ in range(2)]
    gs = [t.cuda() for t in ts]
    norm = d.dcn_clip_grads(gs, 1.0)
    n = norm64(ts)
    assert abs(float(norm) - n) <= 5 * U * n
    for t, g in zip(ts, gs):
        want = t.double() / (n + 1e-6)
        assert ((g.double().cpu() - want).abs() <= want.abs() * (torch.finfo(t.dtype).eps / 2 + 12 * U) + 1e-7).all()


@pytest.mark.parametrize("dtype", list(DT))
def test_max_norm_kind(dtype, cuda_dev):
    ts = tensors(SIZES, DT[dtype], 8)
    ts[3][17, 3] = -2.5
    assert float(d.dcn_grad_norm([t.cuda() for t in ts], norm_type=float("inf"))) == 2.5
    gs = [t.cuda() for t in ts]
    assert float(d.dcn_clip_grads(gs, 1.25, norm_type=float("inf"), eps=1e-20)) == 2.5
    assert all(torch.equal(g.cpu(), t * 0.5) for g, t in zip(gs, ts))


def test_magnitudes_outside_fp32_squares(cuda_dev):
    """Squares that underflow or overflow fp32 still give the norm."""
    for dt in (torch.float32, torch.bfloat16):
        for v in (1e-30, 1e25):
            t = torch.full((30000,), v).to(dt)
            n = norm64([t])
            assert abs(float(d.dcn_grad_norm([t.cuda()])) - n) <= 5 * U * n


def test_non_finite(cuda_dev):
    gs = [torch.ones(100, device="cuda"), torch.ones(70000, device="cuda", dtype=torch.bfloat16)]
    gs[1][69999] = float("nan")
    for kind in (2.0, float("inf")):
        assert math.isnan(float(d.dcn_grad_norm(gs, norm_type=kind)))
    assert math.isnan(float(d.dcn_clip_grads(gs, 1.0)))
    assert all(g.isnan().all() for g in gs)
    gs = [torch.ones(100, device="cuda"), torch.ones(20, device="cuda")]
    gs[0][5] = -float("inf")
    assert math.isinf(float(d.dcn_clip_grads(gs, 1.0)))
    assert gs[0][5].isnan() and (gs[0][:5] == 0).all() and (gs[1] == 0).all()


def test_empty_lists_and_zero_gradients(cuda_dev):
    n = torch.full((), 5.0, device="cuda")
    assert float(d.dcn_grad_norm([], norm=n)) == 0.0
    n.fill_(5.0)
    assert float(d.dcn_clip_grads([], 1.0, norm=n)) == 0.0
    assert float(d.dcn_clip_grads([torch.empty(0, device="cuda")], 1.0)) == 0.0
    z = torch.zeros(33, device="cuda")
    assert float(d.dcn_clip_grads([z], 1.0)) == 0.0 and (z == 0).all()
    g = torch.ones(4, device="cuda")
    d.dcn_clip_grads([g], 0.0)
    assert (g == 0).all()


def test_repeats_bit_for_bit_streams_and_graphs(cuda_dev):
    ts = tensors([100001, 70000, 333], torch.float32, 5)
    gs = [t.cuda() for t in ts]
    lst = d.GradList(gs)
    want = d.dcn_grad_norm(lst)
    for _ in range(3):
        assert torch.equal(d.dcn_grad_norm(lst), want)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = d.dcn_grad_norm(gs)
    s.synchronize()
    assert torch.equal(got, want)
    # two graphs over the same list: each keeps its own partial results
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            n = d.dcn_clip_grads(lst, 1.0)
        graphs.append((g, n))
    graphs[0][0].replay()
    torch.cuda.synchronize()
    check_clip(ts, gs, graphs[0][1], 1.0, 1e-6, torch.float32, 5 * U)
    for g, t in zip(gs, ts):
        g.copy_(t * 3)
    graphs[1][0].replay()
    torch.cuda.synchronize()
    check_clip([t * 3 for t in ts], gs, graphs[1][1], 1.0, 1e-6, torch.float32, 5 * U)


def test_more_than_32_bit_elements(cuda_dev):
    """One tensor of more than 2^32 bf16 elements: offsets are 64-bit."""
    n = (1 << 32) + 5
    t = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    t[-1] = 3.0
    t[0] = 4.0
    assert float(d.dcn_clip_grads([t], 2.5, eps=1e-20)) == 5.0
    assert float(t[-1]) == 1.5 and float(t[0]) == 2.0 and float(t[1 << 31]) == 0.0


def test_refusals(cuda_dev):
    g = torch.ones(64, device="cuda")
    with pytest.raises(ValueError, match="overlap"):
        d.dcn_clip_grads([g, g], 1.0)
    with pytest.raises(ValueError, match="overlap"):
        d.GradList([g[:40], g[30:]])
    with pytest.raises(ValueError, match="overlap"):
        d.GradList([g[:32]], [g[16:48]])
    with pytest.raises(ValueError, match="contiguous"):
        d.GradList([torch.ones(8, 8, device="cuda").t()])
    with pytest.raises(ValueError, match="CUDA"):
        d.GradList([torch.ones(8)])
    with pytest.raises(TypeError):
        d.GradList([g.double()])
    with pytest.raises(ValueError):
        d.GradList([g], [torch.ones(63, device="cuda")])
    with pytest.raises(ValueError):
        d.dcn_grad_norm([])
    with pytest.raises(ValueError):
        d.dcn_grad_norm([g], norm_type=1.0)
    with pytest.raises(ValueError):
        d.dcn_clip_grads(d.GradList([g]), 1.0, out=[g])
    for bad in (dict(max_norm=-1.0), dict(max_norm=float("nan")), dict(max_norm=1.0, eps=0.0)):
        with pytest.raises(d.DcnError):
            d.dcn_clip_grads([g], **bad)
    assert (g == 1).all()


def test_channels_last(cuda_dev):
    """Convolution gradients that lie channels-last are as dense as others; an out buffer lies as its gradient does."""
    g = torch.Generator().manual_seed(31)
    cl, cl3 = torch.channels_last, torch.channels_last_3d
    grads = [torch.randn(8, 5, 3, 3, generator=g).cuda().to(memory_format=cl),
             torch.randn(4, 3, 2, 3, 3, generator=g).cuda().to(memory_format=cl3),
             torch.randn(7, 9, generator=g).cuda(), torch.randn(6, 1, 3, 3, generator=g).cuda()]
    assert not grads[0].is_contiguous() and not grads[1].is_contiguous()
    want = torch.sqrt(sum((t.double() ** 2).sum() for t in grads))
    c = min(1.0, 0.5 / (float(want) + 1e-6))
    out = [torch.empty_like(t, dtype=torch.bfloat16) for t in grads]
    assert out[0].is_contiguous(memory_format=cl)
    norm = d.dcn_clip_grads(grads, 0.5, out=out)
    assert abs(float(norm) - float(want)) <= 4 * 2.0 ** -24 * float(want)
    for t, o in zip(grads, out):
        exact = t.double() * c
        assert ((o.double() - exact).abs() <= exact.abs() * (2.0 ** -8 + 8 * 2.0 ** -24)).all()
    before = [t.clone() for t in grads]
    d.dcn_clip_grads(grads, 0.5)
    for t, b in zip(grads, before):
        assert t.stride() == b.stride()
        exact = b.double() * c
        assert ((t.double() - exact).abs() <= exact.abs() * 8 * 2.0 ** -24).all()
    with pytest.raises(ValueError, match="memory formats"):
        d.GradList([grads[0]], [torch.empty(8, 5, 3, 3, device="cuda")])
    d.GradList([grads[3]], [torch.empty(6, 1, 3, 3, device="cuda").to(memory_format=cl)])  # one channel: both at once
    with pytest.raises(ValueError, match="contiguous"):
        d.GradList([grads[0].permute(1, 0, 2, 3)])
