"""Projection with low-rank adapters of many requests on the GPU against 64 bits.

Tolerance per element (u = 2^-24, uT = finfo(T).eps / 2): the contraction has
cin + rank products, exact in fp32, and every addition loses at most one step,
2u of the running sum, which the sum of magnitudes bounds; with more than 64
rows t = scale * A x may be rounded once (uT, and tiny(T) below its normals); the
result is rounded once.
"""
import pytest
import torch

import deformable_convolution_sampling_dcn_b200 as d

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
DT = {"f16": torch.float16, "bf16": torch.bfloat16}


def make(lens, which, cin, cout, rank, adapters, dtype, seed, bias=True, scale=True, rows=None, first=0):
    """Inputs on the CPU; `rows` more than the requests cover leaves padding behind, `first` before."""
    g = torch.Generator().manual_seed(seed)
    dt = DT[dtype]
    start = [first]
    for n in lens:
        start.append(start[-1] + n)
    rows = start[-1] if rows is None else rows
    s = dict(
        x=torch.randn(rows, cin, generator=g).to(dt), weight=(torch.randn(cout, cin, generator=g) * cin ** -0.5).to(dt),
        bias=(torch.randn(cout, generator=g) * 0.2).to(dt) if bias else None,
        a=(torch.randn(adapters, rank, cin, generator=g) * cin ** -0.5).to(dt),
        b=(torch.randn(adapters, cout, rank, generator=g) * rank ** -0.5).to(dt),
        scale=(0.5 + torch.rand(adapters, generator=g)) if scale else None,
        start=torch.tensor(start, dtype=torch.int32), which=torch.tensor(which, dtype=torch.int32))
    return s


def definition(s):
    """(y, tolerance) in 64 bits."""
    dt = s["x"].dtype
    uT = torch.finfo(dt).eps / 2
    tiny = torch.finfo(dt).smallest_normal * torch.finfo(dt).eps / 2
    x, w = s["x"].double(), s["weight"].double()
    y, mag = x @ w.t(), x.abs() @ w.abs().t()
    if s["bias"] is not None:
        y, mag = y + s["bias"].double(), mag + s["bias"].double().abs()
    tr = torch.zeros_like(y)
    start = s["start"].tolist()
    for i, ad in enumerate(s["which"].tolist()):
        lo, hi = start[i], start[i + 1]
        if ad < 0 or ad >= s["a"].shape[0] or lo >= hi:
            continue
        sc = float(s["scale"][ad]) if s["scale"] is not None else 1.0
        a, b = s["a"][ad].double(), s["b"][ad].double()
        t, tm = sc * (x[lo:hi] @ a.t()), sc * (x[lo:hi].abs() @ a.abs().t())
        y[lo:hi] += t @ b.t()
        mag[lo:hi] += tm @ b.abs().t()
        tr[lo:hi] = (t.abs() * uT + tiny) @ b.abs().t()
    n = x.shape[1] + s["a"].shape[1] + 16
    tol = mag * n * 2 * U + y.abs() * uT + tiny
    if x.shape[0] > 64:
        tol = tol + tr * (1 + 2 * uT)
    return y, tol


def call(s, dev="cuda", **kw):
    t = {k: None if v is None else v.to(dev) for k, v in s.items()}
    return d.dcn_proj_adapters_forward(t["x"], t["weight"], t["bias"], t["a"], t["b"], t["start"], t["which"],
                                       scale=t["scale"], **kw)


def check(s, y, rows=slice(None)):
    torch.cuda.synchronize()
    assert d._binding.take_device_error() == 0
    want, tol = definition(s)
    err = (y.double().cpu() - want).abs()
    ok = err <= tol
    assert ok[rows].all(), (float((err / tol)[rows].max()), int((~ok[rows]).sum()))


# rows of each request, adapter of each, cin, cout, rank, adapters
SMALL = [
    ([1], [0], 8, 8, 8, 1),
    ([1], [-1], 64, 64, 16, 1),
    ([1] * 8, [0, 1, 2, -1, 3, 0, 0, 2], 512, 512, 16, 4),
    ([1] * 9, [2, 1, 2, 1, 0, 0, 0, 2, -1], 520, 136, 24, 3),
    ([1] * 17, list(range(16)) + [-1], 1000, 264, 8, 16),
    ([1] * 48, [i % 7 - 1 for i in range(48)], 2048, 1032, 64, 6),
    ([3, 0, 5, 0, 0, 20, 4], [1, 0, -1, 2, 1, 0, 1], 256, 128, 128, 3),   # short requests, empty ones
    ([64], [0], 4096, 256, 32, 1),
    ([33, 31], [1, 1], 96, 72, 40, 2),
    ([65], [0], 64, 64, 16, 1),
    ([128], [0], 8, 8, 8, 1),
    ([100, 28, 1], [0, 1, 0], 64, 72, 8, 2),
    ([1] * 130, [i % 5 - 1 for i in range(130)], 128, 64, 16, 4),
    ([1] * 256, [i % 33 - 1 for i in range(256)], 1000, 136, 16, 32),       # 32 tiles of adapters
    ([70, 0, 30, 100], [1, 0, 0, -1], 4096, 64, 128, 2),
    ([2] * 100, [i % 3 for i in range(100)], 328, 1032, 48, 3),              # two slots a tile, 96 of its rows
    ([0] * 300 + [5] * 50, [i % 4 - 1 for i in range(350)], 200, 264, 24, 3),  # more requests than rows: a slot a row
    ([66, 190], [0, 1], 2056, 520, 64, 2),
]


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("i", range(len(SMALL)))
def test_few_rows(i, dtype, cuda_dev):
    s = make(*SMALL[i], dtype, 10 + i)
    check(s, call(s))


LARGE = [
    ([257], [0], 64, 64, 16, 1),
    ([384], [0], 8, 8, 8, 1),
    ([200, 56, 1], [0, 1, 0], 64, 72, 8, 2),
    ([1] * 300, [i % 5 - 1 for i in range(300)], 128, 64, 16, 4),           # 256 requests in one tile
    ([127, 1, 128, 0, 2, 0, 254], [0, -1, 1, 1, 2, 0, 1], 200, 136, 24, 3),  # at, before and behind tile borders
    ([1600, 1600, 7], [2, -1, 0], 512, 512, 16, 3),
    ([300, 0, 0, 500, 33], [1, 0, 0, 0, 1], 1000, 520, 64, 2),
    ([700], [0], 520, 264, 128, 1),                                          # two blocks of rank
    ([90, 40, 200], [1, 0, 1], 72, 1032, 72, 2),                             # a ragged second block of rank
    ([20000, 13, 5000], [0, 1, 1], 64, 256, 8, 2),                           # several tiles per CTA
    # few tiles and a long contraction: clusters split it, in 2, 4 and 8 parts
    ([270, 0, 30], [1, 0, 0], 4096, 64, 128, 2),
    ([200, 57], [0, 1], 2056, 136, 24, 2),
    ([900, 1, 99, 500], [0, -1, 2, 1], 1000, 104, 16, 3),
    ([266], [0], 192, 64, 8, 1),                                              # as few blocks as splits
    ([3, 300, 700], [2, 1, 0], 3768, 72, 64, 3),
    ([2000, 700], [0, 1], 520, 328, 40, 2),
]


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("i", range(len(LARGE)))
def test_many_rows(i, dtype, cuda_dev):
    s = make(*LARGE[i], dtype, 30 + i)
    check(s, call(s))


@pytest.mark.parametrize("lens,which", [([5, 6], [0, 1]), ([300, 33], [1, 0])])
def test_without_bias_or_scale(lens, which, cuda_dev):
    s = make(lens, which, 136, 80, 16, 2, "f16", 50, bias=False, scale=False)
    check(s, call(s))


@pytest.mark.parametrize("rows,first,lens", [(40, 0, [7, 12]), (40, 5, [7, 12]), (300, 0, [100, 60]),
                                             (300, 9, [150, 100]), (64, 0, [0, 0]), (500, 0, [0, 0]),
                                             (200, 3, [90, 40])])
def test_rows_of_no_request_stay(rows, first, lens, cuda_dev):
    """Padding before the first and behind the last request is left as it was, whatever x holds there."""
    s = make(lens, [1, 0], 64, 96, 16, 2, "bf16", 60, rows=rows, first=first)
    end = first + sum(lens)
    s["x"][end:] = float("nan")
    s["x"][:first] = float("inf")
    out = torch.full((rows, 96), 7.0, dtype=torch.bfloat16, device="cuda")
    y = call(s, out=out)
    assert y is out
    assert (out[:first] == 7).all() and (out[end:] == 7).all()
    check(s, y, slice(first, end))


@pytest.mark.parametrize("lens", [[4, 4, 4], [60, 40, 100], [60, 40, 200]])
def test_one_requests_infinities_stay_its_own(lens, cuda_dev):
    """NaN and infinities in one request's rows or adapter reach no other request in the same tile."""
    s = make(lens, [0, 1, 2], 64, 64, 16, 3, "f16", 70)
    want, tol = definition(s)
    lo, hi = lens[0], lens[0] + lens[1]
    s["a"][1, 3] = float("inf")
    s["b"][1, 5:9] = float("nan")
    s["x"][lo, 0] = float("inf")
    s["x"][hi - 1, 1] = float("nan")
    y = call(s).double().cpu()
    others = list(range(lo)) + list(range(hi, sum(lens)))
    assert ((y - want).abs() <= tol)[others].all()
    assert not torch.isfinite(y[lo:hi]).all(1).any()


def test_bad_adapter_index_is_reported(cuda_dev):
    for lens in ([3, 4], [100, 90], [300, 90]):
        s = make(lens, [7, 1], 64, 64, 16, 2, "bf16", 80)
        y = call(s)
        torch.cuda.synchronize()
        assert d._binding.take_device_error() == 2
        want, tol = definition(s)  # counts it as none
        assert ((y.double().cpu() - want).abs() <= tol).all()
        s["which"][0] = -2
        call(s)
        torch.cuda.synchronize()
        assert d._binding.take_device_error() == 2
        assert d._binding.take_device_error() == 0


def test_adapter_of_an_empty_request_is_not_looked_at(cuda_dev):
    for lens in ([3, 0, 4], [300, 0, 90]):
        s = make(lens, [0, 9, 1], 64, 64, 16, 2, "bf16", 81)
        y = call(s)
        torch.cuda.synchronize()
        assert d._binding.take_device_error() == 0
        want, tol = definition(s)
        assert ((y.double().cpu() - want).abs() <= tol).all()


def test_more_than_32_bit_elements(cuda_dev):
    """Offsets are 64-bit: the last rows of a batch, and the last adapter, of more than 2^32 elements."""
    s = make([70, 200], [0, 1], 512, 512, 16, 2, "bf16", 82)
    rows = (1 << 32) // 512 + 700
    x = torch.zeros(rows, 512, dtype=torch.bfloat16, device="cuda")
    x[-270:] = s["x"].cuda()
    big = dict(s, x=x, start=torch.tensor([0, rows - 270, rows - 200, rows], dtype=torch.int32),
               which=torch.tensor([-1, 0, 1], dtype=torch.int32))
    y = call(big)
    want, tol = definition(s)
    assert ((y[-270:].double().cpu() - want).abs() <= tol).all()
    assert (y[:-270] == s["bias"].cuda()).all()
    del x, y, big
    n = (1 << 32) // (1024 * 32) + 3
    for lens in ([5, 7], [200, 100]):
        s = make(lens, [1, 0], 1024, 1024, 32, 2, "bf16", 83)
        want, tol = definition(s)
        a = torch.zeros(n, 32, 1024, dtype=torch.bfloat16, device="cuda")
        b = torch.zeros(n, 1024, 32, dtype=torch.bfloat16, device="cuda")
        scale = torch.zeros(n, device="cuda")
        a[-2:], b[-2:], scale[-2:] = s["a"].cuda(), s["b"].cuda(), s["scale"].cuda()
        y = call(dict(s, a=a, b=b, scale=scale, which=s["which"] + (n - 2)))
        assert ((y.double().cpu() - want).abs() <= tol).all()


def test_tables_out_of_range_stay_in_bounds(cuda_dev):
    """Starts outside [0, rows]: cut off; the rows of the well-formed requests are right."""
    for rows in (50, 400):
        s = make([rows // 2, rows - rows // 2], [0, 1], 64, 64, 16, 2, "f16", 81)
        bad = dict(s, start=torch.tensor([-5, rows // 2, rows + 1000], dtype=torch.int32))
        y = call(bad)
        check(s, y)


@pytest.mark.parametrize("n", [1024, 1025, 3000])
def test_many_requests(n, cuda_dev):
    """Request tables in shared memory and beyond it."""
    lens = [(i * 7) % 3 for i in range(n)]
    s = make(lens, [i % 4 - 1 for i in range(n)], 64, 64, 8, 3, "f16", n)
    check(s, call(s))
    lens = [1 if i % (n // 40) == 0 else 0 for i in range(n)]  # few rows, many empty requests
    s = make(lens, [i % 4 - 1 for i in range(n)], 64, 64, 8, 3, "f16", n)
    assert s["x"].shape[0] <= 256
    check(s, call(s))


def test_no_adapters_and_empty(cuda_dev):
    for rows in (5, 200, 400):
        s = make([rows], [-1], 64, 64, 16, 1, "f16", 90)
        s["a"], s["b"], s["scale"] = s["a"][:0], s["b"][:0], s["scale"][:0]
        check(s, call(s))
    s = make([0], [0], 64, 64, 16, 1, "f16", 91)
    assert call(s).shape == (0, 64)
    s = make([], [], 64, 64, 16, 1, "f16", 92, rows=10)
    out = torch.full((10, 64), 3.0, dtype=torch.float16, device="cuda")
    call(s, out=out)
    assert (out == 3).all()


def test_leading_dimensions(cuda_dev):
    """A batch of images: requests are its images, each H * W rows."""
    s = make([30] * 4, [0, 1, -1, 1], 64, 72, 16, 2, "bf16", 93)
    flat = call(s)
    s["x"] = s["x"].view(4, 5, 6, 64)
    y = call(s)
    assert y.shape == (4, 5, 6, 72) and torch.equal(y.view(120, 72), flat)


@pytest.mark.parametrize("lens", [[1] * 20, [50, 100], [200, 100]])
def test_streams_graphs_and_repeats(lens, cuda_dev):
    n = len(lens)
    s = make(lens, [i % 3 - 1 for i in range(n)], 512, 256, 16, 2, "bf16", 94)
    t = {k: v.cuda() for k, v in s.items()}
    args = (t["x"], t["weight"], t["bias"], t["a"], t["b"], t["start"], t["which"])
    want = d.dcn_proj_adapters_forward(*args, scale=t["scale"])
    check(s, want)
    assert torch.equal(d.dcn_proj_adapters_forward(*args, scale=t["scale"]), want)
    # two streams at once, each with its own workspace
    outs = []
    streams = [torch.cuda.Stream() for _ in range(2)]
    for st in streams:
        st.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(st):
            outs += [d.dcn_proj_adapters_forward(*args, scale=t["scale"]) for _ in range(5)]
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in outs)
    # two captured graphs, replayed in turn after the request table changed
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            o = d.dcn_proj_adapters_forward(*args, scale=t["scale"])
        graphs.append((g, o))
    s["which"] = (s["which"] + 2) % 3 - 1
    t["which"].copy_(s["which"])
    for g, o in graphs:
        o.zero_()
        g.replay()
    torch.cuda.synchronize()
    for _, o in graphs:
        check(s, o)


def test_calls_on_several_streams_do_not_block_each_other(cuda_dev):
    """CTA pairs and clusters of several calls share the SMs and their tensor memory; every width of tile, with
    splits, in flight at once on four streams.  A wait that ran out would show in the error word."""
    cases = [make([270, 0, 30], [1, 0, 0], 4096, 64, 128, 2, "f16", 1), make([700], [0], 520, 264, 128, 1, "bf16", 2),
             make([900, 1, 99, 500], [0, -1, 2, 1], 1000, 1000, 64, 3, "f16", 3),
             make([1600, 1600, 7], [2, -1, 0], 512, 512, 16, 3, "bf16", 4)]
    dev = [{k: None if v is None else v.cuda() for k, v in c.items()} for c in cases]
    want = [call(c) for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    outs = [[] for _ in cases]
    torch.cuda.synchronize()
    for _ in range(25):
        for i, (st, t) in enumerate(zip(streams, dev)):
            with torch.cuda.stream(st):
                outs[i].append(d.dcn_proj_adapters_forward(t["x"], t["weight"], t["bias"], t["a"], t["b"], t["start"],
                                                           t["which"], scale=t["scale"]))
    torch.cuda.synchronize()
    assert d._binding.take_device_error() == 0
    for o, w in zip(outs, want):
        assert all(torch.equal(y, w) for y in o)


def test_binding_refusals(cuda_dev):
    s = {k: v.cuda() for k, v in make([4], [0], 64, 64, 16, 1, "f16", 95).items()}

    def go(**kw):
        t = dict(s, **kw)
        return d.dcn_proj_adapters_forward(t["x"], t["weight"], t["bias"], t["a"], t["b"], t["start"], t["which"],
                                           scale=t["scale"], workspace=t.get("ws"))

    with pytest.raises(TypeError):
        go(weight=s["weight"].bfloat16())
    with pytest.raises(ValueError):
        go(weight=s["weight"][:, :32].contiguous())
    with pytest.raises(ValueError):
        go(b=s["b"][:, :32].contiguous())
    with pytest.raises(TypeError):
        go(start=s["start"].long())
    with pytest.raises(ValueError):
        go(start=s["start"][:1])
    with pytest.raises(TypeError):
        go(scale=s["scale"].half())
    with pytest.raises(ValueError, match="CUDA"):
        go(which=s["which"].cpu())
    with pytest.raises(d.DcnError):
        go(ws=torch.empty(16, dtype=torch.uint8, device="cuda"))
    f = {k: v.float() if v.is_floating_point() else v for k, v in s.items()}
    with pytest.raises(d.DcnError) as e:
        d.dcn_proj_adapters_forward(f["x"], f["weight"], f["bias"], f["a"], f["b"], f["start"], f["which"])
    assert e.value.status == d._binding.DCN_ERR_UNSUPPORTED
    odd = {k: v.cuda() for k, v in make([4], [0], 60, 64, 16, 1, "f16", 95).items()}
    with pytest.raises(d.DcnError):
        go(**{k: odd[k] for k in ("x", "weight", "a")})


def definition_32(s):
    """(y, tolerance) where t is held in 32 bits: with more than 64 rows it may be two values of the storage type, off by
    uT^2 |t| (the rounding error, rounded) and half a subnormal of fp16; where eight neighbouring ranks of t go beyond
    2^15, they are scaled down by a power of two to below it, and that is tiny / 2^14 of their largest."""
    dt = s["x"].dtype
    uT = torch.finfo(dt).eps / 2
    tiny = torch.finfo(dt).smallest_normal * uT
    _, tol = definition(dict(s, b=torch.zeros_like(s["b"])))  # for the bias, W and the output's tiny; its tr is zero
    want, _ = definition(s)
    x, start = s["x"].double(), s["start"].tolist()
    n = x.shape[1] + s["a"].shape[1] + 16
    plain, _ = definition(dict(s, b=torch.zeros_like(s["b"])))
    tol = tol - plain.abs() * uT + want.abs() * uT
    for i, ad in enumerate(s["which"].tolist()):
        lo, hi = start[i], start[i + 1]
        if ad < 0 or lo >= hi:
            continue
        sc = float(s["scale"][ad]) if s["scale"] is not None else 1.0
        a, b = s["a"][ad].double(), s["b"][ad].double()
        t, tm = sc * (x[lo:hi] @ a.t()), sc * (x[lo:hi].abs() @ a.abs().t())
        low = torch.clamp(t.abs().view(hi - lo, -1, 8).amax(2).repeat_interleave(8, 1) * 2.0 ** -14, min=1.0) * tiny
        tol[lo:hi] += tm @ b.abs().t() * n * 2 * U + (t.abs() * uT * uT * (1 + 2 * uT) + low) @ b.abs().t()
    return want, tol


# rows of each request, adapter of each, cin, cout, rank, adapters: blocks of 32, 64 and 128 bytes of t, split and unsplit
# contractions, both halves of a pair's tile, rows of no adapter
HELD = [
    ([300], [0], 16, 64, 8, 1), ([200, 9, 300], [0, -1, 1], 16, 136, 16, 2), ([513], [0], 16, 264, 24, 1),
    ([90, 400], [1, 0], 16, 72, 32, 2), ([700, 11], [0, 1], 16, 328, 64, 2), ([257], [0], 16, 64, 104, 1),
    ([800], [0], 16, 512, 128, 1), ([270, 0, 30], [1, 0, 0], 4096, 64, 128, 2), ([200, 57], [0, 1], 2056, 136, 24, 2),
    ([266], [0], 3768, 64, 16, 1), ([20000, 13, 5000], [0, 1, 1], 64, 256, 32, 2),
]


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("i", range(len(HELD)))
def test_t_is_held_in_32_bits(i, dtype, cuda_dev):
    """No rounding of t to the storage type, whose error would show where y is small."""
    s = make(*HELD[i], dtype, 200 + i)
    s["bias"] = None
    s["weight"] = (s["weight"].double() / 64).to(DT[dtype])
    y = call(s)
    torch.cuda.synchronize()
    assert d._binding.take_device_error() == 0
    want, tol = definition_32(s)
    err = (y.double().cpu() - want).abs()
    assert (err <= tol).all(), (float((err / tol).max()), int((err > tol).sum()))


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("i", range(len(HELD)))
def test_t_beyond_the_storage_type(i, dtype, cuda_dev):
    """Values of t past 65504, up to 2^24, in some rows, with a B so small that y is within its type."""
    s = make(*HELD[i], dtype, 230 + i)
    dt = DT[dtype]
    big = torch.rand(s["x"].shape[0], 1, generator=torch.Generator().manual_seed(i)) < 0.4
    s["x"] = torch.where(big, s["x"] * 2.0 ** 12, s["x"]).to(dt)
    s["weight"] = (s["weight"].double() * 2.0 ** -12).to(dt)
    s["a"] = (s["a"].double() * 2.0 ** 8).to(dt)
    s["b"] = (s["b"].double() * 2.0 ** -12).to(dt)
    s["scale"] = s["scale"] * 2.0 ** 2
    y = call(s)
    torch.cuda.synchronize()
    want, tol = definition_32(s)
    assert (want.abs() < 60000).all()
    err = (y.double().cpu() - want).abs()
    assert (err <= tol).all(), (float((err / tol).max()), int((err > tol).sum()))


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("cin,cout,rank", [(64, 72, 16), (64, 72, 40), (4096, 64, 128)])
def test_infinite_t_beside_large_values(cin, cout, rank, dtype, cuda_dev):
    """An infinity in one rank of t gives infinities and NaN where 64 bits do, and no NaN beside them."""
    s = make([200, 100], [0, 1], cin, cout, rank, 2, dtype, 250)
    s["x"][:, 1] = s["x"][:, 1].abs() + 1  # times an infinity of A: of one sign
    s["a"][1, 3, 1] = float("inf")
    s["a"][1, 4] *= 2.0 ** 14
    s["b"][1, ::2, 3] = 0.0
    s["b"][1, :, 4] *= 2.0 ** -10
    y = call(s).double().cpu()
    want, _ = definition(s)
    assert want[200:].isnan().any() and want[200:].isinf().any()
    assert torch.equal(y.isnan(), want.isnan()) and torch.equal(y.isinf(), want.isinf())
    assert torch.equal(y[y.isinf()], want[y.isinf()])


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("rows,first,lens", [(700, 0, [200, 57, 400]), (1500, 3, [900, 0, 590]), (300, 0, [100, 100, 100]),
                                             (2000, 700, [1, 1, 1200])])
def test_least_workspace(rows, first, lens, dtype, cuda_dev):
    """With the least workspace the rows go in passes, which cut requests: the same values, other rows as they were."""
    s = make(lens, [1, 0, 1], 64, 520, 24, 2, dtype, 260, rows=rows, first=first)
    p = d._binding.DadaptParams(rows, 64, 520, 24, 2, 3, 1 if dtype == "f16" else 2)
    least = d.lib().dcn_proj_adapters_workspace_bytes(p)
    full = d.lib().dcn_proj_adapters_workspace_full_bytes(p)
    assert rows * 24 * 2 == least and rows * (24 * 4 + (16 if dtype == "f16" else 0)) == full
    end = first + sum(lens)
    for n in (least, least + 999, full - 1, full):
        out = torch.full((rows, 520), 7.0, dtype=DT[dtype], device="cuda")
        y = call(s, out=out, workspace=torch.empty(n, dtype=torch.uint8, device="cuda"))
        assert (out[:first] == 7).all() and (out[end:] == 7).all()
        check(s, y, slice(first, end))
        want, tol = definition_32(s)
        assert ((y.double().cpu() - want).abs() <= tol)[first:end].all()


def test_both_routes_on_several_streams(cuda_dev):
    """The row route with all of an SM's tensor memory (129 to 256 rows) and little shared memory, beside pairs and
    clusters of the tile route that wait for one another, and beside the fused core + projection."""
    cases = [make([130], [0], 128, 512, 8, 1, "f16", 1), make([1] * 200, [i % 3 - 1 for i in range(200)], 128, 64, 16, 2, "bf16", 2),
             make([270, 0, 30], [1, 0, 0], 4096, 64, 128, 2, "f16", 3), make([700], [0], 520, 264, 128, 1, "bf16", 4),
             make([300], [0], 2048, 64, 16, 1, "f16", 5), make([1600, 1600, 7], [2, -1, 0], 512, 512, 16, 3, "bf16", 6)]
    dev = [{k: None if v is None else v.cuda() for k, v in c.items()} for c in cases]
    want = [call(c) for c in cases]
    g = torch.Generator().manual_seed(7)
    shapes = (2, 20, 20, 64), (2, 20, 20, 4, 9, 2), (2, 20, 20, 4, 9), (512, 64)
    core = [torch.randn(s, generator=g).half().cuda() for s in shapes]

    def fused():
        return d.dcn_core_forward_proj(*core, None, group=4, fused=True)
    want.append(fused())
    outs = [[] for _ in want]
    streams = [torch.cuda.Stream() for _ in want]
    torch.cuda.synchronize()
    for _ in range(25):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                t = dev[i] if i < len(dev) else None
                outs[i].append(fused() if t is None else d.dcn_proj_adapters_forward(
                    t["x"], t["weight"], t["bias"], t["a"], t["b"], t["start"], t["which"], scale=t["scale"]))
    torch.cuda.synchronize()
    assert d._binding.take_device_error() == 0
    for o, y in zip(outs, want):
        assert all(torch.equal(v, y) for v in o)


@pytest.mark.parametrize("pad", [300, 900, 5000, (1 << 20) - 5])
@pytest.mark.parametrize("where", ["end", "middle", "front"])
@pytest.mark.parametrize("lens", [[30, 1, 9], [300, 1, 90], [1000, 7, 1200]])
def test_tables_filled_up_with_empty_requests(lens, where, pad, cuda_dev):
    """A table of a fixed size, as a captured graph keeps it: the empty requests, wherever they are, do not keep a call
    busy (no wait runs out, and the padded end costs next to nothing)."""
    s = make(lens, [1, -1, 0], 64, 520, 16, 2, "bf16", 270, rows=sum(lens) + 5)
    start, which = s["start"].tolist(), s["which"].tolist()
    i = {"end": 3, "middle": 2, "front": 0}[where]
    s["start"] = torch.tensor(start[:i] + [start[i]] * pad + start[i:], dtype=torch.int32)
    s["which"] = torch.tensor(which[:i] + [1] * pad + which[i:], dtype=torch.int32)
    t = {k: v.cuda() for k, v in s.items()}
    args = (t["x"], t["weight"], t["bias"], t["a"], t["b"], t["start"], t["which"])
    out = torch.full((sum(lens) + 5, 520), 7.0, dtype=torch.bfloat16, device="cuda")
    d.dcn_proj_adapters_forward(*args, scale=t["scale"], out=out)
    begin, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    begin.record()
    d.dcn_proj_adapters_forward(*args, scale=t["scale"], out=out)
    end.record()
    torch.cuda.synchronize()
    assert d._binding.take_device_error() == 0
    assert begin.elapsed_time(end) < (5.0 if where == "end" else 500.0)  # ms
    assert (out[sum(lens):] == 7).all()
    short = {"start": torch.tensor(start, dtype=torch.int32), "which": torch.tensor(which, dtype=torch.int32)}
    want, tol = definition(dict(s, **short))
    assert ((out.double().cpu() - want).abs() <= tol)[:sum(lens)].all()


def test_a_table_that_is_not_ascending_ends(cuda_dev):
    """Wrong values are allowed, a call that runs on is not; the next call is right."""
    g = torch.Generator().manual_seed(3)
    for n, rows in ((200, 600), (3000, 600), (3000, 100)):
        s = make([rows], [0], 64, 264, 16, 2, "f16", 271)
        bad = dict(s, start=torch.randint(-50, rows + 50, (n + 1,), generator=g).int(),
                   which=torch.randint(-2, 3, (n,), generator=g).int())
        call(bad)
        torch.cuda.synchronize()
        assert d._binding.take_device_error() in (0, 2)
        check(s, call(s))


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("byte", [0x00, 0x7f, 0xff])
@pytest.mark.parametrize("lens,first,rows", [([90, 0, 60, 5], 3, 170), ([300, 1, 200, 40], 7, 600), ([1] * 4, 0, 4),
                                             ([250, 0, 10, 40], 0, 300)])
def test_what_the_workspace_held_does_not_matter(lens, first, rows, byte, dtype, cuda_dev):
    """NaN, infinities and exponents of earlier calls lie in the workspace, also for rows with no adapter or request."""
    s = make(lens, [1, 0, -1, 0], 520, 136, 24, 2, dtype, 280, rows=rows, first=first)
    p = d._binding.DadaptParams(rows, 520, 136, 24, 2, 4, 1 if dtype == "f16" else 2)
    ws = torch.full((d.lib().dcn_proj_adapters_workspace_full_bytes(p),), byte, dtype=torch.uint8, device="cuda")
    out = torch.full((rows, 136), 7.0, dtype=DT[dtype], device="cuda")
    end = first + sum(lens)
    for _ in range(2):
        y = call(s, out=out, workspace=ws)
        check(s, y, slice(first, end))
        want, tol = definition_32(s)
        assert ((y.double().cpu() - want).abs() <= tol)[first:end].all()
        assert (out[:first] == 7).all() and (out[end:] == 7).all()


def test_large_t_in_captured_calls(cuda_dev):
    """Exponents are of the call: a graph replayed on other inputs, and two of them in flight."""
    sets = [make([300, 40, 200], [0, 1, -1], 64, 136, 16, 2, "f16", 290 + i) for i in range(2)]
    sets[1]["x"][100:320] *= 2.0 ** 10
    for s in sets:
        s["a"] *= 2.0 ** 6
        s["b"] *= 2.0 ** -12
        s["weight"] *= 2.0 ** -4
    t = {k: v.cuda() for k, v in sets[0].items()}
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            o = d.dcn_proj_adapters_forward(t["x"], t["weight"], t["bias"], t["a"], t["b"], t["start"], t["which"],
                                            scale=t["scale"])
        graphs.append((g, o))
    for i in (1, 0, 1):
        for k, v in sets[i].items():
            t[k].copy_(v)
        torch.cuda.synchronize()
        streams = [torch.cuda.Stream() for _ in graphs]
        for (g, _), st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
        torch.cuda.synchronize()
        want, tol = definition_32(sets[i])
        for _, o in graphs:
            assert ((o.double().cpu() - want).abs() <= tol).all()
