"""Host-side checks of the norm and gradient-clipping calls (fake,
never-dereferenced pointers; no call here reaches a kernel launch)."""
import ctypes

import pytest

from deformable_convolution_sampling_dcn_b200 import _binding as B
from deformable_convolution_sampling_dcn_b200 import build as build_mod


@pytest.fixture(scope="module")
def lib():
    build_mod.build()
    return B.lib()


def norm(**kw):
    base = dict(rows=4, cols=64, eps=1e-6, dtype=1, quant=0, group=0)
    base.update(kw)
    return B.DnormParams(**base)


def fwd(lib, p, x=16, res=None, w=None, res_out=None, out=16, out8=None, scale=None, rstd=None):
    return lib.dcn_add_rms_norm_forward(ctypes.byref(p), x, res, w, res_out, out, out8, scale, rstd, None)


@pytest.mark.parametrize("kw,status", [
    (dict(cols=0), B.DCN_ERR_SHAPE), (dict(rows=-1), B.DCN_ERR_SHAPE), (dict(cols=16385), B.DCN_ERR_UNSUPPORTED),
    (dict(eps=0.0), B.DCN_ERR_SHAPE), (dict(eps=-1.0), B.DCN_ERR_SHAPE), (dict(eps=float("nan")), B.DCN_ERR_SHAPE),
    (dict(eps=float("inf")), B.DCN_ERR_SHAPE), (dict(dtype=3), B.DCN_ERR_UNSUPPORTED),
    (dict(quant=3), B.DCN_ERR_UNSUPPORTED), (dict(quant=1, group=64), B.DCN_ERR_UNSUPPORTED),
    (dict(group=128), B.DCN_ERR_SHAPE), (dict(rows=1 << 36, cols=64), B.DCN_ERR_SHAPE),
])
def test_norm_params(lib, kw, status):
    assert fwd(lib, norm(**kw)) == status


def test_norm_pointers(lib):
    p = norm()
    assert lib.dcn_add_rms_norm_forward(None, 16, None, None, None, 16, None, None, None, None) == B.DCN_ERR_NULL
    assert fwd(lib, p, x=None) == B.DCN_ERR_NULL
    assert fwd(lib, p, out=None) == B.DCN_ERR_NULL
    assert fwd(lib, p, res=16) == B.DCN_ERR_NULL                 # residual without residual_out
    assert fwd(lib, p, res_out=16) == B.DCN_ERR_NULL
    assert fwd(lib, p, out8=16, scale=16) == B.DCN_ERR_NULL      # 8-bit buffers without an 8-bit output
    assert fwd(lib, norm(quant=1), out8=16) == B.DCN_ERR_NULL
    assert fwd(lib, norm(quant=2), scale=16) == B.DCN_ERR_NULL
    assert fwd(lib, p, x=17) == B.DCN_ERR_ALIGN
    assert fwd(lib, norm(dtype=0), w=18) == B.DCN_ERR_ALIGN
    assert fwd(lib, norm(quant=1), out8=16, scale=18) == B.DCN_ERR_ALIGN
    assert fwd(lib, p, rstd=18) == B.DCN_ERR_ALIGN
    assert fwd(lib, norm(rows=0), x=None, out=None) == B.DCN_OK


def test_norm_backward_checks(lib):
    f, p = lib.dcn_add_rms_norm_backward, norm()
    need = lib.dcn_add_rms_norm_backward_workspace_bytes(ctypes.byref(p))
    assert need == 64 * 4  # one CTA takes the four rows
    many = lib.dcn_add_rms_norm_backward_workspace_bytes(ctypes.byref(norm(rows=1 << 20)))
    assert many % (64 * 4) == 0 and 148 <= many // (64 * 4) <= 1184  # a row of partial sums per CTA, at most 8 an SM
    assert lib.dcn_add_rms_norm_backward_workspace_bytes(ctypes.byref(norm(rows=1 << 30))) == many
    assert lib.dcn_add_rms_norm_backward_workspace_bytes(ctypes.byref(norm(cols=0))) == -1
    b = ctypes.byref(p)
    assert f(b, None, 16, 16, None, None, 16, None, None, 0, None) == B.DCN_ERR_NULL
    assert f(b, 16, 16, 16, 16, None, 16, None, 16, need, None) == B.DCN_ERR_NULL       # weight without grad_weight
    assert f(b, 16, 16, 16, None, None, 16, 16, 16, need, None) == B.DCN_ERR_NULL
    assert f(b, 16, 16, 16, 16, None, 16, 16, None, 0, None) == B.DCN_ERR_NULL          # no workspace
    assert f(b, 16, 16, 16, 16, None, 16, 16, 16, need - 1, None) == B.DCN_ERR_SHAPE
    assert f(b, 16, 16, 16, 16, None, 16, 16, 16, -1, None) == B.DCN_ERR_SHAPE
    assert f(b, 16, 16, 16, 16, None, 16, 16, 8, need, None) == B.DCN_ERR_ALIGN
    assert f(b, 16, 16, 18, None, None, 16, None, None, 0, None) == B.DCN_ERR_ALIGN
    e = ctypes.byref(norm(rows=0))
    assert f(e, None, None, None, None, None, None, None, None, 0, None) == B.DCN_OK


def grads(ptrs=(64,), numel=(4,), dtypes=(0,), **kw):
    n = len(ptrs)
    p = B.DclipParams(kw.get("count", n), kw.get("kind", 0), kw.get("max_norm", 1.0), kw.get("eps", 1e-6))
    return (p, (ctypes.c_void_p * n)(*ptrs), (ctypes.c_int64 * n)(*numel), (ctypes.c_int32 * n)(*dtypes))


def clip(lib, t, outs=None, od=None, norm=16, ws=16, nbytes=1 << 20):
    p, g, n, dt = t
    o = None if outs is None else (ctypes.c_void_p * len(outs))(*outs)
    odt = None if od is None else (ctypes.c_int32 * len(od))(*od)
    return lib.dcn_clip_grads(ctypes.byref(p), g, n, dt, o, odt, norm, ws, nbytes, None)


def test_clip_checks(lib):
    need = lib.dcn_grad_norm_workspace_bytes(1)
    assert need > 0 and lib.dcn_grad_norm_workspace_bytes(-1) == -1
    assert lib.dcn_grad_norm_workspace_bytes(5000) > lib.dcn_grad_norm_workspace_bytes(900)
    assert clip(lib, grads(), norm=None) == B.DCN_ERR_NULL
    assert clip(lib, grads(), ws=None) == B.DCN_ERR_NULL
    assert clip(lib, grads(), ws=8) == B.DCN_ERR_ALIGN
    assert clip(lib, grads(), norm=18) == B.DCN_ERR_ALIGN
    assert clip(lib, grads(), nbytes=need - 1) == B.DCN_ERR_SHAPE
    assert clip(lib, grads(), nbytes=-1) == B.DCN_ERR_SHAPE
    assert clip(lib, grads(count=-1)) == B.DCN_ERR_SHAPE
    assert clip(lib, grads(kind=2)) == B.DCN_ERR_UNSUPPORTED
    assert clip(lib, grads(max_norm=-1.0)) == B.DCN_ERR_SHAPE
    assert clip(lib, grads(max_norm=float("inf"))) == B.DCN_ERR_SHAPE
    assert clip(lib, grads(eps=0.0)) == B.DCN_ERR_SHAPE
    assert clip(lib, grads(numel=(-1,))) == B.DCN_ERR_SHAPE
    assert clip(lib, grads(numel=(1 << 41,))) == B.DCN_ERR_SHAPE
    assert clip(lib, grads(dtypes=(3,))) == B.DCN_ERR_UNSUPPORTED
    assert clip(lib, grads(ptrs=(None,))) == B.DCN_ERR_NULL
    assert clip(lib, grads(ptrs=(66,))) == B.DCN_ERR_ALIGN
    assert clip(lib, grads(), outs=(None,), od=(0,)) == B.DCN_ERR_NULL
    assert clip(lib, grads(), outs=(66,), od=(0,)) == B.DCN_ERR_ALIGN
    assert clip(lib, grads(), outs=(128,), od=(5,)) == B.DCN_ERR_UNSUPPORTED
    assert clip(lib, grads(), outs=(128,)) == B.DCN_ERR_NULL
    assert clip(lib, grads(), outs=(64,), od=(1,)) == B.DCN_ERR_UNSUPPORTED  # in place in another type
    assert lib.dcn_grad_norm(None, None, None, None, 16, 16, 1 << 20, None) == B.DCN_ERR_NULL


def adapt(**kw):
    base = dict(rows=100, cin=64, cout=64, rank=16, num_adapters=3, num_requests=4, dtype=1)
    base.update(kw)
    return B.DadaptParams(**base)


def proj(lib, p, x=16, w=16, bias=16, a=16, b=16, scale=16, start=16, which=16, out=16, ws=16, nbytes=1 << 30):
    return lib.dcn_proj_adapters_forward(ctypes.byref(p), x, w, bias, a, b, scale, start, which, out, ws, nbytes, None)


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=0), B.DCN_ERR_UNSUPPORTED), (dict(rows=-1), B.DCN_ERR_SHAPE), (dict(cin=0), B.DCN_ERR_SHAPE),
    (dict(cin=60), B.DCN_ERR_UNSUPPORTED), (dict(cout=4), B.DCN_ERR_UNSUPPORTED), (dict(rank=4), B.DCN_ERR_UNSUPPORTED),
    (dict(rank=136), B.DCN_ERR_UNSUPPORTED), (dict(cin=65544), B.DCN_ERR_UNSUPPORTED),
    (dict(rows=(1 << 30) + 1), B.DCN_ERR_SHAPE), (dict(num_adapters=1 << 20, cout=2048), B.DCN_ERR_SHAPE),
    (dict(num_requests=-1), B.DCN_ERR_SHAPE), (dict(num_adapters=-1), B.DCN_ERR_SHAPE),
])
def test_adapter_params(lib, kw, status):
    p = adapt(**kw)
    assert proj(lib, p) == status
    assert lib.dcn_proj_adapters_workspace_bytes(ctypes.byref(p)) == -1


def test_adapter_pointers(lib):
    p = adapt()
    need = lib.dcn_proj_adapters_workspace_bytes(ctypes.byref(p))
    assert lib.dcn_proj_adapters_workspace_bytes(ctypes.byref(adapt(rows=1000))) == 1000 * 16 * 2  # t in the storage type
    # few rows: t in fp32, and fp32 partial sums of 16 rows for one block of the weight
    assert lib.dcn_proj_adapters_workspace_bytes(ctypes.byref(adapt(rows=10))) == (10 * 16 + 2 * 16 * 128) * 4
    for name in ("x", "w", "start", "which", "out", "ws", "a", "b"):
        assert proj(lib, p, **{name: None}) == B.DCN_ERR_NULL, name
    for name in ("x", "w", "bias", "a", "b", "out", "ws"):
        assert proj(lib, p, **{name: 8}) == B.DCN_ERR_ALIGN, name
    for name in ("scale", "start", "which"):
        assert proj(lib, p, **{name: 18}) == B.DCN_ERR_ALIGN, name
    assert proj(lib, p, nbytes=need - 1) == B.DCN_ERR_SHAPE
    assert proj(lib, p, nbytes=-1) == B.DCN_ERR_SHAPE
    assert proj(lib, adapt(rows=0), x=None, out=None) == B.DCN_OK
    assert proj(lib, adapt(num_requests=0), x=None) == B.DCN_OK
    assert lib.dcn_proj_adapters_forward(None, 16, 16, 16, 16, 16, 16, 16, 16, 16, 16, 1 << 20, None) == B.DCN_ERR_NULL


def test_out_is_not_the_new_residual(lib):
    assert fwd(lib, norm(), res=32, res_out=16, out=16) == B.DCN_ERR_UNSUPPORTED


def test_python_refusals_without_a_gpu(lib):
    import torch
    # an empty list takes its device from the norm, which has to be on one
    for call in (lambda n: B.dcn_grad_norm([], norm=n), lambda n: B.dcn_clip_grads([], 1.0, norm=n)):
        with pytest.raises(ValueError, match="CUDA"):
            call(torch.zeros(()))
    # sizes that would not fit the library's 32 bits
    with pytest.raises(ValueError, match="32 bits"):
        B._rows(torch.empty(0, 2 ** 32 + 8))
    assert B._rows(torch.empty(0, 2 ** 31 - 1)) == (0, 2 ** 31 - 1)
    # a workspace on another device than the tensors
    class Elsewhere(torch.Tensor):
        is_cuda = True

        def get_device(self):
            return 1
    other = torch.zeros(64, dtype=torch.uint8).as_subclass(Elsewhere)
    assert B._workspace(other, 1) == (other.data_ptr(), 64)
    with pytest.raises(ValueError, match="workspace is on"):
        B._workspace(other, 0)


def test_adapter_workspaces(lib):
    """The least workspace and the one of a single pass, which holds t of more than 256 rows in 32 bits and, in fp16, 16
    exponents a row."""
    least, full = lib.dcn_proj_adapters_workspace_bytes, lib.dcn_proj_adapters_workspace_full_bytes
    for kw in (dict(rows=1000), dict(rows=257, rank=128), dict(rows=1 << 20, rank=8)):
        p = adapt(**kw)
        q = adapt(dtype=2, **kw)
        assert least(ctypes.byref(p)) == least(ctypes.byref(q)) == p.rows * p.rank * 2
        assert full(ctypes.byref(p)) == p.rows * (p.rank * 4 + 16) and full(ctypes.byref(q)) == p.rows * p.rank * 4
    few = ctypes.byref(adapt(rows=10))
    assert least(few) == full(few)
    assert full(ctypes.byref(adapt(cin=60))) == -1


@pytest.mark.parametrize("rank", [16, 64, 128])
@pytest.mark.parametrize("rows", [80, 128, 256])
def test_single_tokens_take_the_row_route(lib, rows, rank):
    """The row route, whose workspace is one size, where every row is a request of its own, whatever the width; a prompt
    of high rank takes the tiles."""
    def route(**kw):
        p = ctypes.byref(adapt(rows=rows, rank=rank, **kw))
        return "rows" if lib.dcn_proj_adapters_workspace_bytes(p) == lib.dcn_proj_adapters_workspace_full_bytes(p) else "tiles"
    for cin, cout in ((512, 512), (1024, 1024), (1024, 4096), (4096, 1024), (4096, 4096)):
        assert route(cin=cin, cout=cout, num_requests=rows) == "rows"
        assert route(cin=cin, cout=cout, num_requests=1 << 20) == "rows"  # a padded table may hold as many
    assert rank < 128 or rows < 128 or route(cin=4096, cout=4096, num_requests=1) == "tiles"


def test_norm_backward_of_a_frozen_weight(lib):
    f, b = lib.dcn_add_rms_norm_backward_input, ctypes.byref(norm())
    assert f(None, 16, 16, 16, 16, None, 16, None) == B.DCN_ERR_NULL
    for i in range(1, 7):
        if i in (4, 5):  # weight, grad_residual_out
            continue
        args = [b, 16, 16, 16, 16, None, 16, None]
        args[i] = None
        assert f(*args) == B.DCN_ERR_NULL
    for i, bad in ((1, 17), (2, 17), (3, 18), (4, 17), (5, 17), (6, 17)):
        args = [b, 16, 16, 16, 16, None, 16, None]
        args[i] = bad
        assert f(*args) == B.DCN_ERR_ALIGN
    assert f(ctypes.byref(norm(cols=0)), 16, 16, 16, 16, None, 16, None) == B.DCN_ERR_SHAPE
    assert f(ctypes.byref(norm(rows=0)), None, None, None, None, None, None, None) == B.DCN_OK
