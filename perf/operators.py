"""Cases that measure the operators around the sampling core and its projection:

  norm       dcn_add_rms_norm_forward: residual addition + root-mean-square norm, output in the
             storage type or in 8 bits with scales
  norm_bwd   dcn_add_rms_norm_backward: its gradients
  clip       dcn_clip_grads: the global gradient norm over many tensors, and clipping
  adapters   dcn_proj_adapters_forward: the pointwise projection with low-rank adapters of many
             requests beside the shared weight

`own` False computes the plain form with elementary torch operations in 32 bits; True calls the
library.  Shapes follow this repository's workloads (DCNv4 P4: 8 x 40 x 40 pixels of 512 channels,
DCNv3 P3: 16 x 80 x 80 of 256, Sparse4D: 900 anchors of 256 channels, 16-bit projections
512 -> 512) and generic widths around them.
"""
import math

import numpy as np
import torch

own = False

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
ES = {"f32": 4, "f16": 2, "bf16": 2}
EPS = 1e-6
CLIP_EPS = 1e-6
GROUP = 128          # columns that share a scale in group mode
E4M3_MAX, INT8_MAX = 448.0, 127.0
SCALE_MIN = 2.0 ** -126


def listed():
    return [
        # Sparse4D's 900 anchor features between two decoder operators: a small call, latency counts
        dict(name="norm_f32_900x256", op="norm", rows=900, cols=256, dtype="f32", residual=True, quant="", group=0),
        # residual stream after a DCNv3 P3 block at batch 16: the widest map
        dict(name="norm_bf16_102400x256", op="norm", rows=102400, cols=256, dtype="bf16", residual=True, quant="",
             group=0),
        # DCNv4 P4 block output handed to an 8-bit projection, one scale per pixel
        dict(name="norm_e4m3_f16_12800x512", op="norm", rows=12800, cols=512, dtype="f16", residual=True,
             quant="e4m3", group=0),
        # a wide model's rows in int8 with a scale per 128 columns, an odd number of rows
        dict(name="norm_int8_bf16_2047x4096", op="norm", rows=2047, cols=4096, dtype="bf16", residual=True,
             quant="int8", group=GROUP),
        # training: fp32 backward at the DCNv4 P4 shape, and 16-bit at the P3 shape
        dict(name="normbwd_f32_12800x512", op="norm_bwd", rows=12800, cols=512, dtype="f32", residual=True),
        dict(name="normbwd_bf16_102400x256", op="norm_bwd", rows=102400, cols=256, dtype="bf16", residual=True),
        # gradients of one block (weights 512 x 512 and vectors), clipped into its buffers
        dict(name="clip_f32_13", op="clip", tensors=13, total=1100000, dtype="f32", out="f32", max_norm=1.0),
        # gradients of a whole backbone in bf16, clipped into fp32 master gradients
        dict(name="clip_bf16_301", op="clip", tensors=301, total=97000000, dtype="bf16", out="f32", max_norm=25.0),
        # serving: eight requests of one token each on the 512 -> 512 projection
        dict(name="adapters_f16_8x512", op="adapters", rows=8, cin=512, cout=512, rank=16, adapters=8, requests=8,
             dtype="f16", tokens=True),
        # serving: 48 single tokens over a wide projection, some without an adapter
        dict(name="adapters_bf16_48x4096", op="adapters", rows=48, cin=4096, cout=4096, rank=16, adapters=32,
             requests=48, dtype="bf16", tokens=True),
        # eight images of the DCNv4 P4 batch, each fine-tuned for its own user
        dict(name="adapters_f16_12800x512", op="adapters", rows=12800, cin=512, cout=512, rank=16, adapters=6,
             requests=8, dtype="f16", tokens=False),
        # long ragged requests over a wide projection
        dict(name="adapters_bf16_16111x2048", op="adapters", rows=16111, cin=2048, cout=2048, rank=64, adapters=16,
             requests=37, dtype="bf16", tokens=False),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "norm", "norm_bwd", "clip", "adapters", "adapters"])
    if op in ("norm", "norm_bwd"):
        cols = _log(rng, 8, 8192)
        if rng.random() < 0.7:  # channel counts are mostly multiples of 8; the rest are odd
            cols = max(8, cols // 8 * 8)
        rows = _log(rng, 1, 102400)
        rows = max(1, min(rows, 26000000 // cols))
        c = dict(op=op, rows=rows, cols=cols, dtype=rng.choice(["f32", "f16", "bf16"]),
                 residual=rng.random() < 0.75)
        if op == "norm":
            q = rng.choice(["", "", "e4m3", "int8"])
            c.update(quant=q, group=rng.choice([0, GROUP]) if q else 0)
        return c
    if op == "clip":
        dt = rng.choice(["f32", "f16", "bf16"])
        out = rng.choice([dt, "f32"])
        total = min(_log(rng, 4000, 97000000), 582000000 // (ES[dt] + ES[out]))
        return dict(op=op, tensors=min(_log(rng, 1, 301), total // 8), total=total, dtype=dt, out=out,
                    max_norm=rng.choice([0.1, 1.0, 25.0]))
    cin, cout = _log(rng, 64, 4096) // 8 * 8, _log(rng, 64, 4096) // 8 * 8
    tokens = rng.random() < 0.4
    rows = _log(rng, 1, 64) if tokens else _log(rng, 16, 16384)
    rank = rng.choice([8, 16, 24, 32, 64, 128])
    rows = max(1, min(rows, 16111 * (2048 * 2048 + 64 * 4096) // (cin * cout + rank * (cin + cout))))
    return dict(op=op, rows=rows, cin=cin, cout=cout, rank=rank,
                adapters=rng.randint(1, 32), requests=rows if tokens else min(rows, rng.randint(1, 40)),
                dtype=rng.choice(["f16", "bf16"]), tokens=tokens)


# ------------------------------------------------------------------ inputs

def _sizes(case, seed):
    """Element counts of the gradient tensors: most of the elements in a few matrices, many vectors."""
    r = np.random.RandomState(seed % (1 << 31))
    n, total = case["tensors"], case["total"]
    w = np.exp(r.normal(0.0, 2.0, n))
    s = np.maximum(1, np.floor(w / w.sum() * (total - n))).astype(np.int64)
    s[int(np.argmax(s))] += total - int(s.sum())
    return [int(v) for v in s]


def _requests(case, seed):
    """Row starts [requests + 1] and the adapter of each request (-1: none)."""
    r = np.random.RandomState(seed % (1 << 31))
    m, n = case["rows"], case["requests"]
    if case["tokens"]:
        start = np.arange(n + 1)
    else:
        cut = np.sort(r.randint(0, m + 1, n - 1)) if n > 1 else np.zeros(0, np.int64)
        start = np.concatenate([[0], cut, [m]])
    which = r.randint(0, case["adapters"], n)
    which[r.rand(n) < 0.15] = -1
    return start.astype(np.int32), which.astype(np.int32)


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed))

    def normal(*shape, std=1.0, dt=torch.float32):
        return (torch.randn(*shape, generator=g, device=dev) * std).to(dt)

    op, dt = case["op"], DT[case["dtype"]]
    s = {"case": case}
    if op in ("norm", "norm_bwd"):
        r, c = case["rows"], case["cols"]
        s["weight"] = (1.0 + 0.2 * torch.randn(c, generator=g, device=dev)).to(dt)
        if op == "norm":
            s["x"] = normal(r, c, dt=dt)
            s["residual"] = normal(r, c, std=2.0, dt=dt) if case["residual"] else None
        else:
            s["h"] = normal(r, c, std=2.0, dt=dt)
            # the forward's statistic, as it saved it
            s["rstd"] = (s["h"].float().square().mean(-1) + EPS).rsqrt()
            s["grad_out"] = normal(r, c, dt=dt)
            s["grad_residual"] = normal(r, c, std=0.5, dt=dt) if case["residual"] else None
        return s
    if op == "clip":
        sizes = _sizes(case, seed)
        # gradients of very different scales in one flat buffer, as bucketed data-parallel training
        # keeps them: most tensors start on no particular boundary
        flat = normal(case["total"], dt=torch.float32)
        std = torch.exp(torch.randn(len(sizes), generator=g, device=dev)) * 0.02
        flat *= torch.repeat_interleave(std, torch.tensor(sizes, device=dev), output_size=case["total"])
        s["flat"] = flat.to(dt)
        s["out_flat"] = torch.empty(case["total"], dtype=DT[case["out"]], device=dev)
        s["grads"] = list(s["flat"].split(sizes))
        s["out"] = list(s["out_flat"].split(sizes))
        if own:
            import deformable_convolution_sampling_dcn_b200 as dcn
            # the table of gradient and master buffers, which stay in place over a training run
            s["list"] = dcn.GradList(s["grads"], s["out"])
        return s
    start, which = _requests(case, seed)
    m, k, n, r, l = case["rows"], case["cin"], case["cout"], case["rank"], case["adapters"]
    s["x"] = normal(m, k, dt=dt)
    s["weight"] = normal(n, k, std=k ** -0.5, dt=dt)
    s["bias"] = normal(n, std=0.1, dt=dt)
    s["a"] = normal(l, r, k, std=k ** -0.5, dt=dt)
    s["b"] = normal(l, n, r, std=0.5 * r ** -0.5, dt=dt)
    s["scale"] = 0.5 + torch.rand(l, generator=g, device=dev)
    s["start"] = torch.from_numpy(start).to(dev)
    s["which"] = torch.from_numpy(which).to(dev)
    return s


# ------------------------------------------------------------------ plain forms

def _norm_plain(s):
    case = s["case"]
    dt = s["x"].dtype
    h = s["x"].float()
    if s["residual"] is not None:
        h = (h + s["residual"].float()).to(dt).float()
    y = h * torch.rsqrt(h.square().mean(-1, keepdim=True) + EPS) * s["weight"].float()
    res = h.to(dt) if s["residual"] is not None else None
    if not case["quant"]:
        return y.to(dt), res
    q, scale = _quantise(y, case)
    return q, scale, res


def _quantise(y, case):
    r, c = y.shape
    w = case["group"] or c
    g = -(-c // w)
    yp = torch.nn.functional.pad(y, (0, g * w - c)).view(r, g, w)
    top = E4M3_MAX if case["quant"] == "e4m3" else INT8_MAX
    scale = (yp.abs().amax(-1) / top).clamp(min=SCALE_MIN)
    q = (yp / scale[..., None]).view(r, g * w)[:, :c]
    if case["quant"] == "e4m3":
        return q.clamp(-top, top).to(torch.float8_e4m3fn), scale
    return q.round().clamp(-top, top).to(DT[case["dtype"]]), scale


def _norm_bwd_plain(s):
    dt = s["h"].dtype
    h, gy, rstd = s["h"].float(), s["grad_out"].float(), s["rstd"][:, None]
    xhat = h * rstd
    g = gy * s["weight"].float()
    gx = rstd * (g - xhat * (g * xhat).mean(-1, keepdim=True))
    if s["grad_residual"] is not None:
        gx = gx + s["grad_residual"].float()
    return gx.to(dt), (gy * xhat).sum(0).to(dt)


def _clip_plain(s):
    # one sum of squares per tensor, then one over the tensors
    norm = torch.stack([g.float().square().sum(dtype=torch.float64) for g in s["grads"]]).sum().sqrt().float()
    coef = (s["case"]["max_norm"] / (norm + CLIP_EPS)).clamp(max=1.0)
    [o.copy_(g.float() * coef) for g, o in zip(s["grads"], s["out"])]
    return norm, s["out_flat"]


def _adapters_plain(s):
    case = s["case"]
    m, l, r = case["rows"], case["adapters"], case["rank"]
    x = s["x"].float()
    # request of each row, then its adapter as a one-hot row (all zero where it has none)
    req = (torch.arange(m, device=x.device)[:, None] >= s["start"][None, 1:-1]).sum(1)
    hot = (s["which"][req][:, None] == torch.arange(l, device=x.device)).float() * s["scale"]
    t = (x @ s["a"].float().view(l * r, -1).t()).view(m, l, r) * hot[:, :, None]
    y = x @ s["weight"].float().t() + s["bias"].float()
    y = y + t.view(m, l * r) @ s["b"].float().permute(0, 2, 1).reshape(l * r, -1)
    return y.to(s["x"].dtype)


# ------------------------------------------------------------------ the library

def _run_own(s):
    import deformable_convolution_sampling_dcn_b200 as dcn
    case = s["case"]
    op = case["op"]
    if op == "norm":
        o = dcn.dcn_add_rms_norm_forward(s["x"], s["residual"], s["weight"], eps=EPS, quant=case["quant"] or None,
                                         group=case["group"])
        if not case["quant"]:
            return o.out, o.residual_out
        return (o.out8 if case["quant"] == "e4m3" else o.out8.to(s["x"].dtype)), o.scale, o.residual_out
    if op == "norm_bwd":
        return dcn.dcn_add_rms_norm_backward(s["grad_out"], s["h"], s["rstd"], s["weight"],
                                             grad_residual_out=s["grad_residual"])
    if op == "clip":
        return dcn.dcn_clip_grads(s["list"], case["max_norm"], eps=CLIP_EPS), s["out_flat"]
    return dcn.dcn_proj_adapters_forward(s["x"], s["weight"], s["bias"], s["a"], s["b"], s["start"], s["which"],
                                         scale=s["scale"])


def run(state):
    if own:
        return _run_own(state)
    op = state["case"]["op"]
    if op == "norm":
        return _norm_plain(state)
    if op == "norm_bwd":
        return _norm_bwd_plain(state)
    if op == "clip":
        return _clip_plain(state)
    return _adapters_plain(state)


def work(case):
    op, es = case["op"], ES[case["dtype"]]
    if op in ("norm", "norm_bwd"):
        n, c = case["rows"] * case["cols"], case["cols"]
        if op == "norm_bwd":  # grad_out, h and grad_residual in, grad_x out
            return {"bytes": n * es * (4 if case["residual"] else 3) + 4 * case["rows"] + 2 * c * es, "flops": 12 * n}
        b = n * es * (3 if case["residual"] else 1) + c * es  # x, residual and the new residual
        if case["quant"]:
            b += n + 4 * case["rows"] * (-(-c // case["group"]) if case["group"] else 1)
        else:
            b += n * es
        return {"bytes": b, "flops": (8 if case["quant"] else 6) * n}
    if op == "clip":
        return {"bytes": case["total"] * (es + ES[case["out"]]), "flops": 3 * case["total"]}
    m, k, n, r = case["rows"], case["cin"], case["cout"], case["rank"]
    used = min(case["adapters"], case["requests"])
    return {"bytes": es * (m * k + n * k + n + m * n + used * r * (k + n)),
            "flops": 2 * m * n * k + 2 * m * r * (k + n)}


# ------------------------------------------------------------------ 64 bits, from the definitions

def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "norm":
        h = s["x"].double()
        if s["residual"] is not None:
            h = torch.add(h, s["residual"].double()).to(s["x"].dtype).double()  # the stored residual is the input
        ms = torch.einsum("rc,rc->r", h, h) / case["cols"]
        y = torch.einsum("rc,r,c->rc", h, 1.0 / torch.sqrt(ms + EPS), s["weight"].double())
        res = h if s["residual"] is not None else None
        if not case["quant"]:
            return y, res
        top = E4M3_MAX if case["quant"] == "e4m3" else INT8_MAX
        w = case["group"] or case["cols"]
        parts = [p.abs().max(dim=1).values for p in torch.split(y, w, dim=1)]
        scale = torch.clamp(torch.stack(parts, dim=1) / top, min=SCALE_MIN)
        if case["quant"] == "int8":
            return None, scale, res  # whole numbers: the code next to a border is a choice of the last bit
        q = y / torch.repeat_interleave(scale, w, dim=1)[:, :case["cols"]]  # before its rounding to 8 bits
        return torch.clamp(q, -top, top), scale, res
    if op == "norm_bwd":
        h, gy, rs = s["h"].double(), s["grad_out"].double(), s["rstd"].double()
        w = s["weight"].double()
        # d/dh of sum(gy * w * h * rs(h)) with rs = (mean(h^2) + eps)^(-1/2): drs/dh_j = -rs^3 h_j / cols
        dot = torch.einsum("rc,c,rc->r", gy, w, h)
        gx = torch.einsum("rc,c,r->rc", gy, w, rs) - h * (dot * rs ** 3 / case["cols"])[:, None]
        if s["grad_residual"] is not None:
            gx = gx + s["grad_residual"].double()
        return gx, torch.einsum("rc,rc,r->c", gy, h, rs)
    if op == "clip":
        d = s["flat"].double()
        norm = torch.linalg.vector_norm(d)
        return norm, d * min(1.0, case["max_norm"] / (float(norm) + CLIP_EPS))
    x, w = s["x"].double(), s["weight"].double()
    y = x @ w.t() + s["bias"].double()
    start, which = s["start"].tolist(), s["which"].tolist()
    for i, a in enumerate(which):
        lo, hi = start[i], start[i + 1]
        if a >= 0 and hi > lo:
            y[lo:hi] += float(s["scale"][a]) * ((x[lo:hi] @ s["a"][a].double().t()) @ s["b"][a].double().t())
    return y
