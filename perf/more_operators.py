"""Measured cases of the linear with a fused epilogue and of the residual norm.

A pass is one call of an operator as a Float8 training or serving step of a
transformer block makes it: a linear whose bias, activation and residual are
applied where its output tile is finished, the gradient through that
activation behind the next linear's product, the gradient through a bias in
front of a quantize, and the norms after and before a block with the gate and
the residual between them.  With ``own`` false ``run`` computes the same
outputs with elementary torch operations in 32 bits.

Kinds of case:
  linear           serving: y = act(x W^T + bias) + residual for M tokens
  linear_rows      serving: y and its per-token E4M3 codes
  linear_train     the pre-activation z, and the codes of y and its transpose
  linear_bwd       dz = (dY W) act'(z), its codes and the bias's gradient
  bias_bwd         the same of a given dY, without the product
  resnorm          s = alpha x + gate N(b), y = N(s), and the statistics
  resnorm_rows     serving: s and the per-token codes of y
  resnorm_quantize training: s, the codes of y and its transpose, statistics
  resnorm_bwd      dx, db with its codes, and the parameters' gradients

Codes are returned as float8 tensors (the values they stand for, in units of
1 / scale); an amax is a bf16 value and returned as one.  The statistics of
the norm in front of the next block are those of the stream as it is stored:
where that is bf16, a value next to a rounding border moves them by more than
their 32 bits tell, so they are returned of fp32 streams (y and its codes
show them otherwise).
"""
import math

import torch

own = False

EPS = 1e-5
E4M3_MAX, E5M2_MAX = 448.0, 57344.0
ACTS = ("none", "relu", "gelu", "gelu_tanh", "silu", "relu2")
ROOT_2_PI = math.sqrt(2.0 / math.pi)
CUBIC = 0.044715


def listed():
    return [
        # decode: one token through the first linear of a GELU feed-forward
        dict(name="linear_token", kind="linear_rows", M=1, N=14336, K=4096, rowwise=True,
             act="gelu", residual=False),
        # a decode batch of 50 sequences through the second linear, added to
        # the residual stream
        dict(name="linear_batch_residual", kind="linear", M=50, N=4096, K=14336, rowwise=False,
             act="none", residual=True),
        # training forward of an 8B-sized first linear
        dict(name="linear_train_8b", kind="linear_train", M=8192, N=14336, K=4096, rowwise=False,
             act="gelu", store_y=False),
        # a tensor-parallel slice at a ragged token count, rowwise scales
        dict(name="linear_train_odd", kind="linear_train", M=1040, N=1808, K=784, rowwise=True,
             act="silu", store_y=True),
        # gradient of that activation behind the second linear's product
        dict(name="linear_bwd_8b", kind="linear_bwd", M=8192, N=14336, K=4096, rowwise=False,
             act="gelu", e5m2=True),
        # the same on a small ragged block, rowwise scales, E4M3
        dict(name="linear_bwd_odd", kind="linear_bwd", M=528, N=4112, K=400, rowwise=True,
             act="gelu_tanh", e5m2=False),
        # the output gradient of the second linear: codes and bias gradient
        dict(name="bias_bwd_8b", kind="bias_bwd", M=8192, N=4096, rowwise=False, act="none",
             e5m2=True),
        # decode: one token between two blocks
        dict(name="resnorm_token", kind="resnorm_rows", rows=1, cols=4096, rms=True, post=True,
             pre=True, gate=True),
        # a packed prefill of odd count and width, fp32 residual stream
        dict(name="resnorm_odd_f32", kind="resnorm", rows=777, cols=1001, rms=False, post=True,
             pre=True, gate=False, dtype="f32"),
        # training forward between two 8B-sized blocks
        dict(name="resnorm_quantize_8b", kind="resnorm_quantize", rows=8192, cols=4096, rms=True,
             post=True, pre=True, gate=True, rowwise=False),
        # its backward, E5M2 codes of the block's output gradient
        dict(name="resnorm_bwd_8b", kind="resnorm_bwd", rows=8192, cols=4096, rms=True, post=True,
             pre=True, gate=True, dtype="bf16", codes=True, rowwise=False, e5m2=True),
        # backward at an odd token count, fp32 stream, a width that is no
        # multiple of 8
        dict(name="resnorm_bwd_odd_f32", kind="resnorm_bwd", rows=1539, cols=2050, rms=False,
             post=True, pre=True, gate=True, dtype="f32", codes=False),
    ]


def draw(rng):
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    def log16(lo, hi):
        return 16 * log(lo / 16.0, hi / 16.0)

    def coin():
        return rng.random() < 0.5

    kind = rng.choice(("linear", "linear_rows", "linear_train", "linear_bwd", "bias_bwd",
                       "resnorm", "resnorm_rows", "resnorm_quantize", "resnorm_bwd"))
    if kind in ("linear", "linear_rows"):
        return dict(kind=kind, M=log(1, 300), N=log16(512, 14336), K=log16(256, 14336),
                    rowwise=kind == "linear_rows" or coin(), act=rng.choice(ACTS),
                    residual=coin())
    if kind in ("linear_train", "linear_bwd"):
        case = dict(kind=kind, M=log16(64, 8192), N=log16(256, 14336), K=log16(128, 4096),
                    rowwise=coin(), act=rng.choice(ACTS))
        case["store_y" if kind == "linear_train" else "e5m2"] = coin()
        return case
    if kind == "bias_bwd":
        return dict(kind=kind, M=log16(16, 8192), N=log16(256, 14336), rowwise=coin(),
                    act=rng.choice(ACTS), e5m2=coin())
    post = coin()
    case = dict(kind=kind, rms=coin(), post=post, pre=True, gate=coin())
    if kind == "resnorm_rows":
        return dict(case, rows=log(1, 512), cols=log16(256, 16384))
    if kind == "resnorm_quantize":
        return dict(case, rows=log16(16, 8192), cols=log16(256, 8192), rowwise=coin())
    case["pre"] = not post or coin()
    dtype = rng.choice(("bf16", "f32"))
    if kind == "resnorm_bwd" and coin():
        return dict(case, rows=log16(16, 8192), cols=log16(256, 8192), dtype=dtype, codes=True,
                    rowwise=coin(), e5m2=coin())
    case.update(rows=log(1, 8192), cols=log(8, 8192), dtype=dtype)
    return dict(case, codes=False) if kind == "resnorm_bwd" else case


# ----------------------------------------------------------------- inputs --

def _quantize(x, rowwise, fmax, ftype, transposed):
    """Codes (uint8) and fp32 scales of a bf16 matrix, as a program that
    quantized its operands earlier holds them."""
    def codes(v, s):
        return (v.float() * s).clamp(-fmax, fmax).to(ftype).view(torch.uint8)

    if not rowwise:
        s = fmax / x.abs().amax().float().clamp(min=1e-12).reshape(1)
        return (codes(x, s).t().contiguous() if transposed else codes(x, s)), s
    v = x.t().contiguous() if transposed else x
    s = fmax / v.abs().amax(1).float().clamp(min=1e-12)
    return codes(v, s[:, None]), s


def _code_buffers(rows, cols, rowwise):
    nr, nc, na = (rows, cols, rows + cols) if rowwise else (1, 1, 1)
    new = lambda shape, dtype: torch.empty(shape, dtype=dtype, device="cuda")
    return dict(q=new((rows, cols), torch.uint8), qt=new((cols, rows), torch.uint8),
                scale=new(nr, torch.float32), scale_t=new(nc, torch.float32),
                amax=new(na, torch.float32))


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    bf, f32, u8 = torch.bfloat16, torch.float32, torch.uint8

    def normal(shape, sigma=1.0, dtype=bf):
        return (torch.randn(shape, generator=gen, device="cuda") * sigma).to(dtype)

    new = lambda shape, dtype: torch.empty(shape, dtype=dtype, device="cuda")
    kind = case["kind"]
    if kind.startswith("resnorm"):
        return _prepare_resnorm(case, gen, normal, new)
    st = dict(case=case, ws=None)
    M, N, rw = case["M"], case["N"], case["rowwise"]
    if kind == "bias_bwd":
        st.update(dy=normal((M, N), 1e-2), dbias=new(N, f32), codes=_code_buffers(M, N, rw),
                  z=None, dz=None)
        if case["act"] != "none":
            st.update(z=normal((M, N)), dz=new((M, N), bf))
        return st
    K = case["K"]
    e4 = torch.float8_e4m3fn
    if kind == "linear_bwd":
        e5 = case["e5m2"]
        st["dyq"], st["sdy"] = _quantize(normal((M, K), 1e-2), rw, E5M2_MAX if e5 else E4M3_MAX,
                                         torch.float8_e5m2 if e5 else e4, False)
        # the transposed copy of the next linear's weight [K, N]
        st["wtq"], st["swt"] = _quantize(normal((K, N), 0.02), rw, E4M3_MAX, e4, True)
        st.update(z=normal((M, N)), dz=new((M, N), bf), dbias=new(N, bf),
                  codes=_code_buffers(M, N, rw))
        return st
    # weights that give pre-activations of order one, whatever K
    st["xq"], st["sx"] = _quantize(normal((M, K)), rw, E4M3_MAX, e4, False)
    st["wq"], st["sw"] = _quantize(normal((N, K), K ** -0.5), rw, E4M3_MAX, e4, False)
    st.update(bias=normal(N, 0.2), residual=None, y=new((M, N), bf))
    if case.get("residual"):
        st["residual"] = normal((M, N), 2.0)
    if kind == "linear_rows":
        st["codes"] = dict(q=new((M, N), u8), scale=new(M, f32), amax=new(M, f32))
    if kind == "linear_train":
        st.update(z=new((M, N), bf), codes=_code_buffers(M, N, rw))
        if not case["store_y"]:
            st["y"] = None
    return st


def _prepare_resnorm(case, gen, normal, new):
    bf, f32, u8 = torch.bfloat16, torch.float32, torch.uint8
    rows, cols = case["rows"], case["cols"]
    kind = case["kind"]
    stream = f32 if case.get("dtype") == "f32" else bf
    st = dict(case=case, ws=None, alpha=0.875)
    # a residual stream: an offset, and one channel in 64 much larger
    gain = torch.ones(cols, device="cuda")
    gain[::64] = 8.0
    x = torch.randn((rows, cols), generator=gen, device="cuda") * gain + 0.25
    b = normal((rows, cols), 1.5)
    pair = lambda: ((1.0 + 0.1 * normal(cols, 1.0, f32)).to(bf), normal(cols, 0.1))
    st.update(b=b, post=pair() if case["post"] else None, pre=pair() if case["pre"] else None,
              gate=(0.5 + 0.2 * normal(cols, 1.0, f32)).to(bf) if case["gate"] else None)
    stats = {n: new(rows, f32) if case[n.split("_")[1]] else None
             for n in ("mean_post", "rstd_post", "mean_pre", "rstd_pre")}
    if case["rms"]:
        stats.update(mean_post=None, mean_pre=None)
    if kind == "resnorm_rows":
        stats = dict.fromkeys(stats)
    st["stats"] = stats
    if kind != "resnorm_bwd":
        st.update(x=x.to(stream), s=new((rows, cols), stream))
        if kind == "resnorm":
            st["y"] = new((rows, cols), bf) if case["pre"] else None
        elif kind == "resnorm_rows":
            st["codes"] = dict(q=new((rows, cols), u8), scale=new(rows, f32),
                               amax=new(rows, f32))
        else:
            st["codes"] = _code_buffers(rows, cols, case["rowwise"])
        return st
    # backward: the stream behind the block and the statistics that the
    # forward pass left
    s = x.to(stream)
    for name, v in (("post", b), ("pre", s)):
        if case[name]:
            v = v.double()
            mean = torch.zeros_like(v[:, 0]) if case["rms"] else v.mean(1)
            var = (v - mean[:, None]).square().mean(1)
            stats["rstd_" + name] = (var + EPS).rsqrt().float()
            if not case["rms"]:
                stats["mean_" + name] = mean.float()
    grads = dict(dx=new((rows, cols), stream), db=new((rows, cols), bf),
                 dgate=new(cols, f32) if case["gate"] else None)
    for name in ("post", "pre"):
        for p in ("weight", "bias"):
            grads["d%s_%s" % (name, p)] = new(cols, f32) if case[name] else None
    st.update(s=s, dy=normal((rows, cols), 1e-2) if case["pre"] else None,
              ds=normal((rows, cols), 1e-2, stream), grads=grads,
              codes=_code_buffers(rows, cols, case["rowwise"]) if case["codes"] else None)
    return st


def _returned(case, stats):
    """The statistics among the outputs."""
    hidden = {"mean_post", "mean_pre"} if case["rms"] else set()
    if case.get("dtype") != "f32":
        hidden |= {"mean_pre", "rstd_pre"}
    return {n: v for n, v in stats.items() if v is not None and n not in hidden}


# ------------------------------------------------------------- plain form --

def _codes(y, rowwise, fmax, ftype):
    """Codes of a bf16 matrix and of its transpose, and the bf16 amax."""
    v = y.float()
    if not rowwise:
        amax = v.abs().amax().reshape(1)
        q = (v * (fmax / amax.clamp(min=1e-12))).clamp(-fmax, fmax).to(ftype)
        return q, q.t().contiguous(), amax.to(torch.bfloat16)
    ar, ac = v.abs().amax(1), v.abs().amax(0)
    q = (v * (fmax / ar.clamp(min=1e-12))[:, None]).clamp(-fmax, fmax).to(ftype)
    qt = (v * (fmax / ac.clamp(min=1e-12))).clamp(-fmax, fmax).to(ftype).t().contiguous()
    return q, qt, torch.cat((ar, ac)).to(torch.bfloat16)


def _row_codes(y):
    v = y.float()
    amax = v.abs().amax(1)
    q = (v * (E4M3_MAX / amax.clamp(min=1e-12))[:, None]).clamp(-E4M3_MAX, E4M3_MAX)
    return q.to(torch.float8_e4m3fn), amax.to(torch.bfloat16)


def _act(z, act):
    if act == "none":
        return z
    if act == "relu":
        return z.clamp(min=0.0)
    if act == "relu2":
        return z.clamp(min=0.0).square()
    if act == "silu":
        return z / (1.0 + torch.exp(-z))
    if act == "gelu_tanh":
        return z / (1.0 + torch.exp(-2.0 * ROOT_2_PI * (z + CUBIC * z * z * z)))
    return 0.5 * z * torch.erfc(z * -math.sqrt(0.5))


def _slope(z, act):
    if act == "none":
        return torch.ones_like(z)
    if act == "relu":
        return (z > 0).to(z.dtype)
    if act == "relu2":
        return 2.0 * z.clamp(min=0.0)
    if act == "silu":
        s = 1.0 / (1.0 + torch.exp(-z))
        return s * (1.0 + z * (1.0 - s))
    if act == "gelu_tanh":
        s = 1.0 / (1.0 + torch.exp(-2.0 * ROOT_2_PI * (z + CUBIC * z * z * z)))
        return s + z * s * (1.0 - s) * 2.0 * ROOT_2_PI * (1.0 + 3.0 * CUBIC * z * z)
    return (0.5 * torch.erfc(z * -math.sqrt(0.5))
            + z * torch.exp(-0.5 * z * z) * (0.5 * ROOT_2_PI))


def _plain_linear(st):
    case = st["case"]
    e4, bf = torch.float8_e4m3fn, torch.bfloat16
    col = lambda s: s[:, None] if case["rowwise"] else s
    kind, act = case["kind"], case["act"]
    if kind in ("linear_bwd", "bias_bwd"):
        fmax, ft = (E5M2_MAX, torch.float8_e5m2) if case["e5m2"] else (E4M3_MAX, e4)
        if kind == "bias_bwd":
            dh = st["dy"].float()
        else:
            dh = (st["dyq"].view(ft).float() @ st["wtq"].view(e4).float().t() / col(st["sdy"])
                  / st["swt"])
        dz = dh if st["z"] is None else dh * _slope(st["z"].float(), act)
        dzb = dz.to(bf)
        q, qt, amax = _codes(dzb, case["rowwise"], fmax, ft)
        r = dict(dbias=dz.sum(0).to(st["dbias"].dtype), q=q, qt=qt, amax=amax)
        return r if st["dz"] is None else dict(dz=dzb, **r)
    z = (st["xq"].view(e4).float() @ st["wq"].view(e4).float().t() / col(st["sx"]) / st["sw"]
         + st["bias"].float())
    zb = z.to(bf)
    # a linear without an activation is rounded once, behind the residual
    y = z if act == "none" else _act(zb.float(), act)
    if st["residual"] is not None:
        y = y + st["residual"].float()
    y = y.to(bf)
    if kind == "linear":
        return dict(y=y)
    if kind == "linear_rows":
        q, amax = _row_codes(y)
        return dict(y=y, q=q, amax=amax)
    q, qt, amax = _codes(y, case["rowwise"], E4M3_MAX, e4)
    r = dict(z=zb, q=q, qt=qt, amax=amax)
    return dict(y=y, **r) if case["store_y"] else r


def _norm(v, pair, rms):
    mean = torch.zeros_like(v[:, 0]) if rms else v.mean(1)
    d = v - mean[:, None]
    rstd = 1.0 / torch.sqrt((d * d).mean(1) + EPS)
    return d * rstd[:, None] * pair[0].float() + pair[1].float(), mean, rstd


def _norm_bwd(g, v, mean, rstd, rms):
    """Gradient of v behind the normalized values, and those values."""
    xh = (v if rms else v - mean[:, None]) * rstd[:, None]
    t = g - xh * (g * xh).mean(1, keepdim=True)
    if not rms:
        t = t - g.mean(1, keepdim=True)
    return t * rstd[:, None], xh


def _plain_resnorm(st):
    case = st["case"]
    rms, kind = case["rms"], case["kind"]
    bf = torch.bfloat16
    b = st["b"].float()
    gate = 1.0 if st["gate"] is None else st["gate"].float()
    if kind != "resnorm_bwd":
        r = {}
        t = b
        if case["post"]:
            t, r["mean_post"], r["rstd_post"] = _norm(b, st["post"], rms)
        s = (st["alpha"] * st["x"].float() + gate * t).to(st["x"].dtype)
        if case["pre"]:
            y, r["mean_pre"], r["rstd_pre"] = _norm(s.float(), st["pre"], rms)
            y = y.to(bf)
        r = _returned(case, r)
        if kind == "resnorm":
            return dict(r, s=s, y=y) if case["pre"] else dict(r, s=s)
        if kind == "resnorm_rows":
            q, amax = _row_codes(y)
            return dict(s=s, q=q, amax=amax)
        q, qt, amax = _codes(y, case["rowwise"], E4M3_MAX, torch.float8_e4m3fn)
        return dict(r, s=s, q=q, qt=qt, amax=amax)
    stats = st["stats"]
    r = {}
    dt = st["ds"].float()
    if case["pre"]:
        dy = st["dy"].float()
        g, xh = _norm_bwd(dy * st["pre"][0].float(), st["s"].float(), stats["mean_pre"],
                          stats["rstd_pre"], rms)
        dt = dt + g
        r.update(dpre_weight=(dy * xh).sum(0), dpre_bias=dy.sum(0))
    db, t = dt * gate, b
    if case["post"]:
        w, c = st["post"][0].float(), st["post"][1].float()
        db, xh = _norm_bwd(db * w, b, stats["mean_post"], stats["rstd_post"], rms)
        r.update(dpost_weight=(dt * gate * xh).sum(0), dpost_bias=(dt * gate).sum(0))
        t = xh * w + c
    if case["gate"]:
        r["dgate"] = (dt * t).sum(0)
    db = db.to(bf)
    r.update(dx=(st["alpha"] * dt).to(st["s"].dtype), db=db)
    if case["codes"]:
        fmax, ft = ((E5M2_MAX, torch.float8_e5m2) if case["e5m2"]
                    else (E4M3_MAX, torch.float8_e4m3fn))
        r["q"], r["qt"], r["amax"] = _codes(db, case["rowwise"], fmax, ft)
    return r


# ------------------------------------------------- the framework's calls --

def _own_linear(st):
    from float8_mixed_precision_amd import ops
    case = st["case"]
    kind, act, rw = case["kind"], case["act"], case["rowwise"]
    e4, bf = torch.float8_e4m3fn, torch.bfloat16
    if st["ws"] is None:
        st["ws"] = ops.alloc_linear_act_workspace(case["M"], case["N"], rw, "cuda")
    if kind in ("linear_bwd", "bias_bwd"):
        out = ops.Quantized(**st["codes"])
        if kind == "linear_bwd":
            ops.fp8_linear_act_bwd(st["dyq"], st["sdy"], st["wtq"], st["swt"], st["z"], act, rw,
                                   e5m2=case["e5m2"], dz=st["dz"], dbias=st["dbias"], out=out,
                                   workspace=st["ws"])
        else:
            ops.fp8_bias_act_bwd(st["dy"], st["z"], act, rw, e5m2=case["e5m2"], dz=st["dz"],
                                 dbias=st["dbias"], out=out, workspace=st["ws"])
        ft = torch.float8_e5m2 if case["e5m2"] else e4
        r = dict(dbias=st["dbias"], q=out.q.view(ft), qt=out.qt.view(ft), amax=out.amax.to(bf))
        return r if st["dz"] is None else dict(dz=st["dz"], **r)
    args = (st["xq"], st["sx"], st["wq"], st["sw"], st["bias"], act)
    if kind == "linear":
        y = ops.fp8_linear_act_fwd(*args, residual=st["residual"], rowwise=rw, y=st["y"],
                                   workspace=st["ws"])
        return dict(y=y)
    if kind == "linear_rows":
        c = st["codes"]
        out = ops.Quantized(c["q"], None, c["scale"], None, c["amax"])
        y = ops.fp8_linear_act_fwd(*args, residual=st["residual"], rowwise=True, y=st["y"],
                                   out=out, transposed=False, workspace=st["ws"])
        return dict(y=y, q=out.q.view(e4), amax=out.amax.to(bf))
    out = ops.Quantized(**st["codes"])
    y = ops.fp8_linear_act_fwd(*args, rowwise=rw, y=st["y"], z=st["z"], out=out,
                               workspace=st["ws"])
    r = dict(z=st["z"], q=out.q.view(e4), qt=out.qt.view(e4), amax=out.amax.to(bf))
    return dict(y=y, **r) if case["store_y"] else r


def _own_resnorm(st):
    from float8_mixed_precision_amd import ops
    case = st["case"]
    kind, rms = case["kind"], case["rms"]
    e4, bf = torch.float8_e4m3fn, torch.bfloat16
    stats = ops.ResNormStats(**st["stats"])
    if kind == "resnorm":
        ops.fp8_resnorm_fwd(st["b"], st["x"], st["post"], st["pre"], st["gate"], st["alpha"], EPS,
                            rms, s=st["s"], y=st["y"], stats=stats)
        r = _returned(case, st["stats"])
        return dict(r, s=st["s"], y=st["y"]) if case["pre"] else dict(r, s=st["s"])
    if kind == "resnorm_rows":
        c = st["codes"]
        out = ops.Quantized(c["q"], None, c["scale"], None, c["amax"])
        ops.fp8_resnorm_quantize(st["b"], st["x"], st["post"], st["pre"], st["gate"], st["alpha"],
                                 EPS, rms, rowwise=True, transposed=False, s=st["s"], out=out,
                                 want_stats=False)
        return dict(s=st["s"], q=out.q.view(e4), amax=out.amax.to(bf))
    rows, cols = st["b"].shape
    if st["ws"] is None:
        st["ws"] = ops.alloc_resnorm_workspace(rows, cols, "cuda", case.get("rowwise", False))
    if kind == "resnorm_quantize":
        out = ops.Quantized(**st["codes"])
        ops.fp8_resnorm_quantize(st["b"], st["x"], st["post"], st["pre"], st["gate"], st["alpha"],
                                 EPS, rms, rowwise=case["rowwise"], s=st["s"], out=out,
                                 stats=stats, workspace=st["ws"])
        r = _returned(case, st["stats"])
        return dict(r, s=st["s"], q=out.q.view(e4), qt=out.qt.view(e4), amax=out.amax.to(bf))
    out = ops.Quantized(**st["codes"]) if case["codes"] else None
    grads = ops.ResNormGrads(**st["grads"])
    ops.fp8_resnorm_bwd(st["dy"], st["ds"], st["b"], st["s"], stats, st["post"], st["pre"],
                        st["gate"], st["alpha"], rms, grads=grads, out=out,
                        rowwise=case.get("rowwise", False), e5m2=case.get("e5m2", False),
                        workspace=st["ws"])
    r = {n: v for n, v in st["grads"].items() if v is not None}
    if case["codes"]:
        ft = torch.float8_e5m2 if case["e5m2"] else e4
        r.update(q=out.q.view(ft), qt=out.qt.view(ft), amax=out.amax.to(bf))
    return r


def run(state):
    linear = not state["case"]["kind"].startswith("resnorm")
    if own:
        return _own_linear(state) if linear else _own_resnorm(state)
    return _plain_linear(state) if linear else _plain_resnorm(state)


# ------------------------------------------------------------------- work --

def work(case):
    kind = case["kind"]
    if kind.startswith("resnorm"):
        n = case["rows"] * case["cols"]
        e = 4 if case.get("dtype") == "f32" else 2
        params = 2 * case["cols"] * (2 * case["post"] + 2 * case["pre"] + case["gate"])
        norms = case["post"] + case["pre"]
        if kind == "resnorm_bwd":
            extra = 2 * n if case["codes"] else 0
            grads = 4 * case["cols"] * (2 * norms + case["gate"])
            return {"bytes": (2 * case["pre"] + 3 * e + 4) * n + extra + params + grads,
                    "flops": (14 * norms + 4) * n}
        y = {"resnorm": 2 * n if case["pre"] else 0, "resnorm_rows": n,
             "resnorm_quantize": 2 * n}[kind]
        return {"bytes": (2 + 2 * e) * n + y + params + 8 * norms * case["rows"],
                "flops": (8 * norms + 3) * n}
    M, N = case["M"], case["N"]
    mn = M * N
    acted = case["act"] != "none"
    if kind == "bias_bwd":
        return {"bytes": (2 + 4 * acted + 2) * mn + 4 * N, "flops": (4 + 8 * acted) * mn}
    K = case["K"]
    ops = M * K + N * K
    product = 2 * mn * K
    if kind == "linear_bwd":
        return {"bytes": ops + 6 * mn + 2 * N, "flops": product + 14 * mn}
    if kind == "linear_train":
        return {"bytes": ops + (4 + 2 * case["store_y"]) * mn + 2 * N, "flops": product + 12 * mn}
    rows = mn if kind == "linear_rows" else 0
    return {"bytes": ops + (2 + 2 * case["residual"]) * mn + rows + 2 * N,
            "flops": product + 8 * mn}


# ---------------------------------------------------------- 64-bit values --

def _bf16(v):
    """Nearest bf16 value (ties to even) of 64-bit values, kept in 64 bits."""
    _, e = torch.frexp(v)
    step = torch.ldexp(torch.ones_like(v), e - 8)
    return torch.where(v == 0, v, torch.round(v / step) * step)


def _fp8(v, e5m2):
    """Nearest code value, saturating, of 64-bit values."""
    fmax, bits, emin = (E5M2_MAX, 2, -14) if e5m2 else (E4M3_MAX, 3, -6)
    e = torch.frexp(v)[1] - 1
    step = torch.ldexp(torch.ones_like(v), e.clamp(min=emin) - bits)
    return (torch.round(v / step) * step).clamp(-fmax, fmax)


def _exact_codes(y, rowwise, e5m2=False, rows_only=False):
    """y: bf16 values in 64 bits.  The scale is one 32-bit division and the
    scaled value one 32-bit product, as the quantize defines them."""
    fmax = E5M2_MAX if e5m2 else E4M3_MAX

    def one(v, amax):
        top = torch.full_like(amax, fmax, dtype=torch.float32)
        s = torch.div(top, amax.clamp(min=1e-12).float()).double()
        return _fp8((v * s).float().double(), e5m2)

    ar = y.abs().amax(1)
    if rows_only:
        return one(y, ar[:, None]), ar
    if not rowwise:
        amax = ar.amax().reshape(1)
        q = one(y, amax)
        return q, q.t().contiguous(), amax
    ac = y.abs().amax(0)
    return one(y, ar[:, None]), one(y, ac[None, :]).t().contiguous(), torch.cat((ar, ac))


def _exact_act(z, act):
    """act(z) and its derivative in 64 bits."""
    one, zero = torch.ones_like(z), torch.zeros_like(z)
    if act == "none":
        return z, one
    if act in ("relu", "relu2"):
        p = torch.where(z > 0, z, zero)
        return (p, torch.where(z > 0, one, zero)) if act == "relu" else (p * p, 2 * p)
    if act == "silu":
        s = torch.sigmoid(z)
        return z * s, s + z * s * torch.sigmoid(-z)
    if act == "gelu_tanh":
        u = ROOT_2_PI * (z + CUBIC * z.pow(3))
        t = torch.tanh(u)
        # 1 + tanh(u) without the cancellation of large negative u
        half = torch.sigmoid(2 * u)
        return z * half, half + 0.5 * z * (1 - t * t) * ROOT_2_PI * (1 + 3 * CUBIC * z * z)
    cdf = torch.special.ndtr(z)
    return z * cdf, cdf + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)


def _exact_linear(st):
    case, D = st["case"], torch.float64
    kind, rw = case["kind"], case["rowwise"]
    e4 = torch.float8_e4m3fn

    def product(p, fp, sp, q, sq):
        v = p.view(fp).to(D) @ q.view(e4).to(D).t()
        sp, sq = sp.to(D), sq.to(D)
        return v / (sp[:, None] * sq[None, :] if rw else sp * sq)

    if kind in ("linear_bwd", "bias_bwd"):
        e5 = case["e5m2"]
        if kind == "bias_bwd":
            dz = st["dy"].to(D)
        else:
            dz = product(st["dyq"], torch.float8_e5m2 if e5 else e4, st["sdy"], st["wtq"],
                         st["swt"])
        if st["z"] is not None:
            dz = dz * _exact_act(st["z"].to(D), case["act"])[1]
        q, qt, amax = _exact_codes(_bf16(dz), rw, e5)
        r = dict(dbias=dz.sum(0), q=q, qt=qt, amax=amax)
        return r if st["dz"] is None else dict(dz=dz, **r)
    z = product(st["xq"], e4, st["sx"], st["wq"], st["sw"]) + st["bias"].to(D)
    y = z if case["act"] == "none" else _exact_act(_bf16(z), case["act"])[0]
    if st["residual"] is not None:
        y = y + st["residual"].to(D)
    if kind == "linear":
        return dict(y=y)
    if kind == "linear_rows":
        q, amax = _exact_codes(_bf16(y), True, rows_only=True)
        return dict(y=y, q=q, amax=amax)
    q, qt, amax = _exact_codes(_bf16(y), rw)
    r = dict(z=z, q=q, qt=qt, amax=amax)
    return dict(y=y, **r) if case["store_y"] else r


def _exact_resnorm(st):
    case, D = st["case"], torch.float64
    rms, kind = case["rms"], case["kind"]
    b = st["b"].to(D)
    n = b.shape[1]
    gate = torch.ones(n, dtype=D, device=b.device) if st["gate"] is None else st["gate"].to(D)

    def normed(v):
        mean = torch.zeros_like(v[:, :1]) if rms else v.sum(1, keepdim=True) / n
        rstd = ((v - mean).square().sum(1, keepdim=True) / n + EPS).pow(-0.5)
        return (v - mean) * rstd, mean[:, 0], rstd[:, 0]

    if kind != "resnorm_bwd":
        r = {}
        t = b
        if case["post"]:
            xh, r["mean_post"], r["rstd_post"] = normed(b)
            t = xh * st["post"][0].to(D) + st["post"][1].to(D)
        s = st["alpha"] * st["x"].to(D) + gate * t
        # the norm in front of the next block is of the stream as it is stored
        sr = _bf16(s) if st["x"].dtype == torch.bfloat16 else s.float().to(D)
        y = None
        if case["pre"]:
            xh, r["mean_pre"], r["rstd_pre"] = normed(sr)
            y = xh * st["pre"][0].to(D) + st["pre"][1].to(D)
        r = _returned(case, r)
        if kind == "resnorm":
            return dict(r, s=s, y=y) if case["pre"] else dict(r, s=s)
        if kind == "resnorm_rows":
            q, amax = _exact_codes(_bf16(y), True, rows_only=True)
            return dict(s=s, q=q, amax=amax)
        q, qt, amax = _exact_codes(_bf16(y), case["rowwise"])
        return dict(r, s=s, q=q, qt=qt, amax=amax)

    def back(g, v, which):
        """Gradient of v behind its normalized values, and those values."""
        mean, rstd = st["stats"]["mean_" + which], st["stats"]["rstd_" + which].to(D)[:, None]
        xh = (v if rms else v - mean.to(D)[:, None]) * rstd
        d = g - xh * ((g * xh).sum(1, keepdim=True) / n)
        if not rms:
            d = d - g.sum(1, keepdim=True) / n
        return d * rstd, xh

    r = {}
    dt = st["ds"].to(D)
    if case["pre"]:
        dy = st["dy"].to(D)
        d, xh = back(dy * st["pre"][0].to(D), st["s"].to(D), "pre")
        dt = dt + d
        r.update(dpre_weight=(dy * xh).sum(0), dpre_bias=dy.sum(0))
    db, t = dt * gate, b
    if case["post"]:
        w = st["post"][0].to(D)
        db, xh = back(dt * gate * w, b, "post")
        r.update(dpost_weight=gate * (dt * xh).sum(0), dpost_bias=gate * dt.sum(0))
        t = xh * w + st["post"][1].to(D)
    if case["gate"]:
        r["dgate"] = (dt * t).sum(0)
    r.update(dx=st["alpha"] * dt, db=db)
    if case["codes"]:
        r["q"], r["qt"], r["amax"] = _exact_codes(_bf16(db), case["rowwise"], case["e5m2"])
    return r


def exact(case, seed):
    st = prepare(case, seed)
    return _exact_resnorm(st) if case["kind"].startswith("resnorm") else _exact_linear(st)
