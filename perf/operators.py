"""Measured cases of the grouped products' operators: bf16 / fp16 rows times their expert's
weights, the two gradients of that product, MXFP4 quantisation, and the product of MXFP4
rows and weights.

``run`` computes a case in plain torch operations (``own`` false) or through this
package's entry points (``own`` true).  Rows are sorted by expert, as everywhere in this
package: a group list on the device says how many each expert has.

Plain form of every product: the rows are laid into [e, cap, width] (cap = the largest
group) and multiplied in f32 by one batched product; padding rows are zero.
"""
import numpy as np
import torch

own = False

F16, BF16, F32 = "fp16", "bf16", "f32"
_T = {F16: torch.float16, BF16: torch.bfloat16, F32: torch.float32}
DEV = "cuda"
MX = 32                      # elements that share one E8M0 scale
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ---------------------------------------------------------------- cases
def _mm(name, op, m, k, n, e, x, out, wt, gl):
    """op: fwd | dgrad | wgrad | mx4; wt: weights stored (e, n, k); gl: 'ends' or 'counts'."""
    return {"name": name, "op": op, "m": m, "k": k, "n": n, "e": e, "x": x, "out": out, "wt": wt, "gl": gl}


def listed():
    return [
        # one token of a layer with eight of 32 experts chosen: the weights' bytes are all there is
        _mm("fwd_token", "fwd", 8, 2048, 7168, 32, BF16, BF16, False, "counts"),
        # odd sizes on every axis, half precision, weights stored the other way
        _mm("fwd_odd", "fwd", 4099, 1000, 1352, 7, F16, F16, True, "ends"),
        # a training or prefill step's rows on the package's usual expert shape
        _mm("fwd_prefill", "fwd", 32768, 2048, 7168, 32, BF16, BF16, False, "ends"),
        # the input gradient of a short batch
        _mm("dgrad_batch", "dgrad", 1000, 2048, 7168, 16, BF16, BF16, False, "counts"),
        _mm("dgrad_prefill", "dgrad", 32768, 2048, 7168, 32, BF16, BF16, True, "counts"),
        # the weight gradient: odd sizes into f32 (a main gradient), and a training step's
        _mm("wgrad_odd", "wgrad", 777, 520, 264, 5, F16, F32, False, "ends"),
        _mm("wgrad_step", "wgrad", 32768, 2048, 7168, 32, BF16, BF16, False, "counts"),
        # quantise and expand: one decode batch's rows, and a block of f32 master weights
        {"name": "quant_batch", "op": "quant", "m": 16, "k": 7168, "x": BF16},
        {"name": "quant_weights", "op": "quant", "m": 57344, "k": 2048, "x": F32},
        # rows quantised in the call, weights quantised once: a token, odd sizes, a prefill
        _mm("mx4_token", "mx4", 8, 2048, 7168, 32, BF16, BF16, True, "counts"),
        _mm("mx4_odd", "mx4", 1533, 1056, 360, 9, F16, F32, True, "ends"),
        _mm("mx4_prefill", "mx4", 32768, 2048, 7168, 32, BF16, BF16, True, "counts"),
    ]


def _log(rng, lo, hi, step=1):
    """A multiple of `step` in [lo, hi], spread over the logarithm."""
    v = lo * (hi / lo) ** rng.random()
    return int(max(lo, min(hi // step * step, round(v / step) * step)))


def draw(rng):
    op = rng.choice(("fwd", "dgrad", "wgrad", "mx4", "quant"))
    if op == "quant":
        k = _log(rng, 32, 8192, 32)
        return {"op": op, "m": _log(rng, 1, max(1, min(65536, (100 << 20) // k))), "k": k,
                "x": rng.choice((F16, BF16, F32))}
    step = 32 if op == "mx4" else 8
    x = rng.choice((F16, BF16))
    while True:
        c = _mm("", op, _log(rng, 1, 32768), _log(rng, 64, 4096, step), _log(rng, 64, 8192, 8), _log(rng, 1, 64), x,
                rng.choice((x, F32)), op == "mx4" or rng.random() < 0.5, rng.choice(("ends", "counts")))
        if c["e"] * c["k"] * c["n"] <= 450 << 20 and c["m"] * c["k"] * c["n"] <= 440 << 30:
            del c["name"]
            return c


def work(case):
    m, k, x = case["m"], case["k"], 4 if case["x"] == F32 else 2
    if case["op"] == "quant":      # read, write codes and scales, read them, write the values
        return {"bytes": m * k * (2 * x + 1) + m * k // MX * 2, "flops": 2 * m * k}
    n, e, out = case["n"], case["e"], 4 if case["out"] == F32 else 2
    used = min(e, m)               # experts with rows
    flops = 2 * m * k * n
    if case["op"] == "fwd":
        b = m * k * x + used * k * n * x + m * n * out
    elif case["op"] == "dgrad":
        b = m * n * x + used * k * n * x + m * k * out
    elif case["op"] == "wgrad":
        b = m * (k + n) * x + e * k * n * out
    else:
        b = m * k * x + used * n * (k // 2 + k // MX) + m * n * out
    return {"bytes": b, "flops": flops}


# ---------------------------------------------------------------- inputs
def _counts(case, seed):
    """Rows of each expert: distinct experts while there are fewer rows than experts, else
    skewed popularity (Dirichlet), some experts empty."""
    rng = np.random.default_rng(seed * 7919 + 11)
    m, e = case["m"], case["e"]
    if m <= e:
        c = np.zeros(e, np.int64)
        c[rng.permutation(e)[:m]] = 1
        return c
    return rng.multinomial(m, rng.dirichlet(np.full(e, 2.0))).astype(np.int64)


def _normal(gen, shape, dtype, scale=1.0):
    t = torch.empty(shape, dtype=dtype, device=DEV).normal_(generator=gen)
    return t.mul_(scale) if scale != 1.0 else t


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(int(seed))
    t, m, k = _T[case["x"]], case["m"], case["k"]
    s = {"case": case}
    if case["op"] == "quant":
        x = _normal(gen, (m, k), torch.float32)
        x *= torch.exp2(torch.randint(-3, 4, (m, 1), device=DEV, generator=gen).float())   # rows of different size
        s["x"] = x.to(t)
        return s
    n, e = case["n"], case["e"]
    c = _counts(case, int(seed))
    ends = np.cumsum(c)
    group = np.repeat(np.arange(e), c)
    s["cap"] = int(c.max())
    s["slot"] = torch.from_numpy(group * s["cap"] + np.arange(m) - (ends - c)[group]).to(DEV)
    s["group_list"] = torch.from_numpy(ends if case["gl"] == "ends" else c).to(DEV)
    shape = (e, n, k) if case["wt"] else (e, k, n)
    if case["op"] == "fwd":
        s["x"], s["w"] = _normal(gen, (m, k), t), _normal(gen, shape, t, k ** -0.5)
    elif case["op"] == "dgrad":
        s["dy"], s["w"] = _normal(gen, (m, n), t), _normal(gen, shape, t, k ** -0.5)
    elif case["op"] == "wgrad":
        s["x"], s["dy"] = _normal(gen, (m, k), t), _normal(gen, (m, n), t)
    else:
        s["x"] = _normal(gen, (m, k), t)
        w = _normal(gen, (e * n, k), torch.bfloat16, k ** -0.5)
        q, sf = _mx4_codes(w)
        q = q.view(e, n, k // 2, 2)
        s["wq"], s["wsf"] = q[..., 0] | (q[..., 1] << 4), sf.view(e, n, k // MX)
    return s


# ---------------------------------------------------------------- plain forms
def _mx4_scaled(x):
    """Blocks of 32 as f32, and each block's E8M0 code: the exponent of its largest
    magnitude, less 2 (E2M1's largest value is 1.5 * 2^2)."""
    b = x.float().view(x.shape[0], -1, MX)
    a = b.abs().amax(-1)
    sf = torch.where(a > 0, torch.frexp(a)[1] + 124, 0).clamp(0, 254)     # frexp's exponent is the IEEE one + 1
    return b * torch.exp2((127 - sf).float())[..., None], sf


def _mx4_round(v):
    """Magnitudes and signs of the nearest E2M1 values, ties to the even code, 6 at most."""
    a = v.abs()
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    return (torch.round(a / step) * step).clamp(max=6.0)


def _mx4_codes(x):
    """E2M1 codes (one per byte) and E8M0 codes, for inputs."""
    v, sf = _mx4_scaled(x)
    r = _mx4_round(v)
    mag = torch.where(r < 2, 2 * r, torch.where(r < 4, r + 2, r / 2 + 4)).to(torch.uint8)
    return (mag | ((v < 0).to(torch.uint8) << 3)).view(x.shape), sf.to(torch.uint8)


def _mx4_values(x):
    """The values that x's MXFP4 codes and scales stand for, f32."""
    v, sf = _mx4_scaled(x)
    return (torch.sign(v) * _mx4_round(v) * torch.exp2((sf - 127).float())[..., None]).view(x.shape)


def _mx4_expand(q, sf):
    """f32 values of packed codes [..., k/2] and scales [..., k/32]."""
    lut = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=q.device)
    codes = torch.stack((q & 15, q >> 4), -1).view(*sf.shape, MX)
    return (lut[codes.int()] * torch.exp2(sf.float() - 127)[..., None]).view(*q.shape[:-1], -1)


def _padded(s, rows):
    e, cap = s["case"]["e"], s["cap"]
    return torch.zeros(e * cap, rows.shape[1], device=DEV).index_copy_(0, s["slot"], rows.float()).view(e, cap, -1)


def _rows(s, t):
    return t.view(-1, t.shape[-1])[s["slot"]].to(_T[s["case"]["out"]])


def _plain(s):
    c = s["case"]
    if c["op"] == "quant":
        return _mx4_values(s["x"]).to(_T[c["x"]])
    if c["op"] == "fwd":
        w = s["w"].float()
        return _rows(s, torch.bmm(_padded(s, s["x"]), w.transpose(1, 2) if c["wt"] else w))
    if c["op"] == "dgrad":
        w = s["w"].float()
        return _rows(s, torch.bmm(_padded(s, s["dy"]), w if c["wt"] else w.transpose(1, 2)))
    if c["op"] == "wgrad":
        a, b = (s["dy"], s["x"]) if c["wt"] else (s["x"], s["dy"])
        return torch.bmm(_padded(s, a).transpose(1, 2), _padded(s, b)).to(_T[c["out"]])
    return _rows(s, torch.bmm(_padded(s, _mx4_values(s["x"])), _mx4_expand(s["wq"], s["wsf"]).transpose(1, 2)))


# ---------------------------------------------------------------- the package's calls
def _problem(c):
    import quantized_moe_grouped_persistent_b200 as q
    types = {BF16: q.QGMM_T_BF16, F16: q.QGMM_T_F16, F32: q.QGMM_T_F32}
    return q.make_mm_problem(c["m"], c["k"], c["n"], c["e"],
                             x_type=q.QGMM_T_MXFP4 if c["op"] == "mx4" else types[c["x"]], out_type=types[c["out"]],
                             transpose_w=c["wt"],
                             group_list_type=q.QGMM_GROUP_CUMSUM if c["gl"] == "ends" else q.QGMM_GROUP_COUNTS)


def _own(s):
    import quantized_moe_grouped_persistent_b200 as q
    c = s["case"]
    m, k = c["m"], c["k"]
    if c["op"] == "quant":
        codes = torch.empty((m, k // 2), dtype=torch.uint8, device=DEV)
        sf = torch.empty((m, k // MX), dtype=torch.uint8, device=DEV)
        out = torch.empty_like(s["x"])
        q.per_token_quant_mxfp4(s["x"], codes, sf)
        q.mxfp4_dequant(codes, sf, out)
        return out
    if "problem" not in s:         # a program keeps its problem and workspace from call to call
        s["problem"] = _problem(c)
        s["ws"] = torch.empty(q.grouped_mm_workspace(s["problem"]), dtype=torch.uint8, device=DEV)
    p, ws, gl, t = s["problem"], s["ws"], s["group_list"], _T[c["out"]]
    if c["op"] == "fwd":
        y = torch.empty((m, c["n"]), dtype=t, device=DEV)
        q.grouped_mm(p, s["x"], s["w"], gl, y, ws)
        return y
    if c["op"] == "dgrad":
        dx = torch.empty((m, k), dtype=t, device=DEV)
        q.grouped_mm_dgrad(p, s["dy"], s["w"], gl, dx, ws)
        return dx
    if c["op"] == "wgrad":
        dw = torch.empty((c["e"], c["n"], k) if c["wt"] else (c["e"], k, c["n"]), dtype=t, device=DEV)
        q.grouped_mm_wgrad(p, s["x"], s["dy"], gl, dw, ws)
        return dw
    codes = torch.empty((m, k // 2), dtype=torch.uint8, device=DEV)
    sf = torch.empty((m, k // MX), dtype=torch.uint8, device=DEV)
    y = torch.empty((m, c["n"]), dtype=t, device=DEV)
    q.per_token_quant_mxfp4(s["x"], codes, sf)
    q.grouped_mm(p, codes, s["wq"], gl, y, ws, x_scale=sf, w_scale=s["wsf"])
    return y


def run(state):
    return _own(state) if own else _plain(state)


# ---------------------------------------------------------------- 64 bits, from the definition
def _exact_mx4(x):
    """The nearest E2M1 multiple of each block's scale, by comparison with all eight levels."""
    b = x.double().reshape(x.shape[0], -1, MX)
    a = b.abs().amax(-1)
    e = torch.floor(torch.log2(torch.where(a > 0, a, 1.0)))
    e = e + (torch.exp2(e + 1) <= a).double() - (torch.exp2(e) > a).double()       # log2's rounding at powers of two
    scale = torch.exp2(torch.where(a > 0, (e - 2).clamp(min=-127), -127.0))[..., None]
    v = b.abs() / scale
    best, far = torch.zeros_like(v), v.clone()
    for code, level in enumerate(E2M1):
        d = (v - level).abs()
        nearer = (d < far) | ((d == far) & (code % 2 == 0))
        best, far = torch.where(nearer, level, best), torch.where(nearer, d, far)
    return (torch.sign(b) * best * scale).reshape(x.shape)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "quant":
        return torch.cat([_exact_mx4(part) for part in s["x"].split(8192)]).to(_T[case["x"]])
    c = _counts(case, int(seed))
    ends = np.cumsum(c)
    spans = [slice(int(b - n), int(b)) for b, n in zip(ends, c)]
    if case["op"] == "wgrad":
        a, b = (s["dy"], s["x"]) if case["wt"] else (s["x"], s["dy"])
        return torch.stack([(a[r].double().t() @ b[r].double()).float() for r in spans])
    if case["op"] == "mx4":
        x, lut = _exact_mx4(s["x"]), torch.tensor(E2M1 + tuple(-v for v in E2M1), dtype=torch.float64, device=DEV)
    out = torch.empty(case["m"], case["k"] if case["op"] == "dgrad" else case["n"], dtype=torch.float64, device=DEV)
    for g, r in enumerate(spans):
        if r.start == r.stop:
            continue
        if case["op"] == "mx4":
            q = s["wq"][g]
            w = torch.stack((lut[(q & 15).int()], lut[(q >> 4).int()]), -1).reshape(case["n"], -1, MX)
            w = (w * torch.exp2(s["wsf"][g].double() - 127)[..., None]).reshape(case["n"], -1)
            out[r] = x[r] @ w.t()
        elif case["op"] == "fwd":
            w = s["w"][g].double()
            out[r] = s["x"][r].double() @ (w.t() if case["wt"] else w)
        else:
            w = s["w"][g].double()
            out[r] = s["dy"][r].double() @ (w if case["wt"] else w.t())
    return out
