"""The MXFP4 operators and the cases they are measured on.

MXFP4 holds a vector in blocks of 32 elements: E2M1 codes (0, 0.5, 1, 1.5, 2,
3, 4, 6 and a sign), two per byte, element 2i in the low nibble, and one E8M0
scale per block, the power of two 2^(code - 127).  For a block with largest
magnitude A > 0 the scale exponent is floor(log2(A)) - 2, held in [-127, 127];
every element is v / scale rounded to the nearest E2M1 value, ties to the even
code, magnitudes past 6 to 6.

Operators:
  quantize   x -> its codes and scales along the rows, and along the columns
             too where `columnwise`; returned as the values they stand for.
  linear     y = Q(x) W^T for bf16 or fp16 x and MXFP4 weights W.
  train      one linear layer forward and backward from x, W and dy: y =
             Q(x) Q(W)^T, dx = Q(dy) Q(W), dW = Q(dy)^T Q(x), each operand
             quantized along the sum's dimension.
  experts    y[r] = s[r] * Q(x[rows[r]]) W_e^T for the rows r of each expert e,
             offsets[e] <= r < offsets[e + 1].
  experts_grad  dx[r] = Q(dy[r]) W_e and dW_e = sum over e's rows of
             Q(dy[r])^T Q(x[rows[r]]), blocks of 32 rows counted from the
             expert's first.

The plain forms below compute them with elementary torch operations in 32
bits; `exact` computes them again in 64.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def _up(n, m):
    return -(-n // m) * m


# --------------------------------------------------------------- the cases

def listed():
    return [
        # one token's hidden vector: the latency of a quantization while serving
        dict(name="quantize_token", op="quantize", rows=1, cols=4096, dtype="bf16", columnwise=False),
        # sizes that fit no block or tile, from a 32-bit master copy
        dict(name="quantize_odd", op="quantize", rows=1021, cols=2885, dtype="fp32", columnwise=True),
        # the activation of the cast's headline workload, both directions for training
        dict(name="quantize_large", op="quantize", rows=16384, cols=8192, dtype="bf16", columnwise=True),
        # a token through the 2D-quantized weight of the cast's workloads: decoding, bound by the weight's bytes
        dict(name="linear_token", op="linear", tokens=1, inner=8192, outer=28672, dtype="bf16"),
        # a decoding batch through a square projection
        dict(name="linear_batch", op="linear", tokens=48, inner=8192, outer=8192, dtype="bf16"),
        # a prompt of odd length and odd sizes in the other 16-bit type
        dict(name="linear_odd", op="linear", tokens=777, inner=1000, outer=4095, dtype="fp16"),
        # the product that the cast's activation goes into: prompts, at the matrix cores' rate
        dict(name="linear_prefill", op="linear", tokens=16384, inner=8192, outer=8192, dtype="bf16"),
        # a training step of one projection, three products and three quantizations
        dict(name="train_step", op="train", tokens=8192, inner=4096, outer=4096, dtype="bf16"),
        # decoding through 64 experts: few rows each, bound by the weights of the experts that are hit
        dict(name="experts_decode", op="experts", tokens=8, topk=4, experts=64, inner=4096, outer=4096,
             skew=0.5, dtype="bf16"),
        # ragged groups, several of them empty, at sizes that fit no tile
        dict(name="experts_odd", op="experts", tokens=301, topk=3, experts=33, inner=1000, outer=777,
             skew=2.0, dtype="bf16"),
        # the grouped workload's 32768 rows over 64 experts
        dict(name="experts_prefill", op="experts", tokens=4096, topk=8, experts=64, inner=4096, outer=4096,
             skew=0.5, dtype="bf16"),
        # the same experts' gradients at half the rows
        dict(name="experts_grad", op="experts_grad", tokens=4096, topk=4, experts=64, inner=4096, outer=1024,
             skew=0.5, dtype="bf16"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["quantize", "linear", "linear", "train", "experts", "experts", "experts_grad"])
    if op == "quantize":
        while True:
            c = dict(op=op, rows=_log(rng, 1, 16384), cols=_log(rng, 32, 16384),
                     dtype=rng.choice(["bf16", "bf16", "fp16", "fp32"]), columnwise=rng.random() < 0.6)
            if c["rows"] * c["cols"] <= 16384 * 8192:
                return c
    if op == "linear":
        # most weights have whole blocks; some sizes are odd
        while True:
            c = dict(op=op, tokens=_log(rng, 1, 16384), inner=_log(rng, 256, 16384), outer=_log(rng, 64, 28672),
                     dtype=rng.choice(["bf16", "bf16", "fp16"]))
            if rng.random() < 0.6:
                c.update(inner=_up(c["inner"], 32), outer=_up(c["outer"], 16))
            if c["tokens"] * c["inner"] * c["outer"] <= 16384 * 8192 * 8192 and c["inner"] * c["outer"] <= 8192 * 28672:
                return c
    if op == "train":
        while True:
            c = dict(op=op, tokens=_log(rng, 64, 16384), inner=_log(rng, 256, 8192), outer=_log(rng, 256, 8192),
                     dtype="bf16")
            if rng.random() < 0.6:
                c.update(inner=_up(c["inner"], 32), outer=_up(c["outer"], 32))
            if c["tokens"] * c["inner"] * c["outer"] <= 8192 * 4096 * 4096:
                return c
    grad = op == "experts_grad"
    while True:
        e = _log(rng, 4, 128)
        c = dict(op=op, tokens=_log(rng, 16 if grad else 1, 4096), topk=rng.randint(1, min(8, e)), experts=e,
                 inner=_log(rng, 256, 6144), outer=_log(rng, 256, 6144), skew=rng.choice([0.0, 0.5, 1.0, 2.0]),
                 dtype="bf16")
        if rng.random() < 0.6:
            c.update(inner=_up(c["inner"], 32), outer=_up(c["outer"], 32))
        size = c["inner"] * c["outer"]
        if (e * size <= 64 * 4096 * (1024 if grad else 4096)
                and c["tokens"] * c["topk"] * size <= 32768 * 4096 * (1024 if grad else 4096)):
            return c


# ----------------------------------------------------- the format, in torch

def _exponents(amax):
    """Scale exponents of blocks with these largest magnitudes (32-bit)."""
    e = torch.frexp(amax)[1].to(torch.int32) - 1 - 2
    return torch.where(amax > 0, e.clamp(-127, 127), torch.full_like(e, -127))


def _codes(x):
    """Last dimension into blocks of 32: (magnitude codes with sign, uint8
    [..., nb, 32]; scale exponents int32 [..., nb])."""
    n = x.shape[-1]
    x = torch.nn.functional.pad(x.float(), (0, _up(n, 32) - n)).unflatten(-1, (-1, 32))
    e = _exponents(x.abs().amax(-1))
    a = torch.ldexp(x.abs(), -e[..., None])
    # the midpoints between neighbours; a tie goes to the even code
    c = ((a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5))
    return c | ((x < 0).to(torch.uint8) << 3), e


def _grid(device):
    g = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], device=device)
    return torch.cat([g, -g])


def _values(codes, e):
    """32-bit values [..., nb*32] of codes and scale exponents."""
    return torch.ldexp(_grid(codes.device)[codes.long()], e[..., None]).flatten(-2)


def _fake(x):
    """The 32-bit values that x's MXFP4 codes along its last dimension stand for."""
    return _values(*_codes(x))[..., :x.shape[-1]]


def _pack(w):
    """w [..., R, K] -> q [..., R, Kp/2] uint8 and sf [..., Rt, Kt, 128, 4]
    uint8 (Kp: K rounded up to 128, Kt = Kp/128, Rt: 128-row tiles): the four
    scales of a row's 128 elements are together, and so are 128 rows."""
    R, K = w.shape[-2:]
    w = torch.nn.functional.pad(w, (0, _up(K, 128) - K))
    c, e = _codes(w)
    c = c.flatten(-2)
    q = c[..., 0::2] | (c[..., 1::2] << 4)
    sf = torch.nn.functional.pad((e + 127).to(torch.uint8), (0, 0, 0, _up(R, 128) - R))
    sf = sf.unflatten(-1, (-1, 4)).unflatten(-3, (-1, 128)).transpose(-3, -2).contiguous()
    return q.contiguous(), sf


def _unpack(q, sf, K):
    """The 32-bit values [..., R, K] of what _pack made."""
    c = torch.stack([q & 15, q >> 4], -1).flatten(-2).unflatten(-1, (-1, 32))
    e = sf.transpose(-3, -2).flatten(-2).flatten(-3, -2)[..., :q.shape[-2], :].to(torch.int32) - 127
    return _values(c, e)[..., :K]


# ----------------------------------------------------------------- inputs

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _activations(g, rows, cols, dtype):
    """Rows of different scale with a few outliers."""
    x = _randn(g, rows, cols) * torch.exp(0.7 * _randn(g, rows, 1))
    out = torch.rand(rows, cols, generator=g, device="cuda") < 1e-3
    return torch.where(out, x * 20, x).to(dtype)


def _weights(g, *shape):
    return (_randn(g, *shape) * shape[-1] ** -0.5).bfloat16()


def _route(g, case):
    """Each token's topk experts by noisy scores with a bias per expert, the
    rows sorted by expert: offsets int32 [E + 1], rows int32 [R], the router's
    weights fp32 [R], and the host's counts."""
    T, k, E = case["tokens"], case["topk"], case["experts"]
    scores = _randn(g, T, E) + case["skew"] * _randn(g, 1, E)
    top, ids = scores.topk(k, dim=1)
    flat = ids.reshape(-1)
    order = torch.argsort(flat, stable=True)
    counts = torch.bincount(flat, minlength=E)
    offsets = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    offsets[1:] = counts.cumsum(0)
    p = torch.softmax(top, 1).reshape(-1)[order].contiguous()
    return offsets, (order // k).int(), p, counts.tolist()


def prepare(case, seed):
    g, op, dt = _gen(seed), case["op"], DTYPES[case["dtype"]]
    if op == "quantize":
        return dict(case, x=_activations(g, case["rows"], case["cols"], dt))
    T, K, N = case["tokens"], case["inner"], case["outer"]
    x = _activations(g, T, K, dt)
    if op == "linear":
        q, sf = _pack(_weights(g, N, K))
        return dict(case, x=x, w_q=q, w_sf=sf)
    if op == "train":
        return dict(case, x=x, w=_weights(g, N, K), dy=(1e-3 * _activations(g, T, N, torch.float32)).to(dt))
    offsets, rows, p, counts = _route(g, case)
    s = dict(case, x=x, offsets=offsets, rows=rows, counts=counts)
    E, R = case["experts"], T * case["topk"]
    if op == "experts":
        q, sf = _pack(_weights(g, E, N, K))
        return dict(s, w_q=q, w_sf=sf, p=p)
    # the weight's columns, [E, K, N]: what a forward pass's weights are next to
    q, sf = _pack(_weights(g, E, N, K).transpose(1, 2).contiguous())
    return dict(s, wt_q=q, wt_sf=sf, dy=(1e-3 * _activations(g, R, N, torch.float32)).to(dt))


# ------------------------------------------------------------ plain forms

def _slots(counts, device, unit=1):
    """Each expert's rows in a padded batch [E, P]: for row r its flat place,
    and P (a multiple of `unit`)."""
    P = max(unit, _up(max(counts), unit))
    c = torch.tensor(counts, device=device)
    start = c.cumsum(0) - c
    e = torch.repeat_interleave(torch.arange(len(counts), device=device), c)
    return e * P + torch.arange(e.numel(), device=device) - start[e], P


def _batched(v, slot, E, P):
    out = torch.zeros(E * P, v.shape[1], dtype=v.dtype, device=v.device)
    out[slot] = v
    return out.view(E, P, -1)


def _run_plain(s):
    op = s["op"]
    x = s["x"]
    if op == "quantize":
        row = _fake(x).bfloat16()
        return {"row": row, "col": _fake(x.t()).bfloat16()} if s["columnwise"] else {"row": row}
    K = s["inner"]
    if op == "linear":
        return _fake(x).matmul(_unpack(s["w_q"], s["w_sf"], K).t()).to(x.dtype)
    if op == "train":
        w, dy = s["w"], s["dy"]
        return {"y": _fake(x).matmul(_fake(w).t()).to(x.dtype),
                "dx": _fake(dy).matmul(_fake(w.t()).t()).to(x.dtype),
                "dw": _fake(dy.t()).matmul(_fake(x.t()).t())}
    E, counts, rows = s["experts"], s["counts"], s["rows"].long()
    slot, P = _slots(counts, x.device, 32)
    if op == "experts":
        w = _unpack(s["w_q"], s["w_sf"], K).transpose(1, 2).contiguous()
        y = torch.bmm(_batched(_fake(x)[rows], slot, E, P), w).view(E * P, -1)[slot]
        return (s["p"][:, None] * y).to(x.dtype)
    N, dy = s["outer"], s["dy"]
    wt = _unpack(s["wt_q"], s["wt_sf"], N).transpose(1, 2).contiguous()
    dx = torch.bmm(_batched(_fake(dy), slot, E, P), wt).view(E * P, -1)[slot].to(x.dtype)
    dyt = _fake(_batched(dy.float(), slot, E, P).transpose(1, 2))
    xt = _fake(_batched(x[rows].float(), slot, E, P).transpose(1, 2)).transpose(1, 2).contiguous()
    return {"dx": dx, "dw": torch.bmm(dyt.contiguous(), xt)}


def _run_own(s):
    import nvfp4_block_scaled_bf16_amd as nv
    op = s["op"]
    x = s["x"]
    if op == "quantize":
        R, C = x.shape
        o = nv.mx_quantize(x, columnwise=s["columnwise"])
        out = {"row": nv.mx_dequantize(o["row_q"], o["row_sf"], C, torch.bfloat16)}
        if s["columnwise"]:
            out["col"] = nv.mx_dequantize(o["col_q"], o["col_sf"], R, torch.bfloat16)
        return out
    if op == "linear":
        return nv.mx_linear(x, s["w_q"], s["w_sf"])
    if op == "train":
        qx, qw, qd = nv.mx_quantize(x), nv.mx_quantize(s["w"]), nv.mx_quantize(s["dy"])
        return {"y": nv.mx_gemm(qx["row_q"], qx["row_sf"], qw["row_q"], qw["row_sf"], x.dtype),
                "dx": nv.mx_gemm(qd["row_q"], qd["row_sf"], qw["col_q"], qw["col_sf"], x.dtype),
                "dw": nv.mx_gemm(qd["col_q"], qd["col_sf"], qx["col_q"], qx["col_sf"], torch.float32)}
    off, rows = s["offsets"], s["rows"]
    if op == "experts":
        return nv.mx_linear_grouped(x, s["w_q"], s["w_sf"], off, rows=rows, row_scale=s["p"])
    qd = nv.mx_quantize_grouped(s["dy"], off)
    qx = nv.mx_quantize_grouped(x, off, rows=rows, rowwise=False)
    return {"dx": nv.mx_gemm_grouped(qd["row_q"], qd["row_sf"], s["wt_q"], s["wt_sf"], off, out_dtype=x.dtype),
            "dw": nv.mx_wgrad_grouped(qd["col_q"], qd["col_sf"], qx["col_q"], qx["col_sf"], off)}


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ------------------------------------------------------------------- work

def work(case):
    op, b = case["op"], 4 if case["dtype"] == "fp32" else 2
    if op == "quantize":
        n = case["rows"] * case["cols"]
        return {"bytes": n * (b + (4 if case["columnwise"] else 2)), "flops": 0}
    T, K, N = case["tokens"], case["inner"], case["outer"]
    w = N * K * 17 / 32          # codes and scales of one weight
    if op == "linear":
        return {"bytes": T * K * b + w + T * N * b, "flops": 2 * T * K * N}
    if op == "train":            # x, w and dy in; y, dx and a 32-bit dw out
        return {"bytes": 2 * (2 * T * K + 2 * T * N + N * K) + 4 * N * K, "flops": 6 * T * K * N}
    E, R = case["experts"], T * case["topk"]
    if op == "experts":
        # the experts that R even draws of E hit
        hit = E * (1 - (1 - 1 / E) ** R)
        return {"bytes": T * K * b + hit * w + R * N * b + 8 * R, "flops": 2 * R * K * N}
    return {"bytes": T * K * b + R * N * b + E * w + R * K * b + 4 * E * N * K, "flops": 4 * R * K * N}


# ------------------------------------------------------------- in 64 bits

def _exact_fake(x):
    """The values of x's codes along its last dimension, found in 64 bits as
    the nearest of the grid's eight magnitudes to |x| / scale."""
    n = x.shape[-1]
    v = torch.zeros(*x.shape[:-1], _up(n, 32), dtype=torch.float64, device=x.device)
    v[..., :n] = x.double()
    v = v.view(*x.shape[:-1], -1, 32)
    top = v.abs().max(-1, keepdim=True).values
    scale = torch.exp2((torch.floor(torch.log2(top.clamp_min(2.0 ** -1000))) - 2).clamp(-127, 127))
    # log2 in 64 bits could round up to a whole number just below a power of two
    scale = torch.where(scale * 4 > top, (scale / 2).clamp_min(2.0 ** -127), scale)
    a = v.abs() / scale
    best, far = torch.zeros_like(a), a.clone()
    for code, m in enumerate([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]):
        d = (a - m).abs()
        take = (d < far) | ((d == far) & (code % 2 == 0))
        best[take], far[take] = m, d[take]
    return (torch.sign(v) * best * scale).flatten(-2)[..., :n]


def _exact_weight(q, sf, K):
    lo, hi = (q % 16).long(), (q // 16).long()
    mag = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64, device=q.device)
    v = torch.empty(*q.shape[:-1], 2 * q.shape[-1], dtype=torch.float64, device=q.device)
    for i, c in enumerate((lo, hi)):
        v[..., i::2] = mag[c % 8] * (1.0 - 2.0 * (c // 8).double())
    r = torch.arange(q.shape[-2], device=q.device)[:, None]
    b = torch.arange(v.shape[-1] // 32, device=q.device)[None, :]
    scale = torch.exp2(sf[..., r // 128, b // 4, r % 128, b % 4].double() - 127)
    return (v.view(*v.shape[:-1], -1, 32) * scale[..., None]).flatten(-2)[..., :K]


def exact(case, seed):
    s = prepare(case, seed)
    op, x = case["op"], s["x"]
    if op == "quantize":
        out = {"row": _exact_fake(x)}
        if case["columnwise"]:
            out["col"] = _exact_fake(x.t())
        return out
    K, N = case["inner"], case["outer"]
    if op == "linear":
        return _exact_fake(x) @ _exact_weight(s["w_q"], s["w_sf"], K).t()
    if op == "train":
        w, dy = s["w"], s["dy"]
        return {"y": _exact_fake(x) @ _exact_fake(w).t(), "dx": _exact_fake(dy) @ _exact_fake(w.t()).t(),
                "dw": _exact_fake(dy.t()) @ _exact_fake(x.t()).t()}
    o, rows = s["offsets"].tolist(), s["rows"].long()
    R = rows.numel()
    if op == "experts":
        y = torch.zeros(R, N, dtype=torch.float64, device=x.device)
        qx = _exact_fake(x)
        for e in range(case["experts"]):
            if o[e] < o[e + 1]:
                w = _exact_weight(s["w_q"][e], s["w_sf"][e], K)
                y[o[e]:o[e + 1]] = qx[rows[o[e]:o[e + 1]]] @ w.t()
        return y * s["p"].double()[:, None]
    dy = s["dy"]
    dx = torch.zeros(R, K, dtype=torch.float64, device=x.device)
    dw = torch.zeros(case["experts"], N, K, dtype=torch.float64, device=x.device)
    for e in range(case["experts"]):
        a, b = o[e], o[e + 1]
        if a < b:
            dx[a:b] = _exact_fake(dy[a:b]) @ _exact_weight(s["wt_q"][e], s["wt_sf"][e], N).t()
            dw[e] = _exact_fake(dy[a:b].t()) @ _exact_fake(x[rows[a:b]].t()).t()
    return {"dx": dx, "dw": dw}
