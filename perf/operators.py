"""Products on block-scaled operands: the cases that are measured, their plain
forms and their values in 64 bits.

Three operators take what the quantization calls of this library write.

* ``mx_grouped_gemm`` -- rows sorted by expert, each multiplied by its expert's
  weight: out[m, n] = sum_k x[m, k] * w[e, n, k] for offsets[e] <= m <
  offsets[e + 1], with x [M, K] and w [E, N, K] as E4M3 codes and one E8M0
  scale per 32 values along k.  The input gradient is the same product with
  the gradient's rows and the weight quantized along its other axis.
* ``mx_grouped_wgrad`` -- the weights' gradients: dw[e, n, k] = sum over the
  rows m of expert e of g[m, n] * x[m, k], both operands quantized along m
  (codes [N, M] and [K, M], scales per 32 rows), group starts multiples of 32.
* ``nvfp4_gemv`` -- few rows times 4-bit weights: out[r, n] = sum_k x[r, k] *
  w[e(r), n, k], x bf16, w as E2M1 codes (two to a byte, element 2i in the low
  nibble), one E4M3 scale per 16 values along k and one fp32 scale per expert.
  With experts, `share` consecutive output rows read one row of x, and a row
  whose expert id is negative is zero.
"""
import math

import torch

own = False

BF16, F32 = "bf16", "f32"
_OUT = {BF16: torch.bfloat16, F32: torch.float32}


def listed():
    return [
        # One decode step of a small batch: a few rows for each expert, some
        # with none; the weights' bytes and the launch are all there is.
        {"name": "gemm_decode", "op": "gemm", "E": 8, "M": 24, "N": 1024, "K": 2048, "out": BF16},
        # Many small experts on a short prompt: about 64 rows each, unevenly.
        {"name": "gemm_many_experts", "op": "gemm", "E": 64, "M": 4096, "N": 1408, "K": 2048, "out": BF16},
        # Odd numbers of rows and columns, K a multiple of 32 only, fp32 out.
        {"name": "gemm_odd", "op": "gemm", "E": 5, "M": 1013, "N": 1001, "K": 1056, "out": F32},
        # The input gradient of a training step: gradient rows times the
        # weight quantized along its output axis.
        {"name": "gemm_dgrad", "op": "gemm", "E": 8, "M": 8192, "N": 4096, "K": 8192, "out": BF16},
        # The up projection of a training step (the widths of this library's
        # gated workload), two thousand rows for each expert on average.
        {"name": "gemm_large", "op": "gemm", "E": 8, "M": 16384, "N": 14336, "K": 4096, "out": BF16},
        # Weight gradients: a small layer, many small experts, and the partner
        # of gemm_large.
        {"name": "wgrad_small", "op": "wgrad", "E": 4, "M": 256, "N": 520, "K": 352, "out": F32},
        {"name": "wgrad_many_experts", "op": "wgrad", "E": 64, "M": 8192, "N": 1408, "K": 2048, "out": F32},
        {"name": "wgrad_large", "op": "wgrad", "E": 8, "M": 16384, "N": 14336, "K": 4096, "out": BF16},
        # One token through one square projection: the shortest call.
        {"name": "gemv_one", "op": "gemv", "E": 0, "T": 1, "share": 1, "N": 2048, "K": 2048, "out": BF16},
        # One token through a wide layer whose weights exceed the L2 cache.
        {"name": "gemv_wide", "op": "gemv", "E": 0, "T": 1, "share": 1, "N": 28672, "K": 8192, "out": BF16},
        # A batch of thirteen tokens, an odd output width, fp32 out.
        {"name": "gemv_batch", "op": "gemv", "E": 0, "T": 13, "share": 1, "N": 4099, "K": 11008, "out": F32},
        # Eight tokens, four of 64 experts each: the routed form of one step.
        {"name": "gemv_experts", "op": "gemv", "E": 64, "T": 8, "share": 4, "N": 2816, "K": 2048, "out": BF16},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("gemm", "wgrad", "gemv"))
    out = rng.choice((BF16, F32))
    if op == "gemv":
        # One to sixteen tokens, dense or routed to one to eight experts each.
        E = rng.choice((0, 0, _log(rng, 4, 128)))
        T = _log(rng, 1, 16)
        share = _log(rng, 1, min(8, E)) if E else 1
        K = 32 * _log(rng, 16, 448)
        N = _log(rng, 256, 28672)
        # No more weights read, and at most twice as many held, as the widest.
        N = max(64, min(N, 28672 * 8192 // (K * max(1, min(E, T * share), E // 2))))
        return {"op": op, "E": E, "T": T, "share": share, "N": N, "K": K, "out": out}
    E = _log(rng, 1, 64)
    if op == "gemm":
        M = _log(rng, 1, 16384)
        K = 32 * _log(rng, 8, 448)
        N = _log(rng, 64, 14336)
    else:
        M = 32 * _log(rng, 1, 512)
        K = 32 * _log(rng, 8, 256)
        N = 8 * _log(rng, 8, 1792)
    # No more operations, and no more weights, than the largest listed case.
    most = 16384 * 14336 * 4096
    N = max(8, min(N, most // (M * K) // 8 * 8, 8 * 14336 * 4096 // (E * K) // 8 * 8 + N % 8))
    return {"op": op, "E": E, "M": M, "N": N, "K": K, "out": out}


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------

def _mx(x):
    """MXFP8 of x [..., K] fp32 along its last axis: codes and scale bytes,
    both uint8.  Floor rule: the scale is 2^(floor(log2 amax) - 8)."""
    b = x.unflatten(-1, (-1, 32))
    amax = b.abs().amax(-1)
    e = (torch.frexp(amax).exponent - 9).clamp_(-127, 127)
    e = torch.where(amax > 0, e, -127)
    q = (b * torch.exp2(-e.float()).unsqueeze(-1)).clamp_(-448, 448)
    return q.flatten(-2).to(torch.float8_e4m3fn).view(torch.uint8), (e + 127).to(torch.uint8)


def _nv(w):
    """NVFP4 of w [E, N, K] fp32: packed E2M1 codes, E4M3 scale bytes and one
    fp32 scale per expert."""
    g = w.abs().amax((-2, -1)) / 2688
    b = w.unflatten(-1, (-1, 16))
    s = (b.abs().amax(-1) / 6 / g[:, None, None]).clamp_(max=448).to(torch.float8_e4m3fn)
    d = s.float() * g[:, None, None]
    v = b / torch.where(d > 0, d, 1).unsqueeze(-1)
    edges = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=w.device)
    c = torch.bucketize(v.abs().flatten(-2), edges).to(torch.uint8)
    c |= (v.flatten(-2) < 0).to(torch.uint8) << 3
    return c[..., 0::2] | c[..., 1::2] << 4, s.view(torch.uint8), g


def _groups(E, units, gen):
    """E uneven group sizes that add up to `units`, as a router leaves them."""
    p = torch.softmax(torch.randn(E, generator=gen, dtype=torch.float64) * 0.7, 0)
    return torch.bincount(torch.multinomial(p, units, replacement=True, generator=gen), minlength=E)


def _activations(gen, rows, cols):
    """Normal values with one channel in 64 ten times as large."""
    x = torch.randn(rows, cols, generator=gen, device="cuda")
    x[:, torch.randint(cols, (cols // 64,), generator=gen, device="cuda")] *= 10
    return x


def prepare(case, seed):
    cpu = torch.Generator().manual_seed(seed)
    gen = torch.Generator(device="cuda").manual_seed(seed)
    E, N, K = case["E"], case["N"], case["K"]
    st = {"op": case["op"], "dtype": _OUT[case["out"]]}
    if case["op"] == "gemv":
        x = _activations(gen, case["T"], K).bfloat16()
        w = torch.randn(max(E, 1), N, K, generator=gen, device="cuda") * K ** -0.5
        q, s, g = _nv(w.bfloat16().float())
        st.update(x=x, share=case["share"])
        if E:
            # Each token's `share` experts, all different; about one slot in
            # sixteen belongs to an expert that another rank holds.
            ids = torch.rand(case["T"], E, generator=cpu).topk(case["share"], 1).indices
            ids = torch.where(torch.rand(ids.shape, generator=cpu) < 1 / 16, -1, ids)
            st.update(w_q=q, w_s=s, g=g, experts=ids.flatten().int().cuda())
        else:
            st.update(w_q=q[0], w_s=s[0], g=g, experts=None)
        return st
    M, step = case["M"], 32 if case["op"] == "wgrad" else 1
    sizes = _groups(E, M // step, cpu) * step
    offsets = torch.zeros(E + 1, dtype=torch.int32)
    offsets[1:] = sizes.cumsum(0)
    st.update(offsets=offsets.cuda(), most=int(sizes.max()))
    if case["op"] == "gemm":
        st["x_q"], st["x_s"] = _mx(_activations(gen, M, K).bfloat16().float())
        w = torch.randn(E, N, K, generator=gen, device="cuda") * K ** -0.5
        st["w_q"], st["w_s"] = _mx(w.bfloat16().float())
    else:
        g = torch.randn(N, M, generator=gen, device="cuda") * 1e-3
        st["g_q"], st["g_s"] = _mx(g.bfloat16().float())
        st["x_q"], st["x_s"] = _mx(_activations(gen, M, K).bfloat16().float().t().contiguous())
    return st


# ---------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------

def run(state):
    st = state
    if own:
        import fp4_quantization_gb300 as mxq

        if st["op"] == "gemm":
            return mxq.mx_grouped_gemm(st["x_q"], st["x_s"], st["w_q"], st["w_s"], st["offsets"], out_dtype=st["dtype"])
        if st["op"] == "wgrad":
            return mxq.mx_grouped_wgrad(st["g_q"], st["g_s"], st["x_q"], st["x_s"], st["offsets"], out_dtype=st["dtype"])
        return mxq.nvfp4_gemv(st["x"], st["w_q"], st["w_s"], st["g"], experts=st["experts"], share=st["share"], out_dtype=st["dtype"])
    return {"gemm": _plain_gemm, "wgrad": _plain_wgrad, "gemv": _plain_gemv}[st["op"]](st)


def _mx_values(q, s):
    """fp32 values of MXFP8 codes [..., K] with scales [..., K / 32]."""
    scale = torch.where(s == 0, 2.0 ** -127, (s.int() << 23).view(torch.float32))
    return (q.view(torch.float8_e4m3fn).float().unflatten(-1, (-1, 32)) * scale.unsqueeze(-1)).flatten(-2)


def _padded(st, rows):
    """Row numbers of every group, padded to the longest group, and which of
    them are rows of the group."""
    off = st["offsets"].long()
    at = off[:-1, None] + torch.arange(st["most"], device="cuda")
    return at.clamp(max=rows - 1), at < off[1:, None]


def _plain_gemm(st):
    x, w = _mx_values(st["x_q"], st["x_s"]), _mx_values(st["w_q"], st["w_s"])
    at, real = _padded(st, len(x))
    y = torch.bmm(x[at] * real.unsqueeze(-1), w.transpose(1, 2))
    m = torch.arange(len(x), device="cuda")
    off = st["offsets"].long()
    e = torch.searchsorted(off, m, right=True) - 1
    return y[e, m - off[e]].to(st["dtype"])


def _plain_wgrad(st):
    g, x = _mx_values(st["g_q"], st["g_s"]), _mx_values(st["x_q"], st["x_s"])
    at, real = _padded(st, g.shape[1])
    g = g.t()[at] * real.unsqueeze(-1)
    return torch.bmm(g.transpose(1, 2), x.t()[at]).to(st["dtype"])


def _plain_gemv(st):
    q, s, g, ids = st["w_q"], st["w_s"], st["g"], st["experts"]
    x = st["x"].float()
    if ids is not None:
        real = ids >= 0
        e = ids.clamp(min=0).long()
        q, s, g = q[e], s[e], g[e][:, None, None]
        x = x.repeat_interleave(st["share"], 0)
    value = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6], device="cuda")
    w = value[torch.stack((q & 15, q >> 4), -1).flatten(-2).int()]
    w = (w.unflatten(-1, (-1, 16)) * (s.view(torch.float8_e4m3fn).float() * g).unsqueeze(-1)).flatten(-2)
    if ids is None:
        return torch.mm(x, w.t()).to(st["dtype"])
    y = torch.bmm(w, x.unsqueeze(-1)).squeeze(-1)
    return (y * real.unsqueeze(-1)).to(st["dtype"])


# ---------------------------------------------------------------------------
# The definition in 64 bits
# ---------------------------------------------------------------------------

def _decode64(codes, exponent_bits, mantissa_bits, bias):
    """Values of a small float format from its definition, in 64 bits."""
    c = codes.to(torch.int16)
    m = (c & ((1 << mantissa_bits) - 1)).double() / (1 << mantissa_bits)
    e = c >> mantissa_bits & ((1 << exponent_bits) - 1)
    v = torch.where(e > 0, 1 + m, 2 * m) * torch.pow(2.0, (e - bias).double())
    return torch.where(c >> (exponent_bits + mantissa_bits) & 1 > 0, -v, v)


def _mx64(q, s):
    return _decode64(q, 4, 3, 7) * torch.pow(2.0, s.double() - 127).repeat_interleave(32, -1)


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "gemv":
        x, N, K = st["x"].double(), case["N"], case["K"]
        q, s = st["w_q"].view(-1, N, K // 2), st["w_s"].view(-1, N, K // 16)
        ids = [0] * case["T"] if st["experts"] is None else st["experts"].tolist()
        y = torch.zeros(len(ids), N, dtype=torch.float64, device="cuda")
        for e in sorted(set(ids) - {-1}):
            w = torch.empty(N, K, dtype=torch.float64, device="cuda")
            w[:, 0::2] = _decode64(q[e] & 15, 2, 1, 1)
            w[:, 1::2] = _decode64(q[e] >> 4, 2, 1, 1)
            w *= _decode64(s[e], 4, 3, 7).repeat_interleave(16, -1) * st["g"][e].double()
            rows = [r for r, i in enumerate(ids) if i == e]
            y[rows] = x[[r // case["share"] for r in rows]] @ w.t()
        return y
    off = st["offsets"].tolist()
    if case["op"] == "gemm":
        y = torch.zeros(case["M"], case["N"], dtype=torch.float64, device="cuda")
        for e in range(case["E"]):
            a, b = off[e], off[e + 1]
            y[a:b] = _mx64(st["x_q"][a:b], st["x_s"][a:b]) @ _mx64(st["w_q"][e], st["w_s"][e]).t()
        return y
    g, x = _mx64(st["g_q"], st["g_s"]), _mx64(st["x_q"], st["x_s"])
    return torch.stack([g[:, a:b] @ x[:, a:b].t() for a, b in zip(off, off[1:])])


# ---------------------------------------------------------------------------
# What a pass cannot do without
# ---------------------------------------------------------------------------

def work(case):
    E, N, K = case["E"], case["N"], case["K"]
    size = 2 if case["out"] == BF16 else 4
    if case["op"] == "gemv":
        T, share = case["T"], case["share"]
        rows = T * share
        used = E * (1 - (1 - share / E) ** T) if E else 1
        return {"bytes": used * N * (K // 2 + K // 16) + 2 * T * K + rows * N * size, "flops": 2.0 * rows * N * K}
    M = case["M"]
    if case["op"] == "gemm":
        used = E * (1 - (1 - 1 / E) ** M)
        return {"bytes": (M + used * N) * (K + K // 32) + M * N * size, "flops": 2.0 * M * N * K}
    return {"bytes": (N + K) * (M + M // 32) + E * N * K * size, "flops": 2.0 * M * N * K}
