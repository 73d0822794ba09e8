"""A gated mixture-of-experts layer on this library's formats: one training step
in MXFP8 and one decoding step with NVFP4 weights.

    python examples/moe_layer.py

Training (all operands quantized by the library, every product one of its
grouped products):

    x -> MXFP8 -> [gate | up] = x W1^T -> SwiGLU -> MXFP8 -> f = h W2^T
    df -> MXFP8 -> dh = df W2 -> dSwiGLU -> MXFP8 -> dx = d[gate | up] W1
    dW2 = df^T h,  dW1 = d[gate | up]^T x

A token's experts are summed by its router's weights: y = sum_j p_j f_j, so that
df_j = p_j dy and dp_j = dy . f_j.  Without weights every p_j is one.  Rows are sorted
by expert, each expert's padded with zero rows to a multiple of 32, so that no block of
32 rows belongs to two experts.  block_step and block_decode put the residual's
addition, the norm and the router around it.  Decoding multiplies the
few rows of a step with the experts' 4-bit weights where they lie.  dense_step is
the block without experts, whose norm hands its codes to the products.
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import fp4_quantization_gb300 as mxq  # noqa: E402


def sort_rows(experts, num_experts):
    """Where each (token, expert) pair goes: its row in the buffer sorted by
    expert, the group offsets [E + 1] (multiples of 32), and the buffer's rows
    (a bound that needs no copy to the host).  A pair without an expert has row -1,
    which indexes the last one: with such a pair the bound is longer than the groups,
    and that row is no expert's."""
    out = mxq.moe_sort(experts.int().contiguous(), num_experts, align=32)
    return out["rows"].flatten().long(), out["offsets"], len(out["source"])


class MXWeights:
    """An expert stack [E, N, K] in MXFP8 along both axes: rows for the
    products, columns for the input gradients."""

    def __init__(self, w):
        q = [mxq.mx_quantize_rowcol(e) for e in w]
        self.q, self.s, self.q_t, self.s_t = (
            torch.stack([d[k] for d in q]) for k in ("q_row", "s_row", "q_col", "s_col"))


def train_step(x, experts, w1, w2, dy, weights=None, checkpoint=False):
    """x [T, H] bf16, experts [T, k] (-1: none), w1 [E, 2F, H] and w2 [E, H, F]
    as MXWeights, dy [T, H]: y and dx [T, H] (summed over a token's experts) and the
    weights' gradients in fp32; with the router's weights [T, k] fp32, their
    gradient too.  With `checkpoint` the backward pass reads [gate | up], the
    largest activation, in 8 bits, so that its bf16 form need not be kept."""
    T, k = experts.shape
    row, offsets, rows = sort_rows(experts, w1.q.shape[0])

    def scatter(t, weights=None):
        out = torch.zeros(rows, t.shape[1], dtype=torch.bfloat16, device=t.device)
        t = t.repeat_interleave(k, 0)
        out[row] = t if weights is None else (t * weights.view(-1, 1)).bfloat16()
        return out

    def gather(t, weights=None):
        t = t[row].view(T, k, -1).float()
        return (t if weights is None else t * weights.unsqueeze(-1)).sum(1).bfloat16()

    def rows_product(q, w, w_s):
        # The padding after the last group belongs to no expert and stays zero.
        out = torch.zeros(rows, w.shape[1], dtype=torch.bfloat16, device=w.device)
        return mxq.mx_grouped_gemm(q["q_row"], q["s_row"], w, w_s, offsets, out=out)

    xq = mxq.mx_quantize_rowcol(scatter(x))
    gate_up = rows_product(xq, w1.q, w1.s)
    if checkpoint:
        hq = mxq.mx_quantize_gated_save(gate_up)
        saved = hq["x_q"], hq["x_s"]
        del gate_up
    else:
        hq = mxq.mx_quantize_gated(gate_up)
    f = rows_product(hq, w2.q, w2.s)

    gq = mxq.mx_quantize_rowcol(scatter(dy, weights))
    dh = rows_product(gq, w2.q_t, w2.s_t)
    dgq = mxq.mx_quantize_dgated_saved(dh, *saved) if checkpoint else mxq.mx_quantize_dgated(dh, gate_up)
    dx = rows_product(dgq, w1.q_t, w1.s_t)
    dw1 = mxq.mx_grouped_wgrad(dgq["q_col"], dgq["s_col"], xq["q_col"], xq["s_col"], offsets)
    dw2 = mxq.mx_grouped_wgrad(gq["q_col"], gq["s_col"], hq["q_col"], hq["s_col"], offsets)
    if weights is None:
        return gather(f), gather(dx), dw1, dw2
    dweights = (f[row].view(T, k, -1).float() * dy.float().unsqueeze(1)).sum(-1)
    return gather(f, weights), gather(dx), dw1, dw2, dweights


def block_step(x, residual, gamma, router, k, w1, w2, dout):
    """A training step of the block around the layer: out = h + sum_j p_j f_j(y) with
    h = x + residual, y its RMSNorm times gamma [H], and p the softmax of the k
    largest of y router^T [T, E], over their sum.  x, residual, dout [T, H] bf16,
    router [E, H] fp32: out, and the gradients of x (and of the residual alike),
    gamma, the router and both weights."""
    n = mxq.mx_rmsnorm(x, gamma, mxq.OUT_BF16, residual=residual)
    h, y = n["h"], n["y"]
    logits = y.float() @ router.t()
    experts, p = mxq.moe_route(logits, k, mxq.ROUTE_RENORM)
    f, dy, dw1, dw2, dp = train_step(y, experts, w1, w2, dout, p, checkpoint=True)
    dlogits = mxq.moe_route_backward(dp, logits, experts, mxq.ROUTE_RENORM)
    dy = (dy.float() + dlogits @ router).bfloat16()
    back = mxq.mx_rmsnorm_backward(dy, h, n["rstd"], gamma, dh=dout)
    return h + f, back["dx"], back["dweight"], dlogits.t() @ y.float(), dw1, dw2


def dense_step(x, residual, gamma, w1, w2, dout):
    """A training step of a dense block, out = h + f(y) with h = x + residual and y its
    RMSNorm times gamma [H].  The norm's own codes are what the products take: rows
    forward, columns for dW1.  x, residual, dout [T, H] bf16, T a multiple of 32, w1
    [1, 2F, H] and w2 [1, H, F] as MXWeights: out, and the gradients of x (and of the
    residual alike), gamma and both weights."""
    offsets = torch.arange(2, dtype=torch.int32, device=x.device) * len(x)

    def rows_product(q, w, w_s):
        return mxq.mx_grouped_gemm(q["q_row"], q["s_row"], w, w_s, offsets)

    def gradient(g, x):
        return mxq.mx_grouped_wgrad(g["q_col"], g["s_col"], x["q_col"], x["s_col"], offsets)

    n = mxq.mx_rmsnorm(x, gamma, residual=residual)
    hq = mxq.mx_quantize_gated_save(rows_product(n, w1.q, w1.s))
    f = rows_product(hq, w2.q, w2.s)

    gq = mxq.mx_quantize_rowcol(dout)
    dgq = mxq.mx_quantize_dgated_saved(rows_product(gq, w2.q_t, w2.s_t), hq["x_q"], hq["x_s"])
    dy = rows_product(dgq, w1.q_t, w1.s_t)
    back = mxq.mx_rmsnorm_backward(dy, n["h"], n["rstd"], gamma, dh=dout)
    return n["h"] + f, back["dx"], back["dweight"], gradient(dgq, n), gradient(gq, hq)


class NVWeights:
    """An expert stack [E, N, K] in NVFP4 along its rows."""

    def __init__(self, w):
        q = [mxq.nvfp4_quantize_transpose(e, mxq.ROWWISE) for e in w]
        self.q, self.s, self.g = (
            torch.stack([d[k] for d in q]) for k in ("q_row", "s_row", "global_scale"))
        self.g = self.g.flatten()


def decode_step(x, experts, w1, w2, weights=None):
    """x [T, H] bf16, experts [T, k], w1 [E, 2F, H] and w2 [E, H, F] as
    NVWeights, the router's weights [T, k] fp32 or none: y [T, H]."""
    T, k = experts.shape
    ids = experts.flatten().int()
    gate_up = mxq.nvfp4_gemv(x, w1.q, w1.s, w1.g, experts=ids, share=k, out_dtype=torch.float32)
    gate, up = gate_up.chunk(2, 1)
    h = (torch.nn.functional.silu(gate) * up).bfloat16()
    f = mxq.nvfp4_gemv(h, w2.q, w2.s, w2.g, experts=ids, out_dtype=torch.float32).view(T, k, -1)
    return (f if weights is None else f * weights.unsqueeze(-1)).sum(1).bfloat16()


def block_decode(x, residual, gamma, router, k, w1, w2):
    """The block for the few tokens of a decoding step, w1 and w2 as NVWeights."""
    n = mxq.mx_rmsnorm(x, gamma, mxq.OUT_BF16, residual=residual)
    experts, p = mxq.moe_route(n["y"].float() @ router.t(), k, mxq.ROUTE_RENORM)
    return n["h"] + decode_step(n["y"], experts, w1, w2, p)


def main():
    T, k, E, H, F = 512, 2, 8, 512, 1024
    gen = torch.Generator(device="cuda").manual_seed(0)

    def draw(*shape, scale=1.0):
        return (torch.randn(*shape, generator=gen, device="cuda") * scale).bfloat16()

    w1, w2 = draw(E, 2 * F, H, scale=H ** -0.5), draw(E, H, F, scale=F ** -0.5)
    x, dy = draw(T, H), draw(T, H)
    scores, experts = (x.float() @ draw(E, H, scale=H ** -0.5).float().t()).topk(k, 1)
    p = scores.softmax(1)
    y, dx, dw1, dw2, dp = train_step(x, experts, MXWeights(w1), MXWeights(w2), dy, p)
    print("training:", *(f"{n} {tuple(t.shape)} norm {t.float().norm():.4g}"
                         for n, t in (("y", y), ("dx", dx), ("dw1", dw1), ("dw2", dw2), ("dp", dp))))
    z = decode_step(x[:4], experts[:4], NVWeights(w1), NVWeights(w2), p[:4])
    off = (z.float() - y[:4].float()).norm() / y[:4].float().norm()
    print(f"decoding: y {tuple(z.shape)}, {off:.3f} from the MXFP8 rows")
    gamma, router = 1 + 0.1 * draw(H).float(), draw(E, H, scale=H ** -0.5).float()
    out = block_step(x, draw(T, H), gamma, router, k, MXWeights(w1), MXWeights(w2), dy)
    print("block:", *(f"{n} {tuple(t.shape)} norm {t.float().norm():.4g}"
                      for n, t in zip(("out", "dx", "dgamma", "drouter", "dw1", "dw2"), out)))
    out = dense_step(x, draw(T, H), gamma, MXWeights(w1[:1]), MXWeights(w2[:1]), dy)
    print("dense:", *(f"{n} {tuple(t.shape)} norm {t.float().norm():.4g}"
                      for n, t in zip(("out", "dx", "dgamma", "dw1", "dw2"), out)))


if __name__ == "__main__":
    main()
