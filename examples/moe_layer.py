"""A gated mixture-of-experts layer on this library's formats: one training step
in MXFP8 and one decoding step with NVFP4 weights.

    python examples/moe_layer.py

Training (all operands quantized by the library, every product one of its
grouped products):

    x -> MXFP8 -> [gate | up] = x W1^T -> SwiGLU -> MXFP8 -> f = h W2^T
    df -> MXFP8 -> dh = df W2 -> dSwiGLU -> MXFP8 -> dx = d[gate | up] W1
    dW2 = df^T h,  dW1 = d[gate | up]^T x

A token's experts are summed by its router's weights: y = sum_j p_j f_j, so that
df_j = p_j dy and dp_j = dy . f_j.  Without weights every p_j is one.  Rows are sorted by expert, each expert's padded with zero rows to a multiple of
32, so that no block of 32 rows belongs to two experts.  Decoding multiplies the
few rows of a step with the experts' 4-bit weights where they lie.
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import fp4_quantization_gb300 as mxq  # noqa: E402


def sort_rows(experts, num_experts):
    """Where each (token, expert) pair goes: its row in the buffer sorted by
    expert, the group offsets [E + 1] (multiples of 32), and the buffer's rows."""
    flat = experts.flatten()
    sizes = torch.bincount(flat, minlength=num_experts)
    padded = (sizes + 31) // 32 * 32
    offsets = torch.zeros(num_experts + 1, dtype=torch.int32, device=flat.device)
    offsets[1:] = padded.cumsum(0)
    order = flat.argsort(stable=True)
    first = torch.zeros_like(sizes)
    first[1:] = sizes.cumsum(0)[:-1]
    rank = torch.arange(len(flat), device=flat.device) - first[flat[order]]
    row = torch.empty_like(order)
    row[order] = offsets[:-1].long()[flat[order]] + rank
    # A bound that needs no copy to the host: every pair, and 31 rows an expert.
    rows = (len(flat) + 31 * num_experts + 31) // 32 * 32
    return row, offsets, rows


class MXWeights:
    """An expert stack [E, N, K] in MXFP8 along both axes: rows for the
    products, columns for the input gradients."""

    def __init__(self, w):
        q = [mxq.mx_quantize_rowcol(e) for e in w]
        self.q, self.s, self.q_t, self.s_t = (
            torch.stack([d[k] for d in q]) for k in ("q_row", "s_row", "q_col", "s_col"))


def train_step(x, experts, w1, w2, dy, weights=None):
    """x [T, H] bf16, experts [T, k], w1 [E, 2F, H] and w2 [E, H, F] as MXWeights,
    dy [T, H]: y and dx [T, H] (summed over a token's experts) and the
    weights' gradients in fp32; with the router's weights [T, k] fp32, their
    gradient too."""
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
    hq = mxq.mx_quantize_gated(gate_up)
    f = rows_product(hq, w2.q, w2.s)

    gq = mxq.mx_quantize_rowcol(scatter(dy, weights))
    dh = rows_product(gq, w2.q_t, w2.s_t)
    dgq = mxq.mx_quantize_dgated(dh, gate_up)
    dx = rows_product(dgq, w1.q_t, w1.s_t)
    dw1 = mxq.mx_grouped_wgrad(dgq["q_col"], dgq["s_col"], xq["q_col"], xq["s_col"], offsets)
    dw2 = mxq.mx_grouped_wgrad(gq["q_col"], gq["s_col"], hq["q_col"], hq["s_col"], offsets)
    if weights is None:
        return gather(f), gather(dx), dw1, dw2
    dweights = (f[row].view(T, k, -1).float() * dy.float().unsqueeze(1)).sum(-1)
    return gather(f, weights), gather(dx), dw1, dw2, dweights


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


if __name__ == "__main__":
    main()
