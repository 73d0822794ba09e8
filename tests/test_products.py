"""Products on block-scaled operands against their definition in 64 bits.

Two kinds of inputs.  With small whole numbers and power-of-two scales every
partial sum is a multiple of 2^-4 below 2^19, so it is exact in fp32 whatever
the order, and the result must equal the 64-bit value rounded once.  With
random codes and scales the error of n terms added in fp32 in any order, each
addition off by at most one unit in the last place (truncation included), is
at most n 2^-23 sum|terms|.  A bf16 output is that sum rounded, and rounding
keeps order, so it lies between the two ends of that interval rounded alike.
"""
import ctypes

import pytest
import torch

import fp4_quantization_gb300 as mxq
from fp4_quantization_gb300 import _lib

gpu = pytest.mark.gpu

# E4M3 codes of 0, .5, 1, 1.5, 2 and their negatives; E2M1 codes likewise.
E4M3_SMALL = [0x00, 0x30, 0x38, 0x3C, 0x40, 0xB0, 0xB8, 0xBC, 0xC0]
E2M1_SMALL = [0, 1, 2, 3, 4, 9, 10, 11, 12]


# ---------------------------------------------------------------------------
# The definition
# ---------------------------------------------------------------------------

def e4m3_values(q):
    return q.view(torch.float8_e4m3fn).to(torch.float64)


def mx_values(q, s):
    return e4m3_values(q) * torch.pow(2.0, s.double() - 127).repeat_interleave(32, -1)


def nv_values(q, s):
    table = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device=q.device)
    c = torch.stack((q & 15, q >> 4), -1).flatten(-2).long()
    v = table[c & 7] * torch.where(c > 7, -1.0, 1.0)
    return v * e4m3_values(s).repeat_interleave(16, -1)


def pick(gen, codes, *shape):
    t = torch.tensor(codes, dtype=torch.uint8, device="cuda")
    return t[torch.randint(len(codes), shape, generator=gen, device="cuda")]


def mx_operand(gen, exact, *shape):
    """Codes [..., K] and scales [..., K / 32]."""
    scales = (*shape[:-1], shape[-1] // 32)
    if exact:
        return pick(gen, E4M3_SMALL, *shape), pick(gen, [126, 127, 128], *scales)
    q = torch.randint(0, 256, shape, generator=gen, device="cuda", dtype=torch.uint8)
    q = torch.where((q & 0x7F) == 0x7F, q - 1, q)              # no NaN codes
    return q, torch.randint(117, 138, scales, generator=gen, device="cuda", dtype=torch.uint8)


def check(got, want, bound, exact, what=""):
    """want, bound: 64 bits; bound = n 2^-23 sum|terms| per element."""
    assert not torch.isnan(got.double()).any() or torch.isnan(want).any(), what
    if exact:
        ref = want.float().to(got.dtype)
        bad = (got != ref).nonzero()
        assert len(bad) == 0, (f"{what}: {len(bad)} of {got.numel()} differ, first {bad[:4].tolist()}: "
                               f"{got[tuple(bad[0])]} for {ref[tuple(bad[0])]}")
        return
    low, high = ((want + d).float().to(got.dtype) for d in (-bound, bound))
    bad = ((got < low) | (got > high)).nonzero()
    assert len(bad) == 0, (f"{what}: {len(bad)} of {got.numel()} off, first {bad[:4].tolist()}: "
                           f"{got[tuple(bad[0])]} not in {low[tuple(bad[0])]}..{high[tuple(bad[0])]}")


def generator(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def offsets_of(sizes, first=0):
    t = torch.tensor([first, *sizes], dtype=torch.int64).cumsum(0)
    return t.to(torch.int32).cuda()


def dev_err():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


# ---------------------------------------------------------------------------
# mx_grouped_gemm
# ---------------------------------------------------------------------------

GEMM = [
    # name, group sizes, N, K, rows before the first group, rows after the last
    ("one_row", [1], 8, 32, 0, 0),
    ("one_tile", [128], 128, 128, 0, 0),
    ("one_group", [130], 257, 160, 0, 0),
    ("empty_groups", [0, 3, 0, 0, 33, 1, 0], 96, 96, 0, 0),
    ("all_empty", [0, 0, 0], 40, 64, 5, 6),
    ("odd", [127, 129, 1, 255, 64], 1001, 1056, 0, 0),
    ("outside_rows", [5, 300], 130, 544, 7, 200),
    ("long_k", [40, 200], 72, 8192 + 32, 0, 0),
    ("ranges", [33, 130], 160, 3 * 8192 - 64, 0, 0),
    ("ranges_odd", [130, 200], 161, 8192 + 64, 0, 0),
    ("few", [100, 0, 3, 1, 0], 300, 1056, 4, 9),
    ("few_ranges", [5, 40, 0], 203, 2 * 8192 + 96, 0, 0),
    ("few_wide", [(i * 5) % 9 for i in range(40)], 2500, 512, 0, 0),
    ("chunk_edges", [128, 256, 384], 384, 512, 0, 0),
    ("many_tiles", [700, 90, 2000, 1310], 1400, 736, 0, 0),
    ("many_groups", [(i * 37) % 23 for i in range(300)], 48, 224, 0, 0),
    ("wide_pairs", [600, 1, 0, 4000, 256], 4096, 640, 0, 0),
]


@gpu
@pytest.mark.parametrize("exact", [True, False], ids=["exact", "random"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("name,sizes,N,K,before,after", GEMM, ids=[c[0] for c in GEMM])
def test_grouped_gemm(name, sizes, N, K, before, after, dtype, exact):
    gen = generator(len(name) + N + K)
    E, M = len(sizes), before + sum(sizes) + after
    x_q, x_s = mx_operand(gen, exact, M, K)
    w_q, w_s = mx_operand(gen, exact, E, N, K)
    off = offsets_of(sizes, before)
    err = dev_err()
    out = torch.full((M, N), 77.0, dtype=dtype, device="cuda")
    mxq.mx_grouped_gemm(x_q, x_s, w_q, w_s, off, out=out, dev_err=err)
    torch.cuda.synchronize()
    assert err.item() == 0
    x, w = mx_values(x_q, x_s), mx_values(w_q, w_s)
    want = torch.full((M, N), 77.0, dtype=torch.float64, device="cuda")
    bound = torch.zeros_like(want)
    for e in range(E):
        a, b = int(off[e]), int(off[e + 1])
        want[a:b] = x[a:b] @ w[e].t()
        bound[a:b] = K * 2.0 ** -23 * (x[a:b].abs() @ w[e].abs().t())
    check(out, want, bound, exact, name)


# Few tiles of a long contraction: CTAs of a cluster share it.
GEMM_SPLIT = [
    ("one_row", [1], 200, 4096, 0, 0),
    ("few_rows", [31], 1000, 8192 - 32, 1, 2),
    ("few_experts", [3, 0, 9, 1], 513, 2048, 0, 0),
    ("last_range_empty", [5], 128, 128 * 65, 0, 0),
    ("dense", [60], 513, 4096, 3, 4),
    ("dense_odd", [77, 0, 250], 267, 2080, 0, 0),
    ("dense_aligned", [128, 256], 256, 16384, 0, 0),
    ("all_empty", [0, 0], 64, 4096, 50, 50),
]


@gpu
@pytest.mark.parametrize("exact", [True, False], ids=["exact", "random"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("name,sizes,N,K,before,after", GEMM_SPLIT, ids=[c[0] for c in GEMM_SPLIT])
def test_grouped_gemm_shared_contraction(name, sizes, N, K, before, after, dtype, exact):
    test_grouped_gemm(name, sizes, N, K, before, after, dtype, exact)


@gpu
def test_grouped_gemm_shared_contraction_in_place():
    """A view at an odd element, the same bits every time, and nothing written
    where the offsets are wrong."""
    gen = generator(6)
    for M, N, K in ((20, 300, 4096), (90, 300, 4096)):
        x_q, x_s = mx_operand(gen, False, M, K)
        w_q, w_s = mx_operand(gen, False, 1, N, K)
        for dtype in (torch.bfloat16, torch.float32):
            first = mxq.mx_grouped_gemm(x_q, x_s, w_q, w_s, offsets_of([M]), out_dtype=dtype)
            whole = torch.full((M, N + 7), 9.0, dtype=dtype, device="cuda")
            for at in (0, 3, 4):
                whole.fill_(9)
                mxq.mx_grouped_gemm(x_q, x_s, w_q, w_s, offsets_of([M]), out=whole[:, at:at + N])
                assert (whole[:, at:at + N] == first).all()
                assert (whole[:, :at] == 9).all() and (whole[:, at + N:] == 9).all()
            err = dev_err()
            whole.fill_(9)
            mxq.mx_grouped_gemm(x_q, x_s, w_q, w_s, offsets_of([M + 1]), out=whole[:, :N],
                                dev_err=err)
            assert err.item() == mxq.DEVERR_OFFSETS and (whole == 9).all()


@gpu
def test_grouped_gemm_strided_output_and_stream():
    """An output inside a wider matrix, at an odd element, on another stream;
    nothing outside it changes."""
    gen = generator(5)
    M, N, K, E = 333, 200, 320, 3
    x_q, x_s = mx_operand(gen, True, M, K)
    w_q, w_s = mx_operand(gen, True, E, N, K)
    off = offsets_of([100, 0, 233])
    want = mx_values(x_q, x_s) @ torch.cat((mx_values(w_q, w_s)[0], mx_values(w_q, w_s)[2])).t()
    want = torch.cat((want[:100, :N], want[100:, N:]))
    for dtype in (torch.bfloat16, torch.float32):
        for at, width in ((3, 251), (8, 256), (0, 202)):
            side = torch.cuda.Stream()
            whole = torch.full((M, width), 9.0, dtype=dtype, device="cuda")
            side.wait_stream(torch.cuda.current_stream())
            mxq.mx_grouped_gemm(x_q, x_s, w_q, w_s, off, out=whole[:, at:at + N], stream=side)
            torch.cuda.synchronize()
            check(whole[:, at:at + N], want, None, True)
            assert (whole[:, :at] == 9).all() and (whole[:, at + N:] == 9).all()


@gpu
def test_grouped_gemm_matches_quantizer_and_dgrad():
    """Operands straight from mx_quantize_rowcol, forward and input gradient."""
    gen = generator(6)
    E, N, K, M = 3, 256, 192, 416
    off = offsets_of([96, 160, 160])
    x = torch.randn(M, K, generator=gen, device="cuda").bfloat16()
    w = torch.randn(E, N, K, generator=gen, device="cuda").bfloat16()
    g = torch.randn(M, N, generator=gen, device="cuda").bfloat16()
    q = [mxq.mx_quantize_rowcol(w[e]) for e in range(E)]
    xq, gq = mxq.mx_quantize_rowcol(x, mxq.ROWWISE), mxq.mx_quantize_rowcol(g, mxq.ROWWISE)
    w_row = [torch.stack([d[k] for d in q]) for k in ("q_row", "s_row")]
    w_col = [torch.stack([d[k] for d in q]) for k in ("q_col", "s_col")]
    y = mxq.mx_grouped_gemm(xq["q_row"], xq["s_row"], *w_row, off, out_dtype=torch.float32)
    dx = mxq.mx_grouped_gemm(gq["q_row"], gq["s_row"], *w_col, off, out_dtype=torch.float32)
    xv, gv = mx_values(xq["q_row"], xq["s_row"]), mx_values(gq["q_row"], gq["s_row"])
    for e in range(E):
        a, b = int(off[e]), int(off[e + 1])
        for got, rows, wv in ((y, xv, mx_values(w_row[0][e], w_row[1][e])),
                              (dx, gv, mx_values(w_col[0][e], w_col[1][e]))):
            check(got[a:b], rows[a:b] @ wv.t(),
                  wv.shape[1] * 2.0 ** -23 * (rows[a:b].abs() @ wv.abs().t()), False)


@gpu
def test_grouped_gemm_scale_extremes():
    """Scale codes 0 and 254 (2^-127 and 2^127) and the largest codes."""
    x_q = torch.full((2, 64), 0x7E, dtype=torch.uint8, device="cuda")      # 448
    w_q = torch.full((1, 16, 64), 0x7E, dtype=torch.uint8, device="cuda")
    x_s = torch.tensor([[254, 254], [0, 0]], dtype=torch.uint8, device="cuda")
    w_s = torch.tensor([[[0, 0]]], dtype=torch.uint8, device="cuda").repeat(1, 16, 1)
    w_s[0, 8:] = 254
    y = mxq.mx_grouped_gemm(x_q, x_s, w_q, w_s, offsets_of([2]), out_dtype=torch.float32)
    want = torch.tensor([[64 * 448.0 ** 2, float("inf")], [0, 64 * 448.0 ** 2]]).cuda()
    assert torch.equal(y[0, ::8], want[0]) and y[1, 8] == want[1, 1] and y[1, 0] == 0


@gpu
@pytest.mark.parametrize("sizes,N,K", [([40, 3, 200], 300, 416), ([9, 2, 0, 5], 200, 96)],
                         ids=["forward", "few"])
def test_grouped_gemm_keeps_nan_where_it_is(sizes, N, K):
    """A NaN code in a row of x reaches that row alone, a NaN scale (255) of a
    weight row that column of its expert alone, and neither other groups'
    rows in the same tile."""
    gen = generator(15)
    M, E = sum(sizes), len(sizes)
    x_q, x_s = mx_operand(gen, True, M, K)
    w_q, w_s = mx_operand(gen, True, E, N, K)
    off = offsets_of(sizes)
    row, e, col = sizes[0], 0, N - 1            # the second group's first row
    x_q[row, K - 1] = 0x7F
    w_s[e, col, 0] = 255
    y = mxq.mx_grouped_gemm(x_q, x_s, w_q, w_s, off, out_dtype=torch.float32)
    bad = torch.zeros(M, N, dtype=torch.bool, device="cuda")
    bad[row], bad[:sizes[0], col] = True, True
    assert torch.equal(y.isnan(), bad)


@gpu
@pytest.mark.slow
def test_products_past_2_31_elements():
    """Outputs and operands whose element numbers pass 32 bits: the last rows,
    experts and columns against the definition."""
    gen = generator(16)
    M, N, K, E = 70016, 32768, 32, 3
    x_q, x_s = mx_operand(gen, True, M, K)
    w_q, w_s = mx_operand(gen, True, E, N, K)
    off = offsets_of([100, 34900, M - 35000])
    y = mxq.mx_grouped_gemm(x_q, x_s, w_q, w_s, off)
    for rows, e in ((slice(0, 70), 0), (slice(34990, 35000), 1), (slice(M - 130, M), 2)):
        want = mx_values(x_q[rows], x_s[rows]) @ mx_values(w_q[e], w_s[e]).t()
        check(y[rows], want, None, True)
    del y
    E, N, K, M = 40, 8192, 8192, 1280
    g_q, g_s = mx_operand(gen, True, N, M)
    x_q, x_s = mx_operand(gen, True, K, M)
    off = offsets_of([32] * E)
    dw = mxq.mx_grouped_wgrad(g_q, g_s, x_q, x_s, off, out_dtype=torch.bfloat16)
    for e in (0, 31, E - 1):
        a = slice(32 * e, 32 * e + 32)
        want = mx_values(g_q[-300:, a], g_s[-300:, e:e + 1]) @ mx_values(x_q[:, a], x_s[:, e:e + 1]).t()
        check(dw[e, -300:], want, None, True)
    del dw
    E, N, K = 72, 16384, 8192
    q = torch.randint(0, 256, (E, N, K // 2), generator=gen, device="cuda", dtype=torch.uint8)
    s = pick(gen, [0x30, 0x38, 0x40], E, N, K // 16)
    g = torch.ones(E, device="cuda")
    x = nv_rows(gen, True, 2, K)
    ids = torch.tensor([E - 1, 0], dtype=torch.int32, device="cuda")
    y = mxq.nvfp4_gemv(x, q, s, g, experts=ids, out_dtype=torch.float32)
    for r, e in enumerate(ids.tolist()):
        check(y[r, -500:], nv_values(q[e, -500:], s[e, -500:]) @ x[r].double(), None, True)


# ---------------------------------------------------------------------------
# mx_grouped_wgrad
# ---------------------------------------------------------------------------

WGRAD = [
    # name, group sizes, N, K, rows before the first group, rows after the last
    ("one_block", [32], 8, 8, 0, 0),
    ("one_tile", [128], 128, 128, 0, 0),
    ("empty", [0, 0], 24, 40, 0, 0),
    ("empty_groups", [0, 64, 0, 32, 0], 130, 70, 0, 0),
    ("odd_widths", [96, 160, 32, 512], 257, 301, 0, 0),
    ("outside_rows", [64, 96], 64, 96, 32, 160),
    ("long", [4096, 32, 2080], 136, 264, 0, 0),
    ("ranges", [96, 20000, 8192, 32], 264, 136, 0, 0),
    ("scale_alignment", [32 * i for i in (1, 2, 3, 5, 7, 11, 13, 4)], 96, 160, 0, 32),
    ("many_tiles", [256, 320], 1500, 1100, 0, 0),
    ("wide_pairs", [224, 0, 800], 2048, 2304, 0, 0),
    ("many_groups", [32 * (i % 3) for i in range(200)], 40, 136, 0, 0),
]


@gpu
@pytest.mark.parametrize("exact", [True, False], ids=["exact", "random"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("name,sizes,N,K,before,after", WGRAD, ids=[c[0] for c in WGRAD])
def test_grouped_wgrad(name, sizes, N, K, before, after, dtype, exact):
    gen = generator(len(name) + N + K)
    M = before + sum(sizes) + after
    g_q, g_s = mx_operand(gen, exact, N, M)
    x_q, x_s = mx_operand(gen, exact, K, M)
    off = offsets_of(sizes, before)
    err = dev_err()
    dw = mxq.mx_grouped_wgrad(g_q, g_s, x_q, x_s, off, out_dtype=dtype, dev_err=err)
    torch.cuda.synchronize()
    assert err.item() == 0
    g, x = mx_values(g_q, g_s), mx_values(x_q, x_s)
    for e, rows in enumerate(sizes):
        a, b = int(off[e]), int(off[e + 1])
        check(dw[e], g[:, a:b] @ x[:, a:b].t(),
              rows * 2.0 ** -23 * (g[:, a:b].abs() @ x[:, a:b].abs().t()), exact, f"{name} {e}")


# Few tiles of long groups: CTAs of a cluster share their rows.
WGRAD_SPLIT = [
    ("one_tile", [4096], 100, 128, 0, 0),
    ("odd_start", [2048 + 32, 3200, 64], 129, 65, 32, 96),
    ("one_long", [0, 8000, 32, 0], 64, 200, 64, 0),
    ("halves", [5120], 640, 520, 0, 0),
    ("last_range_empty", [128 * 65], 72, 80, 0, 0),
    ("all_empty", [0, 0], 40, 40, 4096, 4096),
]


@gpu
@pytest.mark.parametrize("exact", [True, False], ids=["exact", "random"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("name,sizes,N,K,before,after", WGRAD_SPLIT, ids=[c[0] for c in WGRAD_SPLIT])
def test_grouped_wgrad_shared_contraction(name, sizes, N, K, before, after, dtype, exact):
    test_grouped_wgrad(name, sizes, N, K, before, after, dtype, exact)


@gpu
def test_grouped_wgrad_keeps_nan_where_it_is():
    """NaN codes and scales in the 32 rows after a group's end, which share a
    128-row stage with it, stay out of its gradient."""
    gen = generator(17)
    sizes, N, K = [96, 32, 160], 136, 80
    M, off = sum(sizes), offsets_of(sizes)
    g_q, g_s = mx_operand(gen, True, N, M)
    x_q, x_s = mx_operand(gen, True, K, M)
    g_q[:, 96:128] = 0x7F
    x_s[:, 3] = 255
    dw = mxq.mx_grouped_wgrad(g_q, g_s, x_q, x_s, off)
    assert dw[1].isnan().all()
    g, x = mx_values(g_q, g_s), mx_values(x_q, x_s)
    for e, (a, b) in ((0, (0, 96)), (2, (128, 288))):
        check(dw[e], g[:, a:b] @ x[:, a:b].t(), None, True)


@gpu
def test_gradients_against_differences():
    """dX and dW of L = sum(C * Y) from the products themselves against
    central differences of L.  L is linear in X and in W, so a difference of
    any step is exact but for rounding; operands are small whole numbers, so
    there is none, and the products' values equal the differences."""
    gen = generator(8)
    E, N, K, sizes = 2, 64, 96, [64, 32]
    M, off = sum(sizes), offsets_of(sizes)
    one = lambda *s: torch.full(s, 127, dtype=torch.uint8, device="cuda")  # noqa: E731
    x = pick(gen, E4M3_SMALL, M, K)
    w = pick(gen, E4M3_SMALL, E, N, K)
    c = pick(gen, E4M3_SMALL, M, N)

    def loss(x, w):
        y = mxq.mx_grouped_gemm(x, one(M, K // 32), w, one(E, N, K // 32), off,
                                out_dtype=torch.float32)
        return (y.double() * e4m3_values(c)).sum()

    dx = mxq.mx_grouped_gemm(c, one(M, N // 32), w.transpose(1, 2).contiguous(),
                             one(E, K, N // 32), off, out_dtype=torch.float32)
    dw = mxq.mx_grouped_wgrad(c.t().contiguous(), one(N, M // 32), x.t().contiguous(),
                              one(K, M // 32), off)
    up, down = 0x38, 0xB8                                       # +1, -1
    for i in range(12):
        m, k, e, n = (i * 29) % M, (i * 41) % K, i % E, (i * 13) % N
        for t, grad, at in ((x, dx, (m, k)), (w, dw, (e, n, k))):
            hi, lo = t.clone(), t.clone()
            hi[at], lo[at] = up, down
            a, b = ((hi, w), (lo, w)) if t is x else ((x, hi), (x, lo))
            assert (loss(*a) - loss(*b)).item() / 2 == grad[at].item()


@gpu
def test_bad_offsets_write_nothing():
    gen = generator(9)
    q, s = mx_operand(gen, True, 64, 64)
    w, ws = mx_operand(gen, True, 2, 64, 64)
    for bad in ([0, 40, 30], [0, 32, 65], [-1, 32, 64], [0, 2 ** 31 - 1, 64]):
        off = torch.tensor(bad, dtype=torch.int32, device="cuda")
        err, out = dev_err(), torch.full((64, 64), 5.0, dtype=torch.bfloat16, device="cuda")
        mxq.mx_grouped_gemm(q, s, w, ws, off, out=out, dev_err=err)
        dw = torch.full((2, 64, 64), 5.0, device="cuda")
        err2 = dev_err()
        mxq.mx_grouped_wgrad(q, s, q, s, off, out=dw, dev_err=err2)
        torch.cuda.synchronize()
        assert err.item() == mxq.DEVERR_OFFSETS and err2.item() == mxq.DEVERR_OFFSETS
        assert (out == 5).all() and (dw == 5).all()
    err, dw = dev_err(), torch.full((2, 64, 64), 5.0, device="cuda")
    mxq.mx_grouped_wgrad(q, s, q, s, torch.tensor([0, 16, 64], dtype=torch.int32, device="cuda"),
                         out=dw, dev_err=err)
    torch.cuda.synchronize()
    assert err.item() == mxq.DEVERR_OFFSETS and (dw == 5).all()


@gpu
def test_empty_grouped_calls():
    gen = generator(10)
    q, s = mx_operand(gen, True, 32, 64)
    w, ws = mx_operand(gen, True, 2, 0, 64)
    assert mxq.mx_grouped_gemm(q, s, w, ws, offsets_of([16, 16])).shape == (32, 0)
    e, es = mx_operand(gen, True, 0, 64)
    w, ws = mx_operand(gen, True, 2, 8, 64)
    assert mxq.mx_grouped_gemm(e, es, w, ws, offsets_of([0, 0])).shape == (0, 8)
    z = torch.zeros(32, 0, dtype=torch.uint8, device="cuda")
    zw = torch.zeros(2, 8, 0, dtype=torch.uint8, device="cuda")
    assert (mxq.mx_grouped_gemm(z, z, zw, zw, offsets_of([16, 16])) == 0).all()
    z = torch.zeros(16, 0, dtype=torch.uint8, device="cuda")
    assert (mxq.mx_grouped_wgrad(z, z, z, z, offsets_of([0, 0])) == 0).all()


# ---------------------------------------------------------------------------
# nvfp4_gemv
# ---------------------------------------------------------------------------

def nv_operand(gen, exact, E, N, K):
    shape = (E, N, K // 2)
    if exact:
        q = pick(gen, E2M1_SMALL, *shape) | pick(gen, E2M1_SMALL, *shape) << 4
        s = pick(gen, [0x30, 0x38, 0x40], E, N, K // 16)
        g = torch.tensor([0.5, 1, 2, 4], device="cuda")[torch.arange(E, device="cuda") % 4]
        return q, s, g
    q = torch.randint(0, 256, shape, generator=gen, device="cuda", dtype=torch.uint8)
    s = torch.randint(0, 0x7F, (E, N, K // 16), generator=gen, device="cuda", dtype=torch.uint8)
    return q, s, torch.rand(E, generator=gen, device="cuda") + 0.1


def nv_rows(gen, exact, T, K, spread=False):
    if exact:
        return torch.randint(-2, 3, (T, K), generator=gen, device="cuda").bfloat16()
    x = torch.randn(T, K, generator=gen, device="cuda")
    if spread:      # magnitudes from 2^-40 to 2^40, in runs and singly
        x *= torch.pow(2.0, torch.randint(-40, 41, (T, K), generator=gen, device="cuda").float())
    return x.bfloat16()


GEMV = [
    # T, N, K
    (1, 1, 32), (1, 2048, 2048), (2, 17, 96), (3, 1003, 4128), (4, 128, 16384 + 32),
    (5, 300, 1024), (8, 515, 544), (9, 64, 2080), (13, 259, 11008), (16, 1000, 512),
    (17, 40, 320), (33, 48, 608), (40, 129, 64),
]


def gemv_reference(x, q, s, g, ids, share):
    """Values and bounds in 64 bits: the products of bf16 and E2M1 times E4M3
    have at most 14 bits, sums of K of them carry n units in the last place,
    and the products with the block and tensor scales one each."""
    w = nv_values(q, s)
    T, K = x.shape
    rows = x.double().repeat_interleave(share, 0)
    want = torch.zeros(T * share, w.shape[-2], dtype=torch.float64, device="cuda")
    bound = torch.zeros_like(want)
    for r, e in enumerate([0] * T if ids is None else ids.tolist()):
        if 0 <= e < len(w):
            want[r] = w[e] @ rows[r] * g[e].double()
            bound[r] = (K + 4) * 2.0 ** -23 * (w[e].abs() @ rows[r].abs()) * g[e].double()
    return want, bound


@gpu
@pytest.mark.parametrize("kind", ["exact", "random", "spread"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("T,N,K", GEMV)
def test_gemv(T, N, K, dtype, kind):
    gen = generator(T + N + K)
    x = nv_rows(gen, kind == "exact", T, K, kind == "spread")
    q, s, g = nv_operand(gen, kind == "exact", 1, N, K)
    y = mxq.nvfp4_gemv(x, q[0], s[0], g, out_dtype=dtype)
    want, bound = gemv_reference(x, q, s, g, None, 1)
    check(y, want, bound, kind == "exact")


ROUTED = [
    # E, T, share, N, K
    (4, 1, 1, 64, 64), (8, 3, 2, 1000, 544), (64, 8, 4, 256, 2048), (3, 30, 3, 70, 96),
    (1, 5, 1, 33, 320), (128, 16, 8, 40, 512), (2, 700, 2, 24, 32),
]


@gpu
@pytest.mark.parametrize("exact", [True, False], ids=["exact", "random"])
@pytest.mark.parametrize("E,T,share,N,K", ROUTED)
def test_gemv_experts(E, T, share, N, K, exact):
    gen = generator(E + T + N + K)
    x = nv_rows(gen, exact, T, K)
    q, s, g = nv_operand(gen, exact, E, N, K)
    ids = torch.randint(-1, E + 1, (T * share,), generator=gen, device="cuda").int()
    for some in (ids, torch.full_like(ids, -1), torch.full_like(ids, E - 1)):
        y = mxq.nvfp4_gemv(x, q, s, g, experts=some, share=share, out_dtype=torch.float32)
        want, bound = gemv_reference(x, q, s, g, some, share)
        check(y, want, bound, exact)


@gpu
def test_gemv_strides_and_quantizer():
    """Rows inside a wider matrix, an output at an odd element, operands
    straight from nvfp4_quantize_transpose, on another stream."""
    gen = generator(12)
    T, N, K = 6, 96, 256
    wide = torch.randn(T, 2 * K, generator=gen, device="cuda").bfloat16()
    x = wide[:, 8:8 + K]
    w = torch.randn(N, K, generator=gen, device="cuda").bfloat16()
    nv = mxq.nvfp4_quantize_transpose(w, mxq.ROWWISE)
    out = torch.full((T, N + 9), 3.0, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    mxq.nvfp4_gemv(x, nv["q_row"], nv["s_row"], nv["global_scale"], out=out[:, 5:5 + N], stream=side)
    torch.cuda.synchronize()
    want, bound = gemv_reference(x, nv["q_row"][None], nv["s_row"][None], nv["global_scale"], None, 1)
    check(out[:, 5:5 + N], want, bound, False)
    assert (out[:, :5] == 3).all() and (out[:, 5 + N:] == 3).all()


@gpu
def test_gemv_infinities_and_nan():
    """An infinity in a row of x gives what 64 bits give, and a NaN scale its
    column alone; neither reaches other rows."""
    gen = generator(18)
    T, N, K = 4, 40, 320
    q, s, g = nv_operand(gen, True, 1, N, K)
    x = nv_rows(gen, True, T, K)
    s[0, 7, 3] = 0x7F
    x[1, 100], x[2, 5] = float("inf"), float("nan")
    y = mxq.nvfp4_gemv(x, q[0], s[0], g, out_dtype=torch.float32).double()
    want = (x.double().unsqueeze(1) * nv_values(q, s)).sum(-1) * g.double()
    assert torch.equal(y.isnan(), want.isnan())
    here = ~want.isnan()
    assert torch.equal(y[here], want[here])


@gpu
def test_gemv_edges():
    gen = generator(13)
    q, s, g = nv_operand(gen, True, 2, 24, 64)
    x = nv_rows(gen, True, 2, 64)
    assert mxq.nvfp4_gemv(x[:0], q[0], s[0], g[:1]).shape == (0, 24)
    assert mxq.nvfp4_gemv(x, q[0, :0], s[0, :0], g[:1]).shape == (2, 0)
    none = torch.zeros(2, dtype=torch.int32, device="cuda")
    assert (mxq.nvfp4_gemv(x, q[:0], s[:0], g[:0], experts=none) == 0).all()
    assert (mxq.nvfp4_gemv(x[:, :0], q[0, :, :0], s[0, :, :0], g[:1]) == 0).all()
    assert (mxq.nvfp4_gemv(torch.zeros_like(x), q[0], s[0], g[:1]) == 0).all()
    # The largest finite bf16 beside the smallest, in rows of their own and in one.
    x = torch.zeros(3, 64, device="cuda").bfloat16()
    x[0, 3], x[1, 40] = 3e38, 1e-38
    x[2, 0], x[2, 63] = 2.0 ** 100, 2.0 ** -100
    q, s, g = nv_operand(gen, True, 1, 24, 64)
    y = mxq.nvfp4_gemv(x, q[0], s[0], torch.tensor([2.0 ** -10], device="cuda"), out_dtype=torch.float32)
    want, bound = gemv_reference(x, q, s, torch.tensor([2.0 ** -10], device="cuda"), None, 1)
    assert (((y.double() - want).abs() <= bound) | (want.abs() < 2.0 ** -120)).all()


# ---------------------------------------------------------------------------
# Refusals, on the host
# ---------------------------------------------------------------------------

P = ctypes.c_void_p(256)


def test_grouped_refusals():
    L = _lib.lib()

    def gemm(M=64, N=64, K=64, E=2, flags=0, ldo=64):
        return L.mx_grouped_gemm(P, P, P, P, P, M, N, K, E, flags, P, ldo, None, None)

    def wgrad(M=64, N=64, K=64, E=2, flags=0):
        return L.mx_grouped_wgrad(P, P, P, P, P, M, N, K, E, flags, P, None, None)

    assert gemm(flags=1) == 1 and wgrad(flags=512) == 1
    for bad in (dict(M=-1), dict(N=-1), dict(K=-32), dict(K=40), dict(E=-1), dict(E=513),
                dict(M=2 ** 31), dict(ldo=63)):
        assert gemm(**bad) == 2, bad
    for bad in (dict(M=-32), dict(M=48), dict(N=-1), dict(K=-1), dict(E=513), dict(K=2 ** 31)):
        assert wgrad(**bad) == 2, bad


def test_gemv_refusals():
    L = _lib.lib()

    def gemv(ldx=64, T=1, share=1, N=64, K=64, E=1, flags=0, ldo=64, experts=P):
        return L.nvfp4_gemv(P, ldx, P, P, P, experts, T, share, N, K, E, flags, P, ldo, None, None)

    assert gemv(flags=16) == 1
    for bad in (dict(T=-1), dict(share=0), dict(N=-1), dict(K=40), dict(ldx=32), dict(ldo=63),
                dict(E=-1), dict(experts=None, E=2), dict(experts=None, share=2),
                dict(T=2 ** 20, share=2 ** 20)):
        assert gemv(**bad) == 2, bad


@gpu
def test_device_refusals():
    """What the host can only check with a device present: null and
    misaligned pointers, and the binding's own checks."""
    L = _lib.lib()
    b = torch.zeros(1 << 16, dtype=torch.uint8, device="cuda").data_ptr()
    assert L.mx_grouped_gemm(None, b, b, b, b, 64, 64, 64, 2, 0, b, 64, None, None) == 1
    assert L.mx_grouped_gemm(b, b, b, b, None, 64, 64, 64, 2, 0, b, 64, None, None) == 1
    assert L.mx_grouped_gemm(b + 8, b, b, b, b, 64, 64, 64, 2, 0, b, 64, None, None) == 3
    assert L.mx_grouped_gemm(b, b, b, b, b, 64, 64, 64, 2, 0, b + 1, 64, None, None) == 3
    assert L.mx_grouped_wgrad(b, b, b, b, b, 64, 64, 64, 2, 0, None, None, None) == 1
    assert L.mx_grouped_wgrad(b, b, b, b + 4, b, 64, 64, 64, 2, 0, b, None, None) == 3
    assert L.nvfp4_gemv(None, 64, b, b, b, None, 1, 1, 64, 64, 1, 0, b, 64, None, None) == 1
    assert L.nvfp4_gemv(b, 60, b, b, b, None, 1, 1, 64, 32, 1, 0, b, 64, None, None) == 3
    gen = generator(14)
    q, s = mx_operand(gen, True, 32, 64)
    w, ws = mx_operand(gen, True, 2, 32, 64)
    off = offsets_of([16, 16])
    for args, error in (((q, s, w, ws, off.long()), TypeError), ((q, s, w, ws, off[:2]), ValueError),
                        ((q, s[:, :1], w, ws, off), ValueError), ((q.float(), s, w, ws, off), TypeError),
                        ((q.cpu(), s, w, ws, off), TypeError),
                        ((q, s, w.transpose(1, 2), ws, off), ValueError)):
        with pytest.raises(error):
            mxq.mx_grouped_gemm(*args)
    with pytest.raises(TypeError):
        mxq.mx_grouped_gemm(q, s, w, ws, off, out_dtype=torch.float16)
    with pytest.raises(ValueError):
        mxq.mx_grouped_gemm(q, s, w, ws, off, out=torch.empty(32, 31, device="cuda"))
    x = torch.zeros(2, 64, device="cuda").bfloat16()
    nq, ns, ng = nv_operand(gen, True, 2, 8, 64)
    ids = torch.zeros(2, dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError):
        mxq.nvfp4_gemv(x, nq, ns, ng[:1], experts=ids)
    with pytest.raises(ValueError):
        mxq.nvfp4_gemv(x, nq, ns, ng, experts=ids, share=2)
    with pytest.raises(TypeError):
        mxq.nvfp4_gemv(x.float(), nq, ns, ng, experts=ids)
