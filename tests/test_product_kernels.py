"""Every kernel of the products, and every way through one, against the
definition in 64 bits.

A call's sizes choose its kernel, so a change of that rule can leave a kernel
without a test.  Each case here therefore names the cut that it is there for,
the calls check it on the device they run on, and a test without a device checks
that the cases reach every kernel there is.  Inputs, definitions and bounds are
those of test_products.py.
"""
import pytest
import torch

import fp4_quantization_gb300 as mxq
import test_products as products
from test_products import (GEMM, GEMM_SPLIT, GEMV, ROUTED, WGRAD, WGRAD_SPLIT, check, dev_err, generator,
                           gemv_reference, mx_operand, mx_values, nv_operand, nv_rows, offsets_of)

gpu = pytest.mark.gpu
SMS = 152                # of a GB300
SEGMENT = 8192           # terms of an fp32 sum in one range, at most

PAIR, WIDE, NARROW, FEW = (2, 256, 0, 1), (1, 256, 0, 1), (1, 128, 0, 1), (1, 32, 1, 1)


def cut(op, M, N, K, E, flags=0, num_sms=SMS):
    p = mxq.mxq_product_plan(op, M, N, K, E, flags, num_sms=num_sms)
    return tuple(p[f] for f in ("ctas", "cols", "few", "split"))


def gemm_cut(sizes, N, K, before, after, flags=0, num_sms=SMS):
    return cut(mxq.OP_GROUPED_GEMM, before + sum(sizes) + after, N, K, len(sizes), flags, num_sms)


def wgrad_cut(sizes, N, K, before, after, flags=0, num_sms=SMS):
    return cut(mxq.OP_GROUPED_WGRAD, before + sum(sizes) + after, N, K, len(sizes), flags, num_sms)


def sms_here():
    return torch.cuda.get_device_properties(0).multi_processor_count


# Scale rows are whole 16-byte blocks where K (wgrad: M) is a multiple of 512, output
# rows 16-byte aligned where N (wgrad: K) is a multiple of 8.  "ranges": fp32 sums of
# more than SEGMENT terms, in two or three ranges.
GEMM_KERNELS = [
    # name, cut, group sizes, N, K, rows before the first group, rows after the last
    ("pair", PAIR, [600, 1, 0, 2339, 260], 2304, 2560, 0, 0),
    ("pair_odd", PAIR, [600, 1, 0, 2335, 256], 2303, 2528, 3, 5),
    ("pair_odd_columns", PAIR, [300, 1, 0, 1900, 239], 1501, 2560, 0, 60),
    ("pair_ranges", PAIR, [600, 256, 1100], 2304, 8192 + 96, 0, 0),
    ("pair_ranges_odd", PAIR, [5, 1395, 0, 601], 1501, 2 * 8192 + 32, 7, 0),
    ("pair_ranges_whole", PAIR, [1200, 800], 1600, 8192 + 512, 0, 0),
    ("wide", WIDE, [700, 3, 890], 1504, 1024, 0, 0),
    ("wide_odd", WIDE, [700, 3, 890], 1503, 1056, 2, 6),
    ("wide_ranges", WIDE, [500, 128, 672], 3000, 8192 + 96, 0, 0),
    ("wide_ranges_odd", WIDE, [500, 129, 671], 3001, 8192 + 512, 0, 0),
    ("narrow_ranges", NARROW, [130, 40, 130], 1904, 8192 + 96, 0, 0),
    ("narrow_ranges_odd", NARROW, [130, 1, 169], 1901, 2 * 8192 + 512, 0, 0),
    ("few_odd", FEW, [20, 0, 31, 1, 40], 301, 512, 0, 1),
    ("few_ranges", FEW, [1, 0, 3, 0, 2, 0, 2, 1], 1280, 2 * 8192 + 96, 2, 3),
    ("few_ranges_whole", FEW, [40, 0, 1, 5, 9, 0, 30, 1], 1285, 8192 + 512, 0, 0),
]

WGRAD_KERNELS = [
    ("pair", PAIR, [2720, 96, 5376], 2048, 2304, 0, 0),
    ("pair_odd", PAIR, [2720, 96, 5344], 2047, 2301, 32, 64),
    ("pair_ranges", PAIR, [8640], 1500, 1904, 32, 32),
    ("pair_ranges_odd", PAIR, [16416], 1501, 1899, 96, 0),
    ("wide", WIDE, [992, 32, 1024], 900, 1104, 0, 0),
    ("wide_odd", WIDE, [992, 0, 1088], 899, 1101, 0, 0),
    ("wide_ranges", WIDE, [8640], 1100, 4096, 32, 32),
    ("wide_ranges_odd", WIDE, [8288], 1099, 4095, 32, 0),
    ("narrow_ranges", NARROW, [8640], 1104, 1104, 32, 32),
    ("narrow_ranges_odd", NARROW, [8288], 1101, 1099, 32, 0),
    ("split_odd", (1, 128, 0, 4), [6144, 0, 2080, 64], 130, 65, 32, 2048),
    ("split_odd_whole", (1, 128, 0, 4), [6144, 2016], 129, 131, 32, 0),
    ("narrow_ranges_groups", NARROW, [96, 8448, 0, 32] + [64] * 60, 300, 196, 32, 0),
]

# Kernel by rows (8 or 16), whether a CTA takes items after its first, whether K is
# staged in chunks, then T, N, K.
GEMV_KERNELS = [
    ("one_items_chunks", 8, True, True, 1, 12000, 14336 + 544),
    ("one_items", 8, True, False, 1, 40000, 1056),
    ("two_chunks", 8, True, True, 2, 12001, 8192),
    ("five_chunks", 8, True, True, 5, 40000, 6144),
    ("eight_items_chunks", 8, True, True, 8, 40000, 2048),
    ("nine_items", 16, True, False, 9, 40007, 1312),
    ("thirteen_chunks", 16, False, True, 13, 17109, 4096),
    ("sixteen_items_chunks", 16, True, True, 16, 40000, 1600),
    ("passes_items_chunks", 16, True, True, 35, 40000, 1600),
]

# The same with E, T, share, N, K and how the ids are drawn: evenly, or half of the
# rows to one expert.
ROUTED_KERNELS = [
    ("items_chunks", 8, True, True, 8, 16, 2, 7000, 4096, "even"),
    ("items_chunks_skewed", 8, True, True, 8, 16, 2, 7000, 4096, "skewed"),
    ("cluster_chunks", 8, True, True, 8, 16, 2, 6000, 8192, "even"),
    ("cluster_chunks_skewed", 8, True, True, 8, 16, 2, 6000, 8192, "skewed"),
    ("uneven_chunks", 8, True, True, 64, 16, 8, 600, 7168, "even"),
    ("uneven_chunks_skewed", 8, True, True, 64, 16, 8, 600, 7168, "skewed"),
    ("long_chunks_skewed", 8, True, True, 64, 9, 7, 640, 14336, "skewed"),
    ("items", 8, True, False, 40, 12, 4, 1500, 512, "even"),
    ("items_skewed", 8, True, False, 40, 12, 4, 1500, 512, "skewed"),
    ("sixteen_items", 16, True, False, 3, 20, 2, 13100, 1600, "even"),
    ("sixteen_items_skewed", 16, True, False, 3, 40, 2, 13100, 1600, "skewed"),
    ("sixteen_items_chunks", 16, True, True, 3, 20, 2, 13100, 2400, "even"),
    ("sixteen_chunks_skewed", 16, True, True, 12, 45, 3, 3500, 2400, "skewed"),
    ("experts_1500", 8, True, False, 1500, 100, 4, 130, 64, "even"),
    ("experts_4096", 8, True, False, 4096, 300, 8, 24, 96, "even"),
    ("experts_4096_skewed", 8, True, False, 4096, 64, 8, 24, 96, "skewed"),
]


def room(p):
    """Values of K that a kernel stages at a time, as it computes them."""
    return (44 if p["toks"] == 16 else 28) * 1024 // (2 * p["cap"]) // 256 * 256


def gemv_kernel(rows, N, K, E, num_sms=SMS):
    p = mxq.mxq_product_plan(mxq.OP_NVFP4_GEMV, rows, N, K, E, num_sms=num_sms)
    span = -(-(-(-K // 256)) // p["cluster"]) * 256
    return p["toks"], p["items"] * p["cluster"] > p["grid"], span > room(p)


def test_the_cases_reach_every_kernel():
    """Cuts of the grouped products by kind, with ranges of long fp32 sums and
    without, scale rows aligned or not, output rows aligned or not."""
    kernels, ways = set(), set()
    for kind, find, cases in (
            ("gemm", gemm_cut, [c[1:] for c in GEMM + GEMM_SPLIT] + [c[2:] for c in GEMM_KERNELS]),
            ("wgrad", wgrad_cut, [c[1:] for c in WGRAD + WGRAD_SPLIT] + [c[2:] for c in WGRAD_KERNELS])):
        for sizes, N, K, before, after in cases:
            M = before + sum(sizes) + after
            depth, along, width = (K, K, N) if kind == "gemm" else (max(sizes), M, K)
            for flags in (0, mxq.OUT_F32):
                ctas, cols, few, split = find(sizes, N, K, before, after, flags)
                at = (kind, ctas, cols, few, split > 1)
                kernels.add(at)
                ways.add((at, "scales", along % 512 == 0))
                ways.add((at, "rows", width % (4 if flags else 8) == 0))
                if flags and split == 1:
                    ways.add((at, "ranges", depth > SEGMENT, width % 4 == 0))
    whole = {("gemm", *c[:3]) for c in (PAIR, WIDE, NARROW, FEW)} | {
        ("wgrad", *c[:3]) for c in (PAIR, WIDE, NARROW)}
    split = {("gemm", *NARROW[:3]), ("gemm", *FEW[:3]), ("wgrad", *NARROW[:3])}
    want = {(*k, False) for k in whole} | {(*k, True) for k in split}
    assert kernels == want
    for at in want:
        assert {w[2] for w in ways if w[:2] == (at, "scales")} == {True, False}, at
        assert {w[2] for w in ways if w[:2] == (at, "rows")} == {True, False}, at
        if not at[4]:
            assert {w[2:] for w in ways if w[:2] == (at, "ranges")} >= {
                (False, True), (False, False), (True, True), (True, False)}, at


def test_the_gemv_cases_reach_every_way():
    for name, toks, items, chunks, T, N, K in GEMV_KERNELS:
        assert gemv_kernel(T, N, K, 0) == (toks, items, chunks), name
    for name, toks, items, chunks, E, T, share, N, K, _ in ROUTED_KERNELS:
        assert gemv_kernel(T * share, N, K, E) == (toks, items, chunks), name
    plans = [mxq.mxq_product_plan(mxq.OP_NVFP4_GEMV, r, N, K, E, num_sms=SMS) for r, N, K, E in
             [(c[0], c[1], c[2], 0) for c in GEMV] + [(c[4], c[5], c[6], 0) for c in GEMV_KERNELS]
             + [(c[1] * c[2], c[3], c[4], c[0]) for c in ROUTED]
             + [(c[5] * c[6], c[7], c[8], c[4]) for c in ROUTED_KERNELS]]
    assert {(p["toks"], p["uneven"]) for p in plans} == {(t, u) for t in (8, 16) for u in (0, 1)}
    assert {(p["toks"], p["cluster"]) for p in plans} >= {(t, c) for t in (8, 16) for c in (1, 2, 8)}
    assert {p["tiles"] for p in plans} == {1, 2, 4, 8}


@pytest.mark.parametrize("E,T,share,N,K", [(64, 16, 8, 4096, 7168), (64, 8, 8, 4096, 14336),
                                           (8, 16, 2, 6000, 6144), (64, 8, 4, 2816, 2048),
                                           (128, 16, 1, 2048, 28672)])
def test_routed_rows_share_a_pass(E, T, share, N, K):
    """Each pass over an expert's rows reads its weights, so that a pass takes three
    quarters at least of the rows that the kernel multiplies, however long K is."""
    p = mxq.mxq_product_plan(mxq.OP_NVFP4_GEMV, T * share, N, K, E, num_sms=SMS)
    assert 4 * p["cap"] >= 3 * p["toks"]


def test_plan_refusals():
    for op, M, N, K, E in ((mxq.OP_GROUPED_GEMM, 0, 8, 32, 1), (mxq.OP_GROUPED_GEMM, 8, 8, 40, 1),
                           (mxq.OP_GROUPED_GEMM, 8, 8, 32, 0), (mxq.OP_GROUPED_GEMM, 8, 8, 32, 513),
                           (mxq.OP_GROUPED_WGRAD, 48, 8, 32, 1), (mxq.OP_GROUPED_WGRAD, 64, 8, 0, 1),
                           (mxq.OP_NVFP4_GEMV, 1, 0, 32, 0), (mxq.OP_NVFP4_GEMV, 1, 8, 32, 4097),
                           (mxq.OP_NVFP4_GEMV, 2 ** 31, 8, 32, 0)):
        with pytest.raises(mxq.MxqError) as e:
            mxq.mxq_product_plan(op, M, N, K, E, num_sms=SMS)
        assert e.value.status == 2
    for op, flags, sms in ((mxq.OP_ROWCOL, 0, SMS), (mxq.OP_GROUPED_GEMM, 1, SMS), (mxq.OP_NVFP4_GEMV, 0, 0)):
        with pytest.raises(mxq.MxqError) as e:
            mxq.mxq_product_plan(op, 64, 64, 64, 1, flags, num_sms=sms)
        assert e.value.status == 1


class OnDevice(torch.Tensor):
    """A host tensor that says it lies on a CUDA device (index `at`)."""

    is_cuda = property(lambda self: self.at >= 0)

    def get_device(self):
        return self.at


def on(at, *shape, dtype=torch.uint8):
    t = torch.zeros(*shape, dtype=dtype).as_subclass(OnDevice)
    t.at = at
    return t


def product_calls():
    """Each product's operands by name, with a call of them."""
    gemm = dict(x_q=on(0, 64, 64), x_s=on(0, 64, 2), w_q=on(0, 2, 32, 64), w_s=on(0, 2, 32, 2),
                offsets=on(0, 3, dtype=torch.int32), out=on(0, 64, 32, dtype=torch.bfloat16))
    wgrad = dict(g_q=on(0, 32, 64), g_s=on(0, 32, 2), x_q=on(0, 64, 64), x_s=on(0, 64, 2),
                 offsets=on(0, 3, dtype=torch.int32), out=on(0, 2, 32, 64, dtype=torch.float32))
    gemv = dict(x=on(0, 2, 64, dtype=torch.bfloat16), w_q=on(0, 3, 32, 32), w_s=on(0, 3, 32, 4),
                global_scale=on(0, 3, dtype=torch.float32), experts=on(0, 2, dtype=torch.int32),
                out=on(0, 2, 32, dtype=torch.bfloat16))
    return [(mxq.mx_grouped_gemm, gemm), (mxq.mx_grouped_wgrad, wgrad), (mxq.nvfp4_gemv, gemv)]


def test_bindings_refuse_what_lies_elsewhere(monkeypatch):
    """Operands, outputs and the error word on another device than the first
    operand's, a first operand not on the current device, host memory: none of
    them reaches the library."""
    class Reached(Exception):
        pass

    class Library:
        def __getattr__(self, name):
            def entry(*args):
                raise Reached
            return entry

    monkeypatch.setattr(mxq._lib, "lib", Library)
    monkeypatch.setattr(torch.cuda, "device_count", lambda: 2)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(mxq, "_several", None, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda dev: 0)
    for call, args in product_calls():
        with pytest.raises(Reached):
            call(**args)
        err = on(0, 1, dtype=torch.int32)
        with pytest.raises(Reached):
            call(**args, dev_err=err)
        for name, t in args.items():
            for at, error in ((1, ValueError), (-1, (TypeError, ValueError))):
                other = t.clone().as_subclass(OnDevice)
                other.at = at
                with pytest.raises(error):
                    call(**{**args, name: other})
            with pytest.raises(TypeError):
                call(**{**args, name: t.tolist()})
        with pytest.raises(ValueError):
            call(**args, dev_err=on(1, 1, dtype=torch.int32))
        monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
        with pytest.raises(ValueError):
            call(**args)
        monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
        # Without another device there is nothing to compare.
        monkeypatch.setattr(mxq, "_several", False)
        for bad in (torch.zeros(1, dtype=torch.int32), on(0, 0, dtype=torch.int32), on(0, 4), [0], 0):
            with pytest.raises(TypeError):
                call(**args, dev_err=bad)
        with pytest.raises((TypeError, ValueError)):
            call(**{**args, "out": args["out"].as_subclass(torch.Tensor)})
        monkeypatch.setattr(mxq, "_several", None)


@gpu
@pytest.mark.parametrize("exact", [True, False], ids=["exact", "random"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("name,kernel,sizes,N,K,before,after", GEMM_KERNELS, ids=[c[0] for c in GEMM_KERNELS])
def test_gemm_kernels(name, kernel, sizes, N, K, before, after, dtype, exact):
    flags = mxq.OUT_F32 if dtype == torch.float32 else 0
    assert gemm_cut(sizes, N, K, before, after, flags, sms_here()) == kernel
    products.test_grouped_gemm(name, sizes, N, K, before, after, dtype, exact)


@gpu
@pytest.mark.parametrize("exact", [True, False], ids=["exact", "random"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("name,kernel,sizes,N,K,before,after", WGRAD_KERNELS, ids=[c[0] for c in WGRAD_KERNELS])
def test_wgrad_kernels(name, kernel, sizes, N, K, before, after, dtype, exact):
    flags = mxq.OUT_F32 if dtype == torch.float32 else 0
    assert wgrad_cut(sizes, N, K, before, after, flags, sms_here()) == kernel
    products.test_grouped_wgrad(name, sizes, N, K, before, after, dtype, exact)


@gpu
@pytest.mark.parametrize("sizes,N,K,kernel", [([700, 3, 890], 1504, 1024, WIDE),
                                              ([1200, 800], 1600, 4096, PAIR)], ids=["wide", "pair"])
def test_large_kernels_in_place(sizes, N, K, kernel):
    """Outputs inside a wider matrix at aligned and odd elements, the same bits
    every time, nothing outside them written, nothing at all where the offsets
    are wrong."""
    M, E = sum(sizes), len(sizes)
    assert gemm_cut(sizes, N, K, 0, 0, 0, sms_here()) == kernel
    gen = generator(20)
    x_q, x_s = mx_operand(gen, False, M, K)
    w_q, w_s = mx_operand(gen, False, E, N, K)
    off = offsets_of(sizes)
    late = off.clone()
    late[-1] += 1
    for dtype in (torch.bfloat16, torch.float32):
        first = mxq.mx_grouped_gemm(x_q, x_s, w_q, w_s, off, out_dtype=dtype)
        whole = torch.empty((M, N + 8), dtype=dtype, device="cuda")
        for at in (0, 3, 8):
            whole.fill_(9)
            mxq.mx_grouped_gemm(x_q, x_s, w_q, w_s, off, out=whole[:, at:at + N])
            assert (whole[:, at:at + N] == first).all()
            assert (whole[:, :at] == 9).all() and (whole[:, at + N:] == 9).all()
        err = dev_err()
        whole.fill_(9)
        mxq.mx_grouped_gemm(x_q, x_s, w_q, w_s, late, out=whole[:, :N], dev_err=err)
        assert err.item() == mxq.DEVERR_OFFSETS and (whole == 9).all()


@gpu
def test_large_kernels_keep_nan_where_it_is():
    """NaN codes and scales in the pair kernels: one row and one column of one
    group forward, one group's gradient."""
    gen = generator(21)
    sizes, N, K = [300, 500, 1200], 1600, 4096   # the second group's first row is 300
    assert gemm_cut(sizes, N, K, 0, 0, mxq.OUT_F32, sms_here()) == PAIR
    M, E = sum(sizes), len(sizes)
    x_q, x_s = mx_operand(gen, True, M, K)
    w_q, w_s = mx_operand(gen, True, E, N, K)
    x_q[300, K - 1] = 0x7F
    w_s[0, N - 1, 0] = 255
    y = mxq.mx_grouped_gemm(x_q, x_s, w_q, w_s, offsets_of(sizes), out_dtype=torch.float32)
    bad = torch.zeros(M, N, dtype=torch.bool, device="cuda")
    bad[300], bad[:300, N - 1] = True, True
    assert torch.equal(y.isnan(), bad)
    sizes, N, K = [2720, 96, 5376], 2048, 2304
    assert wgrad_cut(sizes, N, K, 0, 0, 0, sms_here()) == PAIR
    M = sum(sizes)
    g_q, g_s = mx_operand(gen, True, N, M)
    x_q, x_s = mx_operand(gen, True, K, M)
    g_q[:, 2720:2816] = 0x7F
    x_s[:, 85:88] = 255
    dw = mxq.mx_grouped_wgrad(g_q, g_s, x_q, x_s, offsets_of(sizes), out_dtype=torch.bfloat16)
    assert dw[1].isnan().all()
    g, x = mx_values(g_q, g_s), mx_values(x_q, x_s)
    for e, (a, b) in ((0, (0, 2720)), (2, (2816, M))):
        check(dw[e], g[:, a:b] @ x[:, a:b].t(), None, True)


def normal_operand(gen, *shape):
    """Codes and scales of normal values, as the library quantizes them."""
    K, rows = shape[-1], torch.Size(shape[:-1]).numel()
    x = torch.randn(-(-rows // 32) * 32, K, generator=gen, device="cuda").bfloat16()
    d = mxq.mx_quantize_rowcol(x, mxq.ROWWISE)
    return d["q_row"][:rows].view(shape), d["s_row"][:rows].view(*shape[:-1], K // 32)


@gpu
@pytest.mark.parametrize("sizes,N,K", [([700], 1904, 1056), ([300, 400], 1904, 8192), ([130, 170], 1904, 8192),
                                       ([1200, 800], 1600, 8192 + 512), ([16, 5], 4800, 14336),
                                       ([60], 513, 28672), ([700, 3, 890], 1504, 3 * 8192)])
def test_fp32_sums_keep_the_documented_error(sizes, N, K):
    """The errors of fp32 outputs stay below 2^-20 of their norm, in every kernel
    and however long the sums are: they are taken apart before the tensor cores
    have cut off more than that."""
    gen = generator(K + N)
    M, E = sum(sizes), len(sizes)
    x_q, x_s = normal_operand(gen, M, K)
    w_q, w_s = normal_operand(gen, E, N, K)
    off = offsets_of(sizes)
    y = mxq.mx_grouped_gemm(x_q, x_s, w_q, w_s, off, out_dtype=torch.float32).double()
    x, w = mx_values(x_q, x_s), mx_values(w_q, w_s)
    want = torch.cat([x[a:b] @ w[e].t() for e, (a, b) in enumerate(zip(off[:-1].tolist(), off[1:].tolist()))])
    assert (y - want).norm() <= 2.0 ** -20 * want.norm()


@gpu
@pytest.mark.parametrize("M,N,K", [(8192, 2048, 1024), (16384, 1100, 2000), (24576, 512, 512), (9600, 2048, 2304)])
def test_fp32_gradients_keep_the_documented_error(M, N, K):
    gen = generator(M + N)
    g_q, g_s = normal_operand(gen, N, M)
    x_q, x_s = normal_operand(gen, K, M)
    dw = mxq.mx_grouped_wgrad(g_q, g_s, x_q, x_s, offsets_of([M])).double()
    want = mx_values(g_q, g_s) @ mx_values(x_q, x_s).t()
    assert (dw[0] - want).norm() <= 2.0 ** -20 * want.norm()


@gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("K", [1056, 4096, 8192 + 512])
def test_bits_follow_from_the_shared_contraction(K, dtype):
    """A row's bits are the same in calls of any size, from any kernel, as long as
    as many CTAs share a tile's contraction."""
    gen = generator(K)
    flags = mxq.OUT_F32 if dtype == torch.float32 else 0
    x_q, x_s = normal_operand(gen, 2500, K)
    w_q, w_s = normal_operand(gen, 2, 9600, K)
    seen, kernels = {}, set()
    for N in (1504, 9600):
        for sizes in ([7], [32], [33], [300], [700], [1300], [2500], [1200, 1300], [7, 0], [64, 900]):
            M, E = sum(sizes), len(sizes)
            plan = gemm_cut(sizes, N, K, 0, 0, flags, sms_here())
            y = mxq.mx_grouped_gemm(x_q[:M], x_s[:M], w_q[:E, :N].contiguous(), w_s[:E, :N].contiguous(),
                                    offsets_of(sizes), out_dtype=dtype)
            kernels.add(plan)
            first = seen.setdefault(plan[3], y[:7, :1504].clone())
            assert torch.equal(y[:7, :1504], first), (N, sizes, plan)
    assert {k[3] for k in kernels} == ({1} if K == 1056 else {1, 2, 4})
    assert len({k[:3] for k in kernels}) >= 3


@gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
def test_gradient_bits_follow_from_the_shared_contraction(dtype):
    gen = generator(31)
    flags = mxq.OUT_F32 if dtype == torch.float32 else 0
    rows = 9 * 1024 + 32
    g_q, g_s = normal_operand(gen, 2048, rows)
    x_q, x_s = normal_operand(gen, 2304, rows)

    def at(t, before, after, n, unit):
        """The first n rows of an operand, its group `before` rows into the buffer."""
        side = torch.zeros(n, before // unit + t.shape[1] + after // unit, dtype=torch.uint8, device="cuda")
        side[:, before // unit:before // unit + t.shape[1]] = t[:n]
        return side

    seen, kernels = {}, set()
    for N, K in ((256, 128), (512, 512), (1100, 1100), (2048, 2304)):
        for before, after in ((0, 0), (128, 32), (1024, 416)):
            plan = wgrad_cut([rows], N, K, before, after, flags, sms_here())
            kernels.add(plan)
            dw = mxq.mx_grouped_wgrad(at(g_q, before, after, N, 1), at(g_s, before, after, N, 32),
                                      at(x_q, before, after, K, 1), at(x_s, before, after, K, 32),
                                      offsets_of([rows], before), out_dtype=dtype)
            first = seen.setdefault(plan[3], dw[0, :256, :128].clone())
            assert torch.equal(dw[0, :256, :128], first), (N, K, before, plan)
    assert {k[3] for k in kernels} >= {1, 4} and len({k[:3] for k in kernels}) >= 2


@gpu
@pytest.mark.parametrize("exact", [True, False], ids=["exact", "random"])
def test_most_groups(exact):
    """The limit of 512 groups, uneven, some empty."""
    sizes = [(i * 29) % 71 if i % 5 else 0 for i in range(512)]
    products.test_grouped_gemm("most_groups", sizes, 72, 160, 3, 4, torch.float32, exact)
    assert gemm_cut(sizes, 72, 160, 3, 4, num_sms=sms_here())[2] == 1
    sizes = [(i * 53) % 171 if i % 5 else 0 for i in range(512)]
    products.test_grouped_gemm("most_groups", sizes, 72, 160, 3, 4, torch.float32, exact)
    assert gemm_cut(sizes, 72, 160, 3, 4, num_sms=sms_here())[2] == 0
    products.test_grouped_wgrad("most_groups", [32 * (i % 4) for i in range(512)], 40, 72, 0, 32, torch.float32, exact)


@gpu
@pytest.mark.parametrize("kind", ["exact", "random", "spread"])
@pytest.mark.parametrize("name,toks,items,chunks,T,N,K", GEMV_KERNELS, ids=[c[0] for c in GEMV_KERNELS])
def test_gemv_kernels(name, toks, items, chunks, T, N, K, kind):
    assert gemv_kernel(T, N, K, 0, sms_here()) == (toks, items, chunks)
    gen = generator(T + N + K)
    x = nv_rows(gen, kind == "exact", T, K, kind == "spread")
    q, s, g = nv_operand(gen, kind == "exact", 1, N, K)
    want, bound = gemv_reference(x, q, s, g, None, 1)
    for dtype in (torch.float32, torch.bfloat16):
        err = dev_err()
        y = mxq.nvfp4_gemv(x, q[0], s[0], g, out_dtype=dtype, dev_err=err)
        assert err.item() == 0
        check(y, want, bound, kind == "exact", name)


@gpu
@pytest.mark.parametrize("E,T,share,N,K", [(0, 13, 1, 4099, 11008), (0, 1, 1, 2048, 2048), (64, 16, 8, 600, 7168)])
def test_gemv_gives_the_same_bits(E, T, share, N, K):
    gen = generator(33)
    x = nv_rows(gen, False, T, K)
    q, s, g = nv_operand(gen, False, max(E, 1), N, K)
    ids = draw_ids(gen, "skewed", T * share, E) if E else None
    call = lambda: mxq.nvfp4_gemv(x, *((q, s, g) if E else (q[0], s[0], g)), experts=ids, share=share,  # noqa: E731
                                  out_dtype=torch.float32)
    first = call()
    assert all(torch.equal(call(), first) for _ in range(20))


def draw_ids(gen, how, rows, E):
    ids = torch.randint(-1, E + 1, (rows,), generator=gen, device="cuda")
    if how == "skewed":
        half = torch.rand(rows, generator=gen, device="cuda") < 0.5
        ids = torch.where(half, torch.full_like(ids, E // 2), ids)
    return ids.int()


@gpu
@pytest.mark.parametrize("kind", ["exact", "random", "spread"])
@pytest.mark.parametrize("name,toks,items,chunks,E,T,share,N,K,how", ROUTED_KERNELS,
                         ids=[c[0] for c in ROUTED_KERNELS])
def test_gemv_expert_kernels(name, toks, items, chunks, E, T, share, N, K, how, kind):
    assert gemv_kernel(T * share, N, K, E, sms_here()) == (toks, items, chunks)
    gen = generator(E + T + N + K)
    x = nv_rows(gen, kind == "exact", T, K, kind == "spread")
    q, s, g = nv_operand(gen, kind == "exact", E, N, K)
    ids = draw_ids(gen, how, T * share, E)
    for some in (ids, torch.full_like(ids, E - 1)):
        want, bound = gemv_reference(x, q, s, g, some, share)
        err = dev_err()
        y = mxq.nvfp4_gemv(x, q, s, g, experts=some, share=share, out_dtype=torch.float32, dev_err=err)
        assert err.item() == 0
        check(y, want, bound, kind == "exact", name)
