"""mx_rmsnorm and mx_rmsnorm_backward against their formulas in 64 bits.

Errors.  A row's sum of squares adds non-negative terms in chains of at most 64
fp32 operations (16 or 32 in a thread, 5 across a warp, 32 across warps), so it is
off by 64 2^-24 of itself, rstd by half of that, and with its own roundings by less
than 40 2^-24; y has two products more.  In the backward pass mean(g n) is off by
(64 + 3) 2^-24 of the mean of |g n| and n by one rounding; dx adds four operations.
dweight adds M terms, in any order off by (M + 2) 2^-24 of the sum of |terms|.
Outputs are rounded once: bf16 2^-8 of the value, E4M3 as in layer_util."""
import ctypes

import pytest
import torch

import fp4_quantization_gb300 as mxq
from fp4_quantization_gb300 import _lib
from layer_util import check_mx, guarded

gpu = pytest.mark.gpu
U = 2.0 ** -24
EPS = 1e-5


def inputs(M, K, seed, weight=torch.bfloat16, ld=None):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    ld = ld or K
    size = torch.exp(2 * torch.randn(M, 1, generator=gen, device="cuda"))

    def rows():
        return (torch.randn(M, ld, generator=gen, device="cuda") * size).bfloat16()[:, :K]

    w = (1 + 0.5 * torch.randn(K, generator=gen, device="cuda")).to(weight)
    return rows(), rows(), w, gen


def reference(x, residual, w):
    h = x if residual is None else (x.float() + residual.float()).bfloat16()
    n = h.double()
    rstd = (n.square().mean(-1) + EPS) ** -0.5
    return h, rstd, n * rstd.unsqueeze(-1) * w.double()


def check_forward(out, x, residual, w, flags, what=""):
    h, rstd, y = reference(x, residual, w)
    assert ("h" in out) == (residual is not None)
    if residual is not None:
        assert torch.equal(out["h"], h), what
    assert ((out["rstd"].double() - rstd).abs() <= 40 * U * rstd).all(), what
    err = 44 * U * y.abs()
    if flags & mxq.OUT_BF16:
        assert ((out["y"].double() - y).abs() <= 2.0 ** -8 * y.abs() + 2 * err).all(), what
    ceil, tiled = bool(flags & mxq.SCALE_RCEIL), bool(flags & mxq.SCALE_SWIZZLED)
    if flags & mxq.ROWWISE:
        check_mx(out["q_row"], out["s_row"], y, err, ceil, tiled, what + " rows")
    if flags & mxq.COLWISE:
        check_mx(out["q_col"], out["s_col"], y.t().contiguous(), err.t().contiguous(), ceil, tiled, what + " columns")


# One row, odd numbers of rows, every split of a row over warps and lanes, both
# sides of the number of SMs, last blocks and tiles that are ragged.
SHAPES = [(1, 32), (1, 8192), (3, 96), (7, 288), (5, 544), (2, 1056), (150, 2080), (151, 4128), (9, 8224),
          (2, 16416), (1, 32768), (153, 32), (200, 256), (301, 512), (333, 1024), (160, 1920), (311, 4096),
          (155, 8192), (170, 16384), (153, 32736)]


@gpu
@pytest.mark.parametrize("residual", [False, True], ids=["plain", "residual"])
@pytest.mark.parametrize("M,K", SHAPES)
def test_rows(M, K, residual):
    x, r, w, _ = inputs(M, K, M + K, torch.float32 if K % 64 else torch.bfloat16)
    r = r if residual else None
    flags = mxq.ROWWISE | mxq.OUT_BF16 | (mxq.SCALE_RCEIL if M % 2 else 0)
    check_forward(mxq.mx_rmsnorm(x, w, flags, residual=r, eps=EPS), x, r, w, flags)


@gpu
@pytest.mark.parametrize("flags", [1, 2, 3, 512, 1 | 64, 3 | 64, 1 | 128, 2 | 128, 3 | 128 | 64, 3 | 512])
@pytest.mark.parametrize("M,K", [(32, 32), (160, 96), (96, 1056), (192, 4096), (128, 8192), (416, 544)])
def test_outputs(M, K, flags):
    x, r, w, _ = inputs(M, K, M * K)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    for residual in (None, r):
        out = mxq.mx_rmsnorm(x, w, flags, residual=residual, eps=EPS, dev_err=err)
        check_forward(out, x, residual, w, flags)
        # What else is asked for changes no output.
        for one in (1, 2, 512):
            if flags & one and flags & (1 | 2 | 512) != one:
                alone = mxq.mx_rmsnorm(x, w, flags & ~(1 | 2 | 512) | one, residual=residual, eps=EPS)
                for name, t in alone.items():
                    assert torch.equal(t, out[name]), name
    assert err.item() == 0


@gpu
@pytest.mark.parametrize("M", [1, 5, 130])
def test_tiled_rows_pad_with_zeros(M):
    K = 160
    x, _, w, _ = inputs(M, K, 3)
    s, untouched = guarded(mxq.scale_shape(M, K // 32, mxq.SCALE_SWIZZLED), torch.uint8, 77)
    flags = mxq.ROWWISE | mxq.SCALE_SWIZZLED
    check_forward(mxq.mx_rmsnorm(x, w, flags, eps=EPS, s_row=s), x, None, w, flags)
    untouched()


@gpu
def test_strides_in_place_and_guards():
    M, K = 96, 480
    x, r, w, _ = inputs(M, K, 11, ld=K + 24)
    assert not x.is_contiguous()
    flags = 3 | mxq.OUT_BF16
    want = reference(x, r, w)[0]
    outs, checks = {}, []
    for name, shape, dtype in (("h", (M, K), torch.bfloat16), ("y", (M, K), torch.bfloat16), ("rstd", (M,), torch.float32),
                               ("q_row", (M, K), torch.uint8), ("s_row", (M, K // 32), torch.uint8),
                               ("q_col", (K, M), torch.uint8), ("s_col", (K, M // 32), torch.uint8)):
        outs[name], check = guarded(shape, dtype, 7)
        checks.append(check)
    out = mxq.mx_rmsnorm(x, w, flags, residual=r, eps=EPS, **outs)
    check_forward(out, x, r, w, flags)
    for check in checks:
        check()
    # In place over the residual and over x.
    for over in ("residual", "x"):
        a, b = x.clone(memory_format=torch.preserve_format), r.clone(memory_format=torch.preserve_format)
        again = mxq.mx_rmsnorm(a, w, flags, residual=b, eps=EPS, h=b if over == "residual" else a)
        assert torch.equal(again["h"], want)
        for name in ("y", "rstd", "q_row", "s_row", "q_col", "s_col"):
            assert torch.equal(again[name], out[name]), name
    # A window of a wider matrix keeps what is beside it.
    wide = torch.full((M, K + 16), 3.0, dtype=torch.bfloat16, device="cuda")
    mxq.mx_rmsnorm(x, w, mxq.OUT_BF16, residual=r, eps=EPS, y=wide[:, 8:8 + K])
    assert torch.equal(wide[:, 8:8 + K], out["y"])
    assert (wide[:, :8] == 3).all() and (wide[:, 8 + K:] == 3).all()


@gpu
def test_zero_and_extreme_rows():
    K = 256
    x = torch.zeros(64, K, dtype=torch.bfloat16, device="cuda")
    x[1] = 1e-20
    x[2] = 1e15
    x[3, 5] = 1.0
    x[4] = -2.0 ** -133                       # subnormal
    w = torch.linspace(-2, 2, K, device="cuda")
    flags = 3 | mxq.OUT_BF16
    out = mxq.mx_rmsnorm(x, w, flags, eps=EPS)
    # Zeros, of the weight's sign.
    assert not (out["q_row"][0] & 0x7F).any() and not out["s_row"][0].any() and not out["y"][0].any()
    h, rstd, y = reference(x, None, w)
    assert ((out["rstd"].double() - rstd).abs() <= 40 * U * rstd).all()
    # Products below fp32's normal numbers are off by half its smallest step each.
    assert ((out["y"].double() - y).abs() <= 2.0 ** -8 * y.abs() + 90 * U * y.abs() + 2.0 ** -134).all()


@gpu
def test_residual_sum_of_any_bits():
    """h is the bf16 nearest to the fp32 sum, subnormals and overflow included."""
    gen = torch.Generator(device="cuda").manual_seed(12)
    bits = torch.randint(-2 ** 15, 2 ** 15, (2, 512, 2048), generator=gen, device="cuda").to(torch.int16)
    x, r = bits.view(torch.bfloat16)
    r = torch.where(torch.rand(512, 2048, generator=gen, device="cuda") < 0.5, (x.float() * -1.004).bfloat16(), r)
    x, r = (torch.where(t.isfinite(), t, 1.0) for t in (x, r))
    small = torch.randint(0, 256, (2, 64, 2048), generator=gen, device="cuda").to(torch.int16).view(torch.bfloat16)
    x[:64], r[:64] = small[0], -small[1]
    h = mxq.mx_rmsnorm(x, torch.ones(2048, device="cuda"), mxq.OUT_BF16, residual=r)["h"]
    assert torch.equal(h, (x.float() + r.float()).bfloat16())


@gpu
@pytest.mark.parametrize("K", [480, 608, 1536, 2464, 5120, 5632, 7168, 8192, 9728, 10240, 13888, 16384, 20480])
def test_rows_alone_and_among_many(K):
    """A row has the same bits in a call of few rows, of many, and with a residual of zeros."""
    x, _, w, _ = inputs(5000, K, K)
    flags = mxq.ROWWISE | mxq.OUT_BF16
    many = mxq.mx_rmsnorm(x, w, flags, eps=EPS)
    for rows in (slice(0, 1), slice(4700, 5000), slice(1000, 1800)):
        few = mxq.mx_rmsnorm(x[rows], w, flags, eps=EPS)
        for name in few:
            assert torch.equal(few[name], many[name][rows]), (name, rows)
    check_forward(few, x[rows], None, w, flags)
    zeros = torch.zeros(1, K, dtype=torch.bfloat16, device="cuda").expand(5000, K).contiguous()
    past = mxq.mx_rmsnorm(x, w, flags, residual=zeros, eps=EPS)
    assert all(torch.equal(past[name], many[name]) for name in many)
    alone = mxq.mx_rmsnorm(x[:4992], w, mxq.COLWISE, eps=EPS)
    assert torch.equal(alone["rstd"], many["rstd"][:4992])


@gpu
@pytest.mark.parametrize("K", [7648, 7680, 7712, 8160, 8224, 15360, 15392, 16352, 16416])
def test_rows_where_granules_a_thread_change(K):
    test_rows_alone_and_among_many(K)


def back_bounds(dy, h, rstd, w, dh):
    """dx and dweight in 64 bits, and their error bounds."""
    n = h.double() * rstd.double().unsqueeze(-1)
    g = dy.double() * w.double()
    c = (g * n).mean(-1, keepdim=True)
    r = rstd.double().unsqueeze(-1)
    dx = r * (g - n * c)
    c_err = 70 * U * (g * n).abs().mean(-1, keepdim=True)
    err = r * (n.abs() * c_err + 6 * U * (g.abs() + (n * c).abs()))
    if dh is not None:
        dx = dx + dh.double()
        err = err + 2 * U * dx.abs()
    terms = dy.double() * n
    return dx, err, terms.sum(0), (len(dy) + 4) * U * terms.abs().sum(0)


@gpu
@pytest.mark.parametrize("past", [False, True], ids=["plain", "past"])
@pytest.mark.parametrize("M,K", SHAPES + [(1000, 96), (2000, 512)])
def test_backward(M, K, past):
    x, dh, w, gen = inputs(M, K, M + K, torch.float32 if K % 64 else torch.bfloat16)
    dy = torch.randn(M, K, generator=gen, device="cuda").bfloat16()
    dh = dh if past else None
    rstd = (x.float().square().mean(-1) + EPS).rsqrt()
    out = mxq.mx_rmsnorm_backward(dy, x, rstd, w, dh=dh)
    dx, err, dw, dw_err = back_bounds(dy, x, rstd, w, dh)
    assert ((out["dx"].double() - dx).abs() <= 2.0 ** -8 * dx.abs() + 2 * err + 2.0 ** -130).all()
    assert ((out["dweight"].double() - dw).abs() <= dw_err).all()


@gpu
@pytest.mark.parametrize("past", [False, True], ids=["plain", "past"])
@pytest.mark.parametrize("weight", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("M,K", [(14000, 480), (7000, 672), (4000, 2048), (2000, 4064), (1100, 6176), (960, 8192), (800, 10400),
                                 (700, 16384), (480, 16416), (480, 18432), (320, 20480), (330, 32768)])
def test_backward_of_more_rows_than_are_held(M, K, weight, past):
    """Each CTA takes several rows, through every place of its ring."""
    x, dh, w, gen = inputs(M, K, M + K, weight, ld=K + 8)
    dy = torch.randn(M, K + 16, generator=gen, device="cuda").bfloat16()[:, 8:K + 8]
    dh = dh if past else None
    rstd = (x.float().square().mean(-1) + EPS).rsqrt()
    code = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = mxq.mx_rmsnorm_backward(dy, x, rstd, w, dh=dh, dev_err=code)
    assert code.item() == 0
    for rows in range(0, M, 1000):
        at = slice(rows, rows + 1000)
        dx, err, _, _ = back_bounds(dy[at], x[at], rstd[at], w, dh[at] if past else None)
        assert ((out["dx"][at].double() - dx).abs() <= 2.0 ** -8 * dx.abs() + 2 * err + 2.0 ** -130).all()
    _, _, dw, dw_err = back_bounds(dy, x, rstd, w, dh)
    assert ((out["dweight"].double() - dw).abs() <= dw_err).all()
    over = dy.clone(memory_format=torch.preserve_format) if not past else dh.clone(memory_format=torch.preserve_format)
    again = mxq.mx_rmsnorm_backward(dy if past else over, x, rstd, w, dh=over if past else None, dx=over)
    assert torch.equal(over, out["dx"]) and torch.equal(again["dweight"], out["dweight"])


@gpu
def test_backward_in_place_strides_guards():
    M, K = 77, 416
    x, dh, w, gen = inputs(M, K, 5, ld=K + 8)
    dy = torch.randn(M, K + 40, generator=gen, device="cuda").bfloat16()[:, :K]
    rstd = (x.float().square().mean(-1) + EPS).rsqrt()
    dx, check_dx = guarded((M, K), torch.bfloat16, 5)
    dw, check_dw = guarded((K,), torch.float32, 5)
    out = mxq.mx_rmsnorm_backward(dy, x, rstd, w, dh=dh, dx=dx, dweight=dw)
    check_dx()
    check_dw()
    want, err, dwant, dw_err = back_bounds(dy, x, rstd, w, dh)
    assert ((dx.double() - want).abs() <= 2.0 ** -8 * want.abs() + 2 * err).all()
    assert ((dw.double() - dwant).abs() <= dw_err).all()
    for over in ("dy", "dh"):
        a, b = dy.clone(memory_format=torch.preserve_format), dh.clone(memory_format=torch.preserve_format)
        again = mxq.mx_rmsnorm_backward(a, x, rstd, w, dh=b, dx=a if over == "dy" else b)
        assert torch.equal(again["dx"], out["dx"]) and torch.equal(again["dweight"], out["dweight"])


@gpu
def test_backward_against_differences():
    """Central differences of the forward formula in 64 bits, at random entries."""
    M, K = 4, 64
    x, _, w, gen = inputs(M, K, 9, torch.float32)
    dy = torch.randn(M, K, generator=gen, device="cuda").bfloat16()
    rstd = (x.float().square().mean(-1) + EPS).rsqrt()
    out = mxq.mx_rmsnorm_backward(dy, x, rstd, w)

    def loss(h, w):
        return float((h * (h.square().mean(-1, keepdim=True) + EPS) ** -0.5 * w * dy.double()).sum())

    h, wd = x.double(), w.double()
    scale = out["dx"].double().abs().max()
    for i, j in ((0, 0), (1, 17), (2, 63), (3, 40)):
        # The second-order error of the difference is step^2 times a third derivative
        # of order 1 / h^2: 1e-8 for steps of 1e-4 of a row's size.
        step = 1e-4 * float(h[i].abs().mean())
        e = torch.zeros_like(h)
        e[i, j] = step
        slope = (loss(h + e, wd) - loss(h - e, wd)) / (2 * step)
        got = float(out["dx"][i, j])
        assert abs(got - slope) <= 2.0 ** -8 * abs(slope) + 1e-5 * scale
    e = torch.zeros_like(wd)
    e[5] = 1e-3
    slope = (loss(h, wd + e) - loss(h, wd - e)) / 2e-3      # linear in w
    assert abs(float(out["dweight"][5]) - slope) <= 1e-5 * (1 + abs(slope))


@gpu
def test_empty_and_repeatable():
    K = 128
    w = torch.ones(K, device="cuda")
    x = torch.zeros(0, K, dtype=torch.bfloat16, device="cuda")
    out = mxq.mx_rmsnorm(x, w, 3, eps=EPS)
    assert out["q_row"].shape == (0, K) and out["q_col"].shape == (K, 0)
    back = mxq.mx_rmsnorm_backward(x, x, out["rstd"], w, dweight=torch.full((K,), 9.0, device="cuda"))
    assert not back["dweight"].any()
    x, r, w, _ = inputs(700, 1024, 4)
    a = mxq.mx_rmsnorm(x[:224], w, 3, residual=r[:224])
    b = mxq.mx_rmsnorm(x[:224], w, 3, residual=r[:224])
    assert all(torch.equal(a[n], b[n]) for n in a)
    rstd = (x.float().square().mean(-1) + EPS).rsqrt()
    a, b = (mxq.mx_rmsnorm_backward(r, x, rstd, w) for _ in range(2))
    assert all(torch.equal(a[n], b[n]) for n in a)


# ---------------------------------------------------------------------------
# Refusals, on the host
# ---------------------------------------------------------------------------

P = ctypes.c_void_p(4096)


def norm_call(x=P, ldx=64, residual=None, ldr=64, weight=P, M=64, K=64, eps=1e-5, flags=3, h=None, ldh=64, rstd=P,
              y=None, ldy=64, q_row=P, s_row=P, q_col=P, s_col=P):
    return _lib.lib().mx_rmsnorm(x, ldx, residual, ldr, weight, M, K, eps, flags, h, ldh, rstd, y, ldy, q_row, s_row,
                                 q_col, s_col, None, None)


@pytest.mark.parametrize("kw,status", [
    (dict(flags=0), 1), (dict(flags=64), 1), (dict(flags=3 | 4), 1), (dict(flags=3 | 8), 1),
    (dict(eps=0.0), 1), (dict(eps=-1.0), 1), (dict(eps=float("nan")), 1), (dict(eps=float("inf")), 1),
    (dict(M=-1), 2), (dict(M=33), 2), (dict(K=48, ldx=48), 2), (dict(K=32800, ldx=32800), 2), (dict(ldx=32), 2),
    (dict(flags=1, residual=P, ldr=32), 2), (dict(residual=P, h=P, ldh=32), 2), (dict(flags=512, y=P, ldy=8), 2),
    (dict(h=P), 1),                            # h without a residual
    (dict(residual=P), 1),                     # columns read h
    (dict(M=1 << 31, flags=1), 2),
])
def test_forward_refusals(kw, status):
    assert norm_call(**kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(flags=1), 1), (dict(M=-1), 2), (dict(K=48), 2), (dict(K=1 << 16), 2), (dict(lddy=32), 2), (dict(ldh=32), 2),
    (dict(lddx=32), 2), (dict(dh=P, lddh=32), 2), (dict(dweight=ctypes.c_void_p(4100)), 3),
])
def test_backward_refusals(kw, status):
    a = dict(dy=P, lddy=64, h=P, ldh=64, rstd=P, weight=P, dh=None, lddh=64, M=64, K=64, flags=0, dx=P, lddx=64,
             dweight=P, ws=P, ws_bytes=1 << 20, dev_err=None, stream=None)
    a.update(kw)
    if a["K"] > 64:
        a.update(lddy=a["K"], ldh=a["K"], lddx=a["K"])
    assert _lib.lib().mx_rmsnorm_backward(*a.values()) == status


def test_binding_refuses_host_tensors_and_other_types():
    x, w = torch.zeros(32, 64, dtype=torch.bfloat16), torch.ones(64)
    with pytest.raises(TypeError):
        mxq.mx_rmsnorm(x, w)
    with pytest.raises(TypeError):
        mxq.mx_rmsnorm_backward(x, x, torch.ones(32), w)


@gpu
def test_device_refusals():
    x, r, w, _ = inputs(64, 128, 1)
    for bad, err in ((dict(x=x.float()), TypeError), (dict(x=x[:, :100]), mxq.MxqError), (dict(weight=w[:64]), ValueError),
                     (dict(weight=w.half()), TypeError), (dict(residual=r[:32]), ValueError), (dict(h=r), ValueError),
                     (dict(x=x.t()), ValueError), (dict(q_row=torch.empty(64, 64, dtype=torch.uint8, device="cuda")), ValueError),
                     (dict(rstd=torch.empty(64, device="cuda").double()), TypeError), (dict(flags=0), mxq.MxqError),
                     (dict(dev_err=torch.zeros(1)), TypeError), (dict(x=x[:33]), mxq.MxqError)):
        a = dict(x=x, weight=w, flags=3)
        a.update(bad)
        if "x" in bad and bad["x"].shape[1] == 100:
            a["weight"] = torch.ones(100, device="cuda")
        with pytest.raises(err):
            mxq.mx_rmsnorm(**a)
    # Rows that do not start on 16 bytes.
    odd = torch.zeros(64, 132, dtype=torch.bfloat16, device="cuda")[:, :128]
    with pytest.raises(mxq.MxqError):
        mxq.mx_rmsnorm(odd, w)
    rstd = torch.ones(64, device="cuda")
    with pytest.raises(ValueError):
        mxq.mx_rmsnorm_backward(x, x, rstd[:32], w)
    with pytest.raises(mxq.MxqError):
        mxq.mx_rmsnorm_backward(x, x, rstd, w, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
