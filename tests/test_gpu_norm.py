"""GPU parity of the residual RMS norm (csa_rms_norm) against float64.

Tolerances.  fp32 outputs: the sum of squares of dim values in fp32 is within
(dim / threads + 12) * 2^-24 of exact, its root within half of that; rsqrt is
within 2 ulp, the three products within half an ulp each: 64 * 2^-24 relative
covers every dim here.  bf16 outputs add half a bf16 ulp, 2^-8.  Codes: each
within half an E4M3 step of y / scale, widened by the fp32 bound: 2^-4 + 2^-17
relative, 2^-10 + absolute in the subnormal range.
"""
import numpy as np
import pytest

from oracle import codecs
from oracle.paged import rms_norm
from oracle.quant import ue8m0_exponent

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

F32_REL = 64 * 2.0 ** -24
BF16_REL = 2.0 ** -8


@pytest.fixture(scope="module")
def csa():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    import indexer_selected_sparse_csa2_b200 as m
    return m


def _f64(t):
    return t.detach().double().cpu().numpy()


def _check_values(got, want, dtype, what):
    rel = F32_REL + (BF16_REL if dtype == torch.bfloat16 else 0)
    err = np.abs(_f64(got) - want)
    assert np.all(err <= rel * np.abs(want) + 1e-37), (what, float((err / (np.abs(want) + 1e-30)).max()))


def _check_codes(codes, scales, y, kind, what):
    v = codecs.e4m3_decode(codes.cpu().numpy())
    if kind == "plain":
        z = np.clip(y, -448, 448)
    else:
        block = 32 if kind == "ue8m0" else 128
        yb = y.reshape(y.shape[0], -1, block)
        amax = np.abs(yb).max(axis=2)
        if kind == "ue8m0":
            e = scales.cpu().numpy().astype(np.int64) - 127
            lo, hi = (ue8m0_exponent((amax * f).astype(np.float32)) for f in (1 - F32_REL, 1 + F32_REL))
            assert np.all((e >= lo) & (e <= hi)), what       # equal unless amax sits on a power of two's edge
            s = np.ldexp(1.0, e)
        else:
            s = _f64(scales)
            assert np.all(np.abs(s - amax / 448) <= 2 * F32_REL * amax / 448), what
        z = np.clip((yb / np.where(s > 0, s, 1)[:, :, None]).reshape(y.shape), -448, 448)
    err = np.abs(v - z)
    assert np.all(err <= np.maximum(2.0 ** -4 * np.abs(z), 2.0 ** -10) + 2.0 ** -17 * np.abs(z)), (what, float(err.max()))


def _inputs(seed, rows, dim, dtype, outliers=True):
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((rows, dim)).astype(np.float32)
    r = rng.standard_normal((rows, dim)).astype(np.float32)
    if outliers:
        r[:, rng.integers(0, dim, 3)] *= 50
    w = (1 + 0.2 * rng.standard_normal(dim)).astype(np.float32)
    dev = lambda a: torch.from_numpy(a).cuda()  # noqa: E731
    return dev(x).to(dtype), dev(r).to(dtype), dev(w)


CASES = [(1, 16, "plain"), (1, 32, "ue8m0"), (3, 48, "none"), (5, 96, "ue8m0"), (2, 128, "f32"), (33, 512, "ue8m0"),
         (9, 544, "ue8m0"), (17, 1024, "f32"), (4, 1040, "plain"), (7, 1056, "ue8m0"), (3, 1152, "f32"),
         (1, 4096, "ue8m0"), (300, 4096, "ue8m0"), (67, 5120, "f32"), (5, 7168, "ue8m0"), (2, 16384, "f32"),
         (3, 16368, "plain"), (2000, 512, "none"), (2500, 2048, "f32")]


@pytest.mark.parametrize("rows,dim,kind", CASES)
@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("residual", [False, True])
def test_norm(csa, rows, dim, kind, dtype, residual):
    dt = getattr(torch, dtype)
    x, r, w = _inputs(rows * 7 + dim, rows, dim, dt)
    out = torch.full((rows, dim), 77.0, dtype=dt, device="cuda")
    ro = torch.full((rows, dim), 77.0, dtype=dt, device="cuda") if residual else None
    codes = None if kind == "none" else torch.full((rows, dim), 0x7F, dtype=torch.uint8, device="cuda")
    scales = {"ue8m0": lambda: torch.full((rows, dim // 32), 255, dtype=torch.uint8, device="cuda"),
              "f32": lambda: torch.full((rows, dim // 128), -1.0, device="cuda")}.get(kind, lambda: None)()
    csa.csa_rms_norm(csa.rms_norm_args(x=x, residual=r if residual else None, residual_out=ro, weight=w, eps=1e-6,
                                       out=out, codes=codes, scales=scales))
    torch.cuda.synchronize()
    s, y = rms_norm(_f64(x), 1e-6, _f64(w), _f64(r) if residual else None)
    if residual:
        err = np.abs(_f64(ro) - s)
        rel = 2.0 ** -24 + (BF16_REL if dt == torch.bfloat16 else 0)
        assert np.all(err <= rel * np.abs(s) + 1e-37)
    _check_values(out, y, dt, "out")
    if kind != "none":
        _check_codes(codes, scales, y, kind, "codes")


@pytest.mark.parametrize("dim", [240, 256, 272, 528, 768, 784])
def test_norm_around_the_chunks_of_a_lane(csa, dim):
    """Rows where the number of 8-channel chunks a lane holds changes."""
    for dtype in ("float32", "bfloat16"):
        test_norm(csa, 70, dim, "plain", dtype, True)


def test_norm_without_weight_and_with_zero_rows_of_channels(csa):
    x = torch.zeros(4, 256, device="cuda")
    x[1, 3] = 5.0
    x[2] = 1e-20
    codes = torch.full((4, 256), 1, dtype=torch.uint8, device="cuda")
    sc = torch.full((4, 8), 9, dtype=torch.uint8, device="cuda")
    sf = torch.full((4, 2), 9.0, device="cuda")
    c2 = torch.full((4, 256), 1, dtype=torch.uint8, device="cuda")
    csa.csa_rms_norm(csa.rms_norm_args(x=x, eps=1e-6, codes=codes, scales=sc))
    csa.csa_rms_norm(csa.rms_norm_args(x=x, eps=1e-6, codes=c2, scales=sf))
    torch.cuda.synchronize()
    assert torch.all(codes[0] == 0) and torch.all(sc[0] == 0)          # a zero block: exponent -127, zero codes
    assert torch.all(c2[0] == 0) and torch.all(sf[0] == 0)
    _, y = rms_norm(_f64(x), 1e-6)
    _check_codes(codes[1:2], sc[1:2], y[1:2], "ue8m0", "one channel")
    _check_codes(c2[1:2], sf[1:2], y[1:2], "f32", "one channel")
    _check_codes(codes[2:3], sc[2:3], y[2:3], "ue8m0", "tiny")


def test_norm_of_rows_whose_scales_have_no_reciprocal(csa):
    """amax / 448 below 2^-127, zeros beside it: codes stay within half a step
    of y / 2^-126 (E4M3's smallest step is 2^-9)."""
    x = torch.zeros(3, 256, device="cuda")
    x[0, 0], x[0, 1], x[0, 130] = 2.0 ** -125, -(2.0 ** -128), 2.0 ** -121
    x[1, 5] = 2.0 ** -140
    w = torch.ones(256, device="cuda")
    codes = torch.empty(3, 256, dtype=torch.uint8, device="cuda")
    scales = torch.full((3, 2), 9.0, device="cuda")
    csa.csa_rms_norm(csa.rms_norm_args(x=x, weight=w, eps=1.0, codes=codes, scales=scales))
    torch.cuda.synchronize()
    want = _f64(x)                                   # mean(x^2) is nothing beside eps = 1
    v = codecs.e4m3_decode(codes.cpu().numpy())
    s = _f64(scales)
    assert np.array_equal(s, [[2.0 ** -126, 2.0 ** -126], [2.0 ** -126, 0.0], [0.0, 0.0]])
    z = want / 2.0 ** -126
    assert np.all(np.abs(v - z) <= np.maximum(2.0 ** -4 * np.abs(z), 2.0 ** -10) + 2.0 ** -17)


def test_norm_in_place_and_strided(csa):
    rows, dim = 37, 640
    for dt in (torch.float32, torch.bfloat16):
        x, r, w = _inputs(5, rows, dim, dt)
        want_s, want_y = rms_norm(_f64(x), 1e-5, _f64(w), _f64(r))
        xb, rb = torch.zeros(rows, dim + 32, dtype=dt, device="cuda"), torch.zeros(rows, dim + 64, dtype=dt, device="cuda")
        xb[:, :dim], rb[:, :dim] = x, r
        codes = torch.full((rows, dim + 16), 3, dtype=torch.uint8, device="cuda")
        sc = torch.full((rows, dim // 32 + 3), 3, dtype=torch.uint8, device="cuda")
        # the sum back into residual, the norm back into x
        csa.csa_rms_norm(csa.rms_norm_args(x=xb[:, :dim], residual=rb[:, :dim], residual_out=rb[:, :dim], weight=w, eps=1e-5,
                                           out=xb[:, :dim], codes=codes[:, :dim], scales=sc[:, :dim // 32]))
        torch.cuda.synchronize()
        _check_values(rb[:, :dim], want_s, dt, "residual")
        _check_values(xb[:, :dim], want_y, dt, "out")
        _check_codes(codes[:, :dim], sc[:, :dim // 32], want_y, "ue8m0", "codes")
        assert torch.all(codes[:, dim:] == 3) and torch.all(sc[:, dim // 32:] == 3) and torch.all(xb[:, dim:] == 0)


def test_norm_same_bits_whatever_the_other_rows(csa):
    x, r, w = _inputs(11, 900, 1536, torch.bfloat16)
    def go(x, r):
        out, codes = torch.empty_like(x), torch.empty(x.shape, dtype=torch.uint8, device="cuda")
        sc = torch.empty(x.shape[0], x.shape[1] // 32, dtype=torch.uint8, device="cuda")
        csa.csa_rms_norm(csa.rms_norm_args(x=x, residual=r, weight=w, out=out, codes=codes, scales=sc))
        return out, codes, sc
    whole = go(x, r)
    for i in (0, 1, 500, 899):
        for a, b in zip(whole, go(x[i:i + 1], r[i:i + 1])):
            assert torch.equal(a[i:i + 1], b)


@pytest.mark.parametrize("rows,dim,kind", [(7105, 512, "ue8m0"), (7300, 16, "plain"), (14300, 544, "ue8m0"), (9001, 1024, "f32")])
@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
def test_norm_of_more_rows_than_warps(csa, rows, dim, kind, dtype):
    """Short rows from the 7105th on are a warp's second and third ones."""
    test_norm(csa, rows, dim, kind, dtype, True)


@pytest.mark.parametrize("rows,dim", [(7400, 256), (15000, 640), (3000, 2048)])
@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
def test_norm_in_place_where_rows_are_loaded_ahead(csa, rows, dim, dtype):
    """Both outputs over both inputs, bit for bit the separate ones: a row's
    loads go out before the row before it is written."""
    dt = getattr(torch, dtype)
    x, r, w = _inputs(rows, rows, dim, dt)
    out, ro = torch.empty_like(x), torch.empty_like(x)
    csa.csa_rms_norm(csa.rms_norm_args(x=x, residual=r, residual_out=ro, weight=w, out=out))
    csa.csa_rms_norm(csa.rms_norm_args(x=x, residual=r, residual_out=r, weight=w, out=x))
    torch.cuda.synchronize()
    assert torch.equal(x, out) and torch.equal(r, ro)
