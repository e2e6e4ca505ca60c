"""Paged cache, append, attention and residual norm without a GPU: the oracle
against brute force, and the refusals of the C ABI and of the argument builders
(every bad argument is turned down on the host before any launch)."""
import ctypes

import numpy as np
import pytest

from oracle import paged
from oracle.quant import fp8_window_quant_rows

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def csa():
    import __graft_entry__
    __graft_entry__.build()
    import indexer_selected_sparse_csa2_b200 as m
    return m


# -------------------------------------------------------------------- oracle
def test_oracle_norm_against_torch():
    rng = np.random.default_rng(0)
    x, r, w = rng.standard_normal((5, 96)), rng.standard_normal((5, 96)), rng.standard_normal(96)
    s, y = paged.rms_norm(x, 1e-5, w, r)
    t = torch.from_numpy(x + r)
    want = torch.nn.functional.rms_norm(t, (96,), torch.from_numpy(w), float(np.float32(1e-5)))
    assert np.array_equal(s, x + r) and np.allclose(y, want.numpy(), rtol=1e-12, atol=0)
    _, one = paged.rms_norm(np.full((1, 16), 3.0), 0.0)
    assert np.allclose(one, 1.0)


def test_oracle_positions_and_entries():
    cu, kv = np.array([0, 2, 2, 5]), np.array([10, 4, 2])
    assert paged.row_positions(cu, kv) == [(0, 8), (0, 9), (2, -1), (2, 0), (2, 1)]
    table = np.array([[3, 0], [-1, 5], [1, 4]], dtype=np.int32)
    assert paged.entry_of(table, 4, 5, 0, 5) == (0, 1)
    assert paged.entry_of(table, 4, 5, 2, 7) == (4, 3)
    for b, p in ((0, -1), (0, 8), (1, 0), (1, 4)):        # before, past the table, no page, no such page
        assert paged.entry_of(table, 4, 5, b, p) is None


def test_oracle_attention_against_torch_sdpa_and_gathers_pages():
    rng = np.random.default_rng(1)
    T, n, H = 37, 6, 3
    pages = np.zeros((4, 10, 528), dtype=np.uint8)
    raw = fp8_window_quant_rows(rng.standard_normal((T, 512)).astype(np.float32))
    table = np.array([[2, 0, 3, 1]], dtype=np.int32)
    for p in range(T):
        pages[table[0, p // 10], p % 10] = raw[p]
    kp, X = paged.gather(pages, table, 0, range(T))
    assert np.array_equal(kp, np.arange(T))
    q = rng.standard_normal((n, H, 512))
    pos = np.arange(T - n, T)
    for window in (0, 1, 9):
        out, lse, mass, size, total = paged.attend(q, pos, kp, X, 0.05, window)
        see = (kp[None] <= pos[:, None]) & (kp[None] > pos[:, None] - (window or T))
        qt, xt = torch.from_numpy(q).transpose(0, 1), torch.from_numpy(X).expand(H, T, 512)
        want = torch.nn.functional.scaled_dot_product_attention(qt, xt, xt, torch.from_numpy(see), scale=float(np.float32(0.05)))
        assert np.allclose(out, want.transpose(0, 1).numpy(), rtol=1e-10, atol=1e-12)
        assert np.all(mass >= np.abs(out) - 1e-12) and np.all(total >= mass - 1e-12) and np.all(size > 0)
    # a sink is one more logit with a zero value
    sink = np.array([0.5, -np.inf, 3.0])
    o2, l2, *_ = paged.attend(q, pos, kp, X, 0.05, 0, sink)
    o1, l1, *_ = paged.attend(q, pos, kp, X, 0.05)
    with np.errstate(invalid="ignore"):
        assert np.allclose(l2, np.logaddexp(l1, sink[None]))
    assert np.allclose(o2, o1 * np.exp(l1 - l2)[..., None])
    # nothing to see
    o0, l0, *_ = paged.attend(q, np.full(n, -1), kp, X, 0.05)
    assert not o0.any() and np.all(np.isneginf(l0))
    assert np.array_equal(paged.attend(q, np.full(n, -1), kp, X, 0.05, 0, sink)[1], np.tile(sink, (n, 1)))


def test_oracle_planted_mistakes_show():
    """A causal mask off by one and a window off by one change the result."""
    rng = np.random.default_rng(2)
    X, q = rng.standard_normal((20, 512)), rng.standard_normal((1, 2, 512))
    base = paged.attend(q, np.array([9]), np.arange(20), X, 0.05, 4)[0]
    for pos, window in ((10, 4), (8, 4), (9, 5), (9, 3)):
        assert np.abs(paged.attend(q, np.array([pos]), np.arange(20), X, 0.05, window)[0] - base).max() > 1e-2


# ------------------------------------------------------------------ refusals
def _sweep(csa, call, good, cases):
    for field, val, want in cases:
        b = type(good).from_buffer_copy(good)
        at = b
        *path, last = field.split(".")
        for p in path:
            at = getattr(at, p)
        setattr(at, last, val)
        assert call(b) == want, (field, val)


def _kv(csa, k):
    k.pages, k.fmt, k.page_size, k.n_pages = 4096, csa.CSA_FMT_FP8_E4M3_UE8M0X32, 16, 8
    k.row_stride, k.page_stride = 528, 528 * 16
    k.block_table, k.table_stride, k.max_pages, k.B = 4096, 4, 4, 2
    k.cu_q = k.kv_len = 4096


def _kv_cases(csa):
    I, S, A = csa.CSA_ERR_INVALID_ARG, csa.CSA_ERR_SHAPE, csa.CSA_ERR_ALIGNMENT
    return [("kv." + f, v, w) for f, v, w in [
        ("pages", None, I), ("block_table", None, I), ("cu_q", None, I), ("kv_len", None, I), ("fmt", 2, I), ("fmt", 9, I),
        ("page_size", 0, S), ("page_size", 65537, S), ("max_pages", 0, S), ("max_pages", 1 << 27, S), ("n_pages", 0, S),
        ("n_pages", 1 << 31, S), ("table_stride", 3, S), ("B", 0, S), ("B", 65537, S), ("row_stride", 512, S),
        ("row_stride", 536, A), ("page_stride", 8452, A), ("page_stride", -16, S), ("pages", 4104, A),
        ("block_table", 4098, A), ("cu_q", 4097, A), ("kv_len", 4099, A)]]


def test_norm_refusals(csa):
    a = csa.RmsNormArgs()
    a.n_rows, a.dim, a.dtype, a.scale_kind = 4, 256, csa.CSA_SRC_BF16, csa.CSA_SCALE_UE8M0X32
    a.x = a.out = a.codes = a.scales = a.residual = a.residual_out = a.weight = 4096
    a.x_stride = a.out_stride = a.codes_stride = a.residual_stride = a.residual_out_stride = 256
    a.scales_stride, a.eps = 8, 1e-6
    I, S, A = csa.CSA_ERR_INVALID_ARG, csa.CSA_ERR_SHAPE, csa.CSA_ERR_ALIGNMENT
    call = lambda b: csa._rms_norm(ctypes.byref(b), None)  # noqa: E731
    _sweep(csa, call, a, [
        ("dtype", 2, I), ("scale_kind", 3, I), ("scale_kind", -1, I), ("n_rows", -1, S), ("dim", 0, S), ("dim", 16400, S),
        ("dim", 240, S), ("dim", 248, S), ("x", None, I), ("residual", None, I), ("scales", None, I), ("eps", -1.0, I),
        ("eps", float("nan"), I), ("x_stride", 248, S), ("out_stride", 100, S), ("codes_stride", 255, S), ("scales_stride", 7, S),
        ("residual_stride", 0, S), ("residual_out_stride", 8, S), ("x_stride", 260, A), ("codes_stride", 264, A), ("x", 4098, A),
        ("out", 4104, A), ("codes", 4100, A), ("residual", 4097, A), ("residual_out", 4104, A), ("weight", 4104, A),
        ("n_rows", 0, csa.CSA_OK)])
    b = csa.RmsNormArgs.from_buffer_copy(a)
    b.out = b.codes = None
    assert call(b) == I
    b = csa.RmsNormArgs.from_buffer_copy(a)
    b.scale_kind, b.dim = csa.CSA_SCALE_F32X128, 192
    assert call(b) == S
    b.dim, b.scales = 256, 4097
    assert call(b) == A
    assert csa._rms_norm(None, None) == I


def test_paged_append_refusals(csa):
    a = csa.PagedAppendArgs()
    _kv(csa, a.kv)
    a.src, a.src_dtype, a.norm, a.n_rows, a.src_row_stride, a.eps = 4096, csa.CSA_SRC_BF16, 1, 3, 512, 1e-6
    I, S, A = csa.CSA_ERR_INVALID_ARG, csa.CSA_ERR_SHAPE, csa.CSA_ERR_ALIGNMENT
    call = lambda b: csa._paged_append(ctypes.byref(b), None)  # noqa: E731
    _sweep(csa, call, a, _kv_cases(csa) + [
        ("src", None, I), ("src_dtype", 5, I), ("norm", 2, I), ("eps", -1e-9, I), ("n_rows", -1, S), ("n_rows", 1 << 31, S),
        ("src_row_stride", 511, S), ("src_row_stride", 516, A), ("src", 4104, A), ("weight", 4100, A), ("rope_cs", 4104, A),
        ("n_rows", 0, csa.CSA_OK)])
    b = csa.PagedAppendArgs.from_buffer_copy(a)
    b.norm, b.weight = 0, 4096                        # a weight without the norm
    assert call(b) == I
    assert csa._paged_append(None, None) == I


def test_paged_attn_refusals(csa):
    a = csa.PagedAttnArgs()
    _kv(csa, a.kv)
    a.q = a.out = 4096
    a.n_rows, a.H, a.D, a.q_row_stride, a.q_head_stride, a.softmax_scale = 5, 16, 512, 16 * 512, 512, 0.05
    I, S, A = csa.CSA_ERR_INVALID_ARG, csa.CSA_ERR_SHAPE, csa.CSA_ERR_ALIGNMENT
    call = lambda b: csa._paged_attn(ctypes.byref(b), None, 0, None)  # noqa: E731
    size = lambda b: csa._paged_attn_ws(ctypes.byref(b))  # noqa: E731
    need = size(a)
    assert need > 0 and call(a) == csa.CSA_ERR_WORKSPACE
    assert csa._paged_attn(ctypes.byref(a), 4096, need - 1, None) == csa.CSA_ERR_WORKSPACE
    assert csa._paged_attn(ctypes.byref(a), 4104, need, None) == A
    cases = _kv_cases(csa) + [
        ("q", None, I), ("out", None, I), ("H", 0, S), ("H", 129, S), ("D", 256, S), ("window", -1, S), ("n_rows", -1, S),
        ("n_rows", 1 << 27, S), ("n_rows", 1 << 62, S), ("softmax_scale", -0.1, I), ("softmax_scale", float("nan"), I),
        ("softmax_scale", float("inf"), I), ("q_head_stride", 504, S), ("q_head_stride", 516, A), ("q_row_stride", -8, S),
        ("q_row_stride", 8196, A), ("q", 4104, A), ("out", 4098, A), ("lse", 4097, A), ("sink", 4098, A), ("rope_cs", 4104, A)]
    _sweep(csa, call, a, cases + [("n_rows", 0, csa.CSA_OK)])
    _sweep(csa, size, a, [(f, v, 0) for f, v, _ in cases])
    assert csa._paged_attn(None, None, 0, None) == I and csa._paged_attn_ws(None) == 0


def test_paged_attn_scale_stays_where_its_product_with_log2_e_is_finite(csa):
    a = csa.PagedAttnArgs()
    _kv(csa, a.kv)
    a.q = a.out = 4096
    a.n_rows, a.H, a.D, a.q_row_stride, a.q_head_stride = 5, 16, 512, 16 * 512, 512
    for scale, want in ((1e30, csa.CSA_ERR_WORKSPACE), (0.0, csa.CSA_ERR_WORKSPACE), (2e30, csa.CSA_ERR_INVALID_ARG),
                        (2.9e38, csa.CSA_ERR_INVALID_ARG)):
        a.softmax_scale = scale
        assert csa._paged_attn(ctypes.byref(a), None, 0, None) == want


def test_tables_stay_a_tile_below_two_to_the_31_positions(csa):
    a = csa.PagedAttnArgs()
    _kv(csa, a.kv)
    a.q = a.out = 4096
    a.n_rows, a.H, a.D, a.q_row_stride, a.q_head_stride, a.softmax_scale = 5, 16, 512, 16 * 512, 512, 0.05
    a.kv.page_size = 1
    for pages, want in ((2 ** 31 - 128, csa.CSA_ERR_WORKSPACE), (2 ** 31 - 127, csa.CSA_ERR_SHAPE), (2 ** 31 - 1, csa.CSA_ERR_SHAPE)):
        a.kv.max_pages = a.kv.table_stride = pages
        assert csa._paged_attn(ctypes.byref(a), None, 0, None) == want


def test_argument_builders_check_types_and_shapes(csa):
    z = torch.zeros
    with pytest.raises(TypeError):
        csa.rms_norm_args(x=z(2, 64, dtype=torch.float16), out=z(2, 64))
    with pytest.raises(TypeError):
        csa.rms_norm_args(x=z(2, 64), residual=z(2, 64, dtype=torch.bfloat16), out=z(2, 64))
    with pytest.raises(ValueError):
        csa.rms_norm_args(x=z(2, 64), out=z(2, 32))
    with pytest.raises(ValueError):
        csa.rms_norm_args(x=z(2, 64), out=z(64, 2).t())
    with pytest.raises(ValueError):
        csa.rms_norm_args(x=z(2, 64), codes=z(2, 64, dtype=torch.uint8), scales=z(2, 4, dtype=torch.uint8))
    i32 = dict(dtype=torch.int32)
    pages = z(3, 16, 528, dtype=torch.uint8)
    good = dict(pages=pages, block_table=z(2, 3, **i32), cu_q=z(3, **i32), kv_len=z(2, **i32))
    kv = csa.paged_kv(**good)
    assert (kv.fmt, kv.page_size, kv.n_pages, kv.B, kv.max_pages) == (csa.CSA_FMT_FP8_E4M3_UE8M0X32, 16, 3, 2, 3)
    assert csa.paged_kv(**{**good, "pages": z(3, 16, 288, dtype=torch.uint8)}).fmt == csa.CSA_FMT_FP4_E2M1_E4M3X16
    for key, val, err in (("pages", z(3, 16, 512, dtype=torch.uint8), ValueError), ("cu_q", z(2, **i32), ValueError),
                          ("block_table", z(2, 3), TypeError), ("kv_len", z(3, **i32), ValueError),
                          ("cu_q", z(3, dtype=torch.int64), TypeError), ("kv_len", z(4, **i32)[::2], ValueError)):
        with pytest.raises(err):
            csa.paged_kv(**{**good, key: val})
    with pytest.raises(ValueError):
        csa.paged_append_args(src=z(4, 256), kv=kv)
    with pytest.raises(ValueError):
        csa.paged_append_args(src=z(4, 512), kv=kv, rope_cs=z(3, 32, 2))
    q = z(4, 16, 512, dtype=torch.bfloat16)
    with pytest.raises(TypeError):
        csa.paged_attn_args(q=q.float(), kv=kv, out=q, softmax_scale=1.0)
    with pytest.raises(ValueError):
        csa.paged_attn_args(q=q, kv=kv, out=z(4, 16, 1024, dtype=torch.bfloat16)[..., :512], softmax_scale=1.0)
    with pytest.raises(ValueError):
        csa.paged_attn_args(q=q, kv=kv, out=torch.empty_like(q), lse=z(16, 4), softmax_scale=1.0)
    a = csa.paged_attn_args(q=q, kv=kv, out=torch.empty_like(q), softmax_scale=1.0)
    assert (a.n_rows, a.H, a.D, a.q_row_stride, a.q_head_stride, a.window) == (4, 16, 512, 16 * 512, 512, 0)
    # one row, whatever stride a one-row view carries
    one = csa.rms_norm_args(x=z(64, 3).t()[:1].contiguous(), out=z(1, 64))
    assert one.x_stride >= 64 and one.out_stride >= 64


def test_calls_refuse_host_tensors(csa):
    """The builders take CPU tensors; the calls must not hand their addresses to
    a kernel."""
    z = torch.zeros
    kv = csa.paged_kv(pages=z(3, 16, 528, dtype=torch.uint8), block_table=z(2, 3, dtype=torch.int32),
                      cu_q=z(3, dtype=torch.int32), kv_len=z(2, dtype=torch.int32))
    q = z(4, 16, 512, dtype=torch.bfloat16)
    attn = csa.paged_attn_args(q=q, kv=kv, out=torch.empty_like(q), softmax_scale=1.0)
    for call, args in ((csa.csa_rms_norm, csa.rms_norm_args(x=z(2, 64), out=z(2, 64))),
                       (csa.csa_paged_append, csa.paged_append_args(src=z(4, 512), kv=kv)),
                       (csa.csa_paged_attn, attn)):
        with pytest.raises(ValueError, match="CUDA device"):
            call(args)
    with pytest.raises(ValueError, match="CUDA device"):
        csa.csa_paged_attn(attn, workspace=z(1 << 20, dtype=torch.uint8))


def test_attention_refuses_workspaces_it_could_not_write(csa):
    """On the host, on another device than the arguments, and views whose
    element count is not the size of their memory."""
    kv = csa.PagedAttnArgs()
    _kv(csa, kv.kv)
    kv.q = kv.out = 4096
    kv.n_rows, kv.H, kv.D, kv.q_row_stride, kv.q_head_stride, kv.softmax_scale = 5, 16, 512, 16 * 512, 512, 0.05
    need = csa.csa_paged_attn_workspace_size(kv)
    with pytest.raises(ValueError, match="workspace"):
        csa.csa_paged_attn(kv, workspace=torch.zeros(need, dtype=torch.uint8))

    class Workspace:                                  # stands in for a tensor on a GPU
        device = torch.device("cuda", 1)

        def __init__(self, contiguous):
            self.is_contiguous = lambda: contiguous

        def get_device(self):
            return 1

        def numel(self):
            return need

        def element_size(self):
            return 1

    for dev in (None, 1):
        assert csa._workspace_bytes(Workspace(True), dev, "call") == need
        with pytest.raises(ValueError, match="contiguous"):
            csa._workspace_bytes(Workspace(False), dev, "call")
    with pytest.raises(ValueError, match="cuda:0"):
        csa._workspace_bytes(Workspace(True), 0, "call")
    assert csa._workspace_bytes(None, None, "call") == 0
