"""GPU parity of the paged cache: append (csa_paged_append) and attention of
chunks of new tokens (csa_paged_attn) against float64.

Attention tolerance per element, with A = sum_e w_e |x_e| and
Z = max_e scale * sum_d |q_d x_ed|:
  * the weights' rounding to fp16: 2^-11 of each, A 2^-11 in all; where the
    weight is an fp16 subnormal, half of 2^-24 instead, absolute, on a scale
    where the largest weight (<= 1 of the sum) is at least 2^6: 2^-31 for each
    entry, 2^-31 sum_e |x_e| in all;
  * the logits' fp32 accumulation (512 products and the tensor core's own
    alignment, at most 2^-18 of the sum of magnitudes) and the exp2, which
    change weights by 2 * (2^-18 Z + 2^-20) relative;
  * the output's rounding to bf16: 2^-8 |o|;
  * rotated queries are rounded to fp16: 2^-11 of their share of Z, counted on
    the whole of it.
lse: twice the logits' bound plus 2^-20 (1 + |lse|).
"""
import numpy as np
import pytest

from oracle import rope as orope
from oracle.paged import attend, entry_of, gather, rms_norm, row_positions
from oracle.quant import fp4_dequant_rows, fp4_quant_rows, fp8_window_dequant_rows, fp8_window_quant_rows

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

ENTRY = {"fp8": 528, "fp4": 288}


@pytest.fixture(scope="module")
def csa():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    import indexer_selected_sparse_csa2_b200 as m
    assert m.device_status() == 0
    yield m
    torch.cuda.synchronize()
    assert m.device_status() == 0


def _encode(x, fmt):
    return (fp8_window_quant_rows if fmt == "fp8" else fp4_quant_rows)(x)


class Batch:
    """A paged cache and new tokens, on the host and on the device.
    lens: [(new tokens, cache length)]."""

    def __init__(self, seed, lens, H, fmt="fp8", page=16, q_gain=2.0, tail_rows=0, spread=1.0):
        rng = np.random.default_rng(seed)
        self.lens, self.H, self.fmt, self.page = lens, H, fmt, page
        need = [max(1, -(-T // page)) for _, T in lens]
        self.n_pages = sum(need) + 2
        ids = rng.permutation(self.n_pages).astype(np.int32)
        self.table = np.full((len(lens), max(need) + 1), -1, dtype=np.int32)
        at = 0
        # bytes that decode to the largest magnitudes wherever nothing was written
        self.pages = np.full((self.n_pages, page, ENTRY[fmt]), 0x7E, dtype=np.uint8)
        for b, (n, T) in enumerate(lens):
            self.table[b, :need[b]] = ids[at:at + need[b]]
            at += need[b]
            if T > 0:
                e = _encode((rng.standard_normal((T, 512)) * spread).astype(np.float32), fmt)
                for p in range(0, T, page):
                    k = min(page, T - p)
                    self.pages[self.table[b, p // page], :k] = e[p:p + k]
        self.cu = np.concatenate([[0], np.cumsum([n for n, _ in lens])]).astype(np.int32)
        self.kv = np.array([T for _, T in lens], dtype=np.int32)
        self.rows = int(self.cu[-1]) + tail_rows
        self.q = torch.from_numpy((q_gain * rng.standard_normal((max(1, self.rows), H, 512))).astype(np.float32)).to(torch.bfloat16)
        self.sink = rng.standard_normal(H).astype(np.float32)
        self.cs = np.stack([orope.rope_angles(i) for i in range(max(1, self.rows))])

    def device(self, csa):
        dev = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
        self.d = dict(pages=dev(self.pages), block_table=dev(self.table), cu_q=dev(self.cu), kv_len=dev(self.kv))
        return csa.paged_kv(**self.d)

    def want(self, window=0, sink=None, rope=False, scale=512 ** -0.5):
        n = int(self.cu[-1])
        out, mass = np.zeros((n, self.H, 512)), np.zeros((n, self.H, 512))
        lse, size, total = np.zeros((n, self.H)), np.zeros((n, self.H)), np.zeros((n, 1, 512))
        pos = np.array([p for _, p in row_positions(self.cu, self.kv)], dtype=np.int64)
        q = self.q[:n].double().numpy()
        for b in range(len(self.lens)):
            i, j = self.cu[b], self.cu[b + 1]
            if i == j:
                continue
            kp, X = gather(self.pages, self.table, b, range(0, max(0, int(self.kv[b]))))
            qq = q[i:j]
            if rope:
                qq = np.stack([orope.rotate(qq[t], self.cs[i + t]) for t in range(j - i)])
            out[i:j], lse[i:j], mass[i:j], size[i:j], total[i:j] = attend(qq, pos[i:j], kp, X, scale, window, sink)
        if rope:
            out = np.stack([orope.rotate(out[t], self.cs[t], inverse=True) for t in range(n)]) if n else out
            for m in (mass, total):                # a rotated pair's error stays within the pair's sum
                both = m[..., 448::2] + m[..., 449::2]
                m[..., 448::2] = m[..., 449::2] = both
        return out, lse, mass, size, total


def _check(got, got_lse, want, rope=False):
    out, lse, mass, size, total = want
    n = out.shape[0]
    g = got[:n].double().cpu().numpy()
    dl = 2.0 ** -18 * size + 2.0 ** -20 + (2.0 ** -11 * size if rope else 0)
    tol = 2.0 ** -11 * mass + 2.0 ** -31 * total + 2 * dl[..., None] * mass + 2.0 ** -8 * np.abs(out) + 1e-30
    bad = np.abs(g - out) > tol
    assert not bad.any(), (int(bad.sum()), float((np.abs(g - out) / tol).max()), np.argwhere(bad)[:4].tolist())
    if got_lse is not None:
        l = got_lse[:n].double().cpu().numpy()
        assert np.array_equal(np.isneginf(l), np.isneginf(lse))
        fin = np.isfinite(lse)
        assert np.all(np.abs(l[fin] - lse[fin]) <= 2 * dl[fin] + 2.0 ** -20 * (1 + np.abs(lse[fin])))


def _run(csa, B, kv, window=0, sink=None, rope=False, scale=512 ** -0.5, q=None, stream=None, ws=None):
    q = B.q.cuda() if q is None else q
    out = torch.full((q.shape[0], B.H, 512), 3.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((q.shape[0], B.H), 3.0, device="cuda")
    a = csa.paged_attn_args(q=q, kv=kv, out=out, lse=lse, softmax_scale=scale, window=window,
                            sink=None if sink is None else torch.from_numpy(sink).cuda(),
                            rope_cs=torch.from_numpy(B.cs).cuda() if rope else None)
    if ws is None:                                   # whatever the workspace holds
        ws = torch.full((csa.csa_paged_attn_workspace_size(a),), 0xFF, dtype=torch.uint8, device="cuda")
    csa.csa_paged_attn(a, workspace=ws)
    torch.cuda.synchronize()
    assert csa.device_status() == 0
    return out, lse


SMALL = [
    # lens, H, fmt, page, window, sink
    ([(1, 1)], 1, "fp8", 16, 0, False),
    ([(1, 64)], 64, "fp8", 64, 0, False),
    ([(1, 65)], 64, "fp4", 16, 0, True),
    ([(3, 3), (1, 17), (0, 40), (5, 200)], 16, "fp8", 7, 0, True),
    ([(3, 3), (1, 17), (0, 40), (5, 200)], 16, "fp4", 100, 0, False),
    ([(70, 70), (2, 130)], 3, "fp8", 16, 0, False),
    ([(33, 300)], 128, "fp8", 32, 0, True),
    ([(20, 150), (9, 64)], 24, "fp4", 1, 0, True),
    ([(40, 400), (1, 129), (7, 7)], 64, "fp8", 64, 128, True),
    ([(40, 400), (1, 129), (7, 7)], 64, "fp4", 64, 1, False),
    ([(90, 90)], 8, "fp8", 256, 33, False),
    ([(1, 5000)], 64, "fp8", 64, 0, True),
    ([(2, 3001), (1, 1), (1, 900)], 40, "fp4", 64, 0, False),
]


@pytest.mark.parametrize("case", range(len(SMALL)))
def test_attention(csa, case):
    lens, H, fmt, page, window, sink = SMALL[case]
    B = Batch(100 + case, lens, H, fmt, page)
    s = B.sink if sink else None
    out, lse = _run(csa, B, B.device(csa), window, s)
    _check(out, lse, B.want(window, s))


def _thin(lens, H):
    """The same sequences among enough others without new tokens that a call
    has at most 64 (token, head) rows per sequence on average, which is where
    it changes kernels."""
    rows = sum(n for n, _ in lens) * H
    return lens + [(0, 3)] * max(0, -(-rows // 64) - len(lens))


@pytest.mark.parametrize("case", range(len(SMALL)))
def test_attention_with_few_rows_per_sequence(csa, case):
    lens, H, fmt, page, window, sink = SMALL[case]
    B = Batch(300 + case, _thin(lens, H), H, fmt, page)
    s = B.sink if sink else None
    out, lse = _run(csa, B, B.device(csa), window, s, rope=case % 2 == 0)
    _check(out, lse, B.want(window, s, rope=case % 2 == 0), rope=case % 2 == 0)


@pytest.mark.parametrize("fmt", ["fp8", "fp4"])
@pytest.mark.parametrize("scale", [0.0, 1.0])
def test_softmax_scales_with_few_rows(csa, fmt, scale):
    B = Batch(17, _thin([(5, 300), (1, 70)], 16), 16, fmt, 32)
    out, lse = _run(csa, B, B.device(csa), scale=scale)
    _check(out, lse, B.want(scale=scale))


@pytest.mark.parametrize("order", [1, -1])
def test_running_max_with_few_rows(csa, order):
    B = Batch(18, _thin([(4, 900), (2, 700)], 32), 32, "fp8", 16)
    rng = np.random.default_rng(3)
    for b, T in ((0, 900), (1, 700)):
        gain = np.linspace(0.05, 6.0, T)[::order]
        e = _encode((rng.standard_normal((T, 512)) * gain[:, None]).astype(np.float32), "fp8")
        for p in range(0, T, 16):
            k = min(16, T - p)
            B.pages[B.table[b, p // 16], :k] = e[p:p + k]
    out, lse = _run(csa, B, B.device(csa))
    _check(out, lse, B.want())


def test_block_exponents_far_from_one_with_few_rows(csa):
    B = Batch(19, _thin([(1, 200), (2, 100)], 16), 16, "fp8", 16)
    flat = B.pages.reshape(-1, 528)
    rng = np.random.default_rng(4)
    for p in range(200):
        row = flat[B.table[0, p // 16] * 16 + p % 16]
        row[:512] = rng.permutation(np.tile([c for c in range(256) if c & 0x7F != 0x7F], 3))[:512]
        row[512:] = rng.integers(90, 124, 16)
    out, lse = _run(csa, B, B.device(csa), scale=0.02)
    # as in the test above: decoded values on fp16's grid
    want = B.want(scale=0.02)
    size = want[3] + 0.02 * 2.0 ** -7 * np.abs(B.q.double().numpy()).sum(-1)
    _check(out, lse, (want[0], want[1], want[2] + 2.0 ** -13, size, want[4]))


def test_few_rows_that_see_nothing(csa):
    """Tokens before position 0, caches of length 0 and missing pages, single
    tokens each: zero rows, lse = sink or -inf."""
    B = Batch(20, [(1, 0), (1, 20), (1, 16), (1, -3), (1, 33)], 16)
    B.table[1, :] = -1
    B.table[2, 0] = B.n_pages
    for sink in (None, B.sink):
        out, lse = _run(csa, B, B.device(csa), sink=sink)
        _check(out[4:], lse[4:], [x[4:] for x in B.want(sink=sink)])
        assert not out[:4].any()
        ref = torch.full((4, 16), -np.inf) if sink is None else torch.from_numpy(sink).expand(4, 16)
        assert torch.equal(lse[:4].cpu(), ref) if sink is None else torch.allclose(lse[:4].cpu(), ref, rtol=2 ** -20, atol=0)


def test_single_tokens_of_many_sequences_repeat_their_bits(csa):
    """Split over most of the GPU, sequences of very different lengths, more
    than 32 of them; twice the same bits."""
    rng = np.random.default_rng(21)
    lens = [(1, int(x)) for x in rng.integers(1, 700, 70)] + [(1, 9000), (0, 50), (1, 1)]
    B = Batch(21, lens, 64, "fp8", 32, tail_rows=2)
    kv = B.device(csa)
    out, lse = _run(csa, B, kv, sink=B.sink)
    _check(out, lse, B.want(sink=B.sink))
    assert torch.all(out[-2:] == 3.0) and torch.all(lse[-2:] == 3.0)
    again = _run(csa, B, kv, sink=B.sink)
    assert torch.equal(out, again[0]) and torch.equal(lse, again[1])


def test_single_tokens_in_a_graph(csa):
    """A decode step captured once and replayed as the caches grow."""
    B = Batch(22, [(1, 500), (1, 90), (1, 64)], 16, "fp4", 16)
    kv = B.device(csa)
    q = B.q.cuda()
    out = torch.empty((3, 16, 512), dtype=torch.bfloat16, device="cuda")
    lse = torch.empty((3, 16), device="cuda")
    a = csa.paged_attn_args(q=q, kv=kv, out=out, lse=lse, softmax_scale=0.04)
    ws = torch.empty(csa.csa_paged_attn_workspace_size(a), dtype=torch.uint8, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        csa.csa_paged_attn(a, workspace=ws)
    for drop in (0, 37, 63):
        B.kv = np.array([T - drop for _, T in B.lens], dtype=np.int32)
        B.d["kv_len"].copy_(torch.from_numpy(B.kv))
        out.fill_(3.0)
        lse.fill_(3.0)
        g.replay()
        torch.cuda.synchronize()
        _check(out, lse, B.want(scale=0.04))
    assert csa.device_status() == 0


def test_workspace_of_a_larger_call_serves_a_smaller_one(csa):
    B = Batch(23, [(70, 400), (9, 60)], 16, "fp8", 16)
    kv = B.device(csa)
    sizes = []
    for n in (1, 2, 8, 9, 40, 79):
        q = B.q[:n].cuda()
        a = csa.paged_attn_args(q=q, kv=kv, out=torch.empty((n, 16, 512), dtype=torch.bfloat16, device="cuda"), softmax_scale=0.04)
        sizes.append(csa.csa_paged_attn_workspace_size(a))
    assert sizes == sorted(sizes)


@pytest.mark.parametrize("fmt", ["fp8", "fp4"])
@pytest.mark.parametrize("scale", [0.0, 1e-3, 1.0])
def test_softmax_scales(csa, fmt, scale):
    B = Batch(7, [(5, 300), (1, 70)], 16, fmt, 32)
    out, lse = _run(csa, B, B.device(csa), scale=scale)
    _check(out, lse, B.want(scale=scale))


def test_running_max_moves_late_and_early(csa):
    """Key norms that grow and fall along the cache: the rescaling path."""
    for order in (1, -1):
        B = Batch(8, [(4, 900)], 32, "fp8", 16)
        gain = np.linspace(0.05, 6.0, 900)[::order]
        rng = np.random.default_rng(3)
        e = _encode((rng.standard_normal((900, 512)) * gain[:, None]).astype(np.float32), "fp8")
        for p in range(0, 900, 16):
            k = min(16, 900 - p)
            B.pages[B.table[0, p // 16], :k] = e[p:p + k]
        out, lse = _run(csa, B, B.device(csa))
        _check(out, lse, B.want())


def test_block_exponents_far_from_one(csa):
    """FP8 blocks whose scale is outside fp16's powers of two, next to
    ordinary ones, and every E4M3 code."""
    B = Batch(9, [(3, 200)], 16, "fp8", 16)
    flat = B.pages.reshape(-1, 528)
    rng = np.random.default_rng(4)
    for p in range(200):
        row = flat[B.table[0, p // 16] * 16 + p % 16]
        row[:512] = rng.permutation(np.tile([c for c in range(256) if c & 0x7F != 0x7F], 3))[:512]
        row[512:] = rng.integers(90, 124, 16)
    out, lse = _run(csa, B, B.device(csa), scale=0.02)
    # decoded values below 2^-14 are rounded to fp16's 2^-24 grid: 2^-25 on a
    # value, and through the logits 0.02 * sum |q| 2^-25
    want = B.want(scale=0.02)
    size = want[3] + 0.02 * 2.0 ** -7 * np.abs(B.q.double().numpy()).sum(-1)
    _check(out, lse, (want[0], want[1], want[2] + 2.0 ** -13, size, want[4]))


def test_rows_that_see_nothing(csa):
    """Fewer cached tokens than new ones (negative positions), an empty cache,
    pages that are missing: zero rows, lse = sink or -inf."""
    B = Batch(10, [(6, 6), (4, 4), (3, 100)], 16, "fp8", 16)
    B.kv = np.array([2, 0, 100], dtype=np.int32)
    B.table[2, :] = -1
    B.table[2, 1] = B.n_pages + 3
    kv = B.device(csa)
    for sink in (None, B.sink, np.full(16, -np.inf, dtype=np.float32)):
        out, lse = _run(csa, B, kv, sink=sink)
        want = B.want(sink=sink)
        _check(out, lse, want)
        assert torch.all(out[:4] == 0) and torch.all(out[6:] == 0)
        ref = torch.full((7, 16), -np.inf) if sink is None else torch.from_numpy(sink).expand(7, 16)
        assert torch.allclose(lse[6:].cpu(), ref, rtol=1e-6)


def test_missing_pages_are_left_out(csa):
    B = Batch(11, [(5, 500), (2, 90)], 32, "fp4", 16)
    B.table[0, 3] = -1
    B.table[0, 10] = B.n_pages
    B.table[0, 11] = -2 ** 31
    B.table[0, 12] = 2 ** 31 - 1
    B.table[1, 5] = -7                              # the newest tokens' page
    out, lse = _run(csa, B, B.device(csa))
    _check(out, lse, B.want())


def test_cache_longer_than_its_table(csa):
    """kv_len past the table: positions without a page hold no entry."""
    B = Batch(12, [(3, 64)], 16, "fp8", 16)
    B.table = B.table[:, :4].copy()
    B.kv = np.array([100], dtype=np.int32)
    out, lse = _run(csa, B, B.device(csa))
    _check(out, lse, B.want())
    B.kv = np.array([2 ** 31 - 1], dtype=np.int32)
    out, lse = _run(csa, B, B.device(csa))
    kp, X = gather(B.pages, B.table, 0, range(64))
    _check(out, lse, attend(B.q.double().numpy(), np.full(3, 10 ** 9), kp, X, 512 ** -0.5))


def test_rows_behind_the_last_sequence_stay(csa):
    B = Batch(13, [(5, 50), (0, 9), (2, 33)], 16, "fp8", 16, tail_rows=9)
    out, lse = _run(csa, B, B.device(csa))
    _check(out, lse, B.want())
    assert torch.all(out[7:] == 3.0) and torch.all(lse[7:] == 3.0)


@pytest.mark.parametrize("fmt", ["fp8", "fp4"])
def test_rope(csa, fmt):
    B = Batch(14, [(20, 90), (1, 700), (3, 3)], 16, fmt, 16)
    out, lse = _run(csa, B, B.device(csa), rope=True, sink=B.sink)
    _check(out, lse, B.want(rope=True, sink=B.sink), rope=True)


def test_strided_queries_pages_and_entries(csa):
    B = Batch(15, [(9, 140), (1, 31)], 24, "fp8", 16)
    B.device(csa)
    big = torch.full((B.n_pages, 18, 560), 0x7E, dtype=torch.uint8, device="cuda")
    pages = big[:, 1:17, 16:544]
    pages.copy_(B.d["pages"])
    table = torch.full((2, 40), -1, dtype=torch.int32, device="cuda")
    table[:, :B.table.shape[1]] = B.d["block_table"]
    kv = csa.paged_kv(pages=pages, block_table=table[:, :B.table.shape[1]], cu_q=B.d["cu_q"], kv_len=B.d["kv_len"])
    q = torch.full((B.rows, 24, 576), 1e4, dtype=torch.bfloat16, device="cuda")
    q[..., 32:544] = B.q.cuda()
    out, lse = _run(csa, B, kv, q=q[..., 32:544])
    _check(out, lse, B.want())
    qt = B.q.cuda().transpose(0, 1).contiguous().transpose(0, 1)        # heads outermost
    out2, lse2 = _run(csa, B, kv, q=qt)
    assert torch.equal(out, out2) and torch.equal(lse, lse2)


def test_page_offsets_past_32_bits(csa):
    B = Batch(16, [(2, 40)], 16, "fp8", 16)
    B.device(csa)
    stride = (5 << 30) // 2
    buf = torch.zeros(2 * stride + 16 * 528 + 64, dtype=torch.uint8, device="cuda")
    pages = buf.as_strided((3, 16, 528), (stride, 528, 1))
    order = B.table[0, :3]
    for i in range(3):
        pages[i] = B.d["pages"][int(order[i])]
    table = torch.tensor([[0, 1, 2]], dtype=torch.int32, device="cuda")
    kv = csa.paged_kv(pages=pages, block_table=table, cu_q=B.d["cu_q"], kv_len=B.d["kv_len"])
    out, lse = _run(csa, B, kv)
    _check(out, lse, B.want())
    del buf, pages


@pytest.mark.parametrize("H", [16, 128])
def test_positions_up_to_two_to_the_31(csa, H):
    """The last positions a table can have, behind a window."""
    n = 2 ** 31 - 128
    B = Batch(26, [(1, 200)], H, "fp8", 1)
    B.device(csa)
    table = torch.empty((1, n), dtype=torch.int32, device="cuda")          # only its end is read
    table[0, n - 200:] = B.d["block_table"][0, :200]
    kv = csa.paged_kv(pages=B.d["pages"], block_table=table, cu_q=B.d["cu_q"],
                      kv_len=torch.tensor([n], dtype=torch.int32, device="cuda"))
    out, lse = _run(csa, B, kv, window=90)
    _check(out, lse, B.want(window=90))


def test_same_bits_on_every_run(csa):
    B = Batch(17, [(1, 4000), (30, 500), (1, 2)], 64, "fp8", 64)
    kv = B.device(csa)
    first = _run(csa, B, kv)
    for _ in range(3):
        again = _run(csa, B, kv)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


def test_two_streams_at_once(csa):
    P = [Batch(18, [(1, 3000)], 64, "fp8", 64), Batch(19, [(60, 400), (1, 9)], 32, "fp4", 16)]
    kvs = [b.device(csa) for b in P]
    alone = [_run(csa, b, k) for b, k in zip(P, kvs)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    res = []
    for b, k in zip(P, kvs):
        q = b.q.cuda()
        out, lse = torch.empty(b.rows, b.H, 512, dtype=torch.bfloat16, device="cuda"), torch.empty(b.rows, b.H, device="cuda")
        a = csa.paged_attn_args(q=q, kv=k, out=out, lse=lse, softmax_scale=512 ** -0.5)
        res.append((a, torch.empty(csa.csa_paged_attn_workspace_size(a), dtype=torch.uint8, device="cuda"), out, lse))
    torch.cuda.synchronize()
    for _ in range(10):
        for s, (a, ws, _, _) in zip(streams, res):
            csa.csa_paged_attn(a, workspace=ws, stream=s)
    torch.cuda.synchronize()
    for (_, _, out, lse), (o, l) in zip(res, alone):
        assert torch.equal(out, o) and torch.equal(lse, l)


def test_graph_replay_follows_the_lengths(csa):
    B = Batch(20, [(4, 300), (4, 200)], 16, "fp8", 16, tail_rows=4)
    kv = B.device(csa)
    q = B.q.cuda()
    out, lse = torch.zeros(B.rows, 16, 512, dtype=torch.bfloat16, device="cuda"), torch.zeros(B.rows, 16, device="cuda")
    a = csa.paged_attn_args(q=q, kv=kv, out=out, lse=lse, softmax_scale=512 ** -0.5)
    ws = torch.empty(csa.csa_paged_attn_workspace_size(a), dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        csa.csa_paged_attn(a, workspace=ws)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        csa.csa_paged_attn(a, workspace=ws)
    for lens, cu in (([300, 200], [0, 4, 8]), ([17, 200], [0, 9, 12]), ([250, 3], [0, 1, 3])):
        B.cu, B.kv = np.array(cu, dtype=np.int32), np.array(lens, dtype=np.int32)
        B.d["cu_q"].copy_(torch.from_numpy(B.cu))
        B.d["kv_len"].copy_(torch.from_numpy(B.kv))
        g.replay()
        torch.cuda.synchronize()
        _check(out, lse, B.want())


def test_workspace_of_a_call_on_another_stream(csa):
    """Calls without a workspace, on a stream that is not the current one: the
    memory they allocate stays theirs until they are done."""
    B = Batch(27, [(1, 6000), (1, 40)], 64, "fp8", 64)
    kv = B.device(csa)
    want = _run(csa, B, kv)
    q, side = B.q.cuda(), torch.cuda.Stream()
    out, lse = torch.empty(2, 64, 512, dtype=torch.bfloat16, device="cuda"), torch.empty(2, 64, device="cuda")
    a = csa.paged_attn_args(q=q, kv=kv, out=out, lse=lse, softmax_scale=512 ** -0.5)
    torch.cuda.synchronize()
    for _ in range(20):
        csa.csa_paged_attn(a, stream=side)
        for _ in range(4):                           # takes and writes what the current stream may have
            torch.full((csa.csa_paged_attn_workspace_size(a),), 0xFF, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    assert torch.equal(out, want[0]) and torch.equal(lse, want[1])


@pytest.mark.parametrize("fmt", ["fp8", "fp4"])
@pytest.mark.parametrize("H", [16, 128])
def test_bytes_of_entries_that_no_row_sees(csa, H, fmt):
    """NaN codes and scales behind the sequences' ends, before the windows and
    in pages of no sequence change no bit."""
    B = Batch(28, [(1, 300), (3, 77), (1, 1)], H, fmt, 16)
    first = _run(csa, B, B.device(csa), window=50)
    _check(*first, B.want(window=50))
    seen = np.zeros(B.pages.shape[:2], dtype=bool)
    for b, (n, T) in enumerate(B.lens):
        for p in range(max(0, T - n - 49), T):
            seen[B.table[b, p // 16], p % 16] = True
    B.pages[~seen] = 0xFF
    again = _run(csa, B, B.device(csa), window=50)
    assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


@pytest.mark.parametrize("H", [2, 128])
def test_more_than_a_thousand_sequences(csa, H):
    """The plan's sums over groups of sequences, in both kernels."""
    rng = np.random.default_rng(29)
    lens = [(int(n), int(n) + int(T)) for n, T in zip(rng.integers(0, 3, 1100), rng.integers(0, 90, 1100))]
    B = Batch(29, lens, H, "fp4", 16)
    out, lse = _run(csa, B, B.device(csa), sink=B.sink)
    _check(out, lse, B.want(sink=B.sink))


def _check_far_logits(B, out, lse, scale, sink=None):
    """Logits so large that their own error is many units (2^-18 of the sum of
    magnitudes, plus 2^-22 of the logit for its scaling).  A row whose largest
    logit leads the others by 40 beyond both errors takes that entry alone: the
    others' weights are below e^-40, so out is x_e within the weight's and the
    output's rounding, 2^-11 + 2^-8, and e^-40 of the sum of magnitudes; lse is
    the logit within its error.  The other rows are finite, and no larger than
    the largest entry.  A sink is one more logit whose entry is zero.  Returns
    the number of rows with such a leader."""
    led = 0
    g, gl = out.double().cpu().numpy(), lse.double().cpu().numpy()
    q, sc = B.q.double().numpy(), float(np.float32(scale))
    for r, (b, p) in enumerate(row_positions(B.cu, B.kv)):
        kp, X = gather(B.pages, B.table, b, range(0, p + 1))
        X = np.concatenate([X, np.zeros((1, 512))])                 # the sink's
        logit = sc * (q[r] @ X.T)
        err = 2.0 ** -18 * sc * (np.abs(q[r]) @ np.abs(X).T) + 2.0 ** -22 * np.abs(logit)
        logit[:, -1] = -np.inf if sink is None else sink
        assert np.all(np.isfinite(g[r])) and np.all(np.isfinite(gl[r])), (r, p)
        size = np.abs(X).max(0)
        assert np.all(np.abs(g[r]) <= size * (1 + 2.0 ** -7)), (r, p)
        for h in range(B.H):
            e = int(np.argmax(logit[h]))
            rest = np.delete(logit[h] + err[h], e)
            if len(rest) and logit[h, e] - err[h, e] - rest.max() < 40:
                continue
            led += 1
            tol = (2.0 ** -8 + 2.0 ** -11) * np.abs(X[e]) + np.exp(-40.0) * np.abs(X).sum(0)
            assert np.all(np.abs(g[r, h] - X[e]) <= tol), (r, p, h)
            assert abs(gl[r, h] - logit[h, e]) <= err[h, e] + 2.0 ** -20 * (1 + abs(logit[h, e])), (r, p, h)
    return led


def _set_entries(B, b, x):
    e = _encode(x.astype(np.float32), B.fmt)
    for p in range(0, len(e), B.page):
        k = min(B.page, len(e) - p)
        B.pages[B.table[b, p // B.page], :k] = e[p:p + k]


FAR = [(2.0, 1.0, 2.0 ** 20), (2.0, 1.0, 2.0 ** 23), (2.0, 1.0, 1e12), (2.0, 1.0, 1e26), ("most", "most", 1e26)]


@pytest.mark.parametrize("few", [False, True])
@pytest.mark.parametrize("fmt", ["fp8", "fp4"])
@pytest.mark.parametrize("case", range(len(FAR)))
def test_logits_far_past_fp32_integers(csa, case, fmt, few):
    """Logits up to the largest that fp32 holds (times log2 e), with maxima that
    grow along the cache: in base 2 they are past 2^24, where neighbouring fp32
    values are whole units apart."""
    gain, spread, scale = FAR[case]
    lens = [(4, 900), (2, 130), (3, 3)]
    H = 16 if few else 32
    B = Batch(400 + case, _thin(lens, H) if few else lens, H, fmt, 16)
    rng = np.random.default_rng(500 + case)
    top = 6e4 if fmt == "fp8" else 2600.0                  # an FP4 entry decodes to at most 2688
    if gain == "most":
        q = np.clip(rng.standard_normal(B.q.shape) * 2e4, -65024, 65024)
        q[3, 0] = 65024 * np.where(rng.random(512) < 0.5, -1, 1)
        B.q = torch.from_numpy(q.astype(np.float32)).to(torch.bfloat16)
    for b, (n, T) in enumerate(lens):
        if gain == "most":
            x = np.clip(rng.standard_normal((T, 512)) * top / 4, -top, top)
            if b == 0:                                     # the largest products there are, of either sign
                x[333], x[777] = -top * np.sign(q[3, 0]), top * np.sign(q[3, 0])
        else:
            x = rng.standard_normal((T, 512)) * np.linspace(0.05, 6.0, T)[:, None]
        _set_entries(B, b, x)
    kv = B.device(csa)
    for sink in (None, B.sink):
        out, lse = _run(csa, B, kv, sink=sink, scale=scale)
        assert _check_far_logits(B, out, lse, scale, sink) > 9 * H // 2


@pytest.mark.parametrize("few", [False, True])
@pytest.mark.parametrize("scale", [2.0 ** 20, 1e9, 1e26])
def test_far_logits_that_are_all_the_same(csa, few, scale):
    """Every entry of the cache alike: any weights give that entry."""
    B = Batch(410, _thin([(3, 500)], 32) if few else [(3, 500)], 32, "fp8", 16)
    x = np.random.default_rng(9).standard_normal((1, 512))
    _set_entries(B, 0, np.repeat(x, 500, 0))
    out, lse = _run(csa, B, B.device(csa), scale=scale)
    _, X = gather(B.pages, B.table, 0, range(1))
    logit = float(np.float32(scale)) * (B.q.double().numpy() @ X[0])
    size = float(np.float32(scale)) * (np.abs(B.q.double().numpy()) @ np.abs(X[0]))
    # the weights' rounding is the same for all: at most 2^-11, and 2^-8 of the output's
    assert np.all(np.abs(out.double().cpu().numpy() - X[0]) <= (2.0 ** -8 + 2.0 ** -11) * np.abs(X[0]))
    n = np.array([498, 499, 500])[:, None]
    assert np.all(np.abs(lse.double().cpu().numpy() - logit - np.log(n)) <= 2.0 ** -18 * size + 2.0 ** -20 * (1 + np.abs(logit)))


def test_thousands_of_items_of_one_tile_and_of_none(csa):
    """A window of one entry: items as short as they get, over which every warp
    has to keep up or not matter, with items between them that see nothing.  A
    row's output is its own entry (weight 1: rounded by 2^-11 and 2^-8)."""
    B = Batch(31, [(900, 900), (600, 200), (5, 5), (700, 3000)], 128, "fp8", 16)
    q = B.q.cuda()
    for _ in range(3):
        out, lse = _run(csa, B, B.device(csa), window=1, q=q)
    X, seen = torch.zeros(B.rows, 512), np.zeros(B.rows, dtype=bool)
    for r, (b, p) in enumerate(row_positions(B.cu, B.kv)):
        if p >= 0:
            X[r] = torch.from_numpy(gather(B.pages, B.table, b, [p])[1][0])       # E4M3 times a power of two: exact
            seen[r] = True
    X = X.cuda()
    for i in range(0, B.rows, 256):
        x = X[i:i + 256].double()[:, None]
        assert bool(((out[i:i + 256].double() - x).abs() <= (2.0 ** -8 + 2.0 ** -11) * x.abs()).all())
        z = q[i:i + 256].double() * x
        want, size = 512 ** -0.5 * z.sum(-1), 512 ** -0.5 * z.abs().sum(-1)
        on = torch.from_numpy(seen[i:i + 256]).cuda()
        assert bool((((lse[i:i + 256].double() - want).abs() <= 2.0 ** -17 * size + 2.0 ** -18 * (1 + want.abs()))[on]).all())
        assert bool(torch.isneginf(lse[i:i + 256][~on]).all())


@pytest.mark.parametrize("few", [False, True])
@pytest.mark.parametrize("T,gain", [(130, 2.0), (900, 0.5)])
def test_channels_far_larger_than_the_others(csa, T, gain, few):
    """Channels of 20 times the others' size, whose weighted sums cancel: the
    weights' rounding to fp16 shows there, within its bound."""
    lens = [(5, T), (2, 40)]
    B = Batch(420, _thin(lens, 64) if few else lens, 64, "fp8", 64, q_gain=gain)
    rng = np.random.default_rng(5)
    big = rng.choice(512, 16, replace=False)
    for b, (_, n) in enumerate(lens):
        x = rng.standard_normal((n, 512))
        x[:, big] *= 20
        _set_entries(B, b, x)
    out, lse = _run(csa, B, B.device(csa))
    _check(out, lse, B.want())


@pytest.mark.parametrize("few", [False, True])
def test_block_exponents_of_the_largest_entries(csa, few):
    """Exponent bytes 143 to 151, past fp16's powers of two, with the codes that
    stay under 65504 (a bit or four each: exact in fp16), beside bytes 103 and
    on, and 0."""
    B = Batch(421, _thin([(3, 200)], 16) if few else [(3, 200)], 16, "fp8", 16)
    codes = np.array([c for c in range(256) if c & 0x7F != 0x7F])
    size = np.abs(fp8_window_dequant_rows(np.concatenate([np.resize(codes, 512), np.full(16, 127)])[None].astype(np.uint8))[0, :len(codes)])
    rng = np.random.default_rng(6)
    for p in range(200):
        row = B.pages[B.table[0, p // 16], p % 16]
        row[512:] = np.where(rng.random(16) < 0.6, rng.integers(143, 152, 16), rng.integers(103, 143, 16))
        row[512 + p % 16] = 0
        for k in range(16):
            few_bits = codes[size * 2.0 ** (int(row[512 + k]) - 127) < 65504]
            row[32 * k:32 * k + 32] = rng.choice(few_bits, 32)
    x = gather(B.pages, B.table, 0, range(200))[1]
    assert 32768 <= np.abs(x).max() < 65504
    out, lse = _run(csa, B, B.device(csa), scale=1e-6)
    # byte 0 is 2^-127: below 448 * 2^-127, zero in fp16
    want = B.want(scale=1e-6)
    _check(out, lse, (want[0], want[1], want[2] + 2.0 ** -100, want[3], want[4]))


@pytest.mark.parametrize("H", [16, 128])
def test_attention_without_lse(csa, H):
    B = Batch(422, [(1, 700), (1, 0), (1, 33)], H, "fp8", 16)
    kv = B.device(csa)
    for sink in (None, torch.from_numpy(B.sink).cuda()):
        outs = []
        for lse in (None, torch.empty(3, H, device="cuda")):
            out = torch.full((3, H, 512), 3.0, dtype=torch.bfloat16, device="cuda")
            csa.csa_paged_attn(csa.paged_attn_args(q=B.q.cuda(), kv=kv, out=out, lse=lse, softmax_scale=0.04, sink=sink))
            outs.append(out)
        torch.cuda.synchronize()
        assert torch.equal(*outs)


@pytest.mark.parametrize("few", [False, True])
def test_a_query_out_of_range_spoils_its_own_row(csa, few):
    """NaN, infinite and too large queries, and logits past fp32: no bit of the
    other rows of their items changes."""
    lens = [(6, 300), (2, 70)]
    H = 16
    B = Batch(423, _thin(lens, H) if few else lens, H, "fp8", 16)
    B.pages[B.table[0, 0], 5, :512] = 0x7E                # an entry of 448 * 2^7 throughout
    B.pages[B.table[0, 0], 5, 512:] = 134
    kv = B.device(csa)
    for scale in (0.04, 1e30):
        first = _run(csa, B, kv, scale=scale)
        assert bool(torch.isfinite(first[1]).all())
        q, bad = B.q.cuda().clone(), [(0, 0), (1, 15), (4, 7), (7, 3)]
        if scale == 0.04:
            for (r, h), v in zip(bad, (float("nan"), float("inf"), -1e38, 1e30)):
                q[r, h, 3 * h:3 * h + 40] = v
        else:                                              # |<q, x>| about 22 * 6e4 * 57344: times 1e30 past fp32
            for r, h in bad:
                q[r, h] = 6e4 * torch.sign(q[r, h])
        again = _run(csa, B, kv, scale=scale, q=q)
        keep = torch.ones(B.rows, H, dtype=torch.bool, device="cuda")
        for r, h in bad:
            keep[r, h] = False
        assert torch.equal(first[0][keep], again[0][keep]) and torch.equal(first[1][keep], again[1][keep])


# -------------------------------------------------------------------- append
def _append(csa, B, src, n_rows=None, **kw):
    kv = B.device(csa)
    csa.csa_paged_append(csa.paged_append_args(src=src, kv=kv, **kw))
    torch.cuda.synchronize()
    return B.d["pages"].cpu().numpy()


APPENDS = [([(1, 1)], 16), ([(3, 50), (0, 7), (1, 16), (20, 20)], 16), ([(1, 100)] * 40, 7), ([(300, 1000), (5, 5)], 64),
           ([(1, 3)] * 1200, 16)]


@pytest.mark.parametrize("fmt", ["fp8", "fp4"])
@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("case", range(len(APPENDS)))
def test_append_without_norm_is_the_encoder(csa, fmt, dtype, case):
    """Bit for bit the entries of csa_quant_kv's definition, and nothing else touched."""
    lens, page = APPENDS[case]
    B = Batch(30 + case, lens, 1, fmt, page)
    x = torch.from_numpy(np.random.default_rng(case).standard_normal((B.rows + 3, 512)).astype(np.float32) * 5).to(getattr(torch, dtype)).cuda()
    want = B.pages.copy()
    enc = _encode(x.float().cpu().numpy(), fmt)
    for r, (b, p) in enumerate(row_positions(B.cu, B.kv)):
        want[entry_of(B.table, page, B.n_pages, b, p)] = enc[r]
    assert np.array_equal(_append(csa, B, x), want)


@pytest.mark.parametrize("fmt", ["fp8", "fp4"])
@pytest.mark.parametrize("weight", [False, True])
@pytest.mark.parametrize("rope", [False, True])
def test_append_norm_and_rope(csa, fmt, weight, rope):
    """Decoded entries within half a step of the exact normed and rotated row:
    FP8 2^-4 relative or 2^-10 of the block's scale; FP4 half the E2M1 step at
    the value (at most 1/4 of it, or 1/4 of the scale), plus the clipping that
    a scale rounded down by 2^-4 causes; 2^-17 for the fp32 arithmetic."""
    lens = [(9, 60), (30, 30), (1, 77)]
    B = Batch(40, lens, 1, fmt, 16)
    rng = np.random.default_rng(6)
    x = torch.from_numpy((rng.standard_normal((B.rows, 512)) * 4).astype(np.float32)).to(torch.bfloat16).cuda()
    w = (1 + 0.3 * rng.standard_normal(512)).astype(np.float32)
    pages = _append(csa, B, x, norm=True, eps=1e-5, weight=torch.from_numpy(w).cuda() if weight else None,
                    rope_cs=torch.from_numpy(B.cs).cuda() if rope else None)
    _, y = rms_norm(x.double().cpu().numpy(), 1e-5, w if weight else None)
    if rope:
        y = np.concatenate([orope.rotate(y[i:i + 1], B.cs[i]) for i in range(B.rows)])
    raw = np.stack([pages[entry_of(B.table, 16, B.n_pages, b, p)] for b, p in row_positions(B.cu, B.kv)])
    if fmt == "fp8":
        got, s = fp8_window_dequant_rows(raw), np.repeat(np.ldexp(1.0, raw[:, 512:].astype(int) - 127), 32, axis=1)
        tol = np.maximum(2.0 ** -4 * np.abs(y), 2.0 ** -10 * s)
        amax = np.abs(y).reshape(-1, 16, 32).max(2)
        assert np.all(amax <= 448 * s[:, ::32] * (1 + 2.0 ** -17)) and np.all(amax >= 224 * s[:, ::32] * (1 - 2.0 ** -17))
    else:
        got = fp4_dequant_rows(raw)
        amax = np.repeat(np.abs(y).reshape(-1, 32, 16).max(2), 16, axis=1)
        s = amax / 6
        tol = np.maximum(0.25 * s * (1 + 2.0 ** -4), np.minimum(np.abs(y) / 4, s) * (1 + 2.0 ** -4)) + 2.0 ** -4 * np.abs(y)
    assert np.all(np.abs(got - y) <= tol + 2.0 ** -17 * np.abs(y)), float((np.abs(got - y) - tol).max())
    # and the rows' neighbours in their pages stay
    touched = np.zeros(B.pages.shape[:2], dtype=bool)
    for b, p in row_positions(B.cu, B.kv):
        touched[entry_of(B.table, 16, B.n_pages, b, p)] = True
    assert np.array_equal(pages[~touched], B.pages[~touched])


def test_append_skips_what_has_no_entry(csa):
    """Negative positions, missing pages, positions past the table, rows behind
    the last sequence: nothing is written for them."""
    B = Batch(41, [(6, 6), (4, 64), (3, 3)], 1, "fp8", 16, tail_rows=5)
    B.kv = np.array([2, 64, 2 ** 31 - 1], dtype=np.int32)
    B.table[1, 3] = B.n_pages
    x = torch.randn(B.rows, 512, device="cuda")
    want = B.pages.copy()
    enc = _encode(x.cpu().numpy(), "fp8")
    for r in (4, 5):
        want[entry_of(B.table, 16, B.n_pages, 0, r - 4)] = enc[r]
    assert np.array_equal(_append(csa, B, x), want)


class Rows:
    """Packed rows for an append of thousands: a cache of random bytes, a table
    with holes, sequences of the given (new tokens, length), padding rows."""

    def __init__(self, seed, lens, fmt, page, dtype):
        rng = np.random.default_rng(seed)
        self.lens, self.fmt, self.page = lens, fmt, page
        need = [max(0, -(-T // page)) for _, T in lens]
        self.n_pages = sum(need) + 1
        ids = rng.permutation(self.n_pages).astype(np.int32)
        table = np.full((len(lens), max(need) + 1), -1, dtype=np.int32)
        for b, k in enumerate(need):
            table[b, :k] = ids[sum(need[:b]):sum(need[:b]) + k]
        holes = rng.random(table.shape) < 0.02
        self.table = np.where(holes, rng.choice([-1, self.n_pages, 2 ** 31 - 1], table.shape), table).astype(np.int32)
        self.cu = np.concatenate([[0], np.cumsum([n for n, _ in lens])]).astype(np.int32)
        self.kv = np.array([T for _, T in lens], dtype=np.int32)
        self.n = int(self.cu[-1])
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.src = (torch.randn(self.n + 5, 512, generator=g, device="cuda") * 3).to(dtype)
        self.weight = 1 + 0.2 * torch.randn(512, generator=g, device="cuda")
        angle = 6.3 * torch.rand(self.n + 5, 32, generator=g, device="cuda")
        self.cs = torch.stack([angle.cos(), angle.sin()], -1)
        self.pages = torch.randint(0, 256, (self.n_pages, page, ENTRY[fmt]), generator=g, device="cuda", dtype=torch.uint8)

    def places(self):
        """Entry number of every row (-1: none), by sequence."""
        at = np.full(self.n, -1, dtype=np.int64)
        for b, (n, T) in enumerate(self.lens):
            p = np.arange(T - n, T)
            pg = np.where(p >= 0, p // self.page, -1)
            on = (pg >= 0) & (pg < self.table.shape[1])
            g = np.where(on, self.table[b, np.where(on, pg, 0)], -1)
            on &= (g >= 0) & (g < self.n_pages)
            at[self.cu[b]:self.cu[b + 1]] = np.where(on, g.astype(np.int64) * self.page + p % self.page, -1)
        return at

    def append(self, csa, i=0, j=None, **kw):
        """Rows [i, j) (None: all, and the padding) appended to a copy of the
        cache, or to `into`."""
        pages = kw.pop("into", None)
        pages = self.pages.clone() if pages is None else pages
        e = self.n if j is None else j
        cu = np.clip(self.cu, i, e) - i
        kv_len = self.kv - (self.cu[1:] - np.clip(self.cu[1:], i, e))
        dev = lambda a: torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()  # noqa: E731
        kv = csa.paged_kv(pages=pages, block_table=dev(self.table), cu_q=dev(cu), kv_len=dev(kv_len))
        src = self.src[i:] if j is None else self.src[i:j]
        rope = self.cs[i:] if j is None else self.cs[i:j]
        csa.csa_paged_append(csa.paged_append_args(src=src, kv=kv, rope_cs=rope if kw.pop("rope", False) else None, **kw))
        torch.cuda.synchronize()
        return pages


_R = np.random.default_rng(77)
MANY = [  # from 2369 rows on a warp takes several neighbouring ones: 2, 3, 4 and 32 here, the last in several goes
    ([(2000, 2500), (0, 40), (369, 369)], 16),
    ([(1, 1)] * 20 + [(2400, 2300)] + [(0, 9)] * 5 + [(2583, 9000)], 33),
    ([(int(n), int(n) + int(t)) for n, t in zip(_R.integers(0, 250, 75), _R.integers(-20, 300, 75))], 7),
    ([(40000, 40000), (0, 1), (36011, 36100), (3, 3)], 64),
    ([(int(n), int(n)) for n in _R.integers(0, 2100, 80)], 16),
]


@pytest.mark.parametrize("fmt", ["fp8", "fp4"])
@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("case", range(len(MANY)))
def test_append_of_thousands_of_rows(csa, fmt, dtype, case):
    """Entries bit for bit csa_quant_kv's, and with norm and rotation those of
    the same rows appended 1000 at a time (a warp a row); what has no entry, and
    every other byte of the cache, stays."""
    lens, page = MANY[case]
    R = Rows(600 + case, lens, fmt, page, getattr(torch, dtype))
    assert R.n > 2368
    at = torch.from_numpy(R.places()).cuda()
    on = at >= 0
    assert bool(on.any()) and not bool(on.all())
    enc = torch.empty(R.n, ENTRY[fmt], dtype=torch.uint8, device="cuda")
    csa.csa_quant_kv(R.src[:R.n], csa.CSA_FMT_FP8_E4M3_UE8M0X32 if fmt == "fp8" else csa.CSA_FMT_FP4_E2M1_E4M3X16, enc)
    pick = np.random.default_rng(case).integers(0, R.n, 50)
    assert np.array_equal(enc[pick].cpu().numpy(), _encode(R.src[pick].float().cpu().numpy(), fmt))
    want = R.pages.clone()
    want.view(-1, ENTRY[fmt])[at[on]] = enc[on]
    assert torch.equal(R.append(csa), want)
    kw = dict(norm=True, weight=R.weight, eps=1e-5, rope=True)
    parts = R.pages.clone()
    for i in range(0, R.n, 1000):
        R.append(csa, i, min(i + 1000, R.n), into=parts, **kw)
    whole = R.append(csa, **kw)
    assert torch.equal(whole, parts)
    # those are the normed and rotated rows: a sample against float64, as above
    if fmt == "fp8":
        rows = pick[on[pick].cpu().numpy()]
        _, y = rms_norm(R.src[rows].double().cpu().numpy(), 1e-5, R.weight.double().cpu().numpy())
        y = np.concatenate([orope.rotate(y[i:i + 1], R.cs[r].cpu().numpy()) for i, r in enumerate(rows)])
        raw = whole.view(-1, 528)[at[rows]].cpu().numpy()
        s = np.repeat(np.ldexp(1.0, raw[:, 512:].astype(int) - 127), 32, axis=1)
        err = np.abs(fp8_window_dequant_rows(raw) - y)
        assert np.all(err <= np.maximum(2.0 ** -4 * np.abs(y), 2.0 ** -10 * s) + 2.0 ** -17 * np.abs(y))


@pytest.mark.parametrize("H", [2, 72])
def test_the_most_sequences_of_a_call(csa, H):
    """65536 sequences of one entry each, half of them with a new token (H = 2)
    or all (H = 72: the kernel for many rows), behind 7 rows of no sequence:
    append writes every entry, attention gives it back."""
    B, page = 65536, 3
    rng = np.random.default_rng(32)
    n = (rng.random(B) < 0.5).astype(np.int32) if H == 2 else np.ones(B, dtype=np.int32)
    cu = torch.from_numpy((7 + np.concatenate([[0], np.cumsum(n)])).astype(np.int32)).cuda()
    rows = int(cu[-1]) + 6
    g = torch.Generator(device="cuda").manual_seed(32)
    pages = torch.full((B + 1, page, 528), 0x7E, dtype=torch.uint8, device="cuda")
    table = torch.randperm(B + 1, generator=g, device="cuda")[:B].to(torch.int32)[:, None].contiguous()
    kv = csa.paged_kv(pages=pages, block_table=table, cu_q=cu, kv_len=torch.ones(B, dtype=torch.int32, device="cuda"))
    src = torch.randn(rows, 512, generator=g, device="cuda").to(torch.bfloat16)
    enc = torch.empty(rows, 528, dtype=torch.uint8, device="cuda")
    csa.csa_quant_kv(src, csa.CSA_FMT_FP8_E4M3_UE8M0X32, enc)
    csa.csa_paged_append(csa.paged_append_args(src=src, kv=kv))
    on = torch.from_numpy(n).cuda().bool()
    want = torch.full_like(pages, 0x7E)
    want[table[on, 0].long(), 0] = enc[7:-6]
    assert torch.equal(pages, want)
    del want
    q = torch.randn(rows, H, 512, generator=g, device="cuda").to(torch.bfloat16)
    out = torch.full_like(q, 3.0)
    lse = torch.full((rows, H), 3.0, device="cuda")
    csa.csa_paged_attn(csa.paged_attn_args(q=q, kv=kv, out=out, lse=lse, softmax_scale=0.04))
    torch.cuda.synchronize()
    x = enc[:, :512].contiguous().view(torch.float8_e4m3fn).float().view(rows, 16, 32)
    x = (x * torch.exp2(enc[:, 512:].float() - 127)[:, :, None]).view(rows, 512)
    for i in range(0, rows, 4096):
        k = slice(max(i, 7), min(i + 4096, rows - 6))
        o, xx = out[k].double(), x[k].double()[:, None]
        assert bool(((o - xx).abs() <= (2.0 ** -8 + 2.0 ** -11) * xx.abs()).all())
        z = q[k].double() * xx
        l, size = 0.04 * z.sum(-1), 0.04 * z.abs().sum(-1)
        assert bool(((lse[k].double() - l).abs() <= 2.0 ** -17 * size + 2.0 ** -18 * (1 + l.abs())).all())
    for edge in (slice(0, 7), slice(rows - 6, rows)):
        assert bool((out[edge] == 3.0).all()) and bool((lse[edge] == 3.0).all())


@pytest.mark.parametrize("H", [16, 128])
def test_rows_before_the_first_sequence_stay(csa, H):
    B = Batch(33, [(3, 50), (2, 20)], H, "fp8", 16, tail_rows=4)
    kv = B.device(csa)
    want = _run(csa, B, kv, sink=B.sink)
    pages = _append(csa, B, torch.randn(B.rows, 512, generator=torch.Generator("cuda").manual_seed(1), device="cuda"))
    B.device(csa)
    B.d["cu_q"].add_(4)
    kv = csa.paged_kv(**B.d)
    q = torch.roll(B.q.cuda(), 4, 0)
    out, lse = _run(csa, B, kv, sink=B.sink, q=q)
    assert torch.equal(out[4:], want[0][:5]) and torch.equal(lse[4:], want[1][:5])
    assert bool((out[:4] == 3.0).all()) and bool((lse[:4] == 3.0).all())
    src = torch.roll(torch.randn(B.rows, 512, generator=torch.Generator("cuda").manual_seed(1), device="cuda"), 4, 0)
    csa.csa_paged_append(csa.paged_append_args(src=src, kv=kv))
    torch.cuda.synchronize()
    assert np.array_equal(B.d["pages"].cpu().numpy(), pages)


@pytest.mark.parametrize("H", [16, 128])
def test_the_largest_pages(csa, H):
    B = Batch(34, [(2, 66000), (1, 65537), (1, 65536)], H, "fp4", 65536)
    out, lse = _run(csa, B, B.device(csa), window=900)
    kp = [gather(B.pages, B.table, b, range(T - 1000, T)) for b, (_, T) in enumerate(B.lens)]
    q, r = B.q.double().numpy(), 0
    for b, (n, T) in enumerate(B.lens):
        w = attend(q[r:r + n], np.arange(T - n, T), *kp[b], 512 ** -0.5, 900)
        _check(out[r:r + n], lse[r:r + n], w)
        r += n


# ----------------------------------------------------------------- the chain
def test_norm_append_attention_as_a_layer_uses_them(csa):
    """Residual stream -> norm with 8-bit output (decoded as an 8-bit
    projection would) -> latents and queries -> append -> attention, for three
    steps: a prompt, a chunk, single tokens; each step's attention against
    float64 over the cache as the library wrote it."""
    g = torch.Generator(device="cuda").manual_seed(5)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    dim, H, page = 1024, 16, 16
    wk, wq = rnd(dim, 512) / 32, rnd(dim, H * 512) / 32
    wn, wl = 1 + 0.1 * rnd(dim), 1 + 0.1 * rnd(512)
    pages = torch.zeros(40, page, 528, dtype=torch.uint8, device="cuda")
    table = torch.randperm(40, generator=g, device="cuda").to(torch.int32).view(2, 20)
    kv_now = [0, 0]
    residual = None
    for step, new in enumerate(([37, 5], [1, 40], [1, 1], [1, 1])):
        n = sum(new)
        kv_now = [a + b for a, b in zip(kv_now, new)]
        cu = torch.tensor([0, new[0], n], dtype=torch.int32, device="cuda")
        kvl = torch.tensor(kv_now, dtype=torch.int32, device="cuda")
        x, residual = rnd(n, dim).to(torch.bfloat16), rnd(n, dim).to(torch.bfloat16)
        codes = torch.empty(n, dim, dtype=torch.uint8, device="cuda")
        sc = torch.empty(n, dim // 32, dtype=torch.uint8, device="cuda")
        csa.csa_rms_norm(csa.rms_norm_args(x=x, residual=residual, residual_out=residual, weight=wn, codes=codes, scales=sc))
        h = codes.view(torch.float8_e4m3fn).float().view(n, -1, 32) * torch.exp2(sc.float() - 127)[:, :, None]
        h = h.view(n, dim)
        lat, q = (h @ wk).to(torch.bfloat16), (h @ wq).view(n, H, 512).to(torch.bfloat16)
        pos = [kv_now[b] - new[b] + t for b in range(2) for t in range(new[b])]
        cs = torch.from_numpy(np.stack([orope.rope_angles(p) for p in pos]).astype(np.float32)).cuda()
        kv = csa.paged_kv(pages=pages, block_table=table, cu_q=cu, kv_len=kvl)
        csa.csa_paged_append(csa.paged_append_args(src=lat, kv=kv, norm=True, weight=wl, rope_cs=cs))
        out, lse = torch.empty_like(q), torch.empty(n, H, device="cuda")
        csa.csa_paged_attn(csa.paged_attn_args(q=q, kv=kv, out=out, lse=lse, softmax_scale=512 ** -0.5, rope_cs=cs))
        torch.cuda.synchronize()
        B = Batch(0, [(k, t) for k, t in zip(new, kv_now)], H, "fp8", page)
        B.pages, B.table, B.n_pages, B.q, B.cs = pages.cpu().numpy(), table.cpu().numpy(), 40, q.cpu(), cs.cpu().numpy()
        _check(out, lse, B.want(rope=True), rope=True)
        # the newest latents of the cache are the normed, rotated ones
        _, y = rms_norm(lat.double().cpu().numpy(), 1e-6, wl.double().cpu().numpy())
        y = np.concatenate([orope.rotate(y[i:i + 1], B.cs[i]) for i in range(n)])
        raw = np.stack([B.pages[entry_of(B.table, page, 40, b, p)] for b, p in row_positions(B.cu, B.kv)])
        s = np.repeat(np.ldexp(1.0, raw[:, 512:].astype(int) - 127), 32, axis=1)
        err = np.abs(fp8_window_dequant_rows(raw) - y)
        assert np.all(err <= np.maximum(2.0 ** -4 * np.abs(y), 2.0 ** -10 * s) + 2.0 ** -17 * np.abs(y))


def test_norm_append_attention_in_a_graph(csa):
    """The same chain for a decode step, captured once and replayed while the
    caches grow by a token a step, against the chain call by call."""
    lens = [(1, 60), (1, 30), (1, 77)]
    res = []
    for graph in (False, True):
        B = Batch(30, lens, 16, "fp8", 16)
        kv = B.device(csa)
        gen = torch.Generator(device="cuda").manual_seed(5)
        src = torch.randn(3, 512, generator=gen, device="cuda")
        y, q = torch.empty_like(src), B.q.cuda()
        w = torch.rand(512, generator=gen, device="cuda") + 0.5
        cs = torch.from_numpy(B.cs).cuda()
        out, lse = torch.empty(3, 16, 512, dtype=torch.bfloat16, device="cuda"), torch.empty(3, 16, device="cuda")
        n = csa.rms_norm_args(x=src, out=y, weight=w)
        p = csa.paged_append_args(src=y, kv=kv, norm=True, weight=w, rope_cs=cs)
        a = csa.paged_attn_args(q=q, kv=kv, out=out, lse=lse, softmax_scale=0.04, rope_cs=cs)
        ws = torch.empty(csa.csa_paged_attn_workspace_size(a), dtype=torch.uint8, device="cuda")

        def step():
            csa.csa_rms_norm(n)
            csa.csa_paged_append(p)
            csa.csa_paged_attn(a, workspace=ws)

        got = []
        if graph:
            g = torch.cuda.CUDAGraph()
            torch.cuda.synchronize()
            with torch.cuda.graph(g):
                step()
        for i in range(4):
            g.replay() if graph else step()
            torch.cuda.synchronize()
            got.append((out.clone(), lse.clone(), B.d["pages"].clone()))
            B.d["kv_len"].add_(1)
            src.mul_(-1.5)
        res.append(got)
    for one, two in zip(*res):
        assert all(torch.equal(u, v) for u, v in zip(one, two))
    assert csa.device_status() == 0
