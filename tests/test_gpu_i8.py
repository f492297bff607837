"""The 8-bit projection path (gdn_quantize_i8, gdn_add_rms_norm_i8,
gdn_linear_i8) on the GPU against its definition in numpy.

The integers are decided exactly by the definition, and the product's sums are
exact, so integers, residuals and products are compared bit for bit. Scales are
formed in double and rounded to fp32 once: half a step, 2^-24 relative, plus
the double sum's own error (D 2^-53 for D up to 131056: below 2^-35)."""
import numpy as np
import pytest
import torch

import i8_reference as ref
import i8_shapes
import oracle
from linear_attention_recurrence_04_b200 import gdn, inputs
from parity import assert_parity

pytestmark = pytest.mark.gpu

SCALE_RTOL = 2.0 ** -24 * (1 + 2.0 ** -10)
F32, BF16 = torch.float32, torch.bfloat16


def draw_rows(M, D, seed, dtype=F32):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(M, D, generator=g) * torch.exp(torch.randn(M, 1, generator=g))
    x = torch.where(torch.rand(1, D, generator=g) < 0.02, 10 * x, x)
    return x.to(dtype)


def check_rows(q, scale, want_q, want_scale):
    torch.cuda.synchronize()
    assert np.array_equal(q.cpu().numpy(), want_q)
    s = scale.cpu().numpy().astype(np.float64)
    assert np.array_equal(np.isnan(s), np.isnan(want_scale))
    ok = ~np.isnan(s)
    # a scale below the least normal fp32 is off by half a step of 2^-149
    assert np.all(np.abs(s[ok] - want_scale[ok]) <= np.maximum(want_scale[ok] * SCALE_RTOL, 2.0 ** -150))


SHAPES = [(1, 16), (3, 16), (300, 48), (1, 2048), (5, 4112), (130, 2048), (33, 8192), (2, 16384),
          (2, 32768), (3, 32784), (1, 131056), (0, 64), (4, 0)]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("M,D", SHAPES)
def test_quantize(M, D, dtype):
    x = draw_rows(M, D, seed=M + D, dtype=dtype)
    q, s = gdn.quantize_i8(x.cuda())
    if M * D:
        check_rows(q, s, *ref.rows(x.float().numpy())[:2])
    assert q.shape == (M, D) and s.shape == (M,)


@pytest.mark.parametrize("res", [None, F32, BF16])
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("M,D", SHAPES)
def test_add_rms_norm(M, D, dtype, res):
    x = draw_rows(M, D, seed=M + D, dtype=dtype)
    r = None if res is None else 3 * draw_rows(M, D, seed=M + D + 1, dtype=res)
    w = 1 + 0.2 * draw_rows(1, max(D, 1), seed=5)[0, :D]
    q, s, h = gdn.add_rms_norm_i8(x.cuda(), w.cuda(), None if r is None else r.cuda(), eps=1e-5)
    if M * D:
        wq, ws, wh = ref.rows(x.float().numpy(), None if r is None else r.float().numpy(), w.numpy(),
                              1e-5, res is BF16)
        check_rows(q, s, wq, ws)
        if r is not None:
            assert h.dtype == res and np.array_equal(h.float().cpu().numpy(), wh)
    assert (h is None) == (r is None)


@pytest.mark.parametrize("M,D", [(7, 2048), (2, 32784)])
def test_add_rms_norm_in_place_and_first_layer(M, D):
    """residual_out may be the residual; without a residual it receives the
    row in its own type, and the norm reads that rounded row."""
    x, r = draw_rows(M, D, 1), draw_rows(M, D, 2, BF16)
    w = torch.ones(D)
    wq, ws, wh = ref.rows(x.numpy(), r.float().numpy(), w.numpy(), residual_bf16=True)
    rc = r.cuda()
    q, s, h = gdn.add_rms_norm_i8(x.cuda(), w.cuda(), rc, rc)
    check_rows(q, s, wq, ws)
    assert h is rc and np.array_equal(rc.float().cpu().numpy(), wh)
    out = torch.empty(M, D, dtype=BF16, device="cuda")
    q, s, h = gdn.add_rms_norm_i8(x.cuda(), w.cuda(), residual_out=out)
    wq, ws, wh = ref.rows(x.numpy(), None, w.numpy(), residual_bf16=True)
    check_rows(q, s, wq, ws)
    assert np.array_equal(out.float().cpu().numpy(), wh)


def special_rows(D=64):
    x = np.zeros((14, D), np.float32)
    g = np.random.default_rng(3)
    x[1:] = g.standard_normal((13, D))
    x[2, 5] = np.nan
    x[3, 7] = np.inf
    x[4, 9] = -np.inf
    x[5] *= 1e-42                                  # subnormal
    x[6] *= 1e-31
    x[7] *= np.float32(1e38)
    x[8] = 0
    x[8, 3] = 1e-45                                # the least positive number alone
    x[9] = -x[9, 0]                                # every value the largest
    x[10, 1:] = 0
    x[11, :] = -0.0
    x[12, 0] = np.finfo(np.float32).max            # the largest number
    x[13, 2], x[13, 3] = np.nan, np.inf
    return x


def test_special_values():
    """Zero rows, infinities and NaN, subnormal and huge rows."""
    x = special_rows()
    q, s = gdn.quantize_i8(torch.from_numpy(x).cuda())
    check_rows(q, s, *ref.rows(x)[:2])
    s = s.cpu().numpy()
    assert s[0] == 0 and s[11] == 0 and np.isnan(s[[2, 3, 4, 13]]).all()
    w = np.ones(x.shape[1], np.float32)
    q, s, h = gdn.add_rms_norm_i8(torch.from_numpy(x).cuda(), torch.from_numpy(w).cuda(),
                                  residual_out=torch.empty(x.shape, device="cuda"))
    check_rows(q, s, *ref.rows(x, None, w)[:2])
    assert np.array_equal(h.cpu().numpy(), x, equal_nan=True)
    # a residual that brings the NaN; a weight of zero leaves an empty row
    r = np.zeros_like(x)
    r[1, 1] = np.nan
    q, s, _ = gdn.add_rms_norm_i8(torch.from_numpy(x).cuda(), torch.from_numpy(0 * w).cuda(),
                                  torch.from_numpy(r).cuda())
    check_rows(q, s, *ref.rows(x, r, 0 * w)[:2])
    # the products of a row that is not finite are NaN, of an empty row zero
    qx, sx = gdn.quantize_i8(torch.from_numpy(x).cuda())
    y = gdn.linear_i8(qx, sx, torch.ones(3, 64, dtype=torch.int8, device="cuda"),
                      torch.ones(3, device="cuda")).cpu().numpy()
    assert np.isnan(y[[2, 3, 4, 13]]).all() and (y[[0, 11]] == 0).all()


def test_borders():
    """Values on a half and one step to either side of it: with m = 254 s and
    a = (2 k + 1) s, 127 a / m is exactly k + 1/2."""
    rows = []
    for s in (1.0, 3.0, 0.1, 8388607.0, 1e-20, 1.7e-36, 1e30):
        s = np.float32(s)
        s = np.float32(s - np.fmod(s, np.spacing(s) * 256))   # (2 k + 1) s and 254 s exact
        k = np.arange(127, dtype=np.float32)
        a = (2 * k + 1) * s
        row = np.concatenate([[254 * s], a, np.nextafter(a, np.float32(0)),
                              np.nextafter(a, np.float32(np.inf)), -a]).astype(np.float32)
        rows.append(np.pad(row, (0, 512 - row.size)))
    x = np.stack(rows)
    q, s = gdn.quantize_i8(torch.from_numpy(x).cuda())
    check_rows(q, s, *ref.rows(x)[:2])
    assert (ref.rows(x)[0][0, 1:128] == np.rint(np.arange(127) + 0.5)).all()


def test_every_bf16_quotient():
    """Rows of bf16 values with every pair of 8-bit mantissas at every distance
    of exponents that leaves an integer but zero: all their halves are exact."""
    a = torch.arange(128, 256, dtype=F32)
    a = torch.cat([a * 2.0 ** -s for s in range(9)])
    a = torch.cat([a, -a, torch.zeros(16 - (2 * a.numel() + 1) % 16)])
    x = torch.stack([torch.cat([torch.tensor([float(m)]), torch.where(a.abs() <= m, a, 0 * a)])
                     for m in range(128, 256)])
    for scale in (1.0, 2.0 ** -60, 2.0 ** -110, 2.0 ** 112, 2.0 ** 120):
        xb = (x * scale).to(BF16)
        assert torch.equal(xb.double(), x.double() * scale)
        want = ref.rows(xb.float().numpy())
        for t in (xb, xb.float()):
            check_rows(*gdn.quantize_i8(t.cuda()), *want[:2])


@pytest.mark.parametrize("M,D", [(3, 2048), (2, 32784)])
def test_residual_without_its_output(M, D):
    """The C entry point takes a residual and leaves residual_out out."""
    x, r, w = draw_rows(M, D, 1).cuda(), draw_rows(M, D, 2, BF16).cuda(), torch.ones(D, device="cuda")
    q, s = torch.empty(M, D, dtype=torch.int8, device="cuda"), torch.empty(M, device="cuda")
    assert gdn.load_library().gdn_add_rms_norm_i8(
        x.data_ptr(), 0, r.data_ptr(), w.data_ptr(), 1e-6, None, 1, q.data_ptr(), s.data_ptr(), M, D,
        torch.cuda.current_stream().cuda_stream) == 0
    check_rows(q, s, *ref.rows(x.cpu().numpy(), r.float().cpu().numpy(), np.ones(D), residual_bf16=True)[:2])


@pytest.mark.parametrize("M", [1, 4, 1000])
def test_rows_of_no_elements(M):
    """D = 0: the empty row's maximum is 0, so its scale is 0."""
    x, w = torch.empty(M, 0, device="cuda"), torch.empty(0, device="cuda")
    buf = torch.full((M + 1,), 7.0, device="cuda")
    for call in (lambda: gdn.quantize_i8(x, scale=buf[:M]),
                 lambda: gdn.add_rms_norm_i8(x.to(BF16), w, x, scale=buf[:M])):
        buf.fill_(7.0)
        call()
        assert buf.tolist() == [0.0] * M + [7.0]


def test_rows_independent_of_batch():
    x = draw_rows(1000, 2048, 9).cuda()
    q, s = gdn.quantize_i8(x)
    w = torch.ones(2048, device="cuda")
    qn, sn, _ = gdn.add_rms_norm_i8(x, w)
    for r in (0, 499, 999):
        q1, s1 = gdn.quantize_i8(x[r:r + 1].contiguous())
        assert torch.equal(q1[0], q[r]) and torch.equal(s1[0], s[r])
        q1, s1, _ = gdn.add_rms_norm_i8(x[r:r + 1].contiguous(), w)
        assert torch.equal(q1[0], qn[r]) and torch.equal(s1[0], sn[r])


# Rows whose scale lies next to the middle of two fp32 numbers: adding the
# squares in another order (by the thread of a kernel with one group of 8 a
# thread, or with two) moves it to the other one. (seed, weight of element 0)
AT_A_BORDER = [(1308, "0x1.4994cep+3"), (14429, "0x1.8e006cp+3"), (4424, "0x1.7f6314p+3"),
               (10448, "0x1.787908p+3")]


@pytest.mark.parametrize("seed,top", AT_A_BORDER)
def test_norm_scale_independent_of_batch(seed, top):
    """The scale of a row is the same number in every batch, to the last bit:
    alone, below and above 2^20 groups of 8, and in each place of the batch."""
    D = 8192
    row = torch.randn(D, generator=torch.Generator().manual_seed(seed)).clamp(-4, 4)
    row[0] = 1.0
    w = torch.ones(D)
    w[0] = float.fromhex(top)
    row, w = row.cuda(), w.cuda()
    q1, s1, _ = gdn.add_rms_norm_i8(row[None], w)
    check_rows(q1, s1, *ref.rows(row.cpu().numpy()[None], None, w.cpu().numpy())[:2])
    for M in (2, 1023, 1024, 1500):
        q, s, _ = gdn.add_rms_norm_i8(row.expand(M, D).contiguous(), w)
        assert torch.equal(s, s1.expand(M)) and torch.equal(q, q1.expand(M, D))


# (types, D, the number of rows from which a thread takes more groups): the first
# row count on the other side of 2^20 groups of 8, or of the next limit of D
FEW_AND_MANY = [(F32, None, 8192, 1024), (F32, F32, 4112, 2041), (F32, BF16, 6000, 1399),
                (BF16, F32, 4112, 2041), (BF16, BF16, 2048, 4096), (BF16, BF16, 2064, 4065),
                (BF16, BF16, 8192, 1024), (BF16, BF16, 16368, 513), (F32, BF16, 16384, 512),
                (F32, None, 1024, 8192), (BF16, BF16, 2032, 4129)]


@pytest.mark.parametrize("xt,rt,D,M", FEW_AND_MANY)
def test_norm_of_few_and_many_rows(xt, rt, D, M):
    """Whole rows against the definition just below and just above the number
    of rows from which a thread takes more of a row; the residual in place and
    beside it; and every row the same on both sides."""
    x = draw_rows(M, D, D + M, xt)
    r = None if rt is None else 3 * draw_rows(M, D, D + M + 1, rt)
    w = 1 + 0.2 * draw_rows(1, D, seed=5)[0]
    pick = np.r_[0:4, M // 2, M - 3:M]
    want = ref.rows(x.float().numpy()[pick], None if r is None else r.float().numpy()[pick], w.numpy(),
                    residual_bf16=rt is BF16)
    xc, rc, wc = x.cuda(), None if r is None else r.cuda(), w.cuda()
    q, s, h = gdn.add_rms_norm_i8(xc, wc, rc)
    check_rows(q[pick], s[pick], *want[:2])
    assert rt is None or np.array_equal(h[pick].float().cpu().numpy(), want[2])
    few = M - 1
    r2 = None if rt is None else rc[:few].clone()
    q2, s2, h2 = gdn.add_rms_norm_i8(xc[:few], wc, r2, r2)
    assert torch.equal(q2, q[:few]) and torch.equal(s2, s[:few])
    assert rt is None or (h2 is r2 and torch.equal(h2, h[:few]))
    if rt is not None:                                   # the large batch in place too
        q2, s2, _ = gdn.add_rms_norm_i8(xc, wc, rc, rc)
        assert torch.equal(q2, q) and torch.equal(s2, s) and torch.equal(rc, h)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("D,M", [(512, 16384), (528, 15888), (1008, 8323), (1024, 8192), (4096, 2048),
                                 (8208, 1023), (16368, 513)])
def test_quantize_few_and_many_rows(D, M, dtype):
    x = draw_rows(M, D, D + M, dtype)
    pick = np.r_[0:4, M // 2, M - 3:M]
    xc = x.cuda()
    q, s = gdn.quantize_i8(xc)
    check_rows(q[pick], s[pick], *ref.rows(x.float().numpy()[pick])[:2])
    q2, s2 = gdn.quantize_i8(xc[:M - 1])
    assert torch.equal(q2, q[:M - 1]) and torch.equal(s2, s[:M - 1])


# -- the product ------------------------------------------------------------------

def draw_product(M, N, K, seed):
    g = torch.Generator().manual_seed(seed)
    x = torch.randint(-128, 128, (M, K), generator=g, dtype=torch.int8)
    w = torch.randint(-128, 128, (N, K), generator=g, dtype=torch.int8)
    sx = torch.exp(torch.randn(M, generator=g)) / 127
    sw = torch.exp(torch.randn(N, generator=g)) / 127 / max(K, 1) ** 0.5
    return x, sx, w, sw


def check_product(M, N, K, dtype, seed=0, rows=None):
    x, sx, w, sw = draw_product(M, N, K, seed + M + 3 * N + 7 * K)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    pad = torch.full(((M + 2) * N + 8,), 7.0, dtype=dtype, device="cuda")
    y = gdn.linear_i8(x.cuda(), sx.cuda(), w.cuda(), sw.cuda(), pad[:M * N].view(M, N),
                      status=status)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    assert (pad[M * N:] == 7.0).all(), "written behind the last row"
    rows = slice(None) if rows is None else rows
    want = ref.linear(x.numpy()[rows], sx.numpy()[rows], w.numpy(), sw.numpy(), dtype is BF16)
    got = y.float().cpu().numpy()[rows]
    assert np.array_equal(got, want), np.argwhere(got != want)[:4].tolist()


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("M,N,K", [
    (1, 1, 16), (1, 8, 16), (2, 1, 2048), (3, 5, 144), (1, 8192, 2048), (15, 130, 1040),
    (16, 128, 128), (17, 127, 256), (33, 64, 2048), (64, 4096, 2048), (65, 2050, 512),
    (100, 300, 4096), (128, 257, 1008), (129, 64, 2048), (200, 1000, 272), (255, 255, 400),
    (256, 64, 2048), (300, 4100, 1040), (513, 2048, 4096), (777, 2050, 1040), (2049, 33, 160),
])
def test_linear(M, N, K, dtype):
    check_product(M, N, K, dtype)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("M,N,K,tile,splits", i8_shapes.SPLIT)
def test_linear_split(M, N, K, tile, splits, dtype):
    check_product(M, N, K, dtype)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("M,N,K,tokens,warps", i8_shapes.VEC)
def test_linear_vec(M, N, K, tokens, warps, dtype):
    check_product(M, N, K, dtype)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("M,N,K,tile", i8_shapes.PAIR)
def test_linear_pair(M, N, K, tile, dtype):
    check_product(M, N, K, dtype, rows=sorted({*range(0, M, 29), *range(250, 262), M - 2, M - 1}))


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_linear_pair_tiles_ragged(dtype):
    """Enough tiles for every pair of SMs, no size on the tile grid."""
    check_product(2500, 2602, 400, dtype)
    check_product(2501, 2603, 16, dtype)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("M,N,K", [(3, 64, 256), (40, 256, 512), (70, 128, 4096), (2500, 2560, 272),
                                   (2500, 2600, 144), (2500, 2564, 144)])
def test_linear_output_of_least_alignment(M, N, K, dtype):
    """y, x and w begin 16 bytes past a larger boundary, the scales 4."""
    x, sx, w, sw = draw_product(M, N, K, M + N)
    off = lambda t, n: torch.cat([t.new_zeros(n), t.reshape(-1)]).cuda()[n:].view(t.shape)  # noqa: E731
    buf = torch.full((M * N + 40,), 7.0, dtype=dtype, device="cuda")
    n = 16 // buf.element_size()
    y = buf[n:n + M * N].view(M, N)
    gdn.linear_i8(off(x, 16), off(sx, 1), off(w, 16), off(sw, 1), y)
    torch.cuda.synchronize()
    want = ref.linear(x.numpy(), sx.numpy(), w.numpy(), sw.numpy(), dtype is BF16)
    assert np.array_equal(y.float().cpu().numpy(), want)
    assert (buf[:n] == 7).all() and (buf[n + M * N:] == 7).all()


def test_linear_large_sampled():
    check_product(4096, 8192, 2048, F32, rows=[0, 1, 127, 128, 2049, 4095])


def test_linear_many_tiles_a_pair():
    """Several tiles for each pair of SMs: both accumulator sets in turn."""
    check_product(9000, 4100, 48, BF16, rows=list(range(0, 9000, 37)) + [8999])


def test_linear_longest_sums():
    """K at its limit, every product 128 * 128: the largest 32-bit sum."""
    K = 131056
    x = torch.full((3, K), -128, dtype=torch.int8, device="cuda")
    w = torch.full((5, K), -128, dtype=torch.int8, device="cuda")
    one = torch.ones(5, device="cuda")
    y = gdn.linear_i8(x, one[:3], w, one)
    assert (y.cpu().numpy() == np.float32(K * 16384)).all()


def test_linear_empty():
    x = torch.zeros(3, 0, dtype=torch.int8, device="cuda")
    w = torch.zeros(5, 0, dtype=torch.int8, device="cuda")
    y = torch.full((3, 5), 7.0, device="cuda")
    gdn.linear_i8(x, torch.ones(3, device="cuda"), w, torch.ones(5, device="cuda"), y)
    assert torch.count_nonzero(y) == 0
    e = gdn.linear_i8(torch.zeros(0, 16, dtype=torch.int8, device="cuda"), torch.ones(0, device="cuda"),
                      torch.zeros(5, 16, dtype=torch.int8, device="cuda"), torch.ones(5, device="cuda"))
    assert e.shape == (0, 5)


def test_linear_rows_independent_of_batch():
    """A row is the same in every call, whatever form computes it."""
    x, sx, w, sw = (t.cuda() for t in draw_product(4096, 4096, 1024, 13))
    y = gdn.linear_i8(x, sx, w, sw)
    for M in (1, 20, 64, 128, 200, 700):
        assert torch.equal(gdn.linear_i8(x[-M:], sx[-M:], w, sw), y[-M:]), M


# -- as they are used ---------------------------------------------------------------

@pytest.mark.parametrize("M,N,K", [(1, 512, 4096), (8, 300, 1040), (70, 200, 4096), (600, 1024, 256)])
def test_operands_written_by_the_kernel_before(M, N, K):
    """Each call reads what the call just before it wrote, into the same buffers
    again and again: rows and weights in 8 bits, scales, norm weights, and a
    product that is the next residual."""
    g = torch.Generator().manual_seed(M + N)
    xs = [torch.randn(M, K, generator=g).cuda() for _ in range(6)]
    ws = [torch.randn(N, K, generator=g).cuda() for _ in range(6)]
    q, s = torch.empty(M, K, dtype=torch.int8, device="cuda"), torch.empty(M, device="cuda")
    wq, sw = torch.empty(N, K, dtype=torch.int8, device="cuda"), torch.empty(N, device="cuda")
    y = torch.empty(M, N, device="cuda")
    nx = [torch.randn(M, N - N % 16, generator=g).cuda() for _ in range(6)]

    def run(wait):
        got = []
        for x, w, r in zip(xs, ws, nx):
            for call in (lambda: gdn.quantize_i8(x, q, s), lambda: gdn.quantize_i8(w, wq, sw),
                         lambda: got.append(gdn.linear_i8(q, s, wq, sw, y).clone()),
                         lambda: gdn.quantize_i8(w, wq, sw), lambda: gdn.quantize_i8(x, q, s),
                         lambda: got.append(gdn.linear_i8(q, s, wq, sw)),
                         # a norm whose weight the product before it wrote
                         lambda: got.extend(gdn.add_rms_norm_i8(
                             r, gdn.linear_i8(q[:1], s[:1], wq, sw)[0, :r.shape[1]], r))):
                call()
                if wait:
                    torch.cuda.synchronize()
        torch.cuda.synchronize()
        return got

    want = run(True)
    for _ in range(5):
        for a, b in zip(run(False), want):
            assert torch.equal(a, b)

def test_chain_on_a_stream_captured_and_replayed():
    """norm -> product -> quantise -> product on a side stream, captured once
    and replayed on new inputs, two graphs of other buffers interleaved."""
    M, D, N = 5, 2048, 4096
    g = torch.Generator().manual_seed(4)
    w1, w2 = torch.randn(N, D, generator=g).cuda(), torch.randn(D, N, generator=g).cuda()
    q1, s1 = gdn.quantize_i8(w1)
    q2, s2 = gdn.quantize_i8(w2)
    norm_w = torch.ones(D, device="cuda")
    torch.cuda.synchronize()

    def chain(x, r, out, stream=None):
        q, s, _ = gdn.add_rms_norm_i8(x, norm_w, r, r, stream=stream)
        y = gdn.linear_i8(q, s, q1, s1, stream=stream)
        q, s = gdn.quantize_i8(y, stream=stream)
        gdn.linear_i8(q, s, q2, s2, out, stream=stream)

    bufs, graphs = [], []
    for i in range(2):
        x, r = torch.randn(M, D, device="cuda"), torch.zeros(M, D, device="cuda")
        out = torch.empty(M, D, device="cuda")
        chain(x, r, out)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            chain(x, r, out)
        bufs.append((x, r, out))
        graphs.append(graph)
    side = torch.cuda.Stream()
    for it in range(4):
        new = [torch.randn(M, D, generator=torch.Generator().manual_seed(it * 2 + i)) for i in range(2)]
        old = []
        for (x, r, out), n in zip(bufs, new):
            x.copy_(n)
            old.append(r.clone())
        torch.cuda.synchronize()
        for graph in graphs:
            graph.replay()
        torch.cuda.synchronize()
        for (x, r, out), o in zip(bufs, old):
            want_r, want = o.clone(), torch.empty(M, D, device="cuda")
            torch.cuda.synchronize()
            with torch.cuda.stream(side):
                chain(x, want_r, want)
            side.synchronize()
            assert torch.equal(want, out) and torch.equal(want_r, r)
    graphs.clear()


def test_two_streams_at_once():
    """Calls on two streams share nothing."""
    a = [t.cuda() for t in draw_product(64, 4096, 2048, 1)]
    b = [t.cuda() for t in draw_product(700, 2050, 1040, 2)]
    want = [gdn.linear_i8(*a), gdn.linear_i8(*b)]
    outs = [[torch.empty_like(w) for _ in range(8)] for w in want]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for i in range(8):
        for args, o, st in zip((a, b), outs, streams):
            gdn.linear_i8(*args, o[i], stream=st)
    torch.cuda.synchronize()
    for o, w in zip(outs, want):
        assert all(torch.equal(t, w) for t in o)


def test_layer_decode_with_8_bit_projections():
    """One token through a whole recurrent layer: norm with the residual, the
    qkv, z and b | a projections, the fused layer, the output projection. The
    integer stages are compared bit for bit with the definition, the fused
    layer with the oracle, each from the stage before it."""
    B, D, Hk, Hv = 6, 512, 16, 32
    C, HD = 2 * Hk * 128 + Hv * 128, Hv * 128
    d = inputs.forward_inputs(B, 1, D=D, seed=77, state_std=0.05)
    t = {k: torch.from_numpy(np.ascontiguousarray(v)).cuda() for k, v in d.items()}
    x, r = draw_rows(B, D, 31), draw_rows(B, D, 32, BF16)
    norm_w = 1 + 0.1 * draw_rows(1, D, 33)[0]
    wq = {k: gdn.quantize_i8(t[k].float()) for k in ("w_qkv", "w_z", "w_ba", "w_out")}
    q, s, h = gdn.add_rms_norm_i8(x.cuda(), norm_w.cuda(), r.cuda())
    p = {k: gdn.linear_i8(q, s, *wq[k]) for k in ("w_qkv", "w_z", "w_ba")}
    b, a = p["w_ba"][:, :Hv].contiguous(), p["w_ba"][:, Hv:].contiguous()
    ring0, state0 = d["conv_ring"].copy(), d["state"].copy()
    y = gdn.layer_decode(p["w_qkv"], p["w_z"], a, b, t["conv_ring"], t["conv_w"], t["A_log"],
                         t["dt_bias"], t["norm_w"], t["state"], Hk=Hk)
    qy, sy = gdn.quantize_i8(y)
    out = gdn.linear_i8(qy, sy, *wq["w_out"], out_dtype=BF16)
    torch.cuda.synchronize()

    n = lambda v: v.float().cpu().numpy()  # noqa: E731
    for k in wq:
        check_rows(*wq[k], *ref.rows(n(t[k]))[:2])
    rq, rs, rh = ref.rows(x.numpy(), r.float().numpy(), norm_w.numpy(), residual_bf16=True)
    check_rows(q, s, rq, rs)
    assert np.array_equal(n(h), rh)
    for k in p:
        assert np.array_equal(n(p[k]), ref.linear(q.cpu().numpy(), n(s), wq[k][0].cpu().numpy(), n(wq[k][1])))
    o = oracle.load()
    oy, oring, ostate = o.layer_decode(n(p["w_qkv"]), n(p["w_z"]), n(a), n(b), ring0, d["conv_w"],
                                       d["A_log"], d["dt_bias"], d["norm_w"], state0, Hk=Hk)
    assert_parity(n(y), oy, "layer output")
    assert_parity(n(t["state"]), ostate, "state")
    check_rows(qy, sy, *ref.rows(n(y))[:2])
    assert np.array_equal(n(out), ref.linear(qy.cpu().numpy(), n(sy), wq["w_out"][0].cpu().numpy(),
                                             n(wq["w_out"][1]), True))


# -- the layer over positions ---------------------------------------------------------

def layer_reference(d, Hk):
    """What forward_batch_i8 gets and gives, from forward_inputs' arrays: the
    integers and scales, the oracle's y [B, T, Hv*128] in 64 bits from the
    exact projections, the ring and the state."""
    B, T, D = d["hidden"].shape
    qs = {k: ref.rows(d[k].reshape(-1, d[k].shape[-1]))[:2]
          for k in ("hidden", "w_qkv", "w_z", "w_ba", "w_out")}
    qs = {k: (q, s.astype(np.float32)) for k, (q, s) in qs.items()}
    p = {k: ref.linear(*qs["hidden"], *qs[k]).reshape(B, T, -1) for k in ("w_qkv", "w_z", "w_ba")}
    Hv = d["A_log"].shape[0]
    o, ring, state = oracle.load(), d["conv_ring"], d["state"]
    ys = []
    for t in range(T):
        c = lambda v: np.ascontiguousarray(v)  # noqa: E731
        y, ring, state = o.layer_decode(c(p["w_qkv"][:, t]), c(p["w_z"][:, t]),
                                        c(p["w_ba"][:, t, Hv:]), c(p["w_ba"][:, t, :Hv]), ring,
                                        d["conv_w"], d["A_log"], d["dt_bias"], d["norm_w"], state,
                                        Hk=Hk)
        ys.append(y)
    return qs, p, np.stack(ys, 1), ring, state


def output_bound(y, wq, ws):
    """out from y [R, HD] in 64 bits, and how far the call's may be from it. Its
    y is within the parity tests' 1e-5 of this one, so its row maximum m is:
    an integer that both give alike stands for values 127 e / m of itself
    apart (e = 1e-5), and only where 127 y / m lies within 2 * 127 e / m of a
    half may it be one step off. The product adds three roundings."""
    e = 1e-5
    m = np.abs(y).max(1, keepdims=True)
    t = 127.0 * y / m
    q = np.rint(t)
    near = np.abs(np.abs(t - np.floor(t)) - 0.5) <= 2 * 127.0 * e / m
    s = m / 127.0
    w = wq.astype(np.float64) * ws.astype(np.float64)[:, None]
    slack = np.abs(q) * s * (e / m + 2.0 ** -24) + near * s
    out = (q * s) @ w.T
    return out, slack @ np.abs(w).T + 3 * 2.0 ** -24 * np.abs(out)


def run_layer(d, qs, Hk, out_dtype=F32, T=None, t0=0, ring=None, state=None):
    dev = lambda v: torch.from_numpy(np.ascontiguousarray(v)).cuda()  # noqa: E731
    B, Tall, D = d["hidden"].shape
    T = Tall if T is None else T
    hq, hs = qs["hidden"][0].reshape(B, Tall, D), qs["hidden"][1].reshape(B, Tall)
    ring = dev(d["conv_ring"]) if ring is None else ring
    state = dev(d["state"]) if state is None else state
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    w = [dev(v) for k in ("w_qkv", "w_z", "w_ba", "w_out") for v in qs[k]]
    out = gdn.forward_batch_i8(dev(hq[:, t0:t0 + T]), dev(hs[:, t0:t0 + T]), *w, ring,
                               dev(d["conv_w"]), dev(d["A_log"]), dev(d["dt_bias"]),
                               dev(d["norm_w"]), state, Hk=Hk, out_dtype=out_dtype, status=status)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    return out, ring, state


@pytest.mark.parametrize("B,T,D,Hk,Hv,dtype", [
    (2, 37, 256, 16, 32, F32), (1, 5, 64, 16, 32, BF16), (3, 1, 512, 16, 32, F32),
    (2, 3, 48, 1, 1, F32), (1, 2, 64, 72, 72, BF16), (1, 70, 128, 2, 4, F32)])
def test_forward_batch_i8(B, T, D, Hk, Hv, dtype):
    d = inputs.forward_inputs(B, T, D=D, Hk=Hk, Hv=Hv, seed=2000 + B + T + Hv, state_std=0.05)
    qs, p, y, ring_r, state_r = layer_reference(d, Hk)
    out, ring, state = run_layer(d, qs, Hk, dtype)
    want, bound = output_bound(y.reshape(B * T, -1), *qs["w_out"])
    if dtype is BF16:
        bound = bound + torch.finfo(BF16).eps / 2 * (np.abs(want) + bound)
    got = out.double().cpu().numpy().reshape(B * T, D)
    assert np.all(np.abs(got - want) <= bound), np.max(np.abs(got - want) / bound)
    assert_parity(state.cpu().numpy(), state_r, "state")
    # the ring holds raw projections: the exact ones
    raw = np.concatenate([d["conv_ring"], p["w_qkv"]], 1)[:, -ring.shape[1]:]
    assert np.array_equal(ring.cpu().numpy(), raw)


def test_forward_batch_i8_chunks_and_empty():
    """11 positions in one call and as 4 and 7 resumed from the ring and state
    are both the reference's; a call of no positions does nothing."""
    d = inputs.forward_inputs(2, 11, D=96, seed=2100, state_std=0.05)
    qs, _, y, ring_r, state_r = layer_reference(d, 16)
    want, bound = output_bound(y.reshape(22, -1), *qs["w_out"])
    out, ring, state = run_layer(d, qs, 16)
    a, r, s = run_layer(d, qs, 16, T=4)
    b, r, s = run_layer(d, qs, 16, T=7, t0=4, ring=r, state=s)
    for got, st in ((out, state), (torch.cat([a, b], 1), s)):
        assert_parity(st.cpu().numpy(), state_r, "state")
        assert np.all(np.abs(got.double().cpu().numpy().reshape(22, -1) - want) <= bound)
    assert torch.equal(r, ring)
    e, r2, s2 = run_layer(d, qs, 16, T=0, ring=r.clone(), state=s.clone())
    assert e.shape == (2, 0, 96) and torch.equal(r2, r) and torch.equal(s2, s)


def test_linear_many_short_rows():
    """More tokens than a grid's second dimension has blocks of eight."""
    check_product(600_001, 1, 16, BF16)
    check_product(70_000, 9, 48, F32)


# -- shapes, streams, threads, far offsets ---------------------------------------------

def test_leading_dimensions():
    """Rows over any leading dimensions, none of them too, and none at all."""
    x = draw_rows(6, 64, 41).cuda()
    w, ws = gdn.quantize_i8(draw_rows(9, 64, 42).cuda())
    q, s = gdn.quantize_i8(x)
    y = gdn.linear_i8(q, s, w, ws)
    q3, s3, h3 = gdn.add_rms_norm_i8(x.view(2, 3, 64), torch.ones(64, device="cuda"),
                                     torch.zeros(2, 3, 64, device="cuda"))
    assert torch.equal(q3.view(6, 64), q) and s3.shape == (2, 3) and torch.equal(h3.view(6, 64), x)
    q3, s3 = gdn.quantize_i8(x.view(2, 3, 64))
    assert torch.equal(gdn.linear_i8(q3, s3, w, ws), y.view(2, 3, 9))
    q1, s1 = gdn.quantize_i8(x[4])
    assert s1.shape == () and torch.equal(gdn.linear_i8(q1, s1, w, ws), y[4])
    e, es = gdn.quantize_i8(x.new_zeros(2, 0, 64))
    assert gdn.linear_i8(e, es, w, ws).shape == (2, 0, 9)
    # one tensor as both operands
    assert np.array_equal(gdn.linear_i8(w, ws, w, ws).cpu().numpy(),
                          ref.linear(w.cpu().numpy(), ws.cpu().numpy(), w.cpu().numpy(), ws.cpu().numpy()))


def test_outputs_made_on_the_calls_stream():
    """With `stream`, everything the call makes belongs to that stream."""
    x, w = draw_rows(300, 2048, 43).cuda(), draw_rows(700, 2048, 44).cuda()
    wq, ws = gdn.quantize_i8(w)
    want = gdn.linear_i8(*gdn.quantize_i8(x), wq, ws)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    for _ in range(20):
        q, s = gdn.quantize_i8(x, stream=st)
        y = gdn.linear_i8(q, s, wq, ws, stream=st)
        del q, s                                    # their memory may serve this stream again
        st.synchronize()
        assert torch.equal(y, want)


def test_two_host_threads():
    """Calls of several host threads, each on a stream of its own."""
    import threading
    shapes = [(3, 200, 512), (40, 1000, 1040), (300, 520, 256), (700, 2050, 272)]
    args = [[t.cuda() for t in draw_product(*sh, seed=sum(sh))] for sh in shapes]
    want = [gdn.linear_i8(*a) for a in args]
    torch.cuda.synchronize()
    bad = []

    def work(i):
        st = torch.cuda.Stream()
        for _ in range(50):
            for a, w in zip(args[i:] + args[:i], want[i:] + want[:i]):
                y = gdn.linear_i8(*a, stream=st)
                st.synchronize()
                if not torch.equal(y, w):
                    bad.append(i)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(shapes))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad


def test_offsets_past_32_bits():
    """Outputs and rows beyond 2^32 elements: the last ones, and the ones that
    a 32-bit offset would have written."""
    M, N, K = 530_000, 8208, 16
    x, sx, w, sw = draw_product(8, N, K, 45)
    xb = torch.zeros(M, K, dtype=torch.int8, device="cuda")
    xb[-8:] = x.cuda()
    sb = torch.ones(M, device="cuda")
    sb[-8:] = sx.cuda()
    y = gdn.linear_i8(xb, sb, w.cuda(), sw.cuda(), out_dtype=BF16)
    assert np.array_equal(y[-8:].float().cpu().numpy(), ref.linear(x, sx, w, sw, True))
    assert int(torch.count_nonzero(y[:-8])) == 0
    del y, xb, sb
    M, D = 1_050_000, 4096
    xb = torch.zeros(M, D, dtype=BF16, device="cuda")
    x = draw_rows(5, D, 46, BF16)
    xb[-5:] = x.cuda()
    q, s = gdn.quantize_i8(xb)
    check_rows(q[-5:], s[-5:], *ref.rows(x.float().numpy())[:2])
    assert int(torch.count_nonzero(q[:-5])) == 0 and int(torch.count_nonzero(s[:-5])) == 0


@pytest.mark.parametrize("M,K", [(3, 2048), (40, 528), (300, 4112)])
def test_one_tensor_for_two_arguments(M, K):
    """Rows against themselves, and a row added to itself."""
    x = draw_rows(M, K, 77)
    xc = x.cuda()
    q, s = gdn.quantize_i8(xc)
    y = gdn.linear_i8(q, s, q, s)
    qn, sn = q.cpu().numpy(), s.cpu().numpy()
    assert np.array_equal(y.cpu().numpy(), ref.linear(qn, sn, qn, sn))
    w = torch.ones(K)
    got = gdn.add_rms_norm_i8(xc, w.cuda(), xc)
    want = ref.rows(x.numpy(), x.numpy(), w.numpy())
    check_rows(got[0], got[1], *want[:2])
    assert np.array_equal(got[2].cpu().numpy(), want[2]) and torch.equal(xc.cpu(), x)
