"""MXFP4 products on the GPU against 64-bit products of the same codes."""
import numpy as np
import pytest
import torch

import nvfp4_block_scaled_bf16_amd as nv
from tests import mx_ref
from tests.gpu_util import CANARY
from tests.test_gpu_mx_cast import data, groups

pytestmark = pytest.mark.gpu
TYPES = [torch.bfloat16, torch.float16, torch.float32]


def vectors(rng, R, K):
    """(q, sf, values) of R random vectors: codes of every kind, scales over 2^+-6."""
    Kp = mx_ref.up(K, 128)
    codes = rng.integers(0, 16, (R, Kp)).astype(np.uint8)
    codes[:, K:] = 0
    s = rng.integers(121, 134, (R, Kp // 32)).astype(np.uint8)
    q, sf = torch.from_numpy(mx_ref.pack_codes(codes)).cuda(), torch.from_numpy(mx_ref.pack_scales(s)).cuda()
    return q, sf, mx_ref.values(codes, s)


SHAPES = [(1, 1, 1), (1, 5, 40), (1, 4096, 1024), (2, 33, 128), (7, 257, 129), (16, 64, 2048), (17, 100, 300),
          (31, 129, 1000), (33, 31, 384), (64, 640, 512), (65, 128, 256), (100, 1000, 700), (129, 127, 1100),
          (128, 128, 128), (256, 256, 640), (257, 513, 900), (300, 770, 130), (520, 1030, 260), (1025, 300, 1408)]


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_gemm(M, N, K, dtype):
    rng = np.random.default_rng(M * 7919 + N * 31 + K)
    (aq, asf, a), (bq, bsf, b) = vectors(rng, M, K), vectors(rng, N, K)
    mx_ref.check_product(nv.mx_gemm(aq, asf, bq, bsf, dtype), a, b)


@pytest.mark.parametrize("M", [1, 3, 8, 16, 40, 130])
def test_long_sums(M):
    rng = np.random.default_rng(M)
    (aq, asf, a), (bq, bsf, b) = vectors(rng, M, 28673), vectors(rng, 50, 28673)
    mx_ref.check_product(nv.mx_gemm(aq, asf, bq, bsf, torch.float32), a, b)


@pytest.mark.parametrize("M", [1, 2, 9, 33, 64])
@pytest.mark.parametrize("K", [120, 200, 385, 1000, 1150, 2100])      # 1, 2, 4, 8, 9 and 17 steps
def test_few_rows_by_steps(M, K):
    # fewer steps than waves, an odd one left over, in both ways of few rows
    rng = np.random.default_rng(M * 17 + K)
    (aq, asf, a), (bq, bsf, b) = vectors(rng, M, K), vectors(rng, 77, K)
    mx_ref.check_product(nv.mx_gemm(aq, asf, bq, bsf, torch.float32), a, b)
    x = data(rng, M, K, torch.bfloat16)
    fx = np.pad(mx_ref.fake(mx_ref.host64(x)), ((0, 0), (0, b.shape[1] - K)))
    mx_ref.check_product(nv.mx_linear(x, bq, bsf, torch.float32), fx, b)
    off = torch.tensor([0, M // 2, M], dtype=torch.int32, device="cuda")
    w2, s2 = torch.stack([bq, bq]), torch.stack([bsf, bsf])
    mx_ref.check_product(nv.mx_linear_grouped(x, w2, s2, off, out_dtype=torch.float32), fx, b)


def test_large_tiles():
    # enough tiles for every tile shape, checked at whole rows
    rng = np.random.default_rng(3)
    (aq, asf, a), (bq, bsf, b) = vectors(rng, 2500, 384), vectors(rng, 4100, 384)
    got = nv.mx_gemm(aq, asf, bq, bsf, torch.float32)
    mx_ref.check_product(got, a, b)


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("M,N,K", [(1, 300, 1000), (1, 4096, 4096), (2, 96, 31), (5, 130, 257), (8, 777, 8192), (9, 64, 512),
                                   (16, 200, 4100), (17, 64, 512), (33, 140, 900), (130, 600, 333)])
def test_linear_is_cast_and_product(M, N, K, dtype):
    rng = np.random.default_rng(M * 31 + K)
    x = data(rng, M, K + 3, dtype)[:, 1:K + 1]          # a view: row pitch K + 3, off alignment
    wq, wsf, w = vectors(rng, N, K)
    got = nv.mx_linear(x, wq, wsf, torch.float32)
    mx_ref.check_product(got, np.pad(mx_ref.fake(mx_ref.host64(x)), ((0, 0), (0, w.shape[1] - K))), w)
    o = nv.mx_linear(x, wq, wsf)
    assert o.dtype == dtype and torch.allclose(o, got.to(dtype), rtol=0, atol=0, equal_nan=True)


def test_special_scales():
    # a NaN scale in either operand reaches its row or column alone; the least
    # and the largest scales multiply out
    rng = np.random.default_rng(4)
    for M in (4, 150):
        (aq, asf, a), (bq, bsf, b) = vectors(rng, M, 200), vectors(rng, 140, 200)
        asf[0, 1, 2, 0] = 255
        bsf[1, 0, 3, 1] = 255
        got = nv.mx_gemm(aq, asf, bq, bsf, torch.float32).cpu()
        nan = torch.zeros(M, 140, dtype=torch.bool)
        nan[2] = True
        nan[:, 131] = True
        assert torch.equal(torch.isnan(got), nan)
    codes = np.full((3, 128), 2, np.uint8)               # ones
    for sa, sb, want in ((0, 254, 128.0), (254, 0, 128.0), (127, 127, 128.0), (0, 127, 2.0 ** -120), (250, 131, np.inf)):
        q = torch.from_numpy(mx_ref.pack_codes(codes)).cuda()
        f = [torch.from_numpy(mx_ref.pack_scales(np.full((3, 4), s, np.uint8))).cuda() for s in (sa, sb)]
        got = nv.mx_gemm(q, f[0], q, f[1], torch.float32)
        assert (got == want).all(), (sa, sb, got)


def test_empty_sums_and_sizes():
    z = nv.mx_quantize(torch.zeros(4, 0, device="cuda"), columnwise=False)
    assert torch.equal(nv.mx_gemm(z["row_q"], z["row_sf"], z["row_q"], z["row_sf"]).cpu(), torch.zeros(4, 4).bfloat16())
    wq, wsf, _ = vectors(np.random.default_rng(0), 5, 64)
    e = nv.mx_quantize(torch.zeros(0, 64, device="cuda"), columnwise=False)
    assert nv.mx_gemm(e["row_q"], e["row_sf"], wq, wsf).shape == (0, 5)
    assert nv.mx_gemm(wq, wsf, e["row_q"], e["row_sf"]).shape == (5, 0)
    assert nv.mx_linear(torch.zeros(0, 64, device="cuda"), wq, wsf).shape == (0, 5)
    for M in (1, 7, 300, 5000):                          # nothing to sum: zeros
        x = torch.zeros(M, 0, device="cuda")
        assert torch.equal(nv.mx_linear(x, z["row_q"], z["row_sf"]).cpu(), torch.zeros(M, 4))
        off = torch.tensor([0, M // 2, M], dtype=torch.int32, device="cuda")
        got = nv.mx_linear_grouped(x, z["row_q"].expand(2, 4, 0).contiguous(), z["row_sf"].expand(2, 1, 0, 128, 4).contiguous(), off)
        assert torch.equal(got.cpu(), torch.zeros(M, 4))


def grouped_reference(a, b, off, idx=None):
    """Row values of a for every row of out, by group: [(begin, end, values, b_e)]."""
    rows = a if idx is None else np.where(((idx >= 0) & (idx < len(a)))[:, None], a[np.clip(idx, 0, len(a) - 1)], 0.0)
    return [(off[e], off[e + 1], rows[off[e]:off[e + 1]], b[e]) for e in range(len(off) - 1) if off[e] < off[e + 1]]


def experts(rng, E, N, K):
    ops = [vectors(rng, N, K) for _ in range(E)]
    return torch.stack([o[0] for o in ops]), torch.stack([o[1] for o in ops]), [o[2] for o in ops]


CASES = [(1, 1, 1, 1), (4, 9, 33, 70), (3, 40, 64, 256), (64, 20, 48, 300), (33, 300, 100, 200), (5, 700, 257, 384),
         (70, 900, 40, 129), (2, 1100, 300, 140), (130, 200, 20, 64), (8, 2000, 130, 1000)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=str)
@pytest.mark.parametrize("E,R,N,K", CASES)
def test_grouped(E, R, N, K, dtype):
    rng = np.random.default_rng(E * 100 + R)
    off = groups(rng, E, R)
    aq, asf, a = vectors(rng, R, K)
    bq, bsf, b = experts(rng, E, N, K)
    got = nv.mx_gemm_grouped(aq, asf, bq, bsf, torch.from_numpy(off).cuda(), out_dtype=dtype)
    for s, e, av, bv in grouped_reference(a, b, off):
        mx_ref.check_product(got[s:e], av, bv)


@pytest.mark.parametrize("E,R,N,K", CASES)
def test_grouped_rows_and_factors(E, R, N, K):
    rng = np.random.default_rng(E * 101 + R)
    off = groups(rng, E, R)
    A = max(1, R // 3)
    x = data(rng, A, K, torch.bfloat16, wild=False)
    idx = rng.integers(0, A, R).astype(np.int32)
    if R > 8:
        idx[[1, R - 1]] = [-3, A]                       # outside: rows of zeros
    f = rng.standard_normal(R).astype(np.float32)
    f[0] = 0.0
    bq, bsf, b = experts(rng, E, N, K)
    a = np.pad(mx_ref.fake(mx_ref.host64(x)), ((0, 0), (0, b[0].shape[1] - K)))
    args = dict(rows=torch.from_numpy(idx).cuda(), row_scale=torch.from_numpy(f).cuda())
    offd = torch.from_numpy(off).cuda()
    q = nv.mx_quantize(x, columnwise=False)
    got = nv.mx_gemm_grouped(q["row_q"], q["row_sf"], bq, bsf, offd, out_dtype=torch.float32, **args)
    lin = nv.mx_linear_grouped(x, bq, bsf, offd, out_dtype=torch.float32, **args)
    for s, e, av, bv in grouped_reference(a, b, off, idx):
        mx_ref.check_product(got[s:e], av, bv, f[s:e].astype(np.float64))
        mx_ref.check_product(lin[s:e], av, bv, f[s:e].astype(np.float64))


def test_few_rows_to_many_large_experts():
    # up to two rows a group on average, whatever the work of casting them
    rng = np.random.default_rng(12)
    E, R, N, K = 64, 100, 1400, 4000
    off, x = groups(rng, E, R), data(rng, R, K, torch.bfloat16, wild=False)
    (q0, s0, b0), (q1, s1, b1) = vectors(rng, N, K), vectors(rng, N, K)
    bq, bsf = torch.stack([q0, q1] * (E // 2)), torch.stack([s0, s1] * (E // 2))
    a = np.pad(mx_ref.fake(mx_ref.host64(x)), ((0, 0), (0, b0.shape[1] - K)))
    got = nv.mx_linear_grouped(x, bq, bsf, torch.from_numpy(off).cuda(), out_dtype=torch.float32)
    for e in range(E):
        if off[e + 1] > off[e]:
            mx_ref.check_product(got[off[e]:off[e + 1]], a[off[e]:off[e + 1]], (b0, b1)[e % 2])


def test_an_outside_row_is_zero_beside_a_nan():
    # the row that stands in for an index outside must not leak its NaN
    rng = np.random.default_rng(8)
    x = data(rng, 20, 64, torch.bfloat16, wild=False)
    x[0, 3] = x[19, 3] = float("nan")
    bq, bsf, b = experts(rng, 2, 40, 64)
    idx = torch.tensor([-1, 5, 20, 7] * 40, dtype=torch.int32, device="cuda")
    for n in (4, 160):
        off = torch.tensor([0, n // 2, n], dtype=torch.int32, device="cuda")
        got = nv.mx_linear_grouped(x, bq, bsf, off, rows=idx[:n]).float()
        assert (got[0::2] == 0).all() and torch.isfinite(got).all()
        # nor a factor's or a weight's
        f = torch.full((n,), float("inf"), device="cuda")
        wsf = bsf.clone()
        wsf[:, 0, 0, :] = 255
        got = nv.mx_linear_grouped(x, bq, wsf, off, rows=idx[:n], row_scale=f).float()
        assert (got[0::2] == 0).all() and torch.isnan(got[1::2]).all()


@pytest.mark.parametrize("R", [30, 400])
def test_rows_in_no_group_are_not_written(R):
    rng = np.random.default_rng(9)
    aq, asf, a = vectors(rng, R, 100)
    bq, bsf, b = experts(rng, 2, 50, 100)
    out = torch.full((R * 50 * 4 + 256,), CANARY, dtype=torch.uint8, device="cuda")
    off = torch.tensor([3, 10, R - 5], dtype=torch.int32, device="cuda")
    st = nv.lib().nvfp4_mx_gemm_grouped(aq.data_ptr(), asf.data_ptr(), R, None, R, off.data_ptr(), 2, bq.data_ptr(),
                                        bsf.data_ptr(), 50, 100, None, 0, out.data_ptr() + 128,
                                        torch.cuda.current_stream().cuda_stream)
    assert st == 0
    o = out.cpu()
    assert (o[:128 + 3 * 200] == CANARY).all() and (o[128 + (R - 5) * 200:] == CANARY).all()
    v = o[128:128 + R * 200].view(torch.float32).view(R, 50)
    mx_ref.check_product(v[3:10], a[3:10], b[0])
    mx_ref.check_product(v[10:R - 5], a[10:R - 5], b[1])


@pytest.mark.parametrize("M,N,dtype", [(1, 100, torch.bfloat16), (1, 101, torch.float16), (37, 99, torch.bfloat16),
                                       (300, 130, torch.bfloat16), (300, 131, torch.float16), (600, 2049, torch.float32)])
def test_nothing_written_outside(M, N, dtype):
    rng = np.random.default_rng(M + N)
    (aq, asf, a), (bq, bsf, b) = vectors(rng, M, 200), vectors(rng, N, 200)
    size = M * N * torch.empty((), dtype=dtype).element_size()
    for shift in (0, 4):                                # out aligned to its type alone
        buf = torch.full((size + 512,), CANARY, dtype=torch.uint8, device="cuda")
        out = buf[256 + shift:256 + shift + size]
        st = nv.lib().nvfp4_mx_gemm(aq.data_ptr(), asf.data_ptr(), bq.data_ptr(), bsf.data_ptr(), M, N, 200,
                                    nv.mx._TYPES[dtype], out.data_ptr(), torch.cuda.current_stream().cuda_stream)
        assert st == 0
        assert (buf[:256 + shift] == CANARY).all() and (buf[256 + shift + size:] == CANARY).all()
        mx_ref.check_product(out.clone().view(dtype).view(M, N), a, b)


@pytest.mark.parametrize("E,R,N,K", [(1, 1, 1, 1), (3, 50, 33, 40), (9, 400, 130, 70), (70, 600, 40, 140), (2, 1000, 300, 129),
                                     (130, 64, 20, 30), (6, 777, 257, 384)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=str)
def test_wgrad(E, R, N, K, dtype):
    rng = np.random.default_rng(E * 102 + R)
    off = groups(rng, E, R)
    dy, x = data(rng, R, N, torch.bfloat16, wild=False), data(rng, max(1, R // 2), K, torch.bfloat16, wild=False)
    idx = rng.integers(0, x.shape[0], R).astype(np.int32)
    offd, idxd = torch.from_numpy(off).cuda(), torch.from_numpy(idx).cuda()
    d = nv.mx_quantize_grouped(dy, offd)
    q = nv.mx_quantize_grouped(x, offd, rows=idxd, rowwise=False)
    got = nv.mx_wgrad_grouped(d["col_q"], d["col_sf"], q["col_q"], q["col_sf"], offd, dtype)
    assert got.dtype == dtype
    dv, xv = mx_ref.host64(dy), mx_ref.host64(x)[idx]
    for e in range(E):
        s, t = off[e], off[e + 1]
        if s == t:
            assert (got[e] == 0).all()
        else:
            mx_ref.check_product(got[e], mx_ref.fake(dv[s:t].T), mx_ref.fake(xv[s:t].T))


def test_wgrad_with_offsets_out_of_order():
    # more steps asked for than there are: held to what the vectors have (the
    # first group's sum then takes steps that no cast wrote: unspecified)
    x = data(np.random.default_rng(10), 256, 40, torch.bfloat16)
    good = torch.tensor([0, 128, 256], dtype=torch.int32, device="cuda")
    q = nv.mx_quantize_grouped(x, good)
    bad = torch.tensor([0, 2 ** 31 - 1, -7], dtype=torch.int32, device="cuda")
    got = nv.mx_wgrad_grouped(q["col_q"], q["col_sf"], q["col_q"], q["col_sf"], bad)
    torch.cuda.synchronize()
    assert (got[1] == 0).all()


def grid_values(rng, shape):
    """Values of E2M1's grid: exact under any block scale they can get."""
    return rng.choice(np.array([0.5, 1, 1.5, 2, 3, 4, 6, 0]), shape) * rng.choice([-1.0, 1.0], shape)


@pytest.mark.parametrize("T,K,N", [(40, 70, 50), (200, 130, 257)])
def test_gradients_against_differences(T, K, N):
    # f(x, W) = <dy, x W^T> on values that the cast keeps: its change along a
    # step of either argument is the gradient's product with the step.  All
    # sums here are of multiples of 1/8 below 2^20, exact in fp32.
    rng = np.random.default_rng(T)
    x, x2, w, w2, dy = (grid_values(rng, s) for s in ((T, K), (T, K), (N, K), (N, K), (T, N)))
    dev = lambda v: torch.from_numpy(v).to(torch.bfloat16).cuda()  # noqa: E731
    qx, qw, qd = nv.mx_quantize(dev(x)), nv.mx_quantize(dev(w)), nv.mx_quantize(dev(dy))
    f32 = torch.float32

    def f(x, w):
        a, b = nv.mx_quantize(dev(x), columnwise=False), nv.mx_quantize(dev(w), columnwise=False)
        return float((mx_ref.host64(nv.mx_gemm(a["row_q"], a["row_sf"], b["row_q"], b["row_sf"], f32)) * dy).sum())

    dx = mx_ref.host64(nv.mx_gemm(qd["row_q"], qd["row_sf"], qw["col_q"], qw["col_sf"], f32))
    dw = mx_ref.host64(nv.mx_gemm(qd["col_q"], qd["col_sf"], qx["col_q"], qx["col_sf"], f32))
    assert np.array_equal(dx, dy @ w) and np.array_equal(dw, dy.T @ x)
    assert f(x2, w) - f(x, w) == (dx * (x2 - x)).sum()
    assert f(x, w2) - f(x, w) == (dw * (w2 - w)).sum()


def test_expert_gradients_against_differences():
    rng = np.random.default_rng(21)
    T, K, N, E, R = 60, 70, 40, 5, 150
    off = groups(rng, E, R)
    x, dy = grid_values(rng, (T, K)), grid_values(rng, (R, N))
    w, w2 = grid_values(rng, (E, N, K)), grid_values(rng, (E, N, K))
    idx = rng.integers(0, T, R).astype(np.int32)
    dev = lambda v: torch.from_numpy(v).to(torch.bfloat16).cuda()  # noqa: E731
    offd, idxd = torch.from_numpy(off).cuda(), torch.from_numpy(idx).cuda()

    def stack(w, key):
        o = [nv.mx_quantize(dev(v)) for v in w]
        return torch.stack([q[key + "_q"] for q in o]), torch.stack([q[key + "_sf"] for q in o])

    def f(x, w):
        y = nv.mx_linear_grouped(dev(x), *stack(w, "row"), offd, rows=idxd, out_dtype=torch.float32)
        return float((mx_ref.host64(y) * dy).sum())

    qd = nv.mx_quantize_grouped(dev(dy), offd)
    qx = nv.mx_quantize_grouped(dev(x), offd, rows=idxd, rowwise=False)
    dx = mx_ref.host64(nv.mx_gemm_grouped(qd["row_q"], qd["row_sf"], *stack(w, "col"), offd, out_dtype=torch.float32))
    dw = mx_ref.host64(nv.mx_wgrad_grouped(qd["col_q"], qd["col_sf"], qx["col_q"], qx["col_sf"], offd))
    x2 = grid_values(rng, (T, K))
    total = np.zeros((T, K))
    np.add.at(total, idx, dx)                            # a token's rows add up
    assert f(x2, w) - f(x, w) == (total * (x2 - x)).sum()
    assert f(x, w2) - f(x, w) == (dw * (w2 - w)).sum()


def test_outputs_and_operands_past_four_gigabytes():
    rng = np.random.default_rng(30)
    # out: 2^31 + elements, checked in its last rows
    (aq, asf, a), (bq, bsf, b) = vectors(rng, 130, 96), vectors(rng, 32800, 96)
    M = 65600
    big_q = aq.repeat(M // 130 + 1, 1)[:M].contiguous()
    r = torch.arange(M, device="cuda") % 130
    big_sf = torch.zeros(nv.mx_sf_shape(M, 96), dtype=torch.uint8, device="cuda")
    pos = torch.arange(M, device="cuda")
    big_sf[pos // 128, :, pos % 128] = asf[r // 128, :, r % 128]
    got = nv.mx_gemm(big_q, big_sf, bq, bsf)
    last = np.arange(M - 140, M) % 130
    mx_ref.check_product(got[-140:], a[last], b)
    del got, big_q, big_sf
    # an operand of 4.5 GB, its last vectors reached through row indices
    A, K = 560_000, 16384
    q = torch.zeros(A, K // 2, dtype=torch.uint8, device="cuda")
    sf = torch.zeros(nv.mx_sf_shape(A, K), dtype=torch.uint8, device="cuda")
    tq, tsf, t = vectors(rng, 4, K)
    q[-4:] = tq
    for i in range(4):
        at = A - 4 + i
        sf[at // 128, :, at % 128] = tsf[0, :, i]
    wq, wsf, w = vectors(rng, 30, K)
    for n in (4, 200):
        pick = rng.integers(0, 4, n)
        idx = torch.from_numpy((A - 4 + pick).astype(np.int32)).cuda()
        off = torch.tensor([0, n], dtype=torch.int32, device="cuda")
        got = nv.mx_gemm_grouped(q, sf, wq[None], wsf[None], off, rows=idx, out_dtype=torch.float32)
        mx_ref.check_product(got, t[pick], w)
    mx_ref.check_product(nv.mx_gemm(q, sf, wq, wsf, torch.float32)[-4:], t, w)


def test_on_a_stream_and_in_a_graph():
    rng = np.random.default_rng(31)
    x = [data(np.random.default_rng(s), 300, 256, torch.bfloat16) for s in (1, 2)]
    one = [v[:1].contiguous() for v in x]
    wq, wsf, w = vectors(rng, 200, 256)
    bq, bsf, _ = experts(rng, 6, 48, 256)
    off = torch.from_numpy(groups(rng, 6, 300)).cuda()
    buf, buf1 = x[0].clone(), one[0].clone()

    def work():
        q = nv.mx_quantize_grouped(buf, off)
        return (nv.mx_linear(buf, wq, wsf), nv.mx_linear(buf1, wq, wsf), nv.mx_linear_grouped(buf, bq, bsf, off),
                nv.mx_wgrad_grouped(q["col_q"], q["col_sf"], q["col_q"], q["col_sf"], off))

    def eager(i):
        buf.copy_(x[i])
        buf1.copy_(one[i])
        return [t.clone() for t in work()]

    want = [eager(0), eager(1)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = eager(1)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want[1]))
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        out = work()
    for i in (0, 1, 0, 1):
        buf.copy_(x[i])
        buf1.copy_(one[i])
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want[i]))
        assert all(torch.equal(a, b) for a, b in zip(eager(i), want[i]))


def test_the_same_twice():
    rng = np.random.default_rng(32)
    for M, N, K in ((1, 500, 8192), (40, 300, 8192), (700, 900, 1000)):
        (aq, asf, _), (bq, bsf, _) = vectors(rng, M, K), vectors(rng, N, K)
        first = nv.mx_gemm(aq, asf, bq, bsf, torch.float32)
        for _ in range(3):
            assert torch.equal(nv.mx_gemm(aq, asf, bq, bsf, torch.float32), first)
