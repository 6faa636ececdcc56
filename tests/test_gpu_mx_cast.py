"""MXFP4 cast and dequantization on the GPU against the plain reference:
every code and scale byte equal, nothing written outside the outputs."""
import numpy as np
import pytest
import torch

import nvfp4_block_scaled_bf16_amd as nv
from nvfp4_block_scaled_bf16_amd import mx
from tests import mx_ref
from tests.gpu_util import Guarded, U8, assert_bytes_equal, host

pytestmark = pytest.mark.gpu
TYPES = [torch.bfloat16, torch.float16, torch.float32]


def data(rng, M, K, dtype, wild=True):
    x = rng.standard_normal((M, K)) * np.exp(rng.standard_normal((M, 1)))
    if wild and M and K:
        x *= np.exp2(rng.integers(-12, 12, (M, K)))
        x[rng.random((M, K)) < 0.05] = 0.0
        x[rng.random((M, K)) < 0.01] *= -1e-6
    return torch.from_numpy(x).to(dtype).cuda()


def mx_spec(M, K, row=True, col=True):
    spec = {}
    if row:
        spec.update(row_q=(M * mx_ref.up(K, 128) // 2, U8), row_sf=(int(np.prod(nv.mx_sf_shape(M, K))), U8))
    if col:
        spec.update(col_q=(K * mx_ref.up(M, 128) // 2, U8), col_sf=(int(np.prod(nv.mx_sf_shape(K, M))), U8))
    return spec


def cast_guarded(x, row=True, col=True):
    M, K = x.shape
    g = Guarded(mx_spec(M, K, row, col))
    p = [g[k].data_ptr() if k in g else None for k in ("row_q", "row_sf", "col_q", "col_sf")]
    st = nv.lib().nvfp4_mx_quantize(x.data_ptr(), mx._TYPES[x.dtype], M, K, x.stride(0), *p,
                                    torch.cuda.current_stream().cuda_stream)
    assert st == 0, nv.lib().nvfp4_last_error()
    torch.cuda.synchronize()
    g.check_guards()
    return g


def check_cast(out, x64, row=True, col=True):
    for on, name, v in ((row, "row", x64), (col, "col", x64.T)):
        if on:
            c, s = mx_ref.quantize(v)
            sf = mx_ref.pack_scales(s)
            q = mx_ref.pack_codes(c)
            got_q = host(out[name + "_q"]).reshape(q.shape)
            nan = (s == 255).repeat(16, 1)          # a NaN block's codes are unspecified
            assert_bytes_equal(np.where(nan, 0, got_q), q, name + "_q")
            assert_bytes_equal(host(out[name + "_sf"]).reshape(sf.shape), sf, name + "_sf")


SHAPES = [(1, 1), (1, 32), (2, 31), (3, 33), (1, 4096), (127, 129), (128, 128), (129, 127), (300, 1000), (17, 2885),
          (260, 514), (64, 8200)]


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("M,K", SHAPES)
def test_both_directions(M, K, dtype):
    x = data(np.random.default_rng(M * 10007 + K), M, K, dtype)
    check_cast(cast_guarded(x), mx_ref.host64(x))


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("M,K", SHAPES)
@pytest.mark.parametrize("row", [True, False], ids=["row", "col"])
def test_one_direction(M, K, dtype, row):
    x = data(np.random.default_rng(M * 10009 + K), M, K, dtype)
    check_cast(cast_guarded(x, row, not row), mx_ref.host64(x), row, not row)


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("pitch,shift", [(301, 0), (304, 1), (512, 3), (299, 0)])
def test_row_pitch_and_alignment(dtype, pitch, shift):
    # rows begin anywhere: odd pitches and a base off every vector alignment
    base = data(np.random.default_rng(pitch), 70, 520, dtype).reshape(-1)
    x = base[shift:shift + 69 * pitch + 299].as_strided((70, 299), (pitch, 1))
    for row, col in ((True, True), (True, False)):
        check_cast(cast_guarded(x, row, col), mx_ref.host64(x), row, col)


def test_transposed_view_and_repeated_row():
    x = data(np.random.default_rng(5), 90, 70, torch.bfloat16)
    check_cast(nv.mx_quantize(x.t()), mx_ref.host64(x).T)
    check_cast(nv.mx_quantize(x.t(), columnwise=False), mx_ref.host64(x).T, col=False)
    r = x[3:4].expand(40, 70)                       # row pitch 0
    check_cast(nv.mx_quantize(r), mx_ref.host64(r))
    with pytest.raises(ValueError):
        nv.mx_quantize(x[:, ::2])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16], ids=str)
def test_every_16_bit_value_under_every_scale(dtype):
    # row s holds all finite values next to a maximum of exponent s, so that
    # every value meets every scale it can: 31 values and the maximum a block
    v = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(dtype).float()
    v = v[torch.isfinite(v)]
    v = torch.nn.functional.pad(v, (0, -len(v) % 31)).view(-1, 31)
    exps = range(-126, 128, 11) if dtype == torch.bfloat16 else range(-24, 16)
    for e in exps:
        top = 2.0 ** e
        w = torch.where(v.abs() <= top * 1.75, v, torch.zeros_like(v))
        x = torch.cat([w, torch.full((len(w), 1), top)], 1).to(dtype)
        x = x.cuda().contiguous()
        check_cast(nv.mx_quantize(x, columnwise=False), mx_ref.host64(x), col=False)
        t = x.t().contiguous()
        check_cast(nv.mx_quantize(t, rowwise=False), mx_ref.host64(t), row=False)


@pytest.mark.parametrize("dtype", TYPES, ids=str)
def test_zeros_subnormals_and_the_largest(dtype):
    fi = torch.finfo(dtype)
    tiny = torch.tensor([0.0, -0.0, fi.smallest_normal, -fi.smallest_normal / 2, fi.max, -fi.max, fi.eps, 1.0])
    rng = np.random.default_rng(6)
    x = tiny[torch.from_numpy(rng.integers(0, 8, (64, 256)))].to(dtype)
    x[:8] = 0.0
    x[8:16] = (torch.from_numpy(rng.random((8, 256))) * 8 * fi.smallest_normal).to(dtype)
    x[16:24] = -0.0
    x = x.cuda()
    check_cast(cast_guarded(x), mx_ref.host64(x))


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("bad", [float("inf"), -float("inf"), float("nan")])
def test_a_bad_value_spoils_its_block_alone(dtype, bad):
    x = data(np.random.default_rng(7), 200, 300, dtype, wild=False)
    x[5, 40] = bad
    x[199, 299] = bad
    out = cast_guarded(x)
    check_cast(out, mx_ref.host64(x))
    assert int((host(out["row_sf"]) == 255).sum()) == 2 and int((host(out["col_sf"]) == 255).sum()) == 2
    o = nv.mx_quantize(x)
    back = nv.mx_dequantize(o["row_q"], o["row_sf"], 300, dtype)
    nan = torch.isnan(back)
    assert nan[5, 32:64].all() and nan[199, 288:300].all() and int(nan.sum()) == 44


def test_fp32_between_the_grid():
    # fp32 values next to every midpoint, under several scales
    mid = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], np.float32)
    near = np.concatenate([mid, np.nextafter(mid, np.float32(0)), np.nextafter(mid, np.float32(9)), [4.0, 7.9, 6.0]])
    near = np.concatenate([near, -near])[:48]
    x = np.zeros((40, 64), np.float32)
    x[:, :48] = near
    x[:, 48] = x[:, 0] = 4.0
    x *= np.exp2(np.linspace(-120, 120, 40).round()).astype(np.float32)[:, None]
    x = torch.from_numpy(x).cuda()
    check_cast(cast_guarded(x), mx_ref.host64(x))


def groups(rng, E, R, empty=0.3):
    p = rng.dirichlet(np.full(E, 0.5)) * (rng.random(E) > empty)
    p = p / p.sum() if p.sum() > 0 else np.full(E, 1 / E)
    return np.concatenate([[0], np.cumsum(rng.multinomial(R, p))]).astype(np.int32)


def check_grouped_cast(out, x64, off, row=True):
    """x64: the R vectors; each group's columns in steps of its own."""
    R, K = x64.shape
    E = len(off) - 1
    Tp = nv.mx_padded_rows(R, E)
    assert tuple(out["col_q"].shape) == (K, Tp // 2)
    q = host(out["col_q"])
    s = host(out["col_sf"])
    at = 0
    for e in range(E):
        n = off[e + 1] - off[e]
        if n <= 0:
            continue
        c, sc = mx_ref.quantize(x64[off[e]:off[e + 1]].T)
        steps = c.shape[1] // 128
        assert_bytes_equal(q[:, 64 * at:64 * (at + steps)], mx_ref.pack_codes(c), f"group {e} codes")
        assert_bytes_equal(s[:, at:at + steps], mx_ref.pack_scales(sc), f"group {e} scales")
        at += steps
    if row:
        c, sc = mx_ref.quantize(x64)
        assert_bytes_equal(host(out["row_q"])[:off[-1]], mx_ref.pack_codes(c)[:off[-1]], "row_q")
        r, b = np.meshgrid(np.arange(off[-1]), np.arange(sc.shape[1]), indexing="ij")
        got = host(out["row_sf"])[r // 128, b // 4, r % 128, b % 4]
        assert_bytes_equal(got, sc[:off[-1]], "row_sf")


@pytest.mark.parametrize("E,R,K", [(1, 1, 1), (1, 200, 70), (5, 130, 129), (7, 1000, 300), (70, 500, 40), (130, 1500, 33)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=str)
def test_grouped(E, R, K, dtype):
    rng = np.random.default_rng(E * 1000 + R)
    off = groups(rng, E, R)
    x = data(rng, R, K, dtype)
    out = nv.mx_quantize_grouped(x, torch.from_numpy(off).cuda())
    check_grouped_cast(out, mx_ref.host64(x), off)


@pytest.mark.parametrize("rowwise", [True, False])
def test_grouped_with_rows(rowwise):
    rng = np.random.default_rng(11)
    x = data(rng, 90, 200, torch.bfloat16)
    idx = rng.integers(0, 90, 400).astype(np.int32)
    idx[[0, 17, 399]] = [-1, 90, 2 ** 31 - 1]       # outside: rows of zeros
    off = groups(rng, 9, 400)
    v = np.zeros((400, 200))
    inside = (idx >= 0) & (idx < 90)
    v[inside] = mx_ref.host64(x)[idx[inside]]
    out = nv.mx_quantize_grouped(x, torch.from_numpy(off).cuda(), rows=torch.from_numpy(idx).cuda(), rowwise=rowwise)
    check_grouped_cast(out, v, off, rowwise)
    if rowwise:                                      # rows alone take their own kernel
        o = nv.mx_quantize_grouped(x, torch.from_numpy(off).cuda(), rows=torch.from_numpy(idx).cuda(), columnwise=False)
        check_cast(o, v, col=False)


def test_offsets_out_of_order_stay_inside():
    # held to [0, R], a group that ends before it begins is empty
    x = data(np.random.default_rng(12), 300, 64, torch.bfloat16)
    off = torch.tensor([-5, 100, 40, 1000, 2 ** 31 - 1], dtype=torch.int32, device="cuda")
    out = nv.mx_quantize_grouped(x, off)
    torch.cuda.synchronize()
    c, s = mx_ref.quantize(mx_ref.host64(x)[:100].T)
    assert_bytes_equal(host(out["col_q"])[:, :64], mx_ref.pack_codes(c), "first group")


@pytest.mark.parametrize("dtype", TYPES, ids=str)
def test_dequantize_every_code_and_scale(dtype):
    # 255 scales (every code but NaN's) x 16 codes, then odd widths
    codes = np.tile(np.arange(16, dtype=np.uint8), (256, 8))
    s = np.repeat(np.arange(256, dtype=np.uint8)[:, None], 4, 1)
    q, sf = torch.from_numpy(mx_ref.pack_codes(codes)).cuda(), torch.from_numpy(mx_ref.pack_scales(s)).cuda()
    want = torch.from_numpy(mx_ref.values(codes, s)).float().to(dtype)
    for C in (128, 127, 121, 97, 100):
        got = nv.mx_dequantize(q, sf, C, dtype).cpu()
        w = want[:, :C]
        assert got.shape == w.shape and torch.equal(torch.isnan(got), torch.isnan(w))
        assert torch.equal(torch.nan_to_num(got, 0.0), torch.nan_to_num(w, 0.0))


def test_round_trip_is_idempotent():
    x = data(np.random.default_rng(13), 257, 1023, torch.float32)
    o = nv.mx_quantize(x)
    v = nv.mx_dequantize(o["row_q"], o["row_sf"], 1023)
    again = nv.mx_quantize(v, columnwise=False)
    assert torch.equal(nv.mx_dequantize(again["row_q"], again["row_sf"], 1023), v)


def test_empty():
    for shape in ((0, 5), (5, 0), (0, 0)):
        o = nv.mx_quantize(torch.zeros(shape, device="cuda"))
        assert tuple(nv.mx_dequantize(o["row_q"], o["row_sf"], shape[1]).shape) == shape


def test_rows_past_two_gigabytes():
    # the last rows of x lie past 2^31 and 2^32 bytes
    K, M = 4096, 600_000
    x = torch.zeros(M, K, dtype=torch.bfloat16, device="cuda")
    tail = data(np.random.default_rng(14), 3, K, torch.bfloat16)
    x[-3:] = tail
    o = nv.mx_quantize(x, columnwise=False)
    c, s = mx_ref.quantize(mx_ref.host64(tail))
    assert_bytes_equal(host(o["row_q"][-3:]), mx_ref.pack_codes(c), "row_q")
    got = nv.mx_dequantize(o["row_q"], o["row_sf"], K, torch.bfloat16)[-3:]
    assert np.array_equal(mx_ref.host64(got), mx_ref.values(c, s))
    idx = torch.tensor([M - 1, 0, M - 3], dtype=torch.int32, device="cuda")
    g = nv.mx_quantize_grouped(x, torch.tensor([0, 3], dtype=torch.int32, device="cuda"), rows=idx)
    v = mx_ref.host64(x[idx.long()])
    check_grouped_cast(g, v, np.array([0, 3]))
