"""Refusals of the MXFP4 entry points (CPU): every bad argument gets its
documented status before anything is launched, and the binding rejects what the
library would misread."""
import pytest
import torch

import nvfp4_block_scaled_bf16_amd as nv

OK, EINVAL, ESHAPE, EALIGN = 0, 1, 2, 3
F = 0x10000        # an aligned address that is never dereferenced: validation fails first
BF16 = 1
BIG = 1 << 31


def L():
    return nv.lib()


def test_quantize():
    q = L().nvfp4_mx_quantize
    assert q(F, BF16, 16, 16, 16, None, None, None, None, None) == EINVAL          # no direction
    assert b"direction" in L().nvfp4_last_error()
    assert q(F, BF16, 16, 16, 16, F, None, None, None, None) == EINVAL             # half a direction
    assert q(F, BF16, 16, 16, 16, F, F, None, F, None) == EINVAL
    assert q(F, 3, 16, 16, 16, F, F, F, F, None) == EINVAL                         # type
    assert q(F, BF16, -1, 16, 16, F, F, F, F, None) == EINVAL
    assert q(F, BF16, 16, 16, -16, F, F, F, F, None) == EINVAL                     # pitch
    assert q(None, BF16, 16, 16, 16, F, F, F, F, None) == EINVAL
    assert q(F, BF16, 16, (1 << 23) + 1, 1 << 24, F, F, None, None, None) == ESHAPE
    assert q(F, BF16, BIG, 16, 16, F, F, None, None, None) == ESHAPE
    assert q(F, BF16, BIG - 1, 1 << 23, 1 << 23, F, F, F, F, None) == ESHAPE       # tiles
    assert q(F + 1, BF16, 16, 16, 16, F, F, F, F, None) == EALIGN
    assert q(F + 2, 0, 16, 16, 16, F, F, F, F, None) == EALIGN                     # fp32 needs 4
    assert q(F, BF16, 16, 16, 16, F + 8, F, F, F, None) == EALIGN
    assert q(F, BF16, 16, 16, 16, F, F + 2, F, F, None) == EALIGN
    assert q(None, BF16, 0, 16, 16, F, F, F, F, None) == OK                        # nothing to do


def test_quantize_grouped():
    q = L().nvfp4_mx_quantize_grouped
    assert q(F, BF16, 16, 16, 16, None, 16, None, 2, F, F, F, F, None) == EINVAL   # offsets
    assert q(F, BF16, 16, 16, 16, None, 16, F, -1, F, F, F, F, None) == EINVAL
    assert q(F, BF16, 16, 16, 16, None, 17, F, 2, F, F, F, F, None) == EINVAL      # R without rows
    assert q(F, BF16, 16, 16, 16, F, BIG, F, 2, F, F, F, F, None) == ESHAPE
    assert q(F, BF16, 16, 16, 16, F + 2, 17, F, 2, F, F, F, F, None) == EALIGN
    assert q(F, BF16, 16, 16, 16, None, 16, F + 1, 2, F, F, F, F, None) == EALIGN
    assert q(None, BF16, 0, 16, 16, F, 5, F, 2, F, F, F, F, None) == EINVAL        # rows of nothing


def test_dequantize():
    d = L().nvfp4_mx_dequantize
    assert d(F, F, 4, 32, 9, F, None) == EINVAL
    assert d(F, F, -4, 32, 0, F, None) == EINVAL
    assert d(None, F, 4, 32, 0, F, None) == EINVAL
    assert d(F, F, 4, 32, 0, None, None) == EINVAL
    assert d(F + 4, F, 4, 32, 0, F, None) == EALIGN
    assert d(F, F, 4, 32, 0, F + 2, None) == EALIGN
    assert d(None, None, 0, 32, 0, None, None) == OK


def test_gemm():
    g = L().nvfp4_mx_gemm
    assert g(F, F, F, F, -1, 4, 32, BF16, F, None) == EINVAL
    assert g(F, F, F, F, 4, 4, 32, 5, F, None) == EINVAL
    assert g(F, None, F, F, 4, 4, 32, BF16, F, None) == EINVAL
    assert g(F, F, F, F, 4, 4, 32, BF16, None, None) == EINVAL
    assert g(F, F, F, F, 4, 4, (1 << 23) + 1, BF16, F, None) == ESHAPE
    assert g(F, F, F, F, BIG, 4, 32, BF16, F, None) == ESHAPE
    assert g(F, F, F, F, BIG - 1, BIG - 1, 32, BF16, F, None) == ESHAPE
    assert g(F, F, F + 8, F, 4, 4, 32, BF16, F, None) == EALIGN
    assert g(F, F, F, F + 2, 4, 4, 32, BF16, F, None) == EALIGN
    assert g(F, F, F, F, 4, 4, 32, BF16, F + 1, None) == EALIGN
    assert g(None, None, None, None, 0, 4, 32, BF16, None, None) == OK


def test_grouped_and_wgrad():
    g = L().nvfp4_mx_gemm_grouped
    a = lambda **k: list({**dict(aq=F, asf=F, A=8, rows=None, R=8, off=F, E=2, bq=F, bsf=F, N=4, K=32, s=None, t=1, out=F,  # noqa: E731
                                 st=None), **k}.values())
    assert g(*a(off=None)) == EINVAL and g(*a(E=-1)) == EINVAL and g(*a(R=9)) == EINVAL and g(*a(t=3)) == EINVAL
    assert g(*a(bq=None)) == EINVAL and g(*a(out=None)) == EINVAL and g(*a(A=0, rows=F)) == EINVAL
    assert g(*a(s=F + 2)) == EALIGN and g(*a(rows=F + 2)) == EALIGN and g(*a(bsf=F + 1)) == EALIGN
    assert g(*a(N=BIG)) == ESHAPE and g(*a(K=BIG)) == ESHAPE
    assert g(*a(N=0)) == OK and g(*a(E=0)) == OK and g(*a(A=0, R=0)) == OK
    w = L().nvfp4_mx_wgrad_grouped
    assert w(F, F, F, F, 4, 4, 100, F, 2, 0, F, None) == ESHAPE
    assert w(F, F, F, F, 4, 4, (1 << 23) + 128, F, 2, 0, F, None) == ESHAPE
    assert w(F, F, F, F, 4, 4, 128, None, 2, 0, F, None) == EINVAL
    assert w(F, F, F, F, 4, -4, 128, F, 2, 0, F, None) == EINVAL
    assert w(F, F, F, F, BIG - 1, 256, 128, F, 1 << 20, 0, F, None) == ESHAPE
    assert w(F, F, None, F, 4, 4, 128, F, 2, 0, F, None) == EINVAL
    assert w(F, F, F, F, 4, 4, 128, F, 2, 0, F + 2, None) == EALIGN
    assert w(F, F, F, F, 4, 0, 128, F, 2, 0, F, None) == OK


def test_linear_needs_its_workspace():
    f, need = L().nvfp4_mx_linear, L().nvfp4_mx_linear_workspace
    n = need(500, 256, 300)
    assert n > 0 and need(-1, 4, 4) == 0 and need(0, 4, 4) == 0
    assert f(F, BF16, 500, 300, 300, F, F, 256, BF16, F, None, 0, None) == EINVAL
    assert f(F, BF16, 500, 300, 300, F, F, 256, BF16, F, F, n - 1, None) == EINVAL
    assert b"workspace" in L().nvfp4_last_error()
    assert f(F, BF16, 500, 300, 300, F, F, 256, BF16, F, F + 8, n, None) == EALIGN
    assert f(F, BF16, 500, 300, 300, F, None, 256, BF16, F, F, n, None) == EINVAL
    assert f(F, BF16, 500, -3, 300, F, F, 256, BF16, F, F, n, None) == EINVAL
    h, need = L().nvfp4_mx_linear_grouped, L().nvfp4_mx_linear_grouped_workspace
    n = need(500, 700, 4096, 300)
    assert n > 0
    assert h(F, BF16, 500, 300, 300, F, 700, F, 4, F, F, 4096, None, BF16, F, F, n - 1, None) == EINVAL
    assert h(F, BF16, 500, 300, 300, None, 700, F, 4, F, F, 4096, None, BF16, F, F, n, None) == EINVAL
    assert h(F, BF16, 0, 300, 300, F, 700, F, 4, F, F, 4096, None, BF16, F, F, n, None) == EINVAL
    assert h(F, BF16, 500, 300, 300, F, 700, None, 4, F, F, 4096, None, BF16, F, F, n, None) == EINVAL


def test_status_reaches_python():
    with pytest.raises(nv.NVFP4Error) as e:
        nv._check(L().nvfp4_mx_gemm(F, F, F, F, 4, 4, 32, 5, F, None))
    assert e.value.status == EINVAL and "type" in str(e.value)


def test_binding_checks_without_a_gpu():
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    q, sf = torch.zeros(4, 64, dtype=torch.uint8), torch.zeros(1, 1, 128, 4, dtype=torch.uint8)
    off = torch.zeros(3, dtype=torch.int32)
    for call in (lambda: nv.mx_quantize(x), lambda: nv.mx_quantize([1.0]), lambda: nv.mx_dequantize(q, sf, 64),
                 lambda: nv.mx_gemm(q, sf, q, sf), lambda: nv.mx_linear(x, q, sf),
                 lambda: nv.mx_quantize_grouped(x, off), lambda: nv.mx_wgrad_grouped(q, sf, q, sf, off),
                 lambda: nv.mx_linear_grouped(x, q[None], sf[None], off)):
        with pytest.raises(ValueError):
            call()


def test_sizes():
    assert nv.mx_sf_shape(1, 1) == (1, 1, 128, 4) and nv.mx_sf_shape(129, 256) == (2, 2, 128, 4)


def test_padded_rows_cover_every_split():
    # most[E][R]: the longest that E groups of R rows in all can get, by the
    # last group's size
    most = [[0] * 301]
    most[0][1:] = [-1] * 300
    for E in range(1, 6):
        last = most[-1]
        most.append([max(last[R - c] + -(-c // 128) * 128 for c in range(R + 1) if last[R - c] >= 0) for R in range(301)])
        for R in range(301):
            assert nv.mx_padded_rows(R, E) % 128 == 0
            assert most[E][R] <= nv.mx_padded_rows(R, E)
            assert R <= nv.mx_padded_rows(R, E)


def test_another_device_is_made_current_for_the_call(monkeypatch):
    import contextlib

    from nvfp4_block_scaled_bf16_amd import mx

    current, seen = [0], []

    @contextlib.contextmanager
    def device(index):
        last, current[0] = current[0], index
        yield
        current[0] = last

    def fn(*args):
        seen.append((current[0], args))
        return 0

    monkeypatch.setattr(torch.cuda, "current_device", lambda: current[0])
    monkeypatch.setattr(torch.cuda, "device", device)
    monkeypatch.setattr(mx, "_raw_stream", lambda index: 100 + index)
    mx._call(0, fn, 7)
    mx._call(1, fn, 8)
    assert seen == [(0, (7, 100)), (1, (8, 101))] and current == [0]
