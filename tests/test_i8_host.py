"""The 8-bit projection path without a GPU: argument checks of the entry points
(refused on the host before any launch) and of the binding, and the
definition's own properties."""
import numpy as np
import pytest
import torch

import i8_reference as ref
from linear_attention_recurrence_04_b200 import build as gdn_build
from linear_attention_recurrence_04_b200 import gdn

OK, NULL, SHAPE, UNSUP, ALIGN, OVERFLOW, CUDA, ALIAS = range(8)


@pytest.fixture(scope="module")
def lib():
    gdn_build.build()
    return gdn.load_library()


def fake(i):
    """Aligned device addresses 4 GiB apart, never dereferenced."""
    return (i + 1) << 32


def test_quantize_argument_checks(lib):
    def f(x=fake(1), xt=0, q=fake(2), s=fake(3), M=4, D=64):
        return lib.gdn_quantize_i8(x, xt, q, s, M, D, None)
    assert f(M=-1) == SHAPE and f(D=-16) == SHAPE
    assert f(D=24) == UNSUP and f(xt=2) == UNSUP and f(xt=-1) == UNSUP
    assert f(x=0) == NULL and f(q=0) == NULL and f(s=0) == NULL
    assert f(x=fake(1) + 8) == ALIGN and f(q=fake(2) + 4) == ALIGN and f(s=fake(3) + 2) == ALIGN
    assert f(M=1 << 31) == OVERFLOW and f(D=1 << 40) == OVERFLOW
    assert f(q=fake(1) + 64) == ALIAS and f(s=fake(1) + 1020) == ALIAS and f(s=fake(2) + 16) == ALIAS
    assert f(x=0, q=0, s=0, M=0) == OK and f(x=0, q=0, s=0, D=0) == OK
    assert b"" == lib.gdn_last_error()


def test_add_rms_norm_argument_checks(lib):
    def f(x=fake(1), xt=0, r=fake(2), w=fake(3), ro=fake(4), rt=1, q=fake(5), s=fake(6), M=4, D=64):
        return lib.gdn_add_rms_norm_i8(x, xt, r, w, 1e-6, ro, rt, q, s, M, D, None)
    assert f(M=-1) == SHAPE
    assert f(D=8) == UNSUP and f(rt=7) == UNSUP and f(xt=9) == UNSUP
    assert f(w=0) == NULL and f(x=0) == NULL
    assert f(r=fake(2) + 4) == ALIGN and f(ro=fake(4) + 8) == ALIGN and f(w=fake(3) + 4) == ALIGN
    # the residual in place is allowed only as a whole (refused here by x = 0)
    assert f(ro=fake(2) + 16) == ALIAS and f(ro=fake(2), q=fake(2) + 64) == ALIAS
    assert f(ro=fake(2), x=fake(2)) == ALIAS and f(ro=fake(1)) == ALIAS
    assert f(q=fake(3)) == ALIAS and f(s=fake(4)) == ALIAS and f(q=fake(2)) == ALIAS
    assert f(x=0, w=0, q=0, s=0, M=0) == OK


def test_linear_i8_argument_checks(lib):
    def f(x=fake(1), sx=fake(2), w=fake(3), sw=fake(4), y=fake(5), yt=0, M=4, N=4, K=64, st=0):
        return lib.gdn_linear_i8(x, sx, w, sw, y, yt, M, N, K, st, None)
    assert f(M=-1) == SHAPE and f(N=-1) == SHAPE and f(K=-16) == SHAPE
    assert f(K=8) == UNSUP and f(K=131072) == UNSUP and f(yt=2) == UNSUP
    assert f(x=0) == NULL and f(sx=0) == NULL and f(w=0) == NULL and f(sw=0) == NULL and f(y=0) == NULL
    assert f(x=fake(1) + 8) == ALIGN and f(y=fake(5) + 4) == ALIGN and f(sx=fake(2) + 1) == ALIGN
    assert f(st=fake(6) + 2) == ALIGN
    assert f(M=1 << 30) == OVERFLOW and f(N=1 << 40) == OVERFLOW and f(M=1 << 22, N=1 << 24) == OVERFLOW
    assert f(y=fake(1) + 16) == ALIAS and f(y=fake(2)) == ALIAS and f(st=fake(5)) == ALIAS
    assert f(x=0, w=0, y=0, M=0) == OK and f(x=0, w=0, y=0, N=0) == OK


def test_rows_of_no_elements(lib):
    """With D = 0 the scales are still written (as zeros), so their pointer is
    held to its alignment; nothing else is looked at."""
    assert lib.gdn_quantize_i8(0, 0, 0, fake(3) + 2, 4, 0, None) == ALIGN
    assert lib.gdn_add_rms_norm_i8(0, 0, 0, 0, 1e-6, 0, 0, 0, fake(3) + 1, 4, 0, None) == ALIGN
    assert lib.gdn_quantize_i8(0, 0, 0, fake(3) + 2, 0, 0, None) == OK


def test_binding_refuses(lib):
    x = torch.zeros(4, 64)
    i = torch.zeros(4, 64, dtype=torch.int8)
    s = torch.zeros(4)
    with pytest.raises(ValueError):
        gdn.quantize_i8(x)                                   # not a CUDA tensor
    with pytest.raises(TypeError):
        gdn.quantize_i8(x.half())
    with pytest.raises(TypeError):
        gdn.add_rms_norm_i8(i, torch.ones(64))
    with pytest.raises(ValueError):
        gdn.linear_i8(i, s, i[:, :32], s)                    # another K
    with pytest.raises(TypeError):
        gdn.linear_i8(x, s, i, s)
    with pytest.raises(ValueError):
        gdn.linear_i8(i, s, i, s)


def test_definition():
    """Halves go to even, the largest value to 127, q * scale is within half a
    step of the row, and a power of two times the row leaves q alone."""
    x = np.array([[254, 1, 3, 5, -1, -3, -253, 0]], np.float32)
    q, s, _ = ref.rows(x)
    assert q.tolist() == [[127, 0, 2, 2, 0, -2, -126, 0]] and s[0] == 2.0
    g = np.random.default_rng(0)
    x = g.standard_normal((50, 64)).astype(np.float32)
    q, s, _ = ref.rows(x)
    assert (np.abs(q).max(1) == 127).all()
    assert (np.abs(q * s[:, None] - x) <= 0.5 * s[:, None] * (1 + 1e-12)).all()
    assert np.array_equal(ref.rows(x * np.float32(2.0 ** -100))[0], q)
    # the norm's scale makes q * scale the normalised row
    w = (1 + 0.1 * g.standard_normal(64)).astype(np.float32)
    q, s, _ = ref.rows(x, None, w, 1e-6)
    want = x * w / np.sqrt(np.mean(x.astype(np.float64) ** 2, 1) + 1e-6)[:, None]
    assert (np.abs(q * s[:, None] - want) <= 0.5 * s[:, None] * (1 + 1e-6)).all()


def test_forward_batch_i8_argument_checks(lib):
    ws = lib.gdn_forward_batch_workspace_size(2, 3, 16, 32, 128, 128)

    def f(hidden=fake(1), hs=fake(2), w_out=fake(9), D=64, out=fake(20), ot=0, workspace=fake(21),
          bytes_=ws, K=4, Hv=32, B=2, T=3, norm_w=fake(15), st=0):
        return lib.gdn_forward_batch_i8(hidden, hs, fake(3), fake(4), fake(5), fake(6), fake(7),
                                        fake(8), w_out, fake(10), fake(11), fake(12), fake(13),
                                        fake(14), norm_w, 1e-6, 1e-6, fake(16), out, ot, workspace,
                                        bytes_, B, T, D, 16, Hv, 128, 128, K, st, None)
    assert f(D=24) == UNSUP and f(D=0) == UNSUP and f(D=131072) == UNSUP and f(Hv=1024) == UNSUP
    assert f(K=3) == UNSUP and f(ot=5) == UNSUP
    assert f(T=-1) == SHAPE and f(Hv=20) == SHAPE and f(bytes_=ws - 1) == SHAPE
    assert f(B=70000) == OVERFLOW
    assert f(hidden=0) == NULL and f(hs=0) == NULL and f(out=0) == NULL and f(workspace=0) == NULL
    assert f(hidden=fake(1) + 8) == ALIGN and f(workspace=fake(21) + 128) == ALIGN
    assert f(norm_w=fake(15) + 2) == ALIGN and f(st=fake(22) + 1) == ALIGN
    assert f(out=fake(21) + 256) == ALIAS and f(out=fake(1)) == ALIAS and f(out=fake(16)) == ALIAS
    assert f(w_out=fake(11)) == ALIAS                       # the ring is updated in place
    assert f(hidden=0, out=0, T=0) == OK
