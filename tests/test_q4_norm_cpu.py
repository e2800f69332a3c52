"""The RMS norm and the 4-bit linear layer without a GPU: pins of the oracle by
hand and by properties, the host queries, and the refusal of bad arguments
with the documented status before anything touches a device."""
import numpy as np
import pytest

from oracle import q4_norm_oracle as q4o
from oracle import ternary_oracle as orc
from ternary_weight_signed_b200 import binding as tb
from ternary_weight_signed_b200 import build as tbbuild

FAKE = 0x10000  # 16-byte aligned, never dereferenced (validation fails first)


@pytest.fixture(scope="module")
def lib():
    tbbuild.build()
    return tb.load()


# ------------------------------------------------------------------ oracle pins
def test_pack_by_hand():
    codes = np.zeros((1, 128), dtype=np.int8)
    codes[0, :6] = [-8, 7, 0, -1, 3, -5]
    b = q4o.pack(codes)
    assert b.shape == (1, 64)
    assert list(b[0, :4]) == [0xF0, 0x78, 0x3B, 0x88]  # k = 2i low nibble, q + 8
    assert np.array_equal(q4o.unpack(b, 1, 128), codes)


def test_every_byte_unpacks_to_its_nibbles():
    q = q4o.unpack(np.arange(256, dtype=np.uint8), 4, 128).reshape(-1)
    for b in range(256):
        assert q[2 * b] == (b & 15) - 8 and q[2 * b + 1] == (b >> 4) - 8


def test_prepare_by_hand():
    w = np.zeros((1, 256))
    w[0, :5] = [7.0, -7.0, 0.5, 1.5, -2.4]  # s = 1: halves to even
    q, s = q4o.prepare_weights(w)
    assert s[0, 0] == 1.0 and list(q[0, :5]) == [7, -7, 0, 2, -2]
    assert s[0, 1] == 0.0 and not q[0, 128:].any()
    # the scale is rounded down by fp16 and the codes are clipped to the range
    w[0, 0] = 1.0
    w[0, 1:5] = [-1.0, 0, 0, 0]
    q, s = q4o.prepare_weights(w)
    assert s[0, 0] == np.float16(np.float32(1 / 7)) and list(q[0, :2]) == [7, -7]
    w[0, 0] = 1e9
    q, s = q4o.prepare_weights(w)
    assert s[0, 0] == 8188.0 and q[0, 0] == 7


def test_prepare_fold_is_the_rotation():
    rng = np.random.default_rng(3)
    w, signs = rng.standard_normal((3, 1024)), rng.choice([-1, 1], 1024).astype(np.int8)
    x = rng.standard_normal((2, 1024))
    q, s = q4o.prepare_weights(w, signs)
    y = q4o.linear(x, q, s, signs=signs)
    # 4 bits of |w'| up to 4.2 sigma: steps of 0.6 sigma, an error of 0.17 sigma rms
    assert np.linalg.norm(y - x @ w.T) / np.linalg.norm(x @ w.T) < 0.5


def test_norm_by_hand_and_invariants():
    n = q4o.rms_norm(np.array([[3.0, -4.0]]), None, 0.0)
    assert np.allclose(n, np.array([[3.0, -4.0]]) / np.sqrt(12.5), rtol=1e-15)
    n = q4o.rms_norm(np.array([[3.0, -4.0]]), [2.0, 0.5], 12.5)
    assert np.allclose(n, [[6.0 / 5.0, -2.0 / 5.0]], rtol=1e-15)
    rng = np.random.default_rng(4)
    h, d = rng.standard_normal((3, 2048)), rng.choice([-1, 1], 2048).astype(np.int8)
    a, b = q4o.rms_norm(h, None, 1e-30), q4o.rms_norm(h, None, 1e-30, d)
    assert np.allclose((a * a).mean(1), 1.0) and np.allclose((b * b).sum(1), (a * a).sum(1))
    assert np.allclose(orc.rotate(a, d), b)


def test_linear_brute_force():
    rng = np.random.default_rng(5)
    q = rng.integers(-8, 8, (3, 256)).astype(np.int8)
    s = rng.random((3, 2)).astype(np.float16)
    x = rng.integers(-127, 128, (2, 256))
    xs = rng.random((2, 2)).astype(np.float32)
    y = q4o.linear(x, q, s, xs)
    for m in range(2):
        for n in range(3):
            v = sum(float(s[n, k // 128]) * int(q[n, k]) * int(x[m, k]) * float(xs[m, k // 128]) for k in range(256))
            assert abs(y[m, n] - v) < 1e-9 * max(1.0, abs(v))


# ------------------------------------------------------------------ host queries
@pytest.mark.parametrize("n,k", [(1, 128), (3, 384), (17408, 5120)])
def test_packed_bytes(lib, n, k):
    assert tb.tb_q4_packed_bytes(n, k) == n * k // 2


def test_queries_reject(lib):
    for n, k in ((0, 128), (4, 100), (4, 0), (-1, 128)):
        assert tb.tb_q4_packed_bytes(n, k) == 0
        assert tb.tb_q4_linear_workspace(1, n, k) == 0
    assert tb.tb_q4_linear_workspace(0, 4, 128) == 0
    assert tb.tb_q4_linear_workspace(1, 4, 128) > 0
    assert tb.status_string(tb.TB_ERR_VALUE) == "bad value"


# ------------------------------------------------------------------ refusals
def _norm(**kw):
    a = dict(x=FAKE, xt=tb.TB_BF16, residual=FAKE + 4096, residual_out=FAKE + 4096, rt=tb.TB_FP32, weight=FAKE,
             wt=tb.TB_BF16, eps=1e-6, signs=None, m=2, k=1024, y=FAKE + 8192, yt=tb.TB_BF16, y_scales=None,
             scale_group=0)
    a.update(kw)
    return tb.tb_rms_norm(**a, stream=0, check=False)


def test_norm_refusals(lib):
    i8 = dict(yt=tb.TB_INT8, y_scales=FAKE, scale_group=1024)
    assert _norm(x=None) == tb.TB_ERR_NULL
    assert _norm(y=None) == tb.TB_ERR_NULL
    assert _norm(residual=None) == tb.TB_ERR_NULL
    assert _norm(residual_out=None) == tb.TB_ERR_NULL
    assert _norm(**{**i8, "y_scales": None}) == tb.TB_ERR_NULL
    assert _norm(y_scales=FAKE) == tb.TB_ERR_DTYPE
    assert _norm(xt=tb.TB_INT8) == tb.TB_ERR_DTYPE
    assert _norm(rt=tb.TB_E4M3) == tb.TB_ERR_DTYPE
    assert _norm(wt=tb.TB_INT32) == tb.TB_ERR_DTYPE
    assert _norm(yt=tb.TB_INT32) == tb.TB_ERR_DTYPE
    assert _norm(yt=6) == tb.TB_ERR_DTYPE
    assert _norm(m=0) == tb.TB_ERR_SHAPE
    assert _norm(k=0) == tb.TB_ERR_SHAPE
    assert _norm(k=tb.TB_RMS_NORM_MAX_K + 1) == tb.TB_ERR_SHAPE
    assert _norm(k=1536, signs=FAKE) == tb.TB_ERR_SHAPE
    assert _norm(scale_group=128) == tb.TB_ERR_SHAPE              # groups of a floating output
    assert _norm(**{**i8, "scale_group": 0}) == tb.TB_ERR_SHAPE
    assert _norm(**{**i8, "scale_group": 64}) == tb.TB_ERR_SHAPE
    assert _norm(**{**i8, "scale_group": 128}, k=1000) == tb.TB_ERR_SHAPE
    for eps in (0.0, -1e-6, float("nan"), float("inf")):
        assert _norm(eps=eps) == tb.TB_ERR_VALUE
    assert _norm(x=FAKE + 1) == tb.TB_ERR_ALIGN
    assert _norm(residual=FAKE + 2, residual_out=FAKE + 2) == tb.TB_ERR_ALIGN
    assert _norm(weight=FAKE + 1) == tb.TB_ERR_ALIGN
    assert _norm(signs=FAKE + 4) == tb.TB_ERR_ALIGN
    assert _norm(**{**i8, "y_scales": FAKE + 2}) == tb.TB_ERR_ALIGN
    assert _norm(y=FAKE, yt=tb.TB_FP16) == tb.TB_ERR_DTYPE         # in place needs one dtype
    assert _norm(residual=FAKE + 4096, residual_out=FAKE) == tb.TB_ERR_DTYPE


def _lin(**kw):
    a = dict(x=FAKE, xt=tb.TB_BF16, x_scales=None, x_group=0, packed=FAKE, scales=FAKE, m=1, n=256, k=1024, signs=None,
             y=FAKE, yt=tb.TB_BF16, workspace=FAKE, ws_bytes=1 << 30)
    a.update(kw)
    return tb.tb_q4_linear(**a, stream=0, check=False)


def test_linear_refusals(lib):
    i8 = dict(xt=tb.TB_INT8, x_scales=FAKE, x_group=1024)
    for name in ("x", "packed", "scales", "y"):
        assert _lin(**{name: None}) == tb.TB_ERR_NULL
    assert _lin(**{**i8, "x_scales": None}) == tb.TB_ERR_NULL
    assert _lin(x_scales=FAKE) == tb.TB_ERR_DTYPE                  # scales beside a floating x
    assert _lin(**i8, signs=FAKE) == tb.TB_ERR_DTYPE               # rotated before the rounding, not after
    assert _lin(xt=tb.TB_FP32) == tb.TB_ERR_DTYPE
    assert _lin(xt=tb.TB_INT32) == tb.TB_ERR_DTYPE
    assert _lin(yt=tb.TB_INT32) == tb.TB_ERR_DTYPE
    assert _lin(m=0) == tb.TB_ERR_SHAPE
    assert _lin(n=0) == tb.TB_ERR_SHAPE
    assert _lin(k=1000) == tb.TB_ERR_SHAPE
    assert _lin(k=1152, signs=FAKE) == tb.TB_ERR_SHAPE
    assert _lin(x_group=128) == tb.TB_ERR_SHAPE
    assert _lin(**{**i8, "x_group": 256}) == tb.TB_ERR_SHAPE
    assert _lin(x=FAKE + 8) == tb.TB_ERR_ALIGN
    assert _lin(packed=FAKE + 8) == tb.TB_ERR_ALIGN
    assert _lin(scales=FAKE + 1) == tb.TB_ERR_ALIGN
    assert _lin(y=FAKE + 1) == tb.TB_ERR_ALIGN
    assert _lin(signs=FAKE + 4) == tb.TB_ERR_ALIGN
    assert _lin(**{**i8, "x_scales": FAKE + 2}) == tb.TB_ERR_ALIGN
    assert _lin(workspace=None) == tb.TB_ERR_WORKSPACE
    assert _lin(ws_bytes=tb.tb_q4_linear_workspace(1, 256, 1024) - 1) == tb.TB_ERR_WORKSPACE
    assert _lin(workspace=FAKE + 8) == tb.TB_ERR_ALIGN


def test_weights_refusals(lib):
    f = tb.tb_q4_pack
    assert f(None, 4, 128, FAKE, stream=0, check=False) == tb.TB_ERR_NULL
    assert f(FAKE, 4, 100, FAKE, stream=0, check=False) == tb.TB_ERR_SHAPE
    assert f(FAKE, 0, 128, FAKE, stream=0, check=False) == tb.TB_ERR_SHAPE
    assert f(FAKE + 8, 4, 128, FAKE, stream=0, check=False) == tb.TB_ERR_ALIGN
    assert f(FAKE, 4, 128, FAKE, FAKE + 2, stream=0, check=False) == tb.TB_ERR_ALIGN
    f = tb.tb_q4_unpack
    assert f(FAKE, 4, 128, None, stream=0, check=False) == tb.TB_ERR_NULL
    assert f(FAKE, 4, 192, FAKE, stream=0, check=False) == tb.TB_ERR_SHAPE
    assert f(FAKE, 4, 128, FAKE + 4, stream=0, check=False) == tb.TB_ERR_ALIGN
    f, bf = tb.tb_q4_prepare_weights, tb.TB_BF16
    assert f(None, bf, None, 4, 128, FAKE, FAKE, stream=0, check=False) == tb.TB_ERR_NULL
    assert f(FAKE, bf, None, 4, 128, FAKE, None, stream=0, check=False) == tb.TB_ERR_NULL
    assert f(FAKE, tb.TB_E4M3, None, 4, 128, FAKE, FAKE, stream=0, check=False) == tb.TB_ERR_DTYPE
    assert f(FAKE, bf, FAKE, 4, 1536, FAKE, FAKE, stream=0, check=False) == tb.TB_ERR_SHAPE
    assert f(FAKE, bf, None, 4, 64, FAKE, FAKE, stream=0, check=False) == tb.TB_ERR_SHAPE
    assert f(FAKE + 2, bf, None, 4, 128, FAKE, FAKE, stream=0, check=False) == tb.TB_ERR_ALIGN
    assert f(FAKE, bf, None, 4, 128, FAKE + 8, FAKE, stream=0, check=False) == tb.TB_ERR_ALIGN
    assert f(FAKE, bf, FAKE + 4, 4, 1024, FAKE, FAKE, stream=0, check=False) == tb.TB_ERR_ALIGN


def test_path_rejects(lib):
    """What the call would refuse has no path (nor has anything without a device)."""
    p = tb.tb_q4_linear_path
    for a in ((tb.TB_FP32, 1, 4, 128), (tb.TB_BF16, 0, 4, 128), (tb.TB_BF16, 1, 0, 128), (tb.TB_BF16, 1, 4, 100),
              (tb.TB_BF16, 1, 4, 128, True), (tb.TB_INT8, 1, 4, 1024, True), (tb.TB_BF16, 2 ** 31, 4, 128)):
        assert p(*a) == -1
