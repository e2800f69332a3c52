"""GPU parity of the 4-bit linear layer: tb_q4_pack / unpack / prepare_weights
bit for bit, tb_q4_linear against its definition in float64
(oracle/q4_norm_oracle.py), and the chain norm -> 8 bits -> linear.

Tolerances of the linear layer, counted in roundings before the first run.
With T = sum |w| |x'|:
  * fp32 sums.  A chain of at most 160 additions whose partial sums grow to T is
    off by less than 160 / 2 * 2^-24 T < 2^-17 T.
  * up to 16 tokens x' is held in 8-bit planes of a fixed-point number per
    128-group: one for an int8 (exact), three up to 5 tokens, else two.  The
    largest of the group, X, is at least 2^21 steps with three and 2^14 with two,
    so a value is off by half a step, 2^-22 or 2^-15 of X: sum |w| X times that.
  * past 16 tokens a weight and, where x is rotated, x' are rounded to 11 bits:
    independent errors of 2^-11 / sqrt(3) rms each at most, so at most
    2^-11 sqrt(2/3) < 2^-11 of y in relative L2 over a whole output, and at most
    2^-10 T for one.
  * a rotated x': ten levels of fp32 sums of up to sum |x| / 32 of its block, at
    most 2^-21 of that; the terms above with 2^-10 T leave room for it.
y's own type adds eps / 2 of each value."""
import functools

import numpy as np
import pytest
import torch

from oracle import q4_norm_oracle as q4o
from ternary_weight_signed_b200 import binding as tb
from tests.gpu_util import DEV, ensure_lib

pytestmark = pytest.mark.gpu

T = {"bf16": (tb.TB_BF16, torch.bfloat16), "fp16": (tb.TB_FP16, torch.float16), "fp32": (tb.TB_FP32, torch.float32),
     "int8": (tb.TB_INT8, torch.int8), "e4m3": (tb.TB_E4M3, torch.float8_e4m3fn)}


@pytest.fixture(scope="module", autouse=True)
def _lib():
    ensure_lib()
    tb.tb_get_device_fault(clear=True)
    yield
    assert tb.tb_get_device_fault() == 0


def draw_signs(rng, k):
    return torch.from_numpy(rng.choice([-1, 1], k).astype(np.int8))


# ------------------------------------------------------------------ weights
@pytest.mark.parametrize("n,k", [(1, 128), (3, 384), (301, 1024), (5, 5120)])
def test_pack_and_unpack(n, k):
    rng = np.random.default_rng(n)
    codes = rng.integers(-8, 8, (n, k)).astype(np.int8)
    packed = torch.zeros(tb.tb_q4_packed_bytes(n, k), dtype=torch.uint8, device=DEV)
    count = torch.zeros(1, dtype=torch.int32, device=DEV)
    tb.tb_q4_pack(torch.from_numpy(codes).to(DEV), n, k, packed, count)
    assert np.array_equal(packed.cpu().numpy().reshape(n, k // 2), q4o.pack(codes)) and int(count) == 0
    back = torch.full((n, k), 77, dtype=torch.int8, device=DEV)
    tb.tb_q4_unpack(packed, n, k, back)
    assert np.array_equal(back.cpu().numpy(), codes)
    # values outside the range go to its nearer end and are counted
    wild = codes.copy()
    wild[0, [0, 5, 127]] = [8, -9, -128]
    tb.tb_q4_pack(torch.from_numpy(wild).to(DEV), n, k, packed, count)
    assert np.array_equal(packed.cpu().numpy().reshape(n, k // 2), q4o.pack(np.clip(wild, -8, 7))) and int(count) == 3
    tb.tb_q4_pack(torch.from_numpy(wild).to(DEV), n, k, packed)  # no counter


@pytest.mark.parametrize("n,k,folded", [(1, 128, True), (9, 1152, True), (301, 2048, True), (7, 640, True), (1, 1024, False),
                                        (67, 5120, False), (301, 2048, False)])
@pytest.mark.parametrize("wt", ["bf16", "fp16", "fp32"])
def test_prepare_bitexact(n, k, folded, wt):
    rng = np.random.default_rng(n + k)
    v = rng.standard_normal((n, k)) * 0.02 * np.exp(rng.standard_normal((n, 1)))
    v = np.round(v * 2.0 ** 22) / 2.0 ** 22  # fp32 values whose folded sums are exact in fp64
    w = torch.from_numpy(v).to(T[wt][1])
    w[0, :128] = 0
    if k >= 1024:
        w[-1, -1024:] = 0
    signs = None if folded else draw_signs(rng, k)
    packed = torch.zeros(n, k // 2, dtype=torch.uint8, device=DEV)
    scales = torch.zeros(n, k // 128, dtype=torch.float16, device=DEV)
    tb.tb_q4_prepare_weights(w.to(DEV), T[wt][0], signs.to(DEV) if signs is not None else None, n, k, packed, scales)
    q, s = q4o.prepare_weights(w.double().numpy(), None if folded else signs.numpy())
    assert np.array_equal(scales.cpu().numpy().view(np.uint16), s.view(np.uint16))
    assert np.array_equal(packed.cpu().numpy(), q4o.pack(q))


@pytest.mark.parametrize("wt", ["bf16", "fp16"])
@pytest.mark.parametrize("span", [0, 12, 17, 20, 26])
def test_prepare_folded_values_of_many_sizes(wt, span):
    """Blocks whose values span up to 2^span below their largest (short and long
    slices of the exact sums), a block of one value, and blocks of zeros."""
    n, k = 40, 2048
    rng = np.random.default_rng(span)
    v = rng.standard_normal((n, k)) * 2.0 ** -rng.uniform(0, max(span, 1e-9), (n, k)) * 0.05
    v[1, :1024] = 0
    v[2, 1024:2048] = 0
    v[2, 1500] = 0.03
    v[3] *= 1e-3
    w = torch.from_numpy(v).to(T[wt][1])
    signs = draw_signs(rng, k)
    packed = torch.zeros(n, k // 2, dtype=torch.uint8, device=DEV)
    scales = torch.zeros(n, k // 128, dtype=torch.float16, device=DEV)
    for off in (0, 1):  # and from 4 bytes past a 16-byte boundary
        buf = torch.empty(n * k + 2, dtype=w.dtype, device=DEV)
        d = buf[2 * off:2 * off + n * k].view(n, k)
        d.copy_(w)
        tb.tb_q4_prepare_weights(d, T[wt][0], signs.to(DEV), n, k, packed, scales)
        q, s = q4o.prepare_weights(w.double().numpy(), signs.numpy())
        assert np.array_equal(scales.cpu().numpy().view(np.uint16), s.view(np.uint16))
        assert np.array_equal(packed.cpu().numpy(), q4o.pack(q))


@pytest.mark.parametrize("wt", ["bf16", "fp16", "fp32"])
def test_prepare_folded_ties(wt):
    """Two values a and b in a block fold to |a +- b| / 32 everywhere: (21, 7) puts the
    scale on an fp16 number and half the codes on q + 1/2, (7 2^11, 7) the scale
    halfway between two fp16 numbers."""
    n, k = 16, 2048
    rng = np.random.default_rng(7)
    v = np.zeros((n, k))
    for i in range(n):
        for blk in range(2):
            at = 1024 * blk + rng.choice(1024, 2, replace=False)
            pair = ((21.0, 7.0), (7.0 * 2 ** 11, 7.0))[i % 2]
            v[i, at] = np.array(pair) * rng.choice([-1.0, 1.0], 2) * 2.0 ** -int(rng.integers(2, 10))
    w = torch.from_numpy(v).to(T[wt][1])
    assert np.array_equal(w.double().numpy(), v)
    signs = draw_signs(rng, k)
    packed = torch.zeros(n, k // 2, dtype=torch.uint8, device=DEV)
    scales = torch.zeros(n, k // 128, dtype=torch.float16, device=DEV)
    tb.tb_q4_prepare_weights(w.to(DEV), T[wt][0], signs.to(DEV), n, k, packed, scales)
    q, s = q4o.prepare_weights(v, signs.numpy())
    assert np.array_equal(scales.cpu().numpy().view(np.uint16), s.view(np.uint16))
    assert np.array_equal(packed.cpu().numpy(), q4o.pack(q))


@pytest.mark.parametrize("size", [1e9, 30000.0, 1e-6, 3e-7, 1e-9])
def test_prepare_ends_of_the_scale(size):
    rng = np.random.default_rng(2)
    w = torch.from_numpy(rng.standard_normal((3, 256)) * size).float()
    packed = torch.zeros(3, 128, dtype=torch.uint8, device=DEV)
    scales = torch.zeros(3, 2, dtype=torch.float16, device=DEV)
    tb.tb_q4_prepare_weights(w.to(DEV), tb.TB_FP32, None, 3, 256, packed, scales)
    q, s = q4o.prepare_weights(w.double().numpy())
    assert np.array_equal(scales.cpu().numpy(), s) and np.array_equal(packed.cpu().numpy(), q4o.pack(q))


@pytest.mark.parametrize("wt", ["bf16", "fp32"])
def test_prepare_values_on_borders(wt):
    """Every q + 1/2 of a group whose scale is a power of two, and its
    neighbours in the input's type: halves go to even."""
    for scale in (1.0, 2.0 ** -7):
        v = [7.0]
        for q in range(-7, 7):
            b = torch.tensor((q + 0.5) * scale).to(T[wt][1])
            v += [(q + 0.5), torch.nextafter(b, torch.tensor(float("inf")).to(b)).item() / scale,
                  torch.nextafter(b, torch.tensor(-float("inf")).to(b)).item() / scale]
        w = torch.zeros(1, 128)
        w[0, :len(v)] = torch.tensor(v) * scale
        w = w.to(T[wt][1])
        packed = torch.zeros(1, 64, dtype=torch.uint8, device=DEV)
        scales = torch.zeros(1, 1, dtype=torch.float16, device=DEV)
        tb.tb_q4_prepare_weights(w.to(DEV), T[wt][0], None, 1, 128, packed, scales)
        q, s = q4o.prepare_weights(w.double().numpy())
        assert float(scales) == scale == s[0, 0]
        assert np.array_equal(packed.cpu().numpy(), q4o.pack(q))


# ------------------------------------------------------------------ linear
@functools.lru_cache(maxsize=8)
def weights(seed, n, k):
    rng = np.random.default_rng(seed)
    codes = rng.integers(-8, 8, (n, k)).astype(np.int8)
    scales = (np.abs(rng.standard_normal((n, k // 128))) * 0.01).astype(np.float16)
    scales[0, 0] = 0
    packed = torch.from_numpy(q4o.pack(codes)).to(DEV)
    return codes, scales, packed, torch.from_numpy(scales.view(np.int16)).to(DEV)


class Linear:
    def __init__(self, seed, m, n, k, xt="bf16", group=0, signs=False, yt="bf16"):
        rng = np.random.default_rng(1000 + seed)
        self.m, self.n, self.k, self.xt, self.group, self.yt = m, n, k, xt, group, yt
        self.codes, self.scales, self.packed, self.dscales = weights(seed, n, k)
        x = rng.standard_normal((m, k)) * (0.2 + rng.random((m, 1)))
        x[rng.random((m, k)) < 0.01] *= 20.0
        self.xs = None
        if group:
            top = 127.0 if xt == "int8" else 448.0
            xg = x.reshape(m, k // group, group)
            xs = (np.abs(xg).max(2) / top).astype(np.float32)
            x = (xg / xs[:, :, None]).reshape(m, k)
            x = np.clip(np.rint(x), -127, 127) if xt == "int8" else np.clip(x, -448, 448)
            self.xs = torch.from_numpy(xs)
        self.x = torch.from_numpy(x).float().to(T[xt][1])
        self.signs = draw_signs(rng, k) if signs else None

    def run(self, guard=0, stream=None):
        self.dx = self.x.to(DEV)
        self.dxs = self.xs.to(DEV) if self.xs is not None else None
        self.ds = self.signs.to(DEV) if self.signs is not None else None
        self.y = torch.full((self.m + guard, self.n), 77.0, device=DEV).to(T[self.yt][1])
        self.wsb = tb.tb_q4_linear_workspace(self.m, self.n, self.k)
        self.ws = torch.full((self.wsb + 256,), 0xFF, dtype=torch.uint8, device=DEV)
        torch.cuda.synchronize()
        self.call(stream)
        torch.cuda.synchronize()
        assert (self.ws[self.wsb:] == 0xFF).all()
        return self

    def call(self, stream=None):
        tb.tb_q4_linear(self.dx, T[self.xt][0], self.dxs, self.group, self.packed, self.dscales, self.m, self.n, self.k,
                        self.ds, self.y, T[self.yt][0], self.ws, self.wsb, stream=stream)

    def check(self):
        xs = self.xs.numpy() if self.xs is not None else None
        sg = self.signs.numpy() if self.signs is not None else None
        x = self.x.to(torch.float64).numpy()
        ref = q4o.linear(x, self.codes, self.scales, xs, sg)
        xr = np.abs(q4o.orc.rotate(x, sg) if sg is not None else x)
        big = q4o.linear(xr, np.abs(self.codes), self.scales, xs)
        y = self.y[:self.m].cpu().double().numpy()
        fi = torch.finfo(T[self.yt][1])
        tol = np.abs(ref) * fi.eps / 2 + fi.smallest_normal * fi.eps
        if self.m <= 16:
            top = np.repeat(xr.reshape(self.m, -1, 128).max(2), 128, axis=1)
            if self.xt != "int8":
                tol += q4o.linear(top, np.abs(self.codes), self.scales, xs) * 2.0 ** (-22 if self.m <= 5 else -15)
            tol += big * (2.0 ** -17 if sg is None else 2.0 ** -10)
        else:
            tol += big * 2.0 ** -10
            rel = np.linalg.norm(y - ref) / np.linalg.norm(ref)
            assert rel <= 2.0 ** -11 + fi.eps / 2, rel
        assert (np.abs(y - ref) <= tol).all()
        return self


SHAPES = [(1, 1, 128), (1, 7, 256), (1, 1000, 640), (1, 2049, 5120), (2, 64, 384), (3, 129, 1152), (5, 18, 17408),
          (7, 333, 2048), (8, 1000, 1024), (9, 257, 1920), (15, 40, 128), (16, 1001, 1280), (17, 255, 384), (24, 100, 512),
          (31, 129, 2048), (32, 512, 1152), (33, 1001, 1920), (47, 30, 640), (64, 300, 1024), (65, 31, 128), (100, 1, 256),
          (128, 400, 896), (129, 257, 640), (200, 513, 1024), (300, 77, 2176), (513, 600, 256)]
KINDS = [("bf16", 0), ("fp16", 0), ("int8", 1), ("int8", 128), ("e4m3", 1), ("e4m3", 128)]


@pytest.mark.parametrize("m,n,k", SHAPES)
@pytest.mark.parametrize("xt,group", KINDS)
def test_linear(m, n, k, xt, group):
    yt = {"bf16": "bf16", "fp16": "fp16", "int8": "fp32", "e4m3": "bf16"}[xt]
    Linear(n, m, n, k, xt, k if group == 1 else group, False, yt).run().check()


@pytest.mark.parametrize("m,n,k", [(1, 513, 1024), (1, 100, 5120), (4, 77, 2048), (16, 300, 5120), (31, 64, 1024),
                                   (65, 200, 2048), (300, 300, 1024)])
@pytest.mark.parametrize("xt,yt", [("bf16", "fp32"), ("fp16", "fp16")])
def test_linear_rotated(m, n, k, xt, yt):
    Linear(n, m, n, k, xt, 0, True, yt).run().check()


@pytest.mark.parametrize("m", [1, 6, 16, 40, 130])
@pytest.mark.parametrize("yt", ["bf16", "fp16", "fp32"])
def test_output_types_and_rows_behind_the_last(m, yt):
    c = Linear(300, m, 300, 512, "bf16", 0, False, yt).run(guard=3).check()
    assert (c.y[m:].float() == 77.0).all()


def within(y, x, w):
    """The bounds above for an unrotated bf16 x and an fp32 y, on the device."""
    m, k = x.shape
    a = x.double().abs()
    tol = a @ w.abs().T * (2.0 ** -17 if m <= 16 else 2.0 ** -10)
    if m <= 16:
        top = a.view(m, -1, 128).amax(2).repeat_interleave(128, 1)
        tol += top @ w.abs().T * 2.0 ** (-22 if m <= 5 else -15)
    return bool(((y.double() - x.double() @ w.T).abs() <= tol).all())


@pytest.mark.parametrize("m,n,k", [(1, 17408, 5120), (1, 1024, 5120), (4, 5120, 17408), (16, 6144, 5120), (2, 40000, 1024),
                                   (16, 5120, 17408), (20, 4096, 2048)])
def test_linear_full_shapes(m, n, k):
    rng = np.random.default_rng(n)
    packed = torch.randint(0, 256, (n, k // 2), dtype=torch.uint8, device=DEV)
    scales = (torch.randn(n, k // 128, device=DEV).abs() * 0.01).to(torch.float16)
    x = torch.from_numpy(rng.standard_normal((m, k))).to(torch.bfloat16).to(DEV)
    y = torch.full((m, n), float("nan"), device=DEV)
    wsb = tb.tb_q4_linear_workspace(m, n, k)
    ws = torch.empty(wsb, dtype=torch.uint8, device=DEV)
    tb.tb_q4_linear(x, tb.TB_BF16, None, 0, packed, scales, m, n, k, None, y, tb.TB_FP32, ws, wsb)
    w = torch.stack((packed & 15, packed >> 4), -1).view(n, k).double() - 8.0
    w *= scales.double().repeat_interleave(128, 1)
    assert within(y, x, w)
    again = torch.empty_like(y)
    tb.tb_q4_linear(x, tb.TB_BF16, None, 0, packed, scales, m, n, k, None, again, tb.TB_FP32, ws, wsb)
    assert torch.equal(y, again)


def test_weights_past_32_bits():
    """Packed codes of more than 4 GiB: the rows at the end match a call on them alone."""
    n, k = 300000, 32768
    packed = torch.randint(0, 256, (n, k // 2), dtype=torch.uint8, device=DEV)
    scales = (torch.randn(n, k // 128, device=DEV).abs() * 0.01).to(torch.float16)
    for m in (1, 40):
        x = torch.randn(m, k, device=DEV).to(torch.bfloat16)
        y, part = torch.empty(m, n, device=DEV), torch.empty(m, 64, device=DEV)
        wsb = tb.tb_q4_linear_workspace(m, n, k)
        ws = torch.empty(wsb, dtype=torch.uint8, device=DEV)
        tb.tb_q4_linear(x, tb.TB_BF16, None, 0, packed, scales, m, n, k, None, y, tb.TB_FP32, ws, wsb)
        tb.tb_q4_linear(x, tb.TB_BF16, None, 0, packed[-64:], scales[-64:], m, 64, k, None, part, tb.TB_FP32, ws, wsb)
        w = torch.stack((packed[-64:] & 15, packed[-64:] >> 4), -1).view(64, k).double() - 8.0
        w *= scales[-64:].double().repeat_interleave(128, 1)
        for got in (y[:, -64:], part):
            assert within(got, x, w)


@pytest.mark.parametrize("m", [1, 8, 16, 48, 200])
@pytest.mark.parametrize("xt", ["bf16", "fp16"])
def test_no_numbers_stay_in_their_row(m, xt):
    c = Linear(90, m, 90, 640, xt, 0, False, "fp32")
    clean = c.run().y.clone()
    c.x[m // 2, 600] = float("nan")
    bad = c.run().y.clone()
    assert torch.isnan(bad[m // 2]).all()
    keep = [i for i in range(m) if i != m // 2]
    assert torch.equal(bad[keep], clean[keep])
    c.x[m // 2, 600] = float("inf")
    c.run()
    assert not torch.isfinite(c.y[m // 2]).any() and torch.equal(c.y[keep], clean[keep])


@pytest.mark.parametrize("m", [1, 16, 40, 150])
@pytest.mark.parametrize("signs", [False, True])
@pytest.mark.parametrize("size", [1e30, 1e-30])
def test_sizes_beyond_fp16(m, signs, size):
    """bf16 activations far outside fp16's range, some rows of ordinary size, one of zeros."""
    c = Linear(80, m, 80, 1024, "bf16", 0, signs, "fp32")
    c.x[::2] *= size
    if m > 3:
        c.x[3] = 0.0
    c.run().check()
    if m > 3:
        assert not c.y[3].any()


def test_streams_graphs_and_two_at_once():
    """The same bits on another stream, in a replayed graph, and from two calls
    in flight at once with a workspace each."""
    for m, xt, signs in ((1, "bf16", False), (16, "fp16", True), (80, "bf16", False)):
        a, b = (Linear(s, m, 700, 2048, xt, 0, signs, "bf16").run().check() for s in (700, 701))
        want = a.y.clone(), b.y.clone()
        s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
        a.y.zero_(), b.y.zero_()
        torch.cuda.synchronize()
        for _ in range(5):
            a.call(stream=s1)
            b.call(stream=s2)
        torch.cuda.synchronize()
        assert torch.equal(a.y, want[0]) and torch.equal(b.y, want[1])
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            a.call()
            b.call()
            a.call()
        a.y.zero_(), b.y.zero_()
        for _ in range(2):
            g.replay()
        torch.cuda.synchronize()
        assert torch.equal(a.y, want[0]) and torch.equal(b.y, want[1])


# ------------------------------------------------------------------ as they are used together
@pytest.mark.parametrize("m", [1, 5, 16, 33, 140])
@pytest.mark.parametrize("yt,group", [("int8", 128), ("e4m3", 0), ("bf16", None)])
def test_norm_then_linear(m, yt, group):
    """prepare -> (norm with residual and rotation -> 8 bits) -> linear, in one
    stream without a wait between them, twice; against the float64 chain on the
    values the norm stored."""
    n, k = 600, 2048
    rng = np.random.default_rng(m)
    dense = torch.from_numpy(rng.standard_normal((n, k)) * 0.02).to(torch.bfloat16).to(DEV)
    signs = draw_signs(rng, k).to(DEV)
    packed = torch.empty(n, k // 2, dtype=torch.uint8, device=DEV)
    scales = torch.empty(n, k // 128, dtype=torch.float16, device=DEV)
    tb.tb_q4_prepare_weights(dense, tb.TB_BF16, signs, n, k, packed, scales)
    x, r = (torch.from_numpy(rng.standard_normal((m, k))).to(torch.bfloat16).to(DEV) for _ in range(2))
    w = torch.ones(k, dtype=torch.bfloat16, device=DEV)
    group = k if group == 0 else group
    a = torch.empty(m, k, dtype=T[yt][1], device=DEV)
    xs = torch.empty(m, k // group, device=DEV) if group else None
    h, y = torch.empty_like(r), torch.empty(m, n, device=DEV)
    wsb = tb.tb_q4_linear_workspace(m, n, k)
    ws = torch.empty(wsb, dtype=torch.uint8, device=DEV)
    for _ in range(2):
        tb.tb_rms_norm(x, tb.TB_BF16, r, h, tb.TB_BF16, w, tb.TB_BF16, 1e-6, signs, m, k, a, T[yt][0], xs, group or 0)
        tb.tb_q4_linear(a, T[yt][0], xs, group or 0, packed, scales, m, n, k, None, y, tb.TB_FP32, ws, wsb)
    torch.cuda.synchronize()
    q, s = q4o.prepare_weights(dense.double().cpu().numpy(), signs.cpu().numpy())
    assert np.array_equal(packed.cpu().numpy(), q4o.pack(q))
    av = a.to(torch.float64).cpu().numpy()
    ref = q4o.linear(av, q, s, xs.cpu().numpy() if group else None)
    got = y.cpu().double().numpy()
    assert np.linalg.norm(got - ref) <= 2.0 ** -11 * np.linalg.norm(ref)
    # and it is near the dense layer on the norm: 8-bit and 4-bit steps, uniform
    # errors of step / sqrt(12): weights max/7 with max about 2.8 sigma in 128
    # values, 0.12 of sigma; e4m3 2^-4 / sqrt(3) = 0.04; together under 0.15
    norm = q4o.rms_norm((x.float() + r.float()).to(torch.bfloat16).double().cpu().numpy(), None, 1e-6)
    dref = norm @ dense.double().cpu().numpy().T
    assert np.linalg.norm(got - dref) <= 0.15 * np.linalg.norm(dref)


@pytest.mark.parametrize("m", [2, 9, 30, 140])
@pytest.mark.parametrize("yt,group", [("int8", 256), ("int8", 128), ("e4m3", 256), ("e4m3", 128)])
def test_a_row_without_numbers_through_both(m, yt, group):
    """A NaN in a row of x reaches that row of y, and a row of zeros gives zeros."""
    n, k = 70, 256
    c = Linear(77, m, n, k, "bf16", 0, False, "fp32")
    x = torch.randn(m, k, device=DEV).to(torch.bfloat16)
    x[0, 3] = float("nan")
    x[1] = 0.0
    a = torch.empty(m, k, dtype=T[yt][1], device=DEV)
    xs, y = torch.empty(m, k // group, device=DEV), torch.full((m, n), 77.0, device=DEV)
    wsb = tb.tb_q4_linear_workspace(m, n, k)
    ws = torch.empty(wsb, dtype=torch.uint8, device=DEV)
    tb.tb_rms_norm(x, tb.TB_BF16, None, None, 0, None, 0, 1e-6, None, m, k, a, T[yt][0], xs, group)
    tb.tb_q4_linear(a, T[yt][0], xs, group, c.packed, c.dscales, m, n, k, None, y, tb.TB_FP32, ws, wsb)
    assert torch.isnan(y[0]).all() and not y[1].any() and torch.isfinite(y[1:]).all()


@pytest.mark.parametrize("m,n,k", [(64, 3000, 1024), (20, 300, 2048), (200, 600, 1024)])
def test_waits_run_out_and_the_next_call_is_right(m, n, k):
    """With the copies of the weights held back (the library's test hook) every
    wait for them runs out, the call returns and says so, and the next is right."""
    c = Linear(n, m, n, k, "bf16", 0, False, "bf16")
    tb.tb_get_device_fault(clear=True)
    tb.tb_test_stall_copies(1, 20_000_000)
    try:
        c.run()
        code = tb.tb_get_device_fault(clear=True)
    finally:
        tb.tb_test_stall_copies(0, 0)
    assert code == 1, code
    for _ in range(2):
        c.run().check()


@pytest.mark.parametrize("m", [1, 40])
def test_norm_then_ternary_linear(m):
    """The norm with the rotation in front of the ternary layer (signs NULL there)
    gives what the layer gives for the unrotated norm with its signs."""
    n, k = 512, 2048
    rng = np.random.default_rng(50 + m)
    codes = torch.from_numpy(rng.integers(-1, 2, (n, k)).astype(np.int8)).to(DEV)
    packed = torch.empty(tb.tb_packed_bytes("2bit", n, k), dtype=torch.uint8, device=DEV)
    tb.tb_pack_ternary("2bit", codes, n, k, packed)
    scales = (torch.from_numpy(np.abs(rng.standard_normal((n, k // 128))) * 0.02).to(torch.float16)).to(DEV)
    signs = draw_signs(rng, k).to(DEV)
    x = torch.from_numpy(rng.standard_normal((m, k))).to(torch.bfloat16).to(DEV)
    plain, rot = torch.empty(m, k, device=DEV), torch.empty(m, k, device=DEV)
    args = (None, None, 0, None, 0, 1e-6)
    tb.tb_rms_norm(x, tb.TB_BF16, *args, None, m, k, plain, tb.TB_FP32)
    tb.tb_rms_norm(x, tb.TB_BF16, *args, signs, m, k, rot, tb.TB_FP32)
    wsb = tb.tb_ternary_linear_workspace("2bit", m, n, k)
    ws = torch.empty(wsb, dtype=torch.uint8, device=DEV)
    y = [torch.empty(m, n, device=DEV) for _ in range(2)]
    tb.tb_ternary_linear(plain, tb.TB_FP32, packed, scales, "2bit", m, n, k, signs, y[0], tb.TB_FP32, ws, wsb)
    tb.tb_ternary_linear(rot, tb.TB_FP32, packed, scales, "2bit", m, n, k, None, y[1], tb.TB_FP32, ws, wsb)
    # both are within 2e-3 of the exact product in relative L2
    assert float((y[0] - y[1]).norm() / y[0].norm()) <= 4e-3


@pytest.mark.parametrize("m,n,k,xt,signs", [(1, 100, 640, "bf16", False), (1, 17408, 5120, "bf16", False),
                                            (3, 40000, 1024, "fp16", False), (16, 600, 2048, "bf16", True),
                                            (16, 5120, 17408, "int8", False)])
def test_waits_of_the_decode_run_out_and_the_next_call_is_right(m, n, k, xt, signs):
    """The same for up to 16 tokens: one row block a CTA and several, one CTA and
    two that split K, a short K whose partial sums reach past the planes of x."""
    c = Linear(n, m, n, k, xt, k if xt == "int8" else 0, signs, "bf16")
    tb.tb_get_device_fault(clear=True)
    tb.tb_test_stall_copies(1, 20_000_000)
    try:
        c.run()
        code = tb.tb_get_device_fault(clear=True)
    finally:
        tb.tb_test_stall_copies(0, 0)
    assert code == 1, code
    for _ in range(2):
        c.run().check()


@pytest.mark.parametrize("xt,group", [("bf16", 0), ("e4m3", 128)])
def test_the_widest_row(xt, group):
    """K next to 2^31: nothing wraps on the way.  x is zero but for 2,000 places all over
    the row, its ends among them, and the scales are 2^-3: every product is exact."""
    m, n, k = 1, 3, 2 ** 31 - 128
    g = torch.Generator(device=DEV)
    g.manual_seed(5)
    packed = torch.randint(0, 256, (n, k // 2), dtype=torch.uint8, device=DEV, generator=g)
    scales = torch.full((n, k // 128), 0.125, dtype=torch.float16, device=DEV)
    at = torch.randint(0, k, (2000,), device=DEV, generator=g)
    at[:300] = torch.arange(300, device=DEV)
    at[300:600] = k - 1 - torch.arange(300, device=DEV)
    at = at.unique()
    v = torch.randint(-8, 9, at.shape, device=DEV, generator=g).float()
    x = torch.zeros(m, k, dtype=T[xt][1], device=DEV)
    x.view(-1)[at] = v.to(x.dtype)
    xs = torch.ones(m, k // 128, device=DEV) if group else None
    y = torch.full((m, n), float("nan"), device=DEV)
    wsb = tb.tb_q4_linear_workspace(m, n, k)
    ws = torch.empty(wsb, dtype=torch.uint8, device=DEV)
    tb.tb_q4_linear(x, T[xt][0], xs, group, packed, scales, m, n, k, None, y, tb.TB_FP32, ws, wsb)
    c = packed[:, at // 2].long()
    q = torch.where(at % 2 == 0, c & 15, c >> 4).double() - 8.0
    assert torch.equal(y[0].double(), (q * v.double()).sum(1) * 0.125)


def test_prepare_the_widest_rows():
    """Unfolded rows with K next to 2^31, more of them than a block takes: a value
    here and there, the groups between them zero."""
    n, k = 9, 2 ** 31 - 128
    g = torch.Generator(device=DEV)
    g.manual_seed(6)
    w = torch.zeros(n, k, dtype=torch.float16, device=DEV)
    cols = torch.randint(0, k, (300,), device=DEV, generator=g)
    cols[:2] = torch.tensor([0, k - 1], device=DEV)
    groups = torch.unique(cols // 128)
    vals = torch.randn(n, cols.numel(), device=DEV, generator=g).half()
    w[:, cols] = vals
    packed = torch.zeros(n, k // 2, dtype=torch.uint8, device=DEV)
    scales = torch.full((n, k // 128), float("nan"), dtype=torch.float16, device=DEV)
    tb.tb_q4_prepare_weights(w, tb.TB_FP16, None, n, k, packed, scales)
    dense = w.view(n, k // 128, 128)[:, groups].reshape(n, -1).double().cpu().numpy()
    q, s = q4o.prepare_weights(dense)
    assert np.array_equal(scales[:, groups].cpu().numpy(), s)
    assert np.array_equal(packed.view(n, k // 128, 64)[:, groups].reshape(n, -1).cpu().numpy(), q4o.pack(q))
    scales[:, groups] = 0
    packed.view(n, k // 128, 64)[:, groups] = 0x88
    for r in range(n):  # a row at a time: the comparisons need memory too
        assert not scales[r].any() and (packed[r] == 0x88).all()


@pytest.mark.parametrize("m", [3, 16, 17, 60, 130, 300])
@pytest.mark.parametrize("xt", ["int8", "e4m3"])
def test_large_scales_of_an_8_bit_row(m, xt):
    """Finite values near fp32's largest: a scale of 1e36 with codes up to 300."""
    c = Linear(70, m, 70, 640, xt, 128, False, "fp32")
    c.scales = (c.scales.astype(np.float32) * 2.0 ** -7).astype(np.float16)  # keeps y finite
    c.dscales = torch.from_numpy(c.scales.view(np.int16)).to(DEV)
    c.xs[1] = 1e36
    c.x[1] = torch.clamp(c.x[1].float(), -300.0, 300.0).to(c.x.dtype)
    c.run().check()


# ------------------------------------------------------------------ which kernel, and its accuracy
PLANES = {"int8": lambda m: 1, "bf16": lambda m: 3 if m <= 5 else 2}


def widest(xt, m, n):
    """The widest K (a multiple of 1024) that the decode kernel takes."""
    code = T[xt][0]
    lo, hi = 1024, 1 << 18
    assert tb.tb_q4_linear_path(code, m, n, lo) == tb.TB_PATH_GEMV
    if tb.tb_q4_linear_path(code, m, n, hi) == tb.TB_PATH_GEMV:
        return hi
    while hi - lo > 1024:
        mid = (lo + hi) // 2048 * 1024
        lo, hi = (mid, hi) if tb.tb_q4_linear_path(code, m, n, mid) == tb.TB_PATH_GEMV else (lo, mid)
    return lo


@pytest.mark.parametrize("xt", ["bf16", "fp16", "e4m3", "int8"])
@pytest.mark.parametrize("n", [1, 5120, 151936])
def test_path_by_size(xt, n):
    """The sizes that the header names, and one kernel on either side of one limit."""
    p, code = tb.tb_q4_linear_path, T[xt][0]
    for m in range(1, 17):
        k = min((1 << 18) // (m * PLANES.get(xt, PLANES["bf16"])(m)), 1 << 17) // 128 * 128
        assert p(code, m, n, k) == p(code, m, n, 128) == p(code, m, n, 5120) == tb.TB_PATH_GEMV
        w = widest(xt, m, n)
        assert all(p(code, m, n, w + 1024 * j) == tb.TB_PATH_GEMM for j in (1, 2, 9, 500))
        assert p(code, m, n, 17408) == (tb.TB_PATH_GEMV if w >= 17408 else tb.TB_PATH_GEMM)
    assert p(code, 8, n, 17408) == tb.TB_PATH_GEMV and p(code, 17, n, 128) == p(code, 3000, n, 5120) == tb.TB_PATH_GEMM
    assert xt != "int8" or p(code, 15, n, 17408) == tb.TB_PATH_GEMV


class Drawn:
    """A call on normal x, weights and signs made on the device, its product in 64
    bits, and what its relative L2 error may be, counted in independent roundings.

    Decode kernel: a value of x is off by at most half a step of its 128-group,
    uniformly, so y by sqrt(sum_k w^2 step^2 / 12) rms: steps of 2^-21 (three planes) or
    1.004 2^-14 of the group's largest (two; the higher plane holds 127 of 128), none for
    an int8.  fp32: a term of 128 products is rounded twice, and at most 160 sums of
    terms round by 2^-24 / sqrt(3) rms of partial sums that stay under 3 R, R = sqrt(sum
    w^2 x^2): under 24 2^-24 R.  A rotated x' is off by sqrt(11) 2^-24 of its block's rms.
    Else: w and (rotated, or with scales per group) x' are rounded to 11 bits, relative
    errors of at most 2^-11 / sqrt(3) rms each, so sqrt(2/3) 2^-11 R at most.
    Twice that: with 64 rows of W and more the sum of the errors' squares is within a
    factor 4 of its mean (its relative deviation is sqrt(2 / 64) at most)."""

    def __init__(self, seed, m, n, k, xt, group=0, signs=False, size=1.0):
        g = torch.Generator(device=DEV)
        g.manual_seed(seed)
        self.m, self.n, self.k, self.xt, self.group = m, n, k, xt, group
        self.packed = torch.randint(0, 256, (n, k // 2), dtype=torch.uint8, device=DEV, generator=g)
        self.scales = (torch.rand(n, k // 128, device=DEV, generator=g) * 0.01 + 0.001).to(torch.float16)
        x = torch.randn(m, k, device=DEV, generator=g)
        self.xs = None
        if group:
            xg = x.view(m, -1, group)
            self.xs = xg.abs().amax(-1) / (127.0 if xt == "int8" else 448.0)
            x = (xg / self.xs[..., None]).view(m, k)
            x = x.round() if xt == "int8" else x.clamp(-448.0, 448.0)
        self.x = (x * size).to(T[xt][1])
        self.signs = torch.randint(0, 2, (k,), device=DEV, generator=g).mul(2).sub(1).to(torch.int8) if signs else None

    def run(self):
        m, n, k = self.m, self.n, self.k
        y = torch.full((m, n), float("nan"), device=DEV)
        wsb = tb.tb_q4_linear_workspace(m, n, k)
        ws = torch.empty(wsb, dtype=torch.uint8, device=DEV)
        tb.tb_q4_linear(self.x, T[self.xt][0], self.xs, self.group, self.packed, self.scales, m, n, k, self.signs, y,
                        tb.TB_FP32, ws, wsb)
        return y

    def check(self):
        m, n, k = self.m, self.n, self.k
        x = self.x.double()
        if self.group:
            x = x * self.xs.double().repeat_interleave(self.group, 1)
        if self.signs is not None:
            x = torch.from_numpy(q4o.orc.rotate(x.cpu().numpy(), self.signs.cpu().numpy())).to(DEV)
        w = torch.stack((self.packed & 15, self.packed >> 4), -1).view(n, k).double() - 8.0
        w *= self.scales.double().repeat_interleave(128, 1)
        ref = x @ w.T
        w2 = w.square().view(n, -1, 128).sum(-1)  # of a group
        r2 = float((x.square() @ w.square().T).sum())
        if tb.tb_q4_linear_path(T[self.xt][0], m, n, k, self.signs is not None) == tb.TB_PATH_GEMV:
            step = {1: 0.0, 2: 1.004 * 2.0 ** -14, 3: 2.0 ** -21}[PLANES.get(self.xt, PLANES["bf16"])(m)]
            top = x.abs().view(m, -1, 128).amax(-1)
            var = float((top.square() @ w2.T).sum()) * step ** 2 / 12.0 + (24 * 2.0 ** -24) ** 2 * r2
            if self.signs is not None:
                rms2 = x.square().view(m, -1, 1024).mean(-1).repeat_interleave(8, 1)
                var += 11 * 2.0 ** -48 * float((rms2 @ w2.T).sum())
        else:
            var = r2 * 2.0 / 3.0 * 2.0 ** -22
        err = float((self.run().double() - ref).norm())
        assert err <= 2.0 * var ** 0.5, (err, 2.0 * var ** 0.5)
        assert err <= 2e-3 * float(ref.norm())


@pytest.mark.parametrize("m", [3, 5, 9, 16])
@pytest.mark.parametrize("xt,group,signs", [("bf16", 0, False), ("fp16", 0, True), ("int8", 1, False), ("int8", 128, False),
                                            ("e4m3", 1, False), ("e4m3", 128, False)])
def test_accuracy_on_either_side_of_the_limit(m, xt, group, signs):
    """The widest x that the decode kernel takes, and the next one."""
    n = 320
    w = widest(xt, m, n)
    for i, k in enumerate((w, w + 1024)):
        assert tb.tb_q4_linear_path(T[xt][0], m, n, k, signs) == (tb.TB_PATH_GEMV, tb.TB_PATH_GEMM)[i]
        Drawn(k + m, m, n, k, xt, k if group == 1 else group, signs).check()


@pytest.mark.parametrize("m,n,k", [(1, 17408, 5120), (2, 64, 640), (4, 1024, 5120), (5, 513, 17408), (6, 300, 1024),
                                   (11, 2049, 5120), (16, 6144, 5120), (16, 5120, 17408), (13, 100, 1152)])
@pytest.mark.parametrize("xt,group", [("bf16", 0), ("fp16", 0), ("int8", 1), ("int8", 128), ("e4m3", 1), ("e4m3", 128)])
def test_accuracy_up_to_16_tokens(m, n, k, xt, group):
    Drawn(n + m, m, n, k, xt, k if group == 1 else group).check()


@pytest.mark.parametrize("m,n,k", [(1, 1024, 5120), (4, 640, 2048), (5, 300, 17408), (9, 200, 1024), (16, 6144, 5120)])
@pytest.mark.parametrize("xt", ["bf16", "fp16"])
def test_accuracy_of_a_rotated_x(m, n, k, xt):
    Drawn(n + m, m, n, k, xt, 0, True).check()


@pytest.mark.parametrize("m,signs,size", [(1, False, 1.4e-32), (4, True, 1.4e-32), (7, False, 1.4e-32), (16, True, 1.4e-32),
                                          (17, True, 1e-37), (64, True, 1e-37), (100, False, 1e-37), (200, True, 1e-37)])
def test_accuracy_of_tiny_rows(m, signs, size):
    """bf16 rows near the end of its range keep their bits."""
    Drawn(m, m, 320, 2048, "bf16", 0, signs, size).check()
