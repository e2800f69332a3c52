"""GPU parity of tb_rms_norm against its definition in float64
(oracle/q4_norm_oracle.py).

Tolerances, counted in roundings before the first run.  h is the same on both
sides (one fp32 addition and one rounding, done here with those types).  The
kernel's sum of squares adds at most 128 values a thread and joins fewer than
64 partial sums, so inv = 1 / sqrt(mean + eps) is off by less than
(128 + 64) / 2 * 2^-24 + 4 * 2^-24 < 100 * 2^-24 relative, and n by three more:
|n - n*| <= 2^-17 |n*|.  Rotated, the terms' errors and ten levels of sums
add up to at most 2^-17 * 2 * sum_block |n*| / 32.  A floating output adds half
a step of its type; a scale is off by 2^-16 relative (the largest |n| and one
division); a code by half a step and what n and the scale are off by."""
import numpy as np
import pytest
import torch

from oracle import q4_norm_oracle as q4o
from ternary_weight_signed_b200 import binding as tb
from tests.gpu_util import DEV, ensure_lib

pytestmark = pytest.mark.gpu

T = {"bf16": (tb.TB_BF16, torch.bfloat16), "fp16": (tb.TB_FP16, torch.float16), "fp32": (tb.TB_FP32, torch.float32),
     "int8": (tb.TB_INT8, torch.int8), "e4m3": (tb.TB_E4M3, torch.float8_e4m3fn)}
TOP = {"int8": 127.0, "e4m3": 448.0}
EPS = 1e-5


@pytest.fixture(scope="module", autouse=True)
def _lib():
    ensure_lib()
    tb.tb_get_device_fault(clear=True)
    yield
    assert tb.tb_get_device_fault() == 0


def rows(rng, m, k, t):
    x = rng.standard_normal((m, k)) * (0.1 + 3.0 * rng.random((m, 1)))
    x[rng.random((m, k)) < 0.01] *= 20.0
    return torch.from_numpy(x).to(T[t][1])


def offset(t, by):
    """t on the device, its first element `by` elements past an aligned address."""
    if t is None:
        return None
    buf = torch.empty(t.numel() + by, dtype=t.dtype, device=DEV)
    v = buf[by:].view(t.shape)
    v.copy_(t)
    return v


class Norm:
    def __init__(self, seed, m, k, xt="bf16", rt=None, wt="bf16", signs=False, yt="bf16", group=0, by=0):
        rng = np.random.default_rng(seed)
        self.m, self.k, self.xt, self.rt, self.wt, self.yt, self.group = m, k, xt, rt, wt, yt, group
        self.x = rows(rng, m, k, xt)
        self.r = rows(rng, m, k, rt) if rt else None
        self.w = torch.from_numpy(1.0 + 0.3 * rng.standard_normal(k)).to(T[wt][1]) if wt else None
        self.signs = torch.from_numpy(rng.choice([-1, 1], k).astype(np.int8)) if signs else None
        self.by = by

    def run(self, guard=0, stream=None):
        d = offset
        self.dx, self.dr, self.dw = d(self.x, self.by), d(self.r, self.by), d(self.w, self.by)
        self.ds = self.signs.to(DEV) if self.signs is not None else None
        y = torch.full(((self.m + guard) * self.k + self.by,), 77.0, device=DEV).to(T[self.yt][1])
        self.y = y[self.by:]
        self.s = torch.full((self.m + guard, self.k // self.group), 77.0, device=DEV) if self.group else None
        self.ro = torch.full_like(self.dr, 77.0) if self.rt else None
        torch.cuda.synchronize()
        self.call(stream)
        torch.cuda.synchronize()
        return self

    def call(self, stream=None):
        tb.tb_rms_norm(self.dx, T[self.xt][0], self.dr, self.ro, T[self.rt or "bf16"][0], self.dw,
                       T[self.wt or "bf16"][0], EPS, self.ds, self.m, self.k, self.y, T[self.yt][0], self.s,
                       self.group, stream=stream)

    def h(self):
        if self.r is None:
            return self.x
        return (self.x.float() + self.r.float()).to(T[self.rt][1])

    def check(self):
        m, k = self.m, self.k
        h = self.h()
        if self.rt:
            assert torch.equal(self.ro.cpu(), h)
        w = self.w.double().numpy() if self.w is not None else None
        sg = self.signs.numpy() if self.signs is not None else None
        n = q4o.rms_norm(h.double().numpy(), w, EPS, sg)
        err = 2.0 ** -17 * np.abs(n)
        if sg is not None:
            plain = np.abs(q4o.rms_norm(h.double().numpy(), w, EPS)).reshape(m, k // 1024, 1024)
            err = np.repeat(2.0 ** -16 * plain.sum(2) / 32.0, 1024, axis=1)
        y = self.y[:m * k].view(m, k).cpu()
        if not self.group:
            fi = torch.finfo(T[self.yt][1])
            tol = err + np.abs(n) * fi.eps / 2 + fi.smallest_normal * fi.eps  # a subnormal's step
            assert (np.abs(y.double().numpy() - n) <= tol).all()
            return
        s = q4o.group_scales(n, self.group, TOP[self.yt])
        big = np.repeat(err.reshape(m, -1, self.group).max(2), self.group, axis=1)
        sx = np.repeat(s, self.group, axis=1)
        got_s = self.s[:m].cpu().double().numpy()
        assert (np.abs(got_s - s) <= 2.0 ** -16 * s + big[:, ::self.group] / TOP[self.yt]).all()
        v = n / sx
        off = big / sx + np.abs(v) * (2.0 ** -16 + big / (sx * TOP[self.yt]))
        q = y.to(torch.float64).numpy()
        if self.yt == "int8":
            assert (np.abs(q - v) <= 0.5 + off).all() and np.abs(q).max() <= 127
        else:
            assert (np.abs(q - v) <= np.maximum(np.abs(v) * 2.0 ** -4, 2.0 ** -10) * (1 + 2.0 ** -10) + off).all()


SIZES = [(1, 1), (1, 7), (3, 128), (2, 129), (5, 1000), (4, 1024), (1, 5120), (7, 2056), (2, 17408), (3, 8191), (2, 32768),
         (9, 32767), (9, 32759), (9, 16383), (9, 8185), (300, 640)]


@pytest.mark.parametrize("m,k", SIZES)
@pytest.mark.parametrize("xt,rt,yt", [("bf16", "bf16", "bf16"), ("fp16", None, "fp32"), ("fp32", "fp32", "fp16"),
                                      ("bf16", "fp32", "fp32"), ("fp16", "bf16", "bf16")])
def test_floating_output(m, k, xt, rt, yt):
    Norm(k + m, m, k, xt, rt, "bf16", False, yt).run().check()


@pytest.mark.parametrize("m,k", [(1, 1024), (3, 5120), (2, 17408), (2, 32768), (130, 2048)])
@pytest.mark.parametrize("xt,rt,yt", [("bf16", "bf16", "bf16"), ("fp32", None, "fp32"), ("fp16", "fp32", "fp16")])
def test_rotated(m, k, xt, rt, yt):
    Norm(k + m, m, k, xt, rt, "fp32", True, yt).run().check()


@pytest.mark.parametrize("yt", ["int8", "e4m3"])
@pytest.mark.parametrize("m,k,grouped,signs", [(1, 1, False, False), (3, 77, False, False), (2, 128, True, False),
                                               (5, 384, True, False), (5, 384, False, False), (1, 5120, False, True),
                                               (4, 5120, True, True), (2, 8199, False, False), (2, 32768, True, True),
                                               (2, 32768, False, False), (129, 1152, True, False), (1, 17408, True, False)])
@pytest.mark.parametrize("xt,rt", [("bf16", "bf16"), ("fp32", None)])
def test_eight_bits(yt, m, k, grouped, signs, xt, rt):
    Norm(k + m, m, k, xt, rt, "fp16", signs, yt, 128 if grouped else k).run().check()


@pytest.mark.parametrize("m,k,xt,rt,signs,yt,grouped", [
    (1300, 1024, "bf16", "bf16", True, "int8", True), (1190, 1032, "fp16", "fp32", False, "bf16", False),
    (2600, 1024, "fp32", None, False, "fp16", False), (1200, 5120, "bf16", "fp32", False, "e4m3", True),
    (1184, 5120, "bf16", "bf16", True, "bf16", False), (1185, 2048, "fp16", None, True, "e4m3", False),
    (1400, 2560, "bf16", "bf16", False, "int8", False), (1201, 13312, "bf16", None, False, "int8", True),
    (3000, 1000, "fp16", "bf16", False, "bf16", False), (1191, 2051, "bf16", "bf16", False, "bf16", False),
    (1300, 4125, "bf16", "fp32", False, "fp16", False), (1185, 2049, "fp16", None, False, "int8", False),
    (2500, 2063, "fp32", "fp16", False, "e4m3", False), (40, 17, "bf16", "bf16", False, "bf16", False),
    (33, 9, "fp16", "fp32", False, "int8", False), (700, 5, "bf16", "bf16", False, "e4m3", False)])
def test_many_rows(m, k, xt, rt, signs, yt, grouped):
    """Rows that come by copies issued ahead, several a block (and a width just
    under), and rows that start anywhere in 16 bytes."""
    group = 0 if yt not in TOP else (128 if grouped else k)
    c = Norm(k + m, m, k, xt, rt, "bf16", signs, yt, group).run(guard=1)
    c.check()
    # in place over the residual, and y over x where the types allow it
    if rt:
        r = c.dr.clone()
        y = c.dx.clone() if xt == yt else torch.empty_like(c.y[:m * k])
        x = y if xt == yt else c.dx
        s = torch.empty(m, k // group, device=DEV) if group else None
        tb.tb_rms_norm(x, T[xt][0], r, r, T[rt][0], c.dw, tb.TB_BF16, EPS, c.ds, m, k, y, T[yt][0], s, group)
        assert torch.equal(r, c.ro) and torch.equal(y.view(-1).view(torch.uint8), c.y[:m * k].view(torch.uint8))


@pytest.mark.parametrize("yt,group", [("bf16", 0), ("int8", 128), ("e4m3", 1024)])
@pytest.mark.parametrize("signs", [False, True])
def test_unaligned_and_no_weight(yt, group, signs):
    # one element past a 16-byte boundary, and no weight
    Norm(9, 3, 1024, "bf16", "fp16", None, signs, yt, group, by=1).run().check()
    if not signs and group != 128:
        Norm(9, 5, 1023, "bf16", "fp16", "fp32", signs, yt, group and 1023, by=3).run().check()


@pytest.mark.parametrize("yt,group", [("bf16", 0), ("fp32", 0), ("int8", 640), ("e4m3", 128)])
def test_rows_behind_the_last_are_left(yt, group):
    c = Norm(10, 3, 640, "bf16", None, "bf16", False, yt, group).run(guard=2)
    c.check()
    fill = torch.tensor(77.0).to(T[yt][1]).float().item()  # as the type holds it (e4m3: 80)
    assert (c.y[3 * 640:].float() == fill).all()
    if group:
        assert (c.s[3:] == 77.0).all()


@pytest.mark.parametrize("k", [512, 1000, 5120])
def test_in_place(k):
    a = Norm(11, 5, k, "bf16", "bf16", "bf16", False, "bf16").run()
    # y over x, the residual over itself
    x, r = a.dx.clone(), a.dr.clone()
    tb.tb_rms_norm(x, tb.TB_BF16, r, r, tb.TB_BF16, a.dw, tb.TB_BF16, EPS, None, 5, k, x, tb.TB_BF16)
    assert torch.equal(x.view(-1), a.y) and torch.equal(r, a.ro)
    # the residual's sum over x
    x, y = a.dx.clone(), torch.empty_like(a.dx)
    tb.tb_rms_norm(x, tb.TB_BF16, a.dr, x, tb.TB_BF16, a.dw, tb.TB_BF16, EPS, None, 5, k, y, tb.TB_BF16)
    assert torch.equal(y.view(-1), a.y) and torch.equal(x, a.ro)


@pytest.mark.parametrize("signs", [False, True])
@pytest.mark.parametrize("yt,group", [("fp32", 0), ("int8", 1024), ("e4m3", 128)])
def test_zero_rows_and_no_numbers(signs, yt, group):
    """A row of zeros gives zeros (scale 0); a NaN or an infinity spoils its own
    row (or groups of it) and no other."""
    c = Norm(12, 6, 1024, "fp32", None, "fp32", signs, yt, group)
    c.x[1] = 0.0
    c.x[2, 5] = float("nan")
    c.x[4, 900] = float("inf")
    c.run()
    y = c.y.view(6, 1024).float().cpu()
    clean = Norm(12, 6, 1024, "fp32", None, "fp32", signs, yt, group).run()
    for r in (0, 3, 5):
        assert torch.equal(y[r], clean.y.view(6, 1024).float().cpu()[r])
    assert not y[1].any()
    if not group:
        assert torch.isnan(y[2]).all() and torch.isnan(y[4, 900])
        assert torch.isnan(y[4]).all() if signs else not y[4, :900].any()
        return
    s = c.s.cpu()
    assert not s[1].any()
    assert torch.isnan(s[2]).all()
    bad = torch.isnan(s[4])
    assert bad.all() if signs or group == 1024 else (bad.sum() == 1 and bad[7])
    q = y[2]
    assert not q.any() if yt == "int8" else torch.isnan(q).all()


def test_squares_beyond_fp32():
    """Sums of squares that overflow or vanish in fp32 are summed scaled."""
    for size in (1e25, 1e-30):
        c = Norm(13, 2, 1024, "fp32", None, "fp32", False, "fp32")
        c.x *= size
        c.run()
        h = c.x.double().numpy()
        n = q4o.rms_norm(h, c.w.double().numpy(), EPS)
        assert (np.abs(c.y.view(2, 1024).cpu().double().numpy() - n) <= 2.0 ** -17 * np.abs(n) + 1e-45).all()


@pytest.mark.parametrize("yt", ["int8", "e4m3"])
def test_tiny_groups_are_zero(yt):
    c = Norm(14, 1, 256, "fp32", None, None, False, yt, 128)
    c.x[:, 128:] *= 1e-33
    c.run()
    s = c.s.cpu()
    assert s[0, 0] > 0 and s[0, 1] == 0
    assert not c.y.float().cpu()[128:].any()


def test_offsets_past_32_bits():
    m, k = 70000, 32768  # 2.3e9 elements
    x = torch.randn(1, k, device=DEV).to(torch.bfloat16).expand(m, k).contiguous()
    x[-1] *= 3.0
    x[-1, 7] = 9.0
    y = torch.empty(m, k, dtype=torch.uint8, device=DEV)
    s = torch.empty(m, 1, device=DEV)
    tb.tb_rms_norm(x, tb.TB_BF16, None, None, 0, None, 0, EPS, None, m, k, y, tb.TB_INT8, s, k)
    one, so = torch.empty(2, k, dtype=torch.uint8, device=DEV), torch.empty(2, 1, device=DEV)
    pair = torch.stack((x[0], x[-1]))
    tb.tb_rms_norm(pair, tb.TB_BF16, None, None, 0, None, 0, EPS, None, 2, k, one, tb.TB_INT8, so, k)
    assert torch.equal(y[0], one[0]) and torch.equal(y[m - 1], one[1]) and torch.equal(y[m - 2], one[0])
    assert torch.equal(s[[0, m - 1]], so)


def test_streams_graphs_and_repeats():
    c = Norm(15, 33, 5120, "bf16", "bf16", "bf16", True, "e4m3", 128).run()
    c.check()
    want = (c.y.clone(), c.s.clone(), c.ro.clone())
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    for t in (c.y.view(torch.uint8), c.s, c.ro):
        t.zero_()
    st.wait_stream(torch.cuda.current_stream())
    c.call(stream=st)
    st.synchronize()
    assert torch.equal(c.y.view(torch.uint8), want[0].view(torch.uint8)) and torch.equal(c.s, want[1])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.call()
        c.call()
    for t in (c.y.view(torch.uint8), c.s, c.ro):
        t.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(c.y.view(torch.uint8), want[0].view(torch.uint8)) and torch.equal(c.ro, want[2])


@pytest.mark.parametrize("m,k,signs,rt,yt,group", [(2400, 1024, True, "bf16", "bf16", 0), (1300, 5120, False, "fp32", "e4m3", 128),
                                                   (1300, 13312, False, None, "int8", 13312), (1200, 1032, False, "bf16", "fp16", 0)])
def test_waits_run_out_and_the_next_call_is_right(m, k, signs, rt, yt, group):
    """With the copies of the rows held back (the library's test hook) every wait
    for them runs out, the call returns and says so without a value written, and the
    next is right."""
    c = Norm(k + m, m, k, "bf16", rt, "bf16", signs, yt, group)
    tb.tb_get_device_fault(clear=True)
    tb.tb_test_stall_copies(1, 20_000_000)
    try:
        c.run()
        code = tb.tb_get_device_fault(clear=True)
    finally:
        tb.tb_test_stall_copies(0, 0)
    assert code == 1, code
    assert (c.y.float() == torch.tensor(77.0).to(T[yt][1]).float().item()).all()
    for t in (c.ro, c.s):
        assert t is None or (t == 77.0).all()
    for _ in range(2):
        c.run().check()
