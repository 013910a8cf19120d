"""GPU parity of the grouped products and their gradients, through the C ABI.

Most cases are exact: operands are small integers (MXFP4: E2M1 values and scales
2^-2 .. 2^2), so every partial sum is a dyadic number that f32 holds, whatever the
order of summation, and the output must equal the 64-bit result rounded once to its
type, bit for bit: |x|, |w| <= 4 and at most 2^18 terms stay below 2^22; MXFP4 terms are
multiples of 2^-6 (two values in halves, two scales of 2^-2) below 36 * 16, and
at most 2^9 of them stay below 2^19 (24 bits hold 2^-5 .. 2^19; the cases here use
scales whose products keep to multiples of 2^-4).
Seeded normal cases bound the rest: k terms summed in f32 in any order, each addition
off by at most 2^-23 of the running magnitude (the tensor core may truncate), plus
half a step of the output's type.
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

T = {0: torch.bfloat16, 1: torch.float16, 2: torch.float32}
E2M1 = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64)
SENTINEL = 7.0


@pytest.fixture(scope="module")
def q(qgmm):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    qgmm.mm_lib()
    return qgmm


def ints(gen, shape, dtype, lim=4):
    return torch.randint(-lim, lim + 1, shape, generator=gen, device="cuda", dtype=torch.int32).to(dtype)


def gen_of(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def group_list(counts, ends):
    c = torch.tensor(counts, dtype=torch.int64, device="cuda")
    return torch.cumsum(c, 0) if ends else c


def spans(counts):
    at = 0
    for g, c in enumerate(counts):
        yield g, slice(at, at + c)
        at += c


def mat(w, transpose_w):
    return w.transpose(1, 2) if transpose_w else w


def strided(t, ld):
    """`t` with its rows `ld` elements apart inside a sentinel-filled buffer: (view, buffer)."""
    if not ld:
        return t.contiguous(), None
    rows = t.numel() // t.shape[-1]
    buf = torch.full((rows, ld), SENTINEL, dtype=t.dtype, device="cuda")
    buf[:, :t.shape[-1]] = t.reshape(rows, -1)
    return buf, buf


class Case:
    def __init__(self, q, counts, k, n, *, m=None, x_type=0, out_type=2, transpose_w=False, ends=True, accumulate=False,
                 pad=0, seed=1, lim=4):
        self.q, self.counts, self.k, self.n = q, list(counts), k, n
        self.total = sum(counts)
        self.m = self.total if m is None else m
        self.e = len(self.counts)
        self.t = transpose_w
        gen = gen_of(seed)
        dt = T[x_type]
        self.x, self.dy = ints(gen, (self.m, k), dt, lim), ints(gen, (self.m, n), dt, lim)
        self.w = ints(gen, (self.e, n, k) if transpose_w else (self.e, k, n), dt, lim)
        self.out = T[out_type]
        ld = lambda v: v + pad if pad else 0
        self.p = q.make_mm_problem(self.m, k, n, self.e, x_type=x_type, out_type=out_type, transpose_w=transpose_w,
                                   group_list_type=0 if ends else 1, accumulate=accumulate, ld_x=ld(k),
                                   ld_w=ld(k if transpose_w else n), ld_y=ld(n))
        self.gl = group_list(self.counts, ends)
        self.ws = torch.empty(q.grouped_mm_workspace(self.p), dtype=torch.uint8, device="cuda")
        self.ws.random_(generator=gen)

    def _out(self, rows, width, ld):
        return torch.full((rows, ld or width), SENTINEL, dtype=self.out, device="cuda")

    def fwd(self):
        y = self._out(self.m, self.n, self.p.ld_y)
        self.q.grouped_mm(self.p, strided(self.x, self.p.ld_x)[0], strided(self.w, self.p.ld_w)[0], self.gl, y, self.ws)
        return y

    def dgrad(self):
        dx = self._out(self.m, self.k, self.p.ld_x)
        self.q.grouped_mm_dgrad(self.p, strided(self.dy, self.p.ld_y)[0], strided(self.w, self.p.ld_w)[0], self.gl, dx,
                                self.ws)
        return dx

    def wgrad(self, dw=None):
        if dw is None:
            dw = self._out(self.e * self.w.shape[1], self.w.shape[2], self.p.ld_w)
        self.q.grouped_mm_wgrad(self.p, strided(self.x, self.p.ld_x)[0], strided(self.dy, self.p.ld_y)[0], self.gl, dw,
                                self.ws)
        return dw

    def want_rows(self, a, b):
        want = torch.full((self.m, b.shape[2]), SENTINEL, dtype=torch.float64, device="cuda")
        for g, r in spans(self.counts):
            want[r] = a[r].double() @ b[g].double()
        return want.to(self.out)

    def want_dw(self):
        a, b = (self.dy, self.x) if self.t else (self.x, self.dy)
        return torch.stack([a[r].double().t() @ b[r].double() for _, r in spans(self.counts)])

    def check(self):
        """All three calls bit for bit; rows past the total and columns past the width stay."""
        for got, want in ((self.fwd(), self.want_rows(self.x, mat(self.w, self.t))),
                          (self.dgrad(), self.want_rows(self.dy, mat(self.w, self.t).transpose(1, 2)))):
            assert self.status() == 0
            assert torch.equal(got[:, :want.shape[1]], want)
            assert bool((got[:, want.shape[1]:] == SENTINEL).all())
        got, want = self.wgrad(), self.want_dw().to(self.out).reshape(-1, self.w.shape[2])
        assert self.status() == 0
        assert torch.equal(got[:, :want.shape[1]], want)
        assert bool((got[:, want.shape[1]:] == SENTINEL).all())

    def status(self):
        return self.q.device_status(self.ws)


SHAPES = [
    ([1], 8, 8), ([1], 16, 264), ([3], 72, 40), ([0, 1, 0], 64, 136), ([17, 0, 5, 64], 128, 256),
    ([255, 257, 1, 0, 130], 264, 520), ([300], 1000, 96), ([15, 16, 17, 31, 33], 40, 1352), ([1] * 9, 2048, 72),
    ([700, 3], 136, 248), ([64, 0, 0, 400], 512, 512), ([129, 127], 56, 904),
]


@pytest.mark.parametrize("counts,k,n", SHAPES)
@pytest.mark.parametrize("transpose_w", [False, True])
@pytest.mark.parametrize("x_type,out_type", [(0, 2), (1, 1), (0, 0), (1, 2)])
def test_exact_products_and_gradients(q, counts, k, n, transpose_w, x_type, out_type):
    lim = 4 if out_type != 1 else 2          # fp16 holds sums below 2^16: 4 * 4 * 700 terms, 2 * 2 * 2048
    if out_type == 1 and sum(counts) and max(counts) * 4 > 60000:
        pytest.skip("fp16 range")
    Case(q, counts, k, n, x_type=x_type, out_type=out_type, transpose_w=transpose_w, seed=k + n, lim=lim,
         ends=(k + n) % 16 == 0).check()


@pytest.mark.parametrize("transpose_w", [False, True])
def test_strided_rows_leave_the_rest_alone(q, transpose_w):
    Case(q, [40, 0, 300, 9], 136, 200, pad=24, transpose_w=transpose_w, ends=False).check()
    Case(q, [33, 2], 8, 264, pad=8, x_type=1, transpose_w=transpose_w).check()


@pytest.mark.parametrize("counts", [[100, 0, 0, 0, 0], [1, 0, 0, 130, 2, 0, 0, 0], [64, 65, 0, 0, 0, 0]])
def test_few_rows_on_average_with_one_long_group(q, counts):
    """The low tiles of calls with few rows, several of them for one expert."""
    Case(q, counts, 328, 520, ends=False).check()
    Case(q, counts, 328, 520, out_type=0, transpose_w=True).check()
    c = MxCase(q, counts, 1024, 264, out_type=0)
    assert torch.equal(c.run(), c.want().bfloat16())


@pytest.mark.parametrize("ends", [False, True])
def test_rows_past_the_total_are_not_touched(q, ends):
    c = Case(q, [5, 0, 70], 96, 104, m=120, ends=ends)
    c.x[75:], c.dy[75:] = float("nan"), float("inf")   # not read into anything either
    c.check()


def test_no_rows_at_all(q):
    c = Case(q, [0, 0, 0], 64, 72, m=40)
    c.check()
    assert torch.equal(c.wgrad(), torch.zeros_like(c.wgrad()))
    z = Case(q, [0, 0], 64, 72)                          # m = 0
    assert z.fwd().shape[0] == 0 and z.dgrad().shape[0] == 0
    assert not z.wgrad().any()
    assert z.status() == 0


def test_many_experts(q):
    rng = np.random.default_rng(3)
    counts = rng.integers(0, 6, 1024)
    counts[rng.permutation(1024)[:500]] = 0
    counts[77] = 300
    Case(q, counts.tolist(), 64, 48, ends=False).check()


@pytest.mark.parametrize("kind", ["negative", "decreasing", "beyond"])
def test_bad_group_lists_are_reported_and_stay_in_bounds(q, kind):
    gl, ends, flag, counts = {
        "negative": ([5, -3, 10, 0], False, 1, [5, 0, 10, 0]),
        "decreasing": ([20, 10, 30, 40], True, 2, [20, 0, 10, 10]),
        "beyond": ([30, 2 ** 62, 2 ** 62, 7], False, 4, [30, 34, 0, 0]),
    }[kind]
    c = Case(q, counts, 64, 72, m=64, ends=ends)
    c.gl = torch.tensor(gl, dtype=torch.int64, device="cuda")
    for got, want in ((c.fwd(), c.want_rows(c.x, c.w)), (c.dgrad(), c.want_rows(c.dy, c.w.transpose(1, 2))),
                      (c.wgrad(), c.want_dw().float().reshape(-1, 72))):
        assert c.status() == flag
        assert torch.equal(got, want)


def test_nan_and_inf_stay_in_their_expert_and_row(q):
    """Rows next to a group's end are loaded with it; what they hold must not leak."""
    c = Case(q, [37, 20, 3, 130], 136, 264)
    c.x[37:57], c.dy[37:57] = float("nan"), float("inf")
    y, dx, dw = c.fwd(), c.dgrad(), c.wgrad().view(4, 136, 264)
    bad = slice(37, 57)
    keep = torch.ones(c.m, dtype=torch.bool, device="cuda")
    keep[bad] = False
    assert torch.equal(y[keep], c.want_rows(c.x, c.w)[keep]) and bool(y[bad].isnan().all())
    assert torch.equal(dx[keep], c.want_rows(c.dy, c.w.transpose(1, 2))[keep])
    assert not bool(dx[bad].isfinite().any())
    want = c.want_dw().float()
    for g in (0, 2, 3):
        assert torch.equal(dw[g], want[g]), g
    assert bool(dw[1].isnan().all())
    # a NaN weight of one expert reaches that expert's rows only
    c = Case(q, [37, 20, 3, 130], 136, 264)
    c.w[1] = float("nan")
    y = c.fwd()
    assert torch.equal(y[keep], c.want_rows(c.x, c.w)[keep]) and bool(y[bad].isnan().all())


@pytest.mark.parametrize("x_type,out_type", [(0, 2), (0, 0), (1, 1)])
def test_accumulating_weight_gradient(q, x_type, out_type):
    c = Case(q, [40, 0, 9], 72, 136, x_type=x_type, out_type=out_type, accumulate=True, transpose_w=True, lim=2)
    old = ints(gen_of(9), (c.e * 136, 72), c.out, 100)
    got = c.wgrad(old.clone())
    want = (old.double() + c.want_dw().reshape(-1, 72)).to(c.out)
    assert torch.equal(got, want)
    assert torch.equal(c.wgrad(got.clone()), (got.double() + c.want_dw().reshape(-1, 72)).to(c.out))


def test_gradients_agree_with_differences(q):
    """L = sum(y * r): L is linear in x and in w, so an exact difference quotient is the gradient."""
    c = Case(q, [20, 3], 40, 48, lim=2)
    c.dy = ints(gen_of(4), (c.m, 48), torch.bfloat16, 2)
    loss = lambda: float((c.fwd().double() * c.dy.double()).sum())
    dx, dw, base = c.dgrad().double(), c.wgrad().view(2, 40, 48).double(), loss()
    rng = np.random.default_rng(0)
    for _ in range(6):
        i, kk, j = rng.integers(23), rng.integers(40), rng.integers(48)
        c.x[i, kk] += 2
        assert (loss() - base) / 2 == float(dx[i, kk])
        c.x[i, kk] -= 2
        g = 0 if i < 20 else 1
        c.w[g, kk, j] += 2
        assert (loss() - base) / 2 == float(dw[g, kk, j])
        c.w[g, kk, j] -= 2


@pytest.mark.parametrize("counts,k,n,x_type,out_type", [
    ([300, 40, 0, 2000], 2048, 512, 0, 0), ([1000], 520, 1352, 1, 1), ([77, 900], 1000, 264, 0, 2),
    ([8], 7168, 256, 1, 2)])
def test_normal_values_within_the_derived_bound(q, counts, k, n, x_type, out_type):
    c = Case(q, counts, k, n, x_type=x_type, out_type=out_type)
    gen = gen_of(5)
    for t in (c.x, c.dy):
        t.normal_(generator=gen)
    c.w.normal_(generator=gen).mul_(k ** -0.5)
    step = torch.finfo(c.out).eps / 2

    def check(got, a, b):
        want, mag = a.double() @ b.double(), a.double().abs() @ b.double().abs()
        bound = a.shape[1] * 2.0 ** -23 * mag
        bound = bound + step * (want.abs() + bound) + (2.0 ** -24 if c.out == torch.float16 else 0.0)   # fp16 subnormals
        assert bool(((got.double() - want).abs() <= bound).all())

    y, dx, dw = c.fwd(), c.dgrad(), c.wgrad().view(c.w.shape)
    for g, r in spans(counts):
        check(y[r], c.x[r], c.w[g])
        check(dx[r], c.dy[r], c.w[g].t())
        check(dw[g], c.x[r].t(), c.dy[r])


@pytest.mark.parametrize("transpose_w", [False, True])
def test_long_sums_exact(q, transpose_w):
    """f32 sums leave the tensor core every 512 terms (8192 in MXFP4) and are added up outside it."""
    Case(q, [20, 0, 70], 4200, 2056, transpose_w=transpose_w, pad=8).check()
    Case(q, [5000, 30, 2048], 136, 264, transpose_w=transpose_w).check()
    c = Case(q, [4100, 9], 72, 520, accumulate=True, transpose_w=transpose_w)
    old = ints(gen_of(9), (2 * c.w.shape[1], c.w.shape[2]), torch.float32, 100)
    assert torch.equal(c.wgrad(old.clone()), (old.double() + c.want_dw().reshape(old.shape)).float())
    for counts in ([30, 3], [900]):          # gathered and arranged scales
        c = MxCase(q, counts, 16896, 72, spread=1)
        assert torch.equal(c.run(), c.want().float())


@pytest.mark.parametrize("length", [2048, 8192, 40000])
def test_long_f32_sums_do_not_drift(q, length):
    """The tensor core may truncate the running sum at each instruction (16 terms), 2^-24 of it on
    average: 32 of them between rounded additions, and at most 79 such additions (40000 terms),
    2^-24 each, come to less than 128 * 2^-24."""
    c = Case(q, [length], 64, 256)
    gen = gen_of(length)
    c.x.normal_(generator=gen), c.dy.normal_(generator=gen)
    want = c.x.double().t() @ c.dy.double()
    assert float((c.wgrad().double() - want).norm() / want.norm()) <= 128 * 2.0 ** -24
    k = min(length, 65536)
    c = Case(q, [64], k, 256, transpose_w=True)
    c.x.normal_(generator=gen), c.w.normal_(generator=gen)
    want = c.x.double() @ c.w[0].double().t()
    assert float((c.fwd().double() - want).norm() / want.norm()) <= 128 * 2.0 ** -24


def test_repeated_calls_are_bitwise_equal(q):
    c = Case(q, [700, 9, 0, 300], 1024, 264, out_type=0)
    for t in (c.x, c.dy, c.w):
        t.normal_(generator=gen_of(6))
    first = (c.fwd(), c.dgrad(), c.wgrad())
    for _ in range(3):
        for a, b in zip(first, (c.fwd(), c.dgrad(), c.wgrad())):
            assert torch.equal(a, b)
    long = Case(q, [9000, 40], 264, 520)                 # f32, several segments
    for t in (long.x, long.dy):
        t.normal_(generator=gen_of(7))
    first = long.wgrad()
    assert all(torch.equal(first, long.wgrad()) for _ in range(3))


def test_offsets_past_32_bits(q):
    """Weights and weight gradients of more than 2^32 bytes, and rows far apart."""
    e, k, n = 40, 8192, 8192                 # 40 * 8192 * 8192 = 2.7e9 elements
    counts = [0] * e
    counts[0], counts[39] = 2, 3
    c = Case(q, counts, k, n, out_type=0, lim=1)
    y, dx = c.fwd(), c.dgrad()
    assert torch.equal(y, c.want_rows(c.x, c.w))
    assert torch.equal(dx, c.want_rows(c.dy, c.w.transpose(1, 2)))
    dw = c.wgrad().view(e, k, n)
    for g, r in ((0, slice(0, 2)), (39, slice(2, 5))):
        assert torch.equal(dw[g], (c.x[r].double().t() @ c.dy[r].double()).to(c.out))
    assert not bool(dw[1:39].any())
    del c, y, dx, dw
    ld = (1 << 27) + 8                       # 20 rows of it: 2.7e9 elements
    gen = gen_of(8)
    buf = torch.zeros(20 * ld, dtype=torch.bfloat16, device="cuda")
    x = torch.as_strided(buf, (20, 64), (ld, 1))
    x.copy_(ints(gen, (20, 64), torch.bfloat16))
    w = ints(gen, (1, 64, 72), torch.bfloat16)
    p = q.make_mm_problem(20, 64, 72, 1, out_type=2, ld_x=ld)
    ws = torch.empty(q.grouped_mm_workspace(p), dtype=torch.uint8, device="cuda")
    y = torch.empty(20, 72, device="cuda")
    q.grouped_mm(p, x, w, group_list([20], True), y, ws)
    assert torch.equal(y, (x.double() @ w[0].double()).float())


# ---------------------------------------------------------------- MXFP4
def mx_values(codes, sf):
    """64-bit values of packed codes [..., k/2] and scales [..., k/32]."""
    lut = torch.cat([E2M1, -E2M1]).to(codes.device)
    v = torch.stack((lut[(codes & 15).int()], lut[(codes >> 4).int()]), -1).reshape(*sf.shape, 32)
    return (v * torch.exp2(sf.double() - 127)[..., None]).reshape(*codes.shape[:-1], -1)


class MxCase:
    def __init__(self, q, counts, k, n, *, m=None, out_type=2, ends=False, pad=0, seed=2, spread=2):
        self.q, self.counts, self.k, self.n, self.e = q, list(counts), k, n, len(counts)
        self.m = sum(counts) if m is None else m
        gen = gen_of(seed)
        byte = lambda *s: torch.randint(0, 256, s, generator=gen, device="cuda", dtype=torch.int32).to(torch.uint8)
        scale = lambda *s: torch.randint(127, 128 + spread, s, generator=gen, device="cuda",
                                         dtype=torch.int32).to(torch.uint8)
        ldk = k + pad
        self.bx, self.bsx = byte(self.m, ldk // 2), scale(self.m, ldk // 32)
        self.bw, self.bsw = byte(self.e * n, ldk // 2), scale(self.e * n, ldk // 32)
        self.out_type = out_type
        self.p = q.make_mm_problem(self.m, k, n, self.e, x_type=q.QGMM_T_MXFP4, out_type=out_type, transpose_w=True,
                                   group_list_type=0 if ends else 1, ld_x=ldk if pad else 0, ld_w=ldk if pad else 0)
        self.gl = group_list(self.counts, ends)
        self.ws = torch.empty(q.grouped_mm_workspace(self.p), dtype=torch.uint8, device="cuda")

    def run(self):
        y = torch.full((self.m, self.n), SENTINEL, dtype=T[self.out_type], device="cuda")
        self.q.grouped_mm(self.p, self.bx, self.bw, self.gl, y, self.ws, x_scale=self.bsx, w_scale=self.bsw)
        return y

    def want(self):
        x = mx_values(self.bx, self.bsx)[:, :self.k]
        w = mx_values(self.bw, self.bsw).view(self.e, self.n, -1)[..., :self.k]
        want = torch.full((self.m, self.n), SENTINEL, dtype=torch.float64, device="cuda")
        for g, r in spans(self.counts):
            want[r] = x[r] @ w[g].t()
        return want


# terms are multiples of 2^-2 below 36 * 2^spread * 2^spread; k of them fit 24 bits while
# k * 36 * 4^spread * 4 < 2^24
@pytest.mark.parametrize("counts,k,n,spread", [
    ([1], 32, 8, 2), ([1], 64, 264, 2), ([3, 0, 2], 96, 40, 2), ([17, 0, 5, 64], 128, 256, 2), ([300], 1056, 96, 2),
    ([255, 225, 1, 0, 130], 288, 520, 2), ([15, 16, 17, 31, 33], 160, 1352, 2), ([1] * 9, 2048, 72, 2),
    ([700, 3], 544, 248, 2), ([64, 0, 0, 400], 512, 512, 2), ([129, 127], 224, 904, 2), ([40], 7168, 128, 1),
    ([450, 449], 1024, 384, 2)])
@pytest.mark.parametrize("out_type", [0, 1, 2])
def test_mxfp4_exact(q, counts, k, n, spread, out_type):
    c = MxCase(q, counts, k, n, out_type=out_type, spread=spread, seed=k + n, ends=n % 16 == 8)
    want = c.want()
    assert torch.equal(c.run(), want.to(T[out_type]))
    assert q.device_status(c.ws) == 0


def test_mxfp4_scales_vary_over_their_range(q):
    """One block per row and column (k = 32), scale exponents far apart.  All terms of an output
    share one power of two, so their sum is exact wherever f32 holds it as a normal number;
    a term below f32's smallest normal 2^-126 may be rounded or flushed, 32 of them by less
    than 32 * 2^-126 = 2^-121."""
    c = MxCase(q, [50, 20], 32, 72)
    c.bsx[:] = (torch.arange(70, device="cuda")[:, None] % 120 + 10).to(torch.uint8)
    c.bsw[:] = (torch.arange(144, device="cuda")[:, None] % 110 + 20).to(torch.uint8)
    want = c.want()
    assert bool(((c.run().double() - want).abs() <= 2.0 ** -121).all())
    assert float(want.abs().max()) > 2.0 ** -60          # outputs far above that bound are among them


def test_mxfp4_nan_scales_and_strides(q):
    c = MxCase(q, [40, 0, 30], 96, 72, m=90, pad=160)
    c.bsx[45, 1] = 255                       # a row of the third expert
    c.bsx[70:] = 255                         # rows past the total
    c.bsx[:, 3:], c.bsw[:, 3:] = 255, 255    # past k
    y, want = c.run(), c.want().float()
    keep = torch.ones(90, dtype=torch.bool, device="cuda")
    keep[45] = False
    assert torch.equal(y[keep], want[keep]) and bool(y[45].isnan().all())
    w = MxCase(q, [40, 0, 30], 96, 72)
    w.bsw[72 * 2 + 5, 0] = 255               # one column of the third expert
    y, want = w.run(), w.want().float()
    assert bool(y[40:, 5].isnan().all())
    y[40:, 5] = want[40:, 5] = 0
    assert torch.equal(y, want)


def test_mxfp4_normal_values(q):
    """f32 sums of k exact products (every block's scales applied exactly): k * 2^-23 of the
    magnitudes, plus half a bf16 step."""
    gen = gen_of(3)
    counts, k, n = [400, 31, 0, 90], 2048, 264
    x = torch.randn(521, k, generator=gen, device="cuda").bfloat16()
    w = (torch.randn(4 * n, k, generator=gen, device="cuda") * k ** -0.5)
    c = MxCase(q, counts, k, n, out_type=0)
    q.per_token_quant_mxfp4(x, c.bx, c.bsx)
    q.per_token_quant_mxfp4(w, c.bw, c.bsw)
    got, want = c.run().double(), c.want()
    xv, wv = mx_values(c.bx, c.bsx).abs(), mx_values(c.bw, c.bsw).abs().view(4, n, k)
    for g, r in spans(counts):
        bound = k * 2.0 ** -23 * (xv[r] @ wv[g].t())
        assert bool(((got[r] - want[r]).abs() <= bound + 2.0 ** -8 * (want[r].abs() + bound)).all())


# ---------------------------------------------------------------- the quantiser
def quant_want(x):
    """Codes and scales from the definition: nearest of the eight levels, ties to the even code."""
    b = x.double().reshape(-1, 32)
    a = b.abs().amax(-1)
    nan = b.isnan().any(-1)
    fin = torch.where(nan | a.isinf() | (a == 0), 1.0, a)
    exp = torch.floor(torch.log2(fin))
    exp = exp + (torch.exp2(exp + 1) <= fin).double() - (torch.exp2(exp) > fin).double()
    sf = torch.where(a == 0, 0.0, (exp + 125).clamp(min=0))
    sf = torch.where(a.isinf(), 253.0, sf)
    v = b.abs() / torch.exp2(sf - 127)[:, None]
    code, far = torch.zeros_like(v), v.clone()
    for c, level in enumerate(E2M1.tolist()):
        d = (v - level).abs()
        nearer = (d < far) | ((d == far) & (c % 2 == 0))
        code, far = torch.where(nearer, float(c), code), torch.where(nearer, d, far)
    code = torch.where(v.isinf(), 7.0, code) + 8.0 * b.signbit()
    sf, code = torch.where(nan, 255.0, sf), torch.where(nan[:, None], 0.0, code)
    c = code.to(torch.uint8).reshape(-1, 2)
    return (c[:, 0] | (c[:, 1] << 4)), sf.to(torch.uint8)


def quant(q, x):
    k = x.shape[-1]
    codes = torch.empty(*x.shape[:-1], k // 2, dtype=torch.uint8, device="cuda")
    sf = torch.empty(*x.shape[:-1], k // 32, dtype=torch.uint8, device="cuda")
    q.per_token_quant_mxfp4(x, codes, sf)
    return codes, sf


def same_codes(codes, want, sf):
    """Equal codes, but for the sign of a zero code, which the formula leaves to IEEE (a zero's sign is its own)."""
    assert torch.equal(sf[1].flatten(), sf[0].flatten())
    assert torch.equal(codes.flatten(), want.flatten())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("rows,k", [(1, 32), (3, 96), (17, 7168), (1000, 544), (5, 65536), (4099, 1056)])
def test_quant_codes_match_the_definition(q, dtype, rows, k):
    gen = gen_of(rows + k)
    x = (torch.randn(rows, k, generator=gen, device="cuda") *
         torch.exp2(torch.randint(-20, 14, (rows, 1), generator=gen, device="cuda").float()) * 0.01).to(dtype)
    codes, sf = quant(q, x)
    want, wsf = quant_want(x)
    same_codes(codes, want, (wsf, sf))
    out = torch.empty_like(x)
    q.mxfp4_dequant(codes, sf, out)
    assert torch.equal(out, mx_values(codes, sf).to(dtype))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_quant_of_every_16_bit_pattern(q, dtype):
    """Every bit pattern (subnormals, infinities and NaN among them) next to others like it, and
    alone in a block of zeros."""
    bits = torch.arange(65536, device="cuda", dtype=torch.int32).to(torch.int16)
    alone = torch.zeros(65536, 32, dtype=torch.int16, device="cuda")
    alone[:, 5] = bits
    for x in (bits.view(2048, 32), bits.view(32, 2048).t().contiguous(), alone):
        x = x.view(dtype)
        codes, sf = quant(q, x)
        want, wsf = quant_want(x)
        same_codes(codes, want, (wsf, sf))
        out = torch.empty(x.shape, dtype=torch.float32, device="cuda")
        q.mxfp4_dequant(codes, sf, out)
        torch.testing.assert_close(out, mx_values(codes, sf).float().masked_fill(
            (sf == 255).repeat_interleave(32, -1).view(x.shape), float("nan")), rtol=0, atol=0, equal_nan=True)


def test_quant_of_ties_and_f32_extremes(q):
    levels = [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 7.0, 7.9999, 6.0, 0.24999, 0.250001, 4.999, 5.001]
    x = torch.tensor(levels + [-v for v in levels] + [4.0, -4.0, 0.0, -0.0], device="cuda").view(1, 32)
    rows = [x * 2.0 ** s for s in (-126, -120, -30, 0, 40, 124)]
    tiny = torch.full((1, 32), 1e-45, device="cuda")
    tiny[0, 3] = 1.1e-38                                    # a subnormal maximum
    big = torch.full((1, 32), torch.finfo(torch.float32).max, device="cuda")
    inf = x.clone()
    inf[0, 7] = float("inf")
    nan = x.clone()
    nan[0, 9] = float("nan")
    x = torch.cat(rows + [tiny, big, inf, nan, torch.zeros(1, 32, device="cuda")])
    codes, sf = quant(q, x)
    want, wsf = quant_want(x)
    same_codes(codes, want, (wsf, sf))


# ---------------------------------------------------------------- as they are used
def test_train_then_quantise_then_serve(q):
    """One training step of an expert layer (product, both gradients, an update), the updated
    weights quantised, and rows served through the 4-bit product."""
    gen = gen_of(11)
    counts, k, n, e = [70, 0, 133, 21], 256, 320, 4
    m = sum(counts)
    gl = group_list(counts, False)
    master = torch.randn(e, n, k, generator=gen, device="cuda") * k ** -0.5
    w = master.bfloat16()
    x = torch.randn(m, k, generator=gen, device="cuda").bfloat16()
    target = torch.randn(m, n, generator=gen, device="cuda")
    kw = dict(group_list_type=q.QGMM_GROUP_COUNTS, transpose_w=True)
    p = q.make_mm_problem(m, k, n, e, out_type=q.QGMM_T_F32, **kw)
    ws = torch.empty(q.grouped_mm_workspace(p), dtype=torch.uint8, device="cuda")
    y = torch.empty(m, n, device="cuda")
    q.grouped_mm(p, x, w, gl, y, ws)
    dy = (y - target).bfloat16()
    dx, dw = torch.empty(m, k, device="cuda"), torch.empty(e, n, k, device="cuda")
    q.grouped_mm_dgrad(p, dy, w, gl, dx, ws)
    q.grouped_mm_wgrad(p, x, dy, gl, dw, ws)
    # the gradients that autograd finds in 64 bits for the same rounded dy
    xr, wr = x.double().requires_grad_(), w.double().requires_grad_()
    yr = torch.cat([xr[r] @ wr[g].t() for g, r in spans(counts)])
    yr.backward(dy.double())
    for got, want, a, b, depth in ((y, yr, x, w, k), (dx, xr.grad, dy, w, n), (dw, wr.grad, dy, x, max(counts))):
        bound = depth * 2.0 ** -23 * float(a.double().abs().max() * b.double().abs().max()) * depth
        assert float((got.double() - want.detach()).abs().max()) <= bound + 2.0 ** -24 * float(want.detach().abs().max())
    master -= 0.01 * dw
    wq = torch.empty(e, n, k // 2, dtype=torch.uint8, device="cuda")
    wsf = torch.empty(e, n, k // 32, dtype=torch.uint8, device="cuda")
    q.per_token_quant_mxfp4(master, wq, wsf)
    xq, xsf = quant(q, x)
    p4 = q.make_mm_problem(m, k, n, e, x_type=q.QGMM_T_MXFP4, out_type=q.QGMM_T_F32, **kw)
    y4 = torch.empty(m, n, device="cuda")
    q.grouped_mm(p4, xq, wq, gl, y4, ws, x_scale=xsf, w_scale=wsf)
    xv, wv = mx_values(xq, xsf), mx_values(wq, wsf)
    for g, r in spans(counts):
        bound = k * 2.0 ** -23 * (xv[r].abs() @ wv[g].abs().t())
        assert bool(((y4[r].double() - xv[r] @ wv[g].t()).abs() <= bound).all())


def test_quantised_weights_feed_the_mxa8w4_mode(q):
    """per_token_quant_mxfp4's weights are what finalize's QGMM_W_MXFP4 reads."""
    gen = gen_of(12)
    m, k, n, e = 48, 256, 256, 2
    w = torch.randn(e, n, k, generator=gen, device="cuda")
    x = torch.randn(m, k, generator=gen, device="cuda").bfloat16()
    wq, wsf = quant(q, w)
    x8 = torch.empty(m, k, dtype=torch.uint8, device="cuda")
    sx = torch.empty(m, k // 32, dtype=torch.uint8, device="cuda")
    q.per_token_quant_mxfp8(x, x8, sx)
    gl = group_list([20, 28], False)
    prob = q.make_problem(m, k, n, e, m, weight_type=q.QGMM_W_MXFP4, transpose_x2=True, group_list_type=1)
    ws = torch.empty(q.finalize_workspace(prob), dtype=torch.uint8, device="cuda")
    out = torch.empty(m, n, device="cuda")
    q.finalize(prob, x8, wq, wsf, sx, gl, None, None, None, None, out, ws)
    xv = x8.view(torch.float8_e4m3fn).double().view(m, -1, 32) * torch.exp2(sx.double() - 127)[..., None]
    xv, wv = xv.view(m, k), mx_values(wq, wsf)
    for g, r in ((0, slice(0, 20)), (1, slice(20, 48))):
        want, mag = xv[r] @ wv[g].t(), xv[r].abs() @ wv[g].abs().t()
        assert bool(((out[r].double() - want).abs() <= 2 * (k / 32) * 2.0 ** -24 * mag + 1e-5 * mag).all())


def test_captured_and_replayed_on_another_stream(q):
    """One graph of all five calls, replayed with new inputs while an ordinary call with a
    workspace of its own runs on another stream."""
    c = Case(q, [70, 0, 30], 128, 264, ends=False)
    mx = MxCase(q, [40, 60], 128, 72)
    y, dx, dw = c._out(c.m, c.n, 0), c._out(c.m, c.k, 0), c._out(c.e * c.k, c.n, 0)
    y4 = torch.empty(100, 72, device="cuda")
    xb = ints(gen_of(1), (100, 128), torch.bfloat16, 6)

    def calls():
        q.grouped_mm(c.p, c.x, c.w, c.gl, y, c.ws)
        q.grouped_mm_dgrad(c.p, c.dy, c.w, c.gl, dx, c.ws)
        q.grouped_mm_wgrad(c.p, c.x, c.dy, c.gl, dw, c.ws)
        q.per_token_quant_mxfp4(xb, mx.bx, mx.bsx)
        q.grouped_mm(mx.p, mx.bx, mx.bw, mx.gl, y4, mx.ws, x_scale=mx.bsx, w_scale=mx.bsw)

    calls()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        calls()
    other = Case(q, [33, 44], 128, 72, seed=5)
    for seed in (21, 22):
        gen = gen_of(seed)
        c.x.copy_(ints(gen, c.x.shape, c.x.dtype))
        c.dy.copy_(ints(gen, c.dy.shape, c.x.dtype))
        xb.copy_(ints(gen, xb.shape, xb.dtype, 6))
        c.gl.copy_(torch.tensor([seed, 50, 50 - seed], device="cuda"))
        c.counts = [seed, 50, 50 - seed]
        for t in (y, dx, dw, y4):
            t.fill_(float("nan"))
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            graph.replay()
        got = other.fwd()
        torch.cuda.synchronize()
        assert torch.equal(got, other.want_rows(other.x, other.w))
        assert torch.equal(y, c.want_rows(c.x, c.w)) and torch.equal(dx, c.want_rows(c.dy, c.w.transpose(1, 2)))
        assert torch.equal(dw, c.want_dw().float().reshape(-1, c.n))
        assert torch.equal(y4, mx.want().float())
        assert c.status() == 0 and q.device_status(mx.ws) == 0
    del graph


@pytest.mark.parametrize("call", ["fwd", "wgrad", "mxfp4"])
def test_waits_that_run_out_are_reported(q, call, monkeypatch):
    """With no copy issued every wait gives up after its second: the call reports it, and the
    next one on the same workspace is as usual.  (600 rows of one expert take the
    arranged scales, the others the gathered ones.)"""
    c = MxCase(q, [600], 512, 72) if call == "mxfp4" else Case(q, [70, 3], 136, 72)
    run = {"fwd": getattr(c, "fwd", None), "wgrad": getattr(c, "wgrad", None), "mxfp4": getattr(c, "run", None)}[call]
    monkeypatch.setenv("QGMM_TEST_STALL_PRODUCER", "1")
    run()
    assert q.device_status(c.ws) & q.QGMM_DEV_TIMEOUT
    monkeypatch.delenv("QGMM_TEST_STALL_PRODUCER")
    want = {"fwd": lambda: c.want_rows(c.x, c.w), "wgrad": lambda: c.want_dw().float().reshape(-1, 72),
            "mxfp4": lambda: c.want().float()}[call]()
    assert torch.equal(run(), want)
    assert q.device_status(c.ws) == 0


def test_many_tiles_for_every_pair(q):
    """More tiles than pairs by far, ragged, so that both accumulators and the ring wrap many times."""
    rng = np.random.default_rng(5)
    counts = rng.integers(0, 900, 12).tolist()
    Case(q, counts, 264, 2056, out_type=0, lim=2).check()
    c = MxCase(q, counts, 544, 2056, out_type=0)
    assert torch.equal(c.run(), c.want().bfloat16())


def test_binding_refuses_what_does_not_fit(q):
    c = Case(q, [10, 6], 64, 72)
    y = c._out(16, 72, 0)
    bad = [lambda: q.grouped_mm(c.p, c.x[:15], c.w, c.gl, y, c.ws), lambda: q.grouped_mm(c.p, c.x, c.w[:1], c.gl, y, c.ws),
           lambda: q.grouped_mm(c.p, c.x, c.w, c.gl[:1], y, c.ws), lambda: q.grouped_mm(c.p, c.x, c.w, c.gl, y[:15], c.ws),
           lambda: q.grouped_mm_wgrad(c.p, c.x, c.dy, c.gl, torch.empty(2, 64, 64, device="cuda"), c.ws)]
    for call in bad:
        with pytest.raises(q.QgmmError) as err:
            call()
        assert err.value.code == q.QGMM_ERR_SHAPE
    other_order = c.w.transpose(1, 2).contiguous().transpose(1, 2)
    wide = torch.zeros(16, 128, dtype=torch.bfloat16, device="cuda")
    for call in (lambda: q.grouped_mm(c.p, c.x, other_order, c.gl, y, c.ws),
                 lambda: q.grouped_mm(c.p, wide[:, :64], c.w, c.gl, y, c.ws),
                 lambda: q.grouped_mm(c.p, wide[:, ::2], c.w, c.gl, y, c.ws),
                 lambda: q.grouped_mm(c.p, c.x, c.w, torch.zeros(4, dtype=torch.int64, device="cuda")[::2], y, c.ws),
                 lambda: q.grouped_mm_dgrad(c.p, c.dy.t().contiguous().t(), c.w, c.gl, c._out(16, 64, 0), c.ws),
                 lambda: q.per_token_quant_mxfp4(c.x.t(), c.ws[:128].view(64, 2), c.ws)):
        with pytest.raises(q.QgmmError) as err:
            call()
        assert err.value.code == q.QGMM_ERR_SHAPE
    strided = q.make_mm_problem(16, 64, 72, 2, out_type=2, ld_x=128)
    wide[:, :64] = c.x
    q.grouped_mm(strided, wide[:, :64], c.w, c.gl, y, c.ws)
    assert torch.equal(y, c.want_rows(c.x, c.w))
    for call in (lambda: q.grouped_mm(c.p, c.x.half(), c.w, c.gl, y, c.ws),
                 lambda: q.grouped_mm(c.p, c.x, c.w, c.gl.int(), y, c.ws),
                 lambda: q.grouped_mm(c.p, c.x, c.w, c.gl, y.bfloat16(), c.ws)):
        with pytest.raises(q.QgmmError) as err:
            call()
        assert err.value.code == q.QGMM_ERR_DTYPE
    with pytest.raises(q.QgmmError) as err:
        q.grouped_mm(c.p, c.x, c.w, c.gl, y, c.ws[:128])
    assert err.value.code == q.QGMM_ERR_WORKSPACE_TOO_SMALL


# ---------------------------------------------------------------- sums in parts
# Few tiles and a long sum: the parts go through the workspace, which is how a test knows of them.
@pytest.mark.parametrize("counts,k,n", [([1], 4096, 1024), ([3, 0, 2], 40, 2600), ([0, 5], 2104, 264), ([600], 2600, 136),
                                        ([70, 3, 0], 4104, 520), ([0, 64, 65], 8, 9000), ([1] * 9, 16384, 72)])
@pytest.mark.parametrize("x_type,out_type", [(0, 2), (0, 0), (1, 1)])
def test_sums_in_parts_exact(q, counts, k, n, x_type, out_type):
    for transpose_w in (False, True):
        c = Case(q, counts, k, n, m=sum(counts) + 5, x_type=x_type, out_type=out_type, transpose_w=transpose_w,
                 seed=k + n, pad=24 if transpose_w else 0, lim=2)
        assert c.ws.numel() > 256
        c.x[c.total:], c.dy[c.total:] = float("nan"), float("inf")   # rows past the total
        c.check()


@pytest.mark.parametrize("counts,k,n", [([1], 8192, 1024), ([5, 0, 40], 7200, 264), ([900], 16384, 72), ([2] * 9, 8224, 8)])
@pytest.mark.parametrize("out_type", [0, 1, 2])
def test_mxfp4_sums_in_parts_exact(q, counts, k, n, out_type):
    c = MxCase(q, counts, k, n, m=sum(counts) + 7, out_type=out_type, spread=1, seed=k)
    c.bsx[sum(counts):] = 255
    assert torch.equal(c.run(), c.want().to(T[out_type]))
    assert q.device_status(c.ws) == 0


def test_sums_in_parts_of_normal_values(q):
    """As the other normal values: k terms, 2^-23 of the magnitudes each, and half a step of the output."""
    for x_type, out_type, half in ((0, 0, 2.0 ** -8), (1, 1, 2.0 ** -11), (0, 2, 2.0 ** -24)):
        c = Case(q, [20, 0, 3], 8200, 264, x_type=x_type, out_type=out_type, transpose_w=True)
        gen = gen_of(out_type + 1)
        c.x.normal_(generator=gen), c.w.normal_(0, 8200 ** -0.5, generator=gen)
        got = c.fwd()
        for g, r in spans(c.counts):
            want, mag = c.x[r].double() @ c.w[g].double().t(), c.x[r].double().abs() @ c.w[g].double().abs().t()
            bound = 8200 * 2.0 ** -23 * mag
            assert bool(((got[r].double() - want).abs() <= bound + half * (want.abs() + bound)).all())
        assert all(torch.equal(got, c.fwd()) for _ in range(3))


@pytest.mark.parametrize("kind", ["negative", "decreasing", "beyond"])
def test_sums_in_parts_with_bad_group_lists(q, kind):
    gl, ends, flag, counts = {
        "negative": ([5, -3, 10, 0], False, 1, [5, 0, 10, 0]),
        "decreasing": ([20, 10, 30, 40], True, 2, [20, 0, 10, 10]),
        "beyond": ([30, 2 ** 62, 2 ** 62, 7], False, 4, [30, 34, 0, 0]),
    }[kind]
    c = Case(q, counts, 4096, 72, m=64, ends=ends, out_type=0)
    assert c.ws.numel() > 256
    c.gl = torch.tensor(gl, dtype=torch.int64, device="cuda")
    assert torch.equal(c.fwd(), c.want_rows(c.x, c.w))
    assert c.status() == flag
    c.gl = torch.zeros(4, dtype=torch.int64, device="cuda")       # and with no rows at all
    assert bool((c.fwd() == SENTINEL).all()) and c.status() == 0


def test_sums_in_parts_keep_nan_and_inf_in_their_rows(q):
    c = Case(q, [7, 6, 3], 4096, 264)
    c.x[9, 4000], c.x[10, 5] = float("nan"), float("inf")
    got, keep = c.fwd(), [i for i in range(16) if i not in (9, 10)]
    assert torch.equal(got[keep], c.want_rows(c.x, c.w)[keep])
    assert bool(got[9].isnan().all()) and not bool(got[10].isfinite().any())


def test_sums_in_parts_captured_with_shared_workspace(q):
    """Both directions and a product with another number of parts, one after the other on one workspace,
    in two graphs replayed in turn with new rows."""
    a, b = Case(q, [3, 5], 4096, 2600, ends=False), Case(q, [9, 0, 1], 8192, 72, out_type=0)
    ws = torch.empty(max(a.ws.numel(), b.ws.numel()), dtype=torch.uint8, device="cuda")
    a.ws = b.ws = ws
    outs = a._out(8, 2600, 0), a._out(8, 4096, 0), b._out(10, 72, 0)

    def calls():
        q.grouped_mm(a.p, a.x, a.w, a.gl, outs[0], ws)
        q.grouped_mm_dgrad(a.p, a.dy, a.w, a.gl, outs[1], ws)
        q.grouped_mm(b.p, b.x, b.w, b.gl, outs[2], ws)

    calls()
    torch.cuda.synchronize()
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    for g in graphs:
        with torch.cuda.graph(g):
            calls()
    for i, (g, counts) in enumerate(zip(graphs * 2, ([8, 0], [1, 2], [0, 0], [4, 4]))):
        gen = gen_of(30 + i)
        for t in (a.x, a.dy, b.x):
            t.copy_(ints(gen, t.shape, t.dtype))
        a.counts = counts
        a.gl.copy_(torch.tensor(counts, device="cuda"))
        for t in outs:
            t.fill_(SENTINEL)
        g.replay()
        assert torch.equal(outs[0], a.want_rows(a.x, a.w))
        assert torch.equal(outs[1], a.want_rows(a.dy, a.w.transpose(1, 2)))
        assert torch.equal(outs[2], b.want_rows(b.x, b.w))
        assert q.device_status(ws) == 0
    del graphs


def test_sums_in_parts_report_waits_that_run_out(q, monkeypatch):
    c = Case(q, [5, 3], 4096, 72)
    assert c.ws.numel() > 256
    monkeypatch.setenv("QGMM_TEST_STALL_PRODUCER", "1")
    c.fwd()
    assert c.status() & q.QGMM_DEV_TIMEOUT
    monkeypatch.delenv("QGMM_TEST_STALL_PRODUCER")
    assert torch.equal(c.fwd(), c.want_rows(c.x, c.w)) and c.status() == 0


@pytest.mark.parametrize("counts,k,n", [([2600], 64, 256), ([0, 5000, 1, 70, 0], 152, 72), ([0, 12000, 1, 70, 0], 152, 72), ([13, 3, 9024], 264, 520),
                                        ([3000, 3001, 2999], 256, 768), ([40000], 8, 8)])
@pytest.mark.parametrize("x_type,out_type,accumulate", [(0, 2, False), (0, 0, True), (1, 1, False), (1, 2, True)])
def test_weight_gradients_in_parts_exact(q, counts, k, n, x_type, out_type, accumulate):
    """An expert's rows in parts: uneven, empty and unaligned ones, NaN and infinity in the rows of no
    expert; accumulated, what experts without rows hold (a negative zero too) stays bit for bit."""
    for transpose_w in (False, True):
        c = Case(q, counts, k, n, m=sum(counts) + 9, x_type=x_type, out_type=out_type, accumulate=accumulate,
                 transpose_w=transpose_w, pad=16 if transpose_w else 0, ends=transpose_w, seed=k + n, lim=1)
        assert c.ws.numel() > 256 or c.m < 1600 * c.e        # fewer rows an expert are summed whole
        c.x[c.total:], c.dy[c.total:] = float("nan"), float("inf")
        width, rows = c.w.shape[2], c.w.shape[1]
        old = ints(gen_of(9), (c.e * rows, c.p.ld_w or width), c.out, 50)
        old[old == 0] = -0.0
        got = c.wgrad(old.clone())
        assert c.status() == 0
        want = c.want_dw()
        if accumulate:
            want += old[:, :width].view(c.e, rows, width).double()
        want = want.to(c.out).reshape(-1, width)
        assert torch.equal(got[:, :width], want) and torch.equal(got[:, width:], old[:, width:])
        for g, r in spans(counts):
            if accumulate and r.start == r.stop:
                mine = slice(g * rows, (g + 1) * rows)
                assert torch.equal(got[mine].signbit(), old[mine].signbit())


@pytest.mark.parametrize("last", [4100, 8100])
def test_weight_gradients_in_parts_keep_nan_in_their_expert(q, last):
    c = Case(q, [3000, 40, 5, last], 136, 72)
    assert c.ws.numel() > 256 or last == 4100
    c.x[3000:3040], c.dy[3000:3040] = float("nan"), float("inf")
    got, want = c.wgrad().view(4, 136, 72), c.want_dw().float()
    assert all(torch.equal(got[g], want[g]) for g in (0, 2, 3)) and bool(got[1].isnan().all())


@pytest.mark.parametrize("kind", ["negative", "decreasing", "beyond"])
@pytest.mark.parametrize("times", [1, 2])
def test_weight_gradients_in_parts_with_bad_group_lists(q, kind, times):
    gl, ends, flag, counts = {
        "negative": ([500, -3, 5500, 0], False, 1, [500, 0, 5500, 0]),
        "decreasing": ([2000, 1000, 3000, 6000], True, 2, [2000, 0, 1000, 3000]),
        "beyond": ([3000, 2 ** 62, 2 ** 62, 7], False, 4, [3000, 4000, 0, 0]),
    }[kind]
    c = Case(q, [times * v for v in counts], 64, 72, m=7000 * times, ends=ends)
    assert c.ws.numel() > 256 or times == 1
    c.gl = torch.tensor([v if v == 2 ** 62 else times * v for v in gl], dtype=torch.int64, device="cuda")
    assert torch.equal(c.wgrad(), c.want_dw().float().reshape(-1, 72))
    assert c.status() == flag
    c.gl = torch.zeros(4, dtype=torch.int64, device="cuda")
    assert not c.wgrad().any() and c.status() == 0


def test_weight_gradients_in_parts_of_normal_values(q):
    """Sums of up to 9000 terms, 2^-23 of the magnitudes each, and half a step; every time the same bits."""
    for x_type, out_type, half in ((0, 0, 2.0 ** -8), (1, 1, 2.0 ** -11), (0, 2, 2.0 ** -24)):
        c = Case(q, [9000, 3, 2000], 136, 264, x_type=x_type, out_type=out_type)
        for i, t in enumerate((c.x, c.dy)):
            t.normal_(0, 0.25, generator=gen_of(out_type + 3 + i))
        got = c.wgrad()
        assert all(torch.equal(got, c.wgrad()) for _ in range(3))
        for g, r in spans(c.counts):
            x, dy = c.x[r].double(), c.dy[r].double()
            want, bound = x.t() @ dy, 9000 * 2.0 ** -23 * (x.abs().t() @ dy.abs())
            assert bool(((got.view(3, 136, 264)[g].double() - want).abs() <= bound + half * (want.abs() + bound)).all())


def test_weight_gradients_in_parts_captured_and_waits_that_run_out(q, monkeypatch):
    c = Case(q, [3000, 4000], 136, 72, m=7000, ends=False)
    dw = c.wgrad()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        q.grouped_mm_wgrad(c.p, c.x, c.dy, c.gl, dw, c.ws)
    for counts in ([7000, 0], [1, 6000], [64, 6936]):
        c.counts = counts
        c.gl.copy_(torch.tensor(counts, device="cuda"))
        dw.fill_(SENTINEL)
        graph.replay()
        assert torch.equal(dw, c.want_dw().float().reshape(-1, 72)) and c.status() == 0
    monkeypatch.setenv("QGMM_TEST_STALL_PRODUCER", "1")
    c.wgrad()
    assert c.status() & q.QGMM_DEV_TIMEOUT
    monkeypatch.delenv("QGMM_TEST_STALL_PRODUCER")
    assert torch.equal(c.wgrad(), c.want_dw().float().reshape(-1, 72)) and c.status() == 0
    del graph


# ---------------------------------------------------------------- long sums into 16 bits
def shrink(got, want):
    """The share of itself that `got` lost against 64-bit `want`, and six deviations of that share's mean
    over independent roundings of at most half a step each."""
    want = want.flatten()
    lost = float(-((got.flatten().double() - want) * want).sum() / (want * want).sum())
    return lost, 6 * torch.finfo(got.dtype).eps / 2 * float((want ** 4).sum().sqrt() / (want * want).sum())


@pytest.mark.parametrize("length", [16384, 65536])
@pytest.mark.parametrize("call", ["fwd", "dgrad"])
@pytest.mark.parametrize("transpose_w", [False, True])
def test_long_16_bit_sums_do_not_drift(q, length, call, transpose_w):
    """Whole sums (more tiles than the parts' rule takes), taken out of the tensor core every 2048 terms: 128
    instructions, each of which may truncate by 2^-24 of the running sum on average."""
    k, n = (length, 2048) if call == "fwd" else (2048, length)
    c = Case(q, [2048], k, n, x_type=1, out_type=1, transpose_w=transpose_w)
    gen = gen_of(length)
    for t in (c.x, c.dy, c.w):
        t.normal_(0, 0.25, generator=gen)
    w = mat(c.w, transpose_w)[0].double()
    c.ws.fill_(0xA5)
    got, want = (c.fwd(), c.x.double() @ w) if call == "fwd" else (c.dgrad(), c.dy.double() @ w.t())
    assert bool((c.ws[256:] == 0xA5).all())              # not cut into parts
    lost, noise = shrink(got, want)
    assert abs(lost) <= 128 * 2.0 ** -24 + noise


@pytest.mark.parametrize("k,n", [(8264, 2600), (2600, 8264)])
@pytest.mark.parametrize("x_type", [0, 1])
def test_long_16_bit_sums_exact(q, k, n, x_type):
    for transpose_w, counts in ((False, [70, 300, 0, 257, 1]), (True, [15, 600])):
        c = Case(q, counts, k, n, m=sum(counts) + 7, x_type=x_type, out_type=x_type, transpose_w=transpose_w,
                 pad=24 if transpose_w else 0, seed=k, lim=1)
        c.x[c.total:], c.dy[c.total:] = float("nan"), float("inf")
        c.check()


@pytest.mark.parametrize("rows,x_type", [(1 << 18, 1), (1 << 19, 1), (1 << 19, 0)])
@pytest.mark.parametrize("transpose_w", [False, True])
def test_long_16_bit_weight_gradients_do_not_drift(q, rows, x_type, transpose_w):
    """As above: whole sums, taken out every 8192 rows (fp16) or 32768 (bf16), 16 rows an instruction."""
    c = Case(q, [rows], 1600, 2040, x_type=x_type, out_type=x_type, transpose_w=transpose_w)
    assert 2 * -(-1600 // 256) * -(-2040 // 256) > 74    # tiles: not cut into parts
    gen = gen_of(rows)
    for t in (c.x, c.dy):
        t.normal_(0, 0.125, generator=gen)
    want = torch.zeros(1600, 2040, dtype=torch.float64, device="cuda")
    for at in range(0, rows, 1 << 14):
        part = slice(at, at + (1 << 14))
        want += c.x[part].double().t() @ c.dy[part].double()
    got = c.wgrad()
    lost, noise = shrink(got, want.t() if transpose_w else want)
    assert abs(lost) <= (512 if x_type else 2048) * 2.0 ** -24 + noise


@pytest.mark.parametrize("counts,k,n", [([32768], 1608, 1544), ([32769], 1608, 1544), ([33000, 0, 65537, 70], 776, 1032),
                                        ([300] * 37 + [70001], 264, 520), ([10] * 240 + [66001], 264, 136)])
@pytest.mark.parametrize("x_type,accumulate", [(0, False), (1, True), (0, True)])
def test_long_16_bit_weight_gradients_exact(q, counts, k, n, x_type, accumulate):
    """One segment, barely two, several; one and two epilogue groups; next to experts without rows, and
    NaN and infinity in the rows of no expert."""
    for transpose_w in (False, True):
        c = Case(q, counts, k, n, m=sum(counts) + 9, x_type=x_type, out_type=x_type, accumulate=accumulate,
                 transpose_w=transpose_w, pad=16 if transpose_w else 0, ends=transpose_w, seed=k + n, lim=1)
        c.x[c.total:], c.dy[c.total:] = float("nan"), float("inf")
        c.ws.fill_(255)                                  # NaN wherever f32 sums are kept
        width, rows = c.w.shape[2], c.w.shape[1]
        old = ints(gen_of(9), (c.e * rows, c.p.ld_w or width), c.out, 50)
        got = c.wgrad(old.clone())
        assert c.status() == 0
        want = c.want_dw() + (old[:, :width].view(c.e, rows, width).double() if accumulate else 0)
        assert torch.equal(got[:, :width], want.to(c.out).reshape(-1, width))
        assert torch.equal(got[:, width:], old[:, width:])


def test_long_16_bit_weight_gradients_keep_nan_in_their_expert(q):
    c = Case(q, [66000, 40, 140000, 65540], 776, 1032, out_type=0, lim=2)
    c.x[66000:66040], c.dy[66000:66040] = float("nan"), float("inf")
    c.dy[66040 + 65540, 5] = float("nan")
    got, want = c.wgrad().view(4, 776, 1032), c.want_dw().bfloat16()
    assert torch.equal(got[0], want[0]) and torch.equal(got[3], want[3]) and bool(got[1].isnan().all())
    assert bool(got[2, :, 5].isnan().all())
    got[2, :, 5] = want[2, :, 5] = 0
    assert torch.equal(got[2], want[2])
    assert all(torch.equal(c.wgrad().view(4, 776, 1032)[3], want[3]) for _ in range(3))


def test_a_weight_gradient_of_more_than_a_second(q):
    """The rows past the last expert's end are cleared when its tiles come, here after more than a second
    of tiles of whole stages: a limit that counted from the kernel's start would report a wait that ran out."""
    torch.cuda.empty_cache()
    free = torch.cuda.mem_get_info()[0]
    block, times, width = 8192, 32, 65536                # 2.3e15 operations
    rows = block * times
    if free < 100 << 30:
        pytest.skip("needs 90 GB")
    base = [ints(gen_of(s), (block, width), torch.bfloat16, 1) for s in (1, 2)]
    last = [ints(gen_of(s), (8, width), torch.bfloat16, 1) for s in (3, 4)]
    x, dy = (torch.cat([b] * times + [l]) for b, l in zip(base, last))
    dw = torch.empty(2, width, width, dtype=torch.bfloat16, device="cuda")
    p = q.make_mm_problem(rows + 8, width, width, 2)
    ws = torch.empty(q.grouped_mm_workspace(p), dtype=torch.uint8, device="cuda")
    gl = group_list([rows, 8], True)
    start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    start.record()
    q.grouped_mm_wgrad(p, x, dy, gl, dw, ws)
    end.record()
    assert q.device_status(ws) == 0
    assert start.elapsed_time(end) > 1100                # else this shows nothing
    del x, dy
    for at in (0, 256, 32768 + 100, width - 128):
        r = slice(at, at + 128)
        assert torch.equal(dw[0, r], (times * (base[0][:, r].t().float() @ base[1].float())).bfloat16())
        assert torch.equal(dw[1, r], (last[0][:, r].t().float() @ last[1].float()).bfloat16())
    del dw, base, last
    torch.cuda.empty_cache()


def test_a_refused_launch_is_not_the_next_calls(q):
    """A launch on the default stream while a stream that waits for it is captured fails on the host;
    the calls after it succeed, and are reported so."""
    import ctypes as C
    rt = C.CDLL("libcudart.so.12")                       # the one that torch has loaded
    whole, parts, none = Case(q, [70, 3], 136, 72), Case(q, [3], 8192, 264), Case(q, [0, 0], 64, 72)
    for c in (whole, parts, none):
        c.fwd()
    calls = [(c, c._out(c.m, c.n, 0)) for c in (whole, parts, none)]
    torch.cuda.synchronize()
    for c, y in calls:
        stream, graph = C.c_void_p(), C.c_void_p()
        assert rt.cudaStreamCreate(C.byref(stream)) == 0
        assert rt.cudaStreamBeginCapture(stream, 0) == 0
        try:
            with pytest.raises(q.QgmmError) as err:
                q.grouped_mm(whole.p, whole.x, whole.w, whole.gl, calls[0][1], whole.ws, stream=0)
        finally:
            assert rt.cudaStreamEndCapture(stream, C.byref(graph)) != 0 and not graph.value
            rt.cudaGetLastError()
            assert rt.cudaStreamDestroy(stream) == 0
        assert err.value.code == q.QGMM_ERR_CUDA
        q.grouped_mm(c.p, c.x, c.w, c.gl, y, c.ws)
        assert torch.equal(y, c.want_rows(c.x, c.w)) and c.status() == 0


# ---------------------------------------------------------------- which sums are whole
def parts_written(c, call):
    """Whether `call` used the workspace past its head, where the parts of a sum go."""
    c.ws.fill_(0xA5)
    call()
    torch.cuda.synchronize()
    return bool((c.ws[256:] != 0xA5).any())


@pytest.mark.parametrize("counts,k,n,cut", [
    ([1], 4096, 1024, "fwd"), ([3, 0, 2], 40, 2600, "dgrad"), ([70, 3, 0], 4104, 520, "fwd"), ([1] * 9, 16384, 72, "fwd"),
    ([0, 64, 65], 8, 9000, "dgrad"), ([0, 5000, 1, 70, 0], 152, 72, ""), ([0, 12000, 1, 70, 0], 152, 72, "wgrad"),
    ([2600], 64, 256, "wgrad"), ([40000], 8, 8, "wgrad"), ([3000, 40, 5, 4100], 136, 72, "wgrad"), ([700, 3], 136, 248, ""),
    ([5, 3], 4096, 4104, "fwd dgrad"), ([2048], 65536, 2048, "")])
def test_each_direction_is_cut_where_the_rule_says(q, counts, k, n, cut):
    c = Case(q, counts, k, n)
    assert " ".join(d for d in ("fwd", "dgrad", "wgrad") if parts_written(c, getattr(c, d))) == cut


@pytest.mark.parametrize("call", ["fwd", "dgrad", "wgrad"])
def test_whole_f32_sums_do_not_drift(q, call):
    """128 segments of 512 terms: 32 instructions each, which may truncate by 2^-24 of the running sum on
    average; the additions between them and the output are rounded."""
    long, wide = 65536, 2048
    c = Case(q, [long if call == "wgrad" else wide], long if call == "fwd" else wide, long if call == "dgrad" else wide)
    gen = gen_of(12)
    for t in (c.x, c.dy, c.w):
        t.normal_(0, 0.25, generator=gen)
    assert not parts_written(c, getattr(c, call))
    got = getattr(c, call)()
    want = {"fwd": lambda: c.x.double() @ c.w[0].double(), "dgrad": lambda: c.dy.double() @ c.w[0].double().t(),
            "wgrad": lambda: c.x.double().t() @ c.dy.double()}[call]()
    lost, noise = shrink(got, want)
    assert abs(lost) <= 32 * 2.0 ** -24 + noise
    # 128 roundings of half a step and the drift, in the norm
    assert float((got.double() - want).norm() / want.norm()) <= (32 + 128 ** 0.5) * 2.0 ** -24


@pytest.mark.parametrize("k", [8192, 65536])
def test_mxfp4_f32_sums_of_scattered_scales_do_not_drift(q, k):
    """Blocks up to 2^10 apart in scale, where sums are no longer exact: segments of 8192 terms are 128
    instructions, the additions between them rounded."""
    gen = gen_of(k)
    c = MxCase(q, [700, 1348], k, 1024)
    spread = lambda *s: torch.exp2(10 * torch.rand(*s, k // 32, generator=gen, device="cuda") - 5).repeat_interleave(32, -1)
    q.per_token_quant_mxfp4(torch.randn(2048, k, generator=gen, device="cuda") * spread(2048), c.bx, c.bsx)
    q.per_token_quant_mxfp4(torch.randn(2048, k, generator=gen, device="cuda") * spread(2048), c.bw, c.bsw)
    got, want = c.run(), c.want()
    lost, noise = shrink(got, want)
    assert abs(lost) <= 128 * 2.0 ** -24 + noise
    assert float((got.double() - want).norm() / want.norm()) <= (128 + 8 ** 0.5) * 2.0 ** -24


@pytest.mark.parametrize("rows", [64, 4096])
def test_f32_accumulation_keeps_subnormals(q, rows):
    """Whole sums are added by a reducing copy, parts in registers: both as IEEE adds them."""
    x, dy = (torch.zeros(rows, w, dtype=torch.bfloat16, device="cuda") for w in (64, 256))
    x[0], dy[0] = 2.0 ** -70, 2.0 ** -70                 # their product is 2^-140
    p = q.make_mm_problem(rows, 64, 256, 1, out_type=2, accumulate=True)
    ws = torch.empty(q.grouped_mm_workspace(p), dtype=torch.uint8, device="cuda")
    old = torch.tensor([2.0 ** -130, -2.0 ** -130, 2.0 ** -149, 1.5 * 2.0 ** -126, 2.0 ** -126, 0.0, -2.0 ** -140, 1.0], device="cuda")
    dw = old.repeat(64, 32).view(1, 64, 256).clone()
    q.grouped_mm_wgrad(p, x, dy, group_list([rows], True), dw, ws)
    want = (old.double() + 2.0 ** -140).float().repeat(64, 32).view(1, 64, 256)
    assert torch.equal(dw, want)


@pytest.mark.parametrize("call,length,instructions", [("fwd", 65536, 128), ("dgrad", 65536, 128), ("wgrad", 1 << 18, 512)])
def test_long_fp16_sums_of_one_sign(q, call, length, instructions):
    """Where the terms have one sign the running sum grows to its end, half of it on average, and an
    instruction may lose half of 2^-23 of it with each of its 16 products and with the sum so far."""
    wide = 2048
    c = Case(q, [length if call == "wgrad" else wide], length if call == "fwd" else wide, length if call == "dgrad" else wide,
             x_type=1, out_type=1)
    gen = gen_of(length)
    for t in (c.x, c.dy, c.w):
        t.uniform_(0, 0.5, generator=gen)
    assert not parts_written(c, getattr(c, call)) or call == "wgrad"
    got = getattr(c, call)()
    if call == "wgrad":
        want = sum(c.x[at:at + 16384].double().t() @ c.dy[at:at + 16384].double() for at in range(0, length, 16384))
    else:
        want = c.x.double() @ c.w[0].double() if call == "fwd" else c.dy.double() @ c.w[0].double().t()
    lost, noise = shrink(got, want)
    assert abs(lost) <= instructions * 17 / 4 * 2.0 ** -23 + noise
