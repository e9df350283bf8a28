"""Low-rank adapters beside the projection on the GPU (forward and backward)
and the gradient of the projection's input, against the formulas in 64 bits.

Most cases are exact: activations, factors and gradients are small integers
(times powers of two), so that every product and sum has an exact fp32 value
(below 2^24 units) and the result differs from the formula by its one rounding
to fp16, which the reference repeats; a single missing or misplaced term
shows. The others use normal values and the bound

    |err| <= 2^-11 |ref| + 2^-25 + c,

one fp16 rounding (half a step, also of the smallest subnormal) and c for the
fp32 sums: a sum of h products is rounded h times, on the tensor cores toward
zero once per 16 products, each time by at most 2^-23 of a partial sum that
is at most |x| |a| (Cauchy-Schwarz): together below 16 sqrt(h) 2^-24 |x| |a|
for h <= 16384, and the same again for the second product.
"""
import numpy as np
import pytest
import torch

from mixed_precision_int8_b200 import binding as L, build

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    build.build()
    L.load_library()
    yield


def ints(gen, shape, hi, density=1.0, dtype=torch.float16):
    t = torch.randint(-hi, hi + 1, shape, generator=gen, device="cuda")
    if density < 1.0:
        t = t * (torch.rand(shape, generator=gen, device="cuda") < density)
    return t.to(dtype)


class Case:
    """A batch with integer values whose sums stay exact."""

    def __init__(self, s, h, o, n, r, layout, ranks, seed=0, real=False):
        g = torch.Generator(device="cuda").manual_seed(seed + 31 * s + h)
        self.s, self.h, self.o, self.n, self.r = s, h, o, n, r
        if real:
            self.X = torch.randn(s, h, generator=g, device="cuda").half()
            self.A = (torch.randn(n, r, h, generator=g, device="cuda") * h ** -0.5).half()
            self.B = (torch.randn(n, r, o, generator=g, device="cuda") * 0.05).half()
            self.base = torch.randn(s, o, generator=g, device="cuda").half()
            self.dbase = torch.randn(s, h, generator=g, device="cuda").half()
            self.dY = (torch.randn(s, o, generator=g, device="cuda") * 0.1).half()
            self.scale = 0.5 + torch.rand(n, generator=g, device="cuda")
        else:
            self.X = ints(g, (s, h), 4)
            self.A = ints(g, (n, r, h), 2, 0.25)
            self.B = ints(g, (n, r, o), 2, 0.25)
            self.base = ints(g, (s, o), 100)
            self.dbase = ints(g, (s, h), 100)
            self.dY = ints(g, (s, o), 3, 0.5)
            self.scale = torch.tensor([2.0 ** -(a % 5) for a in range(n)], device="cuda")
        if layout == "requests":
            cuts = sorted(torch.randint(0, s + 1, (n - 1,), generator=g, device="cuda").tolist())
            ids = [sum(i >= c for c in cuts) for i in range(s)]
        elif layout == "requests_bare":
            cuts = sorted(torch.randint(0, s + 1, (n,), generator=g, device="cuda").tolist())
            ids = [sum(i >= c for c in cuts) - 1 for i in range(s)]
        elif layout == "mixed":  # any order, rows without an adapter among them
            ids = torch.randint(-1, n, (s,), generator=g, device="cuda").tolist()
        elif layout == "wild":  # ids that name no adapter
            ids = [(-1, n, 2 ** 31 - 1, -2 ** 31, 0)[i % 5] for i in range(s)]
        else:  # none
            ids = [-1] * s
        self.ids_list = [a if 0 <= a < n else -1 for a in ids]
        self.ids = torch.tensor(ids, dtype=torch.int32, device="cuda")
        self.rank_list = [r] * n if ranks == "full" else [(7 * a + 3) % (r + 1) for a in range(n)]
        self.ranks = None if ranks == "full" else torch.tensor(
            self.rank_list, dtype=torch.int32, device="cuda")
        self.ad = L.Adapters(self.A, self.B, self.scale, self.ranks)

    def rows(self, a):
        return torch.tensor([i for i, x in enumerate(self.ids_list) if x == a],
                            dtype=torch.long, device="cuda")

    def reference(self):
        """(out, v, dX, dA, dB) in 64 bits."""
        d = torch.float64
        out, dX = self.base.to(d), self.dbase.to(d)
        v = torch.zeros(self.s, self.r, dtype=d, device="cuda")
        dA = torch.zeros(self.A.shape, dtype=d, device="cuda")
        dB = torch.zeros(self.B.shape, dtype=d, device="cuda")
        for a in sorted(set(self.ids_list) - {-1}):
            rows, k = self.rows(a), self.rank_list[a]
            A, B, c = self.A[a, :k].to(d), self.B[a, :k].to(d), float(self.scale[a])
            X, dY = self.X[rows].to(d), self.dY[rows].to(d)
            v[rows, :k] = X @ A.T
            out[rows] += c * (v[rows, :k] @ B)
            g = dY @ B.T
            dX[rows] += c * (g @ A)
            dA[a, :k] = c * (g.T @ X)
            dB[a, :k] = c * (v[rows, :k].T @ dY)
        return out, v, dX, dA, dB


def same(got, ref, dtype):
    """Equal as values of the type, the reference rounded once."""
    assert got.dtype == dtype
    assert torch.equal(got, ref.to(dtype))


def bits(t):
    return t.view(torch.int16)


# sizes: one row, the row kernels' limits (128 rows, the work, backward 64 rows
# per adapter held), tiles of 128 rows and the rows around their edges, widths that end inside a tile, ranks that are no
# multiple of 16, more adapters in a tile than accumulators
CASES = [
    (1, 16, 16, 1, 8, "requests", "full"),
    (1, 528, 272, 3, 8, "mixed", "mixed"),
    (7, 4096, 1040, 16, 16, "mixed", "mixed"),
    (16, 1040, 2064, 3, 64, "mixed", "full"),
    (17, 1040, 2064, 3, 24, "mixed", "mixed"),
    (32, 272, 784, 40, 128, "mixed", "mixed"),
    (33, 272, 784, 40, 128, "mixed", "mixed"),
    (33, 272, 784, 1, 128, "mixed", "mixed"),
    (64, 512, 528, 64, 8, "mixed", "full"),
    (128, 528, 784, 40, 24, "mixed", "mixed"),
    (65, 528, 512, 2, 40, "requests", "full"),
    (128, 2064, 784, 2, 16, "requests_bare", "mixed"),
    (64, 528, 784, 1, 24, "requests", "full"),
    (65, 528, 784, 1, 24, "requests", "full"),
    (70, 12288, 16400, 1, 64, "mixed", "mixed"),
    (127, 16400, 12288, 2, 64, "requests", "full"),
    (129, 784, 2064, 2, 16, "requests", "full"),
    (200, 1024, 784, 150, 64, "mixed", "mixed"),
    (300, 528, 272, 4, 128, "requests_bare", "full"),
    (513, 1040, 1296, 3, 64, "requests", "mixed"),
    (700, 272, 272, 2, 8, "none", "full"),
    (300, 272, 528, 5, 24, "wild", "full"),
    # wide features: clusters of 16, and several that share a tile's adapters
    (150, 8208, 528, 5, 24, "mixed", "mixed"),
    (260, 528, 16400, 12, 128, "mixed", "mixed"),
    (300, 16400, 8208, 7, 16, "requests_bare", "full"),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c)))
def test_forward_exact(case):
    c = Case(*case)
    out, v, _, _, _ = c.reference()
    got_v = torch.full((c.s, c.r), 7.0, device="cuda")
    ws = L.AdapterWorkspace(c.s, c.h, c.o, c.n, c.r)
    got = L.llmint8_adapters_forward(c.X, c.ad, c.ids, base=c.base, v=got_v, workspace=ws)
    same(got, out, torch.float16)
    same(got_v, v, torch.float32)
    # without a base, and without v kept
    bare = L.llmint8_adapters_forward(c.X, c.ad, c.ids, workspace=ws)
    same(bare, out - c.base.double(), torch.float16)
    # in place, between rows that are not the call's
    buf = torch.full((c.s + 2, c.o), 5.0, dtype=torch.float16, device="cuda")
    buf[1:-1] = c.base
    L.llmint8_adapters_forward(c.X, c.ad, c.ids, base=buf[1:-1], out=buf[1:-1], workspace=ws)
    same(buf[1:-1], out, torch.float16)
    assert (buf[0] == 5).all() and (buf[-1] == 5).all()
    assert L.llmint8_read_device_status(ws) == 0


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c)))
def test_backward_exact(case):
    c = Case(*case)
    _, v, dX, dA, dB = c.reference()
    ws = L.AdapterWorkspace(c.s, c.h, c.o, c.n, c.r)
    for keep in (v.float(), None):
        got = L.llmint8_adapters_backward(c.X, c.dY, c.ad, c.ids, v=keep, base=c.dbase,
                                          workspace=ws)
        same(got[0], dX, torch.float16)
        same(got[1], dA, torch.float32)
        same(got[2], dB, torch.float32)
    # each output alone; dX in place of the gradient it is added to
    d = c.dbase.clone()
    one = L.llmint8_adapters_backward(None, c.dY, c.ad, c.ids, base=d, dX=d, workspace=ws,
                                      want=(True, False, False))
    assert one[1] is None and one[2] is None
    same(d, dX, torch.float16)
    one = L.llmint8_adapters_backward(c.X, c.dY, c.ad, c.ids, workspace=ws,
                                      want=(False, True, False))
    same(one[1], dA, torch.float32)
    one = L.llmint8_adapters_backward(None, c.dY, c.ad, c.ids, v=v.float(), workspace=ws,
                                      want=(False, False, True))
    same(one[2], dB, torch.float32)
    one = L.llmint8_adapters_backward(None, c.dY, c.ad, c.ids, workspace=ws,
                                      want=(True, False, False))
    same(one[0], dX - c.dbase.double(), torch.float16)
    assert L.llmint8_read_device_status(ws) == 0


# more rows than one pass over the blocks of rows looks through (512 blocks of
# 64), shared by adapters at random places: a CTA's share of a pass may end on
# an odd block
@pytest.mark.parametrize("s,h,o,n,r,layout", [
    (33345, 48, 272, 3, 8, "requests"), (33345, 272, 48, 3, 64, "mixed"),
    (66001, 48, 16, 5, 24, "requests_bare"), (66001, 16, 528, 1, 16, "requests"),
    (100000, 16, 16, 2, 128, "requests")])
def test_factor_gradients_of_many_rows_exact(s, h, o, n, r, layout):
    c = Case(s, h, o, n, r, layout, "full")
    _, v, dX, dA, dB = c.reference()
    g = sum(torch.where((c.ids == a)[:, None], c.dY.double() @ c.B[a].double().T, 0.0)
            for a in range(n))
    # every partial sum is below 2^24 units: exact in fp32, whatever its order
    assert (g.abs().T @ c.X.double().abs()).max() < 2 ** 24
    assert (v.abs().T @ c.dY.double().abs()).max() < 2 ** 24
    ws = L.AdapterWorkspace(s, h, o, n, r)
    for keep in (v.float(), None):
        got = L.llmint8_adapters_backward(c.X, c.dY, c.ad, c.ids, v=keep, base=c.dbase,
                                          workspace=ws)
        same(got[0], dX, torch.float16)
        same(got[1], dA, torch.float32)
        same(got[2], dB, torch.float32)
    assert L.llmint8_read_device_status(ws) == 0


def test_rows_of_unused_slots_and_other_adapters_never_reach_a_result():
    """NaN and infinities in unused rank slots, in adapters without rows, in
    rows without an adapter and in one request's own row stay where they are."""
    for s, layout in ((12, "mixed"), (300, "mixed"), (300, "requests_bare")):
        c = Case(s, 528, 784, 4, 16, layout, "mixed", seed=3)
        out, v, dX, dA, dB = c.reference()
        for a in range(c.n):
            c.A[a, c.rank_list[a]:] = float("nan")
            c.B[a, c.rank_list[a]:] = float("inf")
        for i, a in enumerate(c.ids_list):
            if a < 0:
                c.X[i] = float("nan")
                c.dY[i] = float("inf")
        got_v = torch.empty(c.s, c.r, device="cuda")
        same(L.llmint8_adapters_forward(c.X, c.ad, c.ids, base=c.base, v=got_v), out,
             torch.float16)
        same(got_v, v, torch.float32)
        for keep in (got_v, None):
            got = L.llmint8_adapters_backward(c.X, c.dY, c.ad, c.ids, v=keep, base=c.dbase)
            same(got[0], dX, torch.float16)
            same(got[1], dA, torch.float32)
            same(got[2], dB, torch.float32)
        # one adapter goes bad, and one row of another: everything else holds
        bad = max(set(c.ids_list) - {-1}, key=lambda a: (c.rank_list[a] > 0, a))
        row = next(i for i, a in enumerate(c.ids_list) if a >= 0 and a != bad)
        c.A[bad] = float("nan")
        c.X[row, 3] = float("inf")
        c.dY[row, 5] = float("nan")
        clean = torch.tensor([i for i, a in enumerate(c.ids_list) if a != bad and i != row],
                             device="cuda")
        same(L.llmint8_adapters_forward(c.X, c.ad, c.ids, base=c.base)[clean], out[clean],
             torch.float16)
        got = L.llmint8_adapters_backward(c.X, c.dY, c.ad, c.ids, v=v.float(), base=c.dbase)
        same(got[0][clean], dX[clean], torch.float16)
        for a in set(range(c.n)) - {bad, c.ids_list[row]}:
            same(got[1][a], dA[a], torch.float32)
            same(got[2][a], dB[a], torch.float32)


@pytest.mark.parametrize("s", [12, 300])
def test_gradients_of_adapters_without_rows_are_zeros_whatever_their_scale(s):
    c = Case(s, 528, 784, 4, 16, "mixed", "full")
    c.ids[c.ids == 2] = 1
    c.scale[2] = float("nan")
    got = L.llmint8_adapters_backward(c.X, c.dY, c.ad, c.ids, base=c.dbase)
    c.scale[2] = 1.0
    ref = L.llmint8_adapters_backward(c.X, c.dY, c.ad, c.ids, base=c.dbase)
    for a, b in zip(got, ref):
        assert torch.equal(a, b)
    assert not got[1][2].any() and not got[2][2].any()


def test_rows_without_an_adapter_keep_the_bits_of_their_base():
    for s in (9, 200):
        c = Case(s, 272, 528, 2, 8, "mixed", "full", seed=5)
        free = torch.tensor([i for i, a in enumerate(c.ids_list) if a < 0], device="cuda")
        c.base[free] = torch.randint(-2 ** 15, 2 ** 15, (len(free), c.o),
                                     device="cuda").to(torch.int16).view(torch.float16)
        got = L.llmint8_adapters_forward(c.X, c.ad, c.ids, base=c.base)
        assert torch.equal(bits(got)[free], bits(c.base)[free])


def sum_bound(h):
    return 16 * h ** 0.5 * 2.0 ** -24


REAL = [(5, 2064, 1040, 4, 16, "mixed", "full"), (200, 2064, 1040, 4, 16, "mixed", "mixed"),
        (517, 4096, 2064, 2, 64, "requests", "full")]


@pytest.mark.parametrize("case", REAL, ids=lambda c: "-".join(map(str, c)))
@pytest.mark.parametrize("size", [1.0, 2.0 ** -20, 2.0 ** 10])
def test_real_values_and_their_range(case, size):
    """Normal values; gradients and activations so small or large that v and g
    leave the fp16 range while the results do not."""
    c = Case(*case, real=True)
    c.X, c.dY = (c.X * min(size, 2.0 ** 8)).half(), (c.dY * size).half()
    c.A, c.B = (c.A / min(size, 2.0 ** 8)).half(), (c.B / max(size, 1.0)).half()
    if size < 1:
        c.A = (c.A * size).clamp(-6e4, 6e4).half()
    c.ad = L.Adapters(c.A, c.B, c.scale, c.ranks)
    out, v, dX, dA, dB = c.reference()
    got_v = torch.empty(c.s, c.r, device="cuda")
    got = L.llmint8_adapters_forward(c.X, c.ad, c.ids, base=c.base, v=got_v)
    gX, gA, gB = L.llmint8_adapters_backward(c.X, c.dY, c.ad, c.ids, v=got_v, base=c.dbase)
    d = torch.float64
    for i_rows, a in [(c.rows(a), a) for a in sorted(set(c.ids_list) - {-1})]:
        k, sc = c.rank_list[a], float(c.scale[a])
        A, B = c.A[a, :k].to(d), c.B[a, :k].to(d)
        X, dY = c.X[i_rows].to(d), c.dY[i_rows].to(d)
        nv = X.norm(dim=1)[:, None] * A.norm(dim=1)  # bound of |v|
        ng = dY.norm(dim=1)[:, None] * B.norm(dim=1)
        e = sum_bound(max(c.h, c.o))
        assert ((got_v[i_rows, :k].to(d) - v[i_rows, :k]).abs() <= e * nv).all()
        half = lambda ref: 2.0 ** -11 * ref.abs() + 2.0 ** -25
        lim = half(out[i_rows]) + 2 * e * sc * (nv @ B.abs())
        assert ((got[i_rows].to(d) - out[i_rows]).abs() <= lim).all()
        lim = half(dX[i_rows]) + 2 * e * sc * (ng @ A.abs())
        assert ((gX[i_rows].to(d) - dX[i_rows]).abs() <= lim).all()
        # fp32 results: no rounding but the sums' (over at most 16384 rows)
        lim = 2 * e * sc * (ng.T @ X.abs())
        assert ((gA[a, :k].to(d) - dA[a, :k]).abs() <= lim).all()
        lim = 2 * e * sc * (nv.T @ dY.abs())
        assert ((gB[a, :k].to(d) - dB[a, :k]).abs() <= lim).all()


def test_gradients_against_differences():
    """out is linear in X, A and B one at a time: with integers, the change of
    sum(out * dY) for a step in one of them is the gradient times the step."""
    c = Case(150, 272, 528, 3, 16, "mixed", "mixed", seed=9)
    c.scale.fill_(1.0)

    def loss():
        out = L.llmint8_adapters_forward(c.X, c.ad, c.ids)
        assert out.abs().max() < 2048  # integers below 2^11 are fp16 values
        return float((out.double() * c.dY.double()).sum())

    dX, dA, dB = L.llmint8_adapters_backward(c.X, c.dY, c.ad, c.ids)
    at = loss()
    rng = np.random.default_rng(1)
    row = next(i for i, a in enumerate(c.ids_list) if a >= 0 and c.rank_list[a] > 0)
    a = c.ids_list[row]
    for t, grad, lead in ((c.X, dX, (row,)), (c.A, dA, (a, 0)), (c.B, dB, (a, 0))):
        for _ in range(4):
            where = lead + (int(rng.integers(t.shape[-1])),)
            t[where] += 1
            assert loss() - at == float(grad[where])
            t[where] -= 1


def test_ranks_outside_their_slots_are_clamped():
    for s in (9, 300):
        c = Case(s, 272, 528, 3, 16, "mixed", "mixed", seed=6)
        c.rank_list = [0, 16, 5]
        c.ranks.copy_(torch.tensor([-7, 2 ** 31 - 1, 5]))
        out, _, dX, dA, dB = c.reference()
        same(L.llmint8_adapters_forward(c.X, c.ad, c.ids, base=c.base), out, torch.float16)
        got = L.llmint8_adapters_backward(c.X, c.dY, c.ad, c.ids, base=c.dbase)
        same(got[0], dX, torch.float16)
        same(got[1], dA, torch.float32)
        same(got[2], dB, torch.float32)


def test_no_rows():
    c = Case(4, 272, 528, 2, 8, "mixed", "full")
    X0 = c.X[:0]
    assert L.llmint8_adapters_forward(X0, c.ad, c.ids[:0]).shape == (0, c.o)
    dX, dA, dB = L.llmint8_adapters_backward(X0, c.dY[:0], c.ad, c.ids[:0],
                                             workspace=L.AdapterWorkspace(1, 272, 528, 2, 8))
    assert dX.shape == (0, c.h) and not dA.any() and not dB.any()


def test_offsets_past_32_bits():
    # factors of more than 2^31 elements
    n, r, h, o = 350, 128, 49152, 16
    A = torch.zeros(n, r, h, dtype=torch.float16, device="cuda")
    B = torch.zeros(n, r, o, dtype=torch.float16, device="cuda")
    assert A.numel() > 2 ** 31
    A[n - 1, r - 1, h - 2:] = 1
    B[n - 1, r - 1] = 2
    ad = L.Adapters(A, B, torch.ones(n, device="cuda"))
    for s in (3, 150):
        X = torch.ones(s, h, dtype=torch.float16, device="cuda")
        ids = torch.full((s,), n - 1, dtype=torch.int32, device="cuda")
        out = L.llmint8_adapters_forward(X, ad, ids)
        assert (out == 4).all()
        dX, _, _ = L.llmint8_adapters_backward(None, out, ad, ids, want=(True, False, False))
        assert (dX[:, -2:] == 16 * 4 * 2).all() and not dX[:, :-2].any()
    del A, B, ad
    # outputs and gradients of more than 2^31 elements
    s, h, o = 45000, 16, 49152
    assert s * o > 2 ** 31
    X = torch.zeros(s, h, dtype=torch.float16, device="cuda")
    X[-1] = 1
    A = torch.ones(1, 8, h, dtype=torch.float16, device="cuda")
    B = torch.ones(1, 8, o, dtype=torch.float16, device="cuda")
    ad = L.Adapters(A, B, torch.ones(1, device="cuda"))
    ids = torch.zeros(s, dtype=torch.int32, device="cuda")
    out = L.llmint8_adapters_forward(X, ad, ids)
    assert (out[-1] == 128).all() and not out[:-1].any()
    out.zero_()
    out[-1, -1] = 1
    dX, dA, dB = L.llmint8_adapters_backward(X, out, ad, ids)
    assert (dX[-1] == 8).all() and not dX[:-1].any()
    assert (dA == 1).all()
    assert (dB[0, :, -1] == 16).all() and not dB[0, :, :-1].any()


def test_another_stream_and_a_captured_graph_with_its_chain():
    """Projection, adapters, their backward and the input's gradient captured
    in one graph and replayed on other inputs, next to eager calls."""
    s, h, o, n, r = 150, 528, 784, 3, 16
    c = Case(s, h, o, n, r, "mixed", "mixed", seed=2)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out = L.llmint8_adapters_forward(c.X, c.ad, c.ids, base=c.base, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    same(out, c.reference()[0], torch.float16)
    W = torch.randn(h, o, device="cuda").half()
    pw = L.llmint8_prepare_weight(W)
    mm, ad_ws, bw = L.Workspace(s, h, o), L.AdapterWorkspace(s, h, o, n, r), \
        L.BackwardWorkspace(s, h, o)

    def chain(X, ids):
        y = L.llmint8_matmul(X, pw, 6.0, workspace=mm)
        v = torch.empty(s, r, device="cuda")
        out = L.llmint8_adapters_forward(X, c.ad, ids, base=y, out=y, v=v, workspace=ad_ws)
        dX = L.llmint8_matmul_backward(c.dY, pw, workspace=bw)
        dX, dA, dB = L.llmint8_adapters_backward(X, c.dY, c.ad, ids, v=v, base=dX, dX=dX,
                                                 workspace=ad_ws)
        return out, dX, dA, dB

    X, ids = c.X.clone(), c.ids.clone()
    chain(X, ids)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = chain(X, ids)
    for seed in (4, 5):
        d = Case(s, h, o, n, r, "mixed", "mixed", seed=seed)
        X.copy_(d.X)
        ids.copy_(d.ids)
        graph.replay()
        for got, ref in zip(held, chain(d.X, d.ids)):
            assert torch.equal(got, ref)
    for ws in (mm, ad_ws, bw):
        assert L.llmint8_read_device_status(ws) == 0


# ---------------------------------------------- gradient of the projection's input

BWD = [(1, 16, 16), (5, 528, 272), (16, 1040, 4096), (64, 512, 512), (131, 272, 1040),
       (256, 784, 528), (257, 2064, 272), (600, 528, 2064), (129, 4096, 4096),
       (1100, 4112, 528), (4353, 1296, 272)]


def backward_case(s, h, o, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed + s)
    wq = torch.randint(-127, 128, (o, h), generator=g, device="cuda").to(torch.int8)
    # column scales 127 * 2^-k: the recovered weight is the code times 2^-k
    aw = 127.0 * torch.pow(2.0, -torch.randint(0, 3, (o,), generator=g, device="cuda").float())
    dY = ints(g, (s, o), 2, min(1.0, 400.0 / o))
    base = ints(g, (s, h), 100)
    w = L.PreparedWeight(wq, aw)
    ref = dY.double() @ (wq.double() * (aw.double() / 127)[:, None])
    return w, dY, base, ref


@pytest.mark.parametrize("s,h,o", BWD)
def test_input_gradient_exact(s, h, o):
    w, dY, base, ref = backward_case(s, h, o)
    ws = L.BackwardWorkspace(s, h, o)
    same(L.llmint8_matmul_backward(dY, w, workspace=ws), ref, torch.float16)
    same(L.llmint8_matmul_backward(dY, w, base=base, workspace=ws), ref + base.double(),
         torch.float16)
    buf = torch.full((s + 2, h), 5.0, dtype=torch.float16, device="cuda")
    buf[1:-1] = base
    L.llmint8_matmul_backward(dY, w, base=buf[1:-1], out=buf[1:-1], workspace=ws)
    same(buf[1:-1], ref + base.double(), torch.float16)
    assert (buf[0] == 5).all() and (buf[-1] == 5).all()
    assert L.llmint8_read_device_status(ws) == 0


@pytest.mark.parametrize("s,h,o", [(9, 1040, 2064), (300, 1040, 2064), (513, 528, 12288)])
def test_input_gradient_of_a_prepared_weight(s, h, o):
    """Normal weights: against the recovered fp16 weight, with the fp32 sums'
    bound over o products."""
    g = torch.Generator(device="cuda").manual_seed(o)
    W = (torch.randn(h, o, generator=g, device="cuda") * 0.02).half()
    pw = L.llmint8_prepare_weight(W)
    dY = (torch.randn(s, o, generator=g, device="cuda") * 0.1).half()
    dY[0, 3] = float("inf")  # reaches its own row only
    WR = (pw.wq.float() * pw.aw[:, None] / 127).half().double()
    got = L.llmint8_matmul_backward(dY, pw)
    assert not got[0].isfinite().all()
    ref = dY[1:].double() @ WR
    lim = 2.0 ** -11 * ref.abs() + 2.0 ** -25 \
        + sum_bound(o) * dY[1:].double().norm(dim=1)[:, None] * WR.norm(dim=0)
    assert ((got[1:].double() - ref).abs() <= lim).all()
    assert torch.equal(got, L.llmint8_matmul_backward(dY, pw)) or got[0].isnan().any()
    assert torch.equal(got[1:], L.llmint8_matmul_backward(dY, pw)[1:])


def test_input_gradient_recovers_weights_of_any_size():
    """One-hot gradients read the recovered weights themselves: within half an
    fp16 step of code * aw / 127 (and 2^-6 of one for the factor), and, where
    that is subnormal, two roundings of half of 2^-24; column scales from the
    largest binary16 number to the smallest, and zero."""
    h, scales = 272, [65504.0, 127.0, 1.0, 0.08, 6e-5, 1e-6, 2.0 ** -23, 2.0 ** -24, 0.0]
    o = 16 * ((len(scales) + 15) // 16)
    aw = torch.tensor(scales + [1.0] * (o - len(scales)), device="cuda").half().float()
    g = torch.Generator(device="cuda").manual_seed(8)
    wq = torch.randint(-127, 128, (o, h), generator=g, device="cuda").to(torch.int8)
    wq[:, :255] = torch.arange(-127, 128, device="cuda").to(torch.int8)
    got = L.llmint8_matmul_backward(torch.eye(o, dtype=torch.float16, device="cuda"),
                                    L.PreparedWeight(wq, aw)).double()
    ref = wq.double() * aw.double()[:, None] / 127
    lim = 2.0 ** -11 * (1 + 2.0 ** -6) * ref.abs() + 2.0 ** -24
    assert ((got - ref).abs() <= lim).all()
    # the two smallest scales are one or two steps of 2^-24 at their largest codes
    assert torch.equal(got[6, [0, 254]], torch.tensor([-1.0, 1.0], device="cuda").double()
                       * 2.0 ** -23)
    assert torch.equal(got[7, [0, 254]], torch.tensor([-1.0, 1.0], device="cuda").double()
                       * 2.0 ** -24)
    assert not got[8].any()


def test_input_gradient_no_rows():
    w, dY, _, _ = backward_case(4, 272, 528)
    assert L.llmint8_matmul_backward(dY[:0], w).shape == (0, 272)


# More units of work than CTA pairs (74): pairs that take a second and a third
# unit, on one accumulator after the other (up to 256 rows) or on both at once,
# with odd numbers of stages between them; whole tiles alone, with others
# behind them, and with others cut along the reduction; parts on every pair
MANY_UNITS = [(131, 19216, 272), (200, 18944, 336), (150, 42000, 272), (200, 10256, 4112),
              (4353, 2576, 1296), (4353, 4112, 272), (513, 14208, 208), (1537, 12304, 144),
              (1025, 37888, 80)]


@pytest.mark.parametrize("s,h,o", MANY_UNITS)
def test_input_gradient_of_many_units_exact(s, h, o):
    test_input_gradient_exact(s, h, o)


@pytest.mark.parametrize("s,h,o", [(131, 19216, 272), (4353, 2576, 1296)])
def test_input_gradient_of_many_units_repeats_itself(s, h, o):
    """The same bits from every one of many calls, with normal values, on one
    workspace, and next to another stream's calls."""
    g = torch.Generator(device="cuda").manual_seed(h)
    W = (torch.randn(h, o, generator=g, device="cuda") * 0.02).half()
    pw = L.llmint8_prepare_weight(W)
    dY = (torch.randn(s, o, generator=g, device="cuda") * 0.1).half()
    base = torch.randn(s, h, generator=g, device="cuda").half()
    ws, other_ws = L.BackwardWorkspace(s, h, o), L.BackwardWorkspace(s, h, o)
    first = L.llmint8_matmul_backward(dY, pw, base=base, workspace=ws)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(50):
        other = L.llmint8_matmul_backward(dY, pw, base=base, workspace=other_ws, stream=side)
        assert torch.equal(bits(L.llmint8_matmul_backward(dY, pw, base=base, workspace=ws)),
                           bits(first))
        torch.cuda.current_stream().wait_stream(side)
        assert torch.equal(bits(other), bits(first))
        side.wait_stream(torch.cuda.current_stream())
    for w in (ws, other_ws):
        assert L.llmint8_read_device_status(w) == 0


def test_input_gradient_of_a_row_with_an_infinity_repeats_itself():
    """That row's values repeat themselves too, its NaN in the same places."""
    s, h, o = 300, 1040, 2064
    g = torch.Generator(device="cuda").manual_seed(4)
    pw = L.llmint8_prepare_weight((torch.randn(h, o, generator=g, device="cuda") * 0.02).half())
    dY = (torch.randn(s, o, generator=g, device="cuda") * 0.1).half()
    dY[0, 3] = float("inf")
    got, again = (L.llmint8_matmul_backward(dY, pw) for _ in range(2))
    assert torch.equal(got.isnan(), again.isnan())
    assert torch.equal(got.nan_to_num(0.5), again.nan_to_num(0.5))
    # inf times the recovered weight: its sign, or NaN where the code is zero
    codes = pw.wq[3].int()
    assert (got[0].isnan() == (codes == 0)).all()
    assert torch.equal(got[0][codes != 0], codes[codes != 0].sign() * torch.tensor(
        float("inf"), dtype=torch.float16, device="cuda"))


@pytest.mark.parametrize("s,h,o", [(77, 1040, 49152), (520, 528, 49152)])
@pytest.mark.parametrize("sign", ["mixed", "positive"])
def test_input_gradient_of_a_long_reduction(s, h, o, sign):
    """49152 products per sum. On the tensor cores a sum is rounded toward zero
    once per 16 of them, each time by at most 2^-23 of a partial sum, and where
    it is cut into parts (at most 16) once more for each: together below
    (o / 16 + 16) 2^-23 of the largest partial sum, which is the result itself
    where every term is positive and at most |dY| |WR| else."""
    g = torch.Generator(device="cuda").manual_seed(s)
    wq = torch.randint(-127, 128, (o, h), generator=g, device="cuda").to(torch.int8)
    aw = (0.08 + 0.01 * torch.rand(o, generator=g, device="cuda")).half().float()
    dY = (torch.randn(s, o, generator=g, device="cuda") * 0.01).half()
    if sign == "positive":
        wq, dY = wq.abs(), dY.abs()
    got = L.llmint8_matmul_backward(dY, L.PreparedWeight(wq, aw)).double()
    WR = (wq.float() * (aw[:, None] / 127)).half().double()
    ref = dY.double() @ WR
    lim = 2.0 ** -11 * ref.abs() + 2.0 ** -25
    if sign == "positive":
        lim += (o / 16 + 16) * 2.0 ** -23 * ref
    else:
        lim += (o / 16 + 16) * 2.0 ** -23 * dY.double().norm(dim=1)[:, None] * WR.norm(dim=0)
    assert ((got - ref).abs() <= lim).all()


# as many adapters as a call takes, more than most rows can name
@pytest.mark.parametrize("s", [100, 300])
def test_most_adapters(s):
    case = (s, 32, 48, 65535, 8, "mixed", "mixed")
    test_forward_exact(case)
    test_backward_exact(case)


@pytest.mark.parametrize("s", [12, 300])
def test_infinities_reach_their_own_results_only(s):
    """An infinity of X, dY or a factor: what it enters is infinite or NaN,
    everything else keeps its bits."""
    c = Case(s, 528, 784, 3, 16, "mixed", "full", seed=7)
    ref = L.llmint8_adapters_backward(c.X, c.dY, c.ad, c.ids, base=c.dbase)
    row = next(i for i, a in enumerate(c.ids_list) if a == 1)
    c.dY[row, 5] = float("inf")
    dX, dA, dB = L.llmint8_adapters_backward(c.X, c.dY, c.ad, c.ids, base=c.dbase)
    v = c.X[row].double() @ c.A[1].double().T
    others = torch.arange(s, device="cuda") != row
    assert torch.equal(dX[others], ref[0][others]) and not dX[row].isfinite().any()
    for got, want in ((dA, ref[1]), (dB, ref[2])):
        assert torch.equal(got[[0, 2]], want[[0, 2]])
    keep = torch.arange(c.o, device="cuda") != 5
    assert torch.equal(dB[1][:, keep], ref[2][1][:, keep])
    assert not dB[1][v != 0, 5].isfinite().any()
    c.dY[row, 5] = 0
    c.B[1, 2, 9] = float("-inf")
    out = L.llmint8_adapters_forward(c.X, c.ad, c.ids, base=c.base)
    got_v = c.X.double() @ c.A[1].double().T
    hit = (c.ids == 1) & (got_v[:, 2] != 0)
    assert not out[hit, 9].isfinite().any()
    c.B[1, 2, 9] = 0
    want = L.llmint8_adapters_forward(c.X, c.ad, c.ids, base=c.base)
    mine = (c.ids == 1)[:, None] & (torch.arange(c.o, device="cuda") == 9)
    assert torch.equal(out[~mine], want[~mine])
