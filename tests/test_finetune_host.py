"""Host-side checks of the operators next to the projection that need no GPU:
workspace sizes and the refusal of invalid arguments before anything is
enqueued. Placeholder pointers are never dereferenced; the calls are skipped
when a GPU is visible."""
import ctypes
import math

import pytest
import torch

from mixed_precision_int8_b200 import binding, build

FAKE = ctypes.c_void_p(1 << 20)  # 256-byte aligned, never dereferenced
ODD = ctypes.c_void_p((1 << 20) + 2)
BIG = 1 << 40

needs_no_gpu = pytest.mark.skipif(torch.cuda.is_available(),
                                  reason="placeholder pointers: CPU box only")


@pytest.fixture(scope="module")
def lib():
    build.build()
    return binding.load_library()


def test_workspace_sizes(lib):
    assert lib.llmint8_adapters_workspace_size(0, 256, 256, 1, 8) > 0
    assert (lib.llmint8_adapters_workspace_size(4096, 256, 256, 1, 64)
            > lib.llmint8_adapters_workspace_size(16, 256, 256, 1, 64))
    for bad in ((-1, 256, 256, 1, 8), (2 ** 31 - 1023, 256, 256, 1, 8), (4, 250, 256, 1, 8),
                (4, 256, 8, 1, 8), (4, 256, 256, 0, 8), (4, 256, 256, 65536, 8),
                (4, 256, 256, 1, 0), (4, 256, 256, 1, 12), (4, 256, 256, 1, 136)):
        assert lib.llmint8_adapters_workspace_size(*bad) == 0
    assert lib.llmint8_matmul_backward_workspace_size(128, 256, 256) > 0
    assert lib.llmint8_matmul_backward_workspace_size(-1, 256, 256) == 0
    assert lib.llmint8_matmul_backward_workspace_size(1, 256, 250) == 0
    assert lib.llmint8_layernorm_workspace_size(128, 256) > 0
    assert lib.llmint8_layernorm_workspace_size(128, 133160) == 0
    assert lib.llmint8_grad_list_size(0) > 0
    assert lib.llmint8_grad_list_size(-1) == 0
    assert lib.llmint8_grad_list_size(2 ** 24 + 1) == 0


def _adapters(h=256, o=256, n=2, r=8, a=FAKE, b=FAKE, scale=FAKE, rank=None):
    return binding.llmint8_adapters(h, o, n, r, a, b, scale, rank)


@needs_no_gpu
def test_adapters_forward_refusals(lib):
    def call(ad=None, s=4, X=FAKE, ids=FAKE, base=FAKE, out=ctypes.c_void_p(1 << 24), v=None,
             ws=FAKE, nb=BIG):
        ad = ad if ad is not None else _adapters()
        return lib.llmint8_adapters_forward(X, s, ctypes.byref(ad), ids, base, out, v, ws, nb,
                                            None)
    assert lib.llmint8_adapters_forward(FAKE, 4, None, FAKE, None, FAKE, None, FAKE, BIG,
                                        None) == -1
    for kw in ("a", "b", "scale"):
        assert call(_adapters(**{kw: None})) == -1
    for kw in (dict(h=250), dict(o=8), dict(n=0), dict(n=65536), dict(r=4), dict(r=12),
               dict(r=136)):
        assert call(_adapters(**kw)) == -2
    for kw in (dict(a=ODD), dict(b=ODD), dict(scale=ODD), dict(rank=ODD)):
        assert call(_adapters(**kw)) == -3
    assert call(s=-1) == -2 and call(s=2 ** 31 - 1023) == -2
    for kw in ("X", "ids", "out", "ws"):
        assert call(**{kw: None}) == -1
    for kw in ("X", "ids", "base", "out", "v", "ws"):
        assert call(**{kw: ODD}) == -3
    need = lib.llmint8_adapters_workspace_size(4, 256, 256, 2, 8)
    assert call(nb=need - 1) == -4
    # an output that overlaps its base without being it
    assert call(base=ctypes.c_void_p((1 << 24) + 512)) == -7
    assert call(X=ctypes.c_void_p(1 << 24)) == -7
    assert call(s=0, X=None, ids=None, out=None, ws=None) == 0


@needs_no_gpu
def test_adapters_backward_refusals(lib):
    far = [ctypes.c_void_p((k + 16) << 24) for k in range(3)]

    def call(ad=None, s=4, X=FAKE, dY=FAKE, ids=FAKE, v=FAKE, base=FAKE, dX=far[0], dA=far[1],
             dB=far[2], ws=FAKE, nb=BIG):
        ad = ad if ad is not None else _adapters()
        return lib.llmint8_adapters_backward(X, dY, s, ctypes.byref(ad), ids, v, base, dX, dA,
                                             dB, ws, nb, None)
    assert call(_adapters(r=12)) == -2
    for kw in ("dY", "ids", "ws"):
        assert call(**{kw: None}) == -1
    assert call(X=None) == -1  # needed for dA
    assert call(X=None, dA=None, v=None) == -1  # and for v
    for kw in ("X", "dY", "ids", "v", "base", "dX", "dA", "dB", "ws"):
        assert call(**{kw: ODD}) == -3
    assert call(nb=lib.llmint8_adapters_workspace_size(4, 256, 256, 2, 8) - 1) == -4
    assert call(dX=FAKE, base=None) == -7  # the gradient's own rows
    assert call(base=ctypes.c_void_p((16 << 24) + 256)) == -7
    assert call(s=-1) == -2


@needs_no_gpu
def test_matmul_backward_refusals(lib):
    def call(w=None, s=4, dY=FAKE, base=None, dX=ctypes.c_void_p(1 << 24), ws=FAKE, nb=BIG):
        w = w if w is not None else binding.llmint8_weight(256, 256, FAKE, FAKE)
        return lib.llmint8_matmul_backward(dY, s, ctypes.byref(w), base, dX, ws, nb, None)
    assert lib.llmint8_matmul_backward(FAKE, 4, None, None, FAKE, FAKE, BIG, None) == -1
    assert call(binding.llmint8_weight(256, 256, None, FAKE)) == -1
    assert call(binding.llmint8_weight(250, 256, FAKE, FAKE)) == -2
    assert call(binding.llmint8_weight(256, 256, ODD, FAKE)) == -3
    for kw in ("dY", "dX", "ws"):
        assert call(**{kw: None}) == -1
    for kw in ("dY", "base", "dX", "ws"):
        assert call(**{kw: ODD}) == -3
    assert call(nb=lib.llmint8_matmul_backward_workspace_size(4, 256, 256) - 1) == -4
    assert call(dX=FAKE) == -7  # overlaps dY
    assert call(base=ctypes.c_void_p((1 << 24) + 256)) == -7
    assert call(s=-1) == -2
    assert call(s=0, dY=None, dX=None, ws=None) == 0


@needs_no_gpu
def test_layernorm_refusals(lib):
    def fwd(x=FAKE, xt=0, s=4, h=256, g=FAKE, b=FAKE, pt=0, eps=1e-5, y=FAKE, mean=FAKE,
            rstd=FAKE):
        return lib.llmint8_layernorm_forward(x, xt, s, h, g, b, pt, eps, y, mean, rstd, None)
    assert fwd(h=250) == -2 and fwd(h=133160) == -2 and fwd(s=-1) == -2
    assert fwd(xt=2) == -7 and fwd(pt=2) == -7 and fwd(xt=-1) == -7
    for bad in (-1.0, math.nan, math.inf):
        assert fwd(eps=bad) == -7
    for kw in ("x", "g", "y"):
        assert fwd(**{kw: None}) == -1
    for kw in ("x", "g", "b", "y", "mean", "rstd"):
        assert fwd(**{kw: ODD}) == -3
    assert fwd(s=0, x=None, g=None, y=None) == 0

    def bwd(dy=FAKE, x=FAKE, xt=0, s=4, h=256, g=FAKE, pt=0, mean=FAKE, rstd=FAKE, dx=FAKE,
            dg=FAKE, db=FAKE, ws=FAKE, nb=BIG):
        return lib.llmint8_layernorm_backward(dy, x, xt, s, h, g, pt, mean, rstd, dx, dg, db,
                                              ws, nb, None)
    assert bwd(h=250) == -2 and bwd(xt=2) == -7 and bwd(pt=3) == -7
    for kw in ("dy", "x", "g", "mean", "rstd", "ws"):
        assert bwd(**{kw: None}) == -1
    for kw in ("dy", "x", "g", "mean", "rstd", "dx", "dg", "db", "ws"):
        assert bwd(**{kw: ODD}) == -3
    assert bwd(nb=lib.llmint8_layernorm_workspace_size(4, 256) - 1) == -4


@needs_no_gpu
def test_clip_refusals(lib):
    lst = binding.llmint8_grad_list(FAKE, BIG, 1, 1)
    init = lib.llmint8_grad_list_init
    item = binding.llmint8_grad(FAKE, FAKE, 10, 1)

    def one(**kw):
        g = binding.llmint8_grad(kw.get("grad", FAKE), kw.get("out", FAKE), kw.get("n", 10),
                                 kw.get("type", 1))
        return init(ctypes.byref(g), 1, ctypes.byref(lst), None)
    assert init(None, 1, ctypes.byref(lst), None) == -1
    assert init(ctypes.byref(item), 1, None, None) == -1
    assert init(ctypes.byref(item), -1, ctypes.byref(lst), None) == -2
    assert one(type=3) == -7 and one(n=-1) == -2 and one(grad=None) == -1
    assert one(grad=ODD) == -3 and one(out=ODD) == -3
    assert one(out=ctypes.c_void_p((1 << 20) + 4)) == -7  # a shifted overlap
    far = ctypes.c_void_p(1 << 24)

    def two(a, b):
        pair = (binding.llmint8_grad * 2)(a, b)
        return init(pair, 2, ctypes.byref(lst), None)
    G = binding.llmint8_grad
    assert two(G(FAKE, None, 10, 1), G(FAKE, None, 10, 1)) == -7  # one tensor twice
    assert two(G(FAKE, far, 10, 1), G(far, None, 10, 1)) == -7  # an output that is read
    assert two(G(FAKE, far, 10, 1), G(FAKE, ctypes.c_void_p((1 << 24) + 36), 10, 1)) == -7
    # read twice into outputs of their own: allowed (and then no usable device)
    assert two(G(FAKE, far, 10, 1), G(FAKE, ctypes.c_void_p((1 << 24) + 40), 10, 1)) in (-5, -8)
    small = binding.llmint8_grad_list(FAKE, lib.llmint8_grad_list_size(1) - 1, 0, 0)
    assert init(ctypes.byref(item), 1, ctypes.byref(small), None) == -4
    off = binding.llmint8_grad_list(ODD, BIG, 0, 0)
    assert init(ctypes.byref(item), 1, ctypes.byref(off), None) == -3
    clip = lib.llmint8_clip_grads
    assert clip(None, 1.0, FAKE, None) == -1
    assert clip(ctypes.byref(lst), 1.0, None, None) == -1
    for bad in (-1.0, math.nan):
        assert clip(ctypes.byref(lst), bad, FAKE, None) == -7
    assert clip(ctypes.byref(lst), 1.0, ctypes.c_void_p((1 << 20) + 1), None) == -3
    assert clip(ctypes.byref(small), 1.0, FAKE, None) != 0


def test_binding_refuses_tensors_it_cannot_take():
    A = torch.zeros(2, 8, 32, dtype=torch.float16)
    with pytest.raises(ValueError):
        binding.Adapters(A, A, torch.ones(2))  # not on a GPU
    with pytest.raises(ValueError):
        binding.Adapters(A[0], A, torch.ones(2))
    with pytest.raises(ValueError):
        binding.llmint8_layernorm_forward(torch.zeros(4, 32), torch.ones(32))
    with pytest.raises(ValueError):
        binding.llmint8_layernorm_forward(torch.zeros(32), torch.ones(32))
    with pytest.raises(ValueError, match="on a CUDA device"):
        binding.GradList([torch.zeros(8)])


def _overlapping(base_args, spans, allowed, call):
    """Every output moved onto the last byte's place of every other tensor (or
    onto its first) is refused; `allowed` pairs may be the same tensor."""
    outs = [k for k, (_, written) in spans.items() if written]
    for out in outs:
        for other, (size, _) in spans.items():
            if other == out:
                continue
            for shift in (0, size - 16 if size > 16 else 0):
                if shift == 0 and (out, other) in allowed:
                    continue
                at = base_args[other].value + shift
                args = dict(base_args, **{out: ctypes.c_void_p(at // 16 * 16)})
                assert call(**args) == -7, (out, other, shift)


def _places(names):
    return {k: ctypes.c_void_p((i + 4) << 26) for i, k in enumerate(names)}


@needs_no_gpu
def test_outputs_that_overlap_are_refused(lib):
    s, h, o, n, r = 40, 256, 528, 2, 8
    size = dict(X=2 * s * h, dY=2 * s * o, ids=4 * s, base=2 * s * o, out=2 * s * o, v=4 * s * r,
                a=2 * n * r * h, b=2 * n * r * o, scale=4 * n, rank=4 * n, dX=2 * s * h,
                dA=4 * n * r * h, dB=4 * n * r * o)

    def ad(a, b, scale, rank):
        return ctypes.byref(binding.llmint8_adapters(h, o, n, r, a, b, scale, rank))

    def forward(X, ids, base, out, v, a, b, scale, rank):
        return lib.llmint8_adapters_forward(X, s, ad(a, b, scale, rank), ids, base, out, v, FAKE,
                                            BIG, None)
    names = ("X", "ids", "base", "out", "v", "a", "b", "scale", "rank")
    spans = {k: (size[k], k in ("out", "v")) for k in names}
    assert forward(**_places(names)) in (-5, -8)  # sound, but for the GPU
    _overlapping(_places(names), spans, {("out", "base")}, forward)

    def backward(X, dY, ids, v, base, dX, dA, dB, a, b, scale, rank):
        return lib.llmint8_adapters_backward(X, dY, s, ad(a, b, scale, rank), ids, v, base, dX,
                                             dA, dB, FAKE, BIG, None)
    names = ("X", "dY", "ids", "v", "base", "dX", "dA", "dB", "a", "b", "scale", "rank")
    size["base"] = 2 * s * h
    spans = {k: (size[k], k in ("dX", "dA", "dB")) for k in names}
    assert backward(**_places(names)) in (-5, -8)
    _overlapping(_places(names), spans, {("dX", "base")}, backward)

    def matmul(dY, wq, aw, base, dX):
        w = binding.llmint8_weight(h, o, wq, aw)
        return lib.llmint8_matmul_backward(dY, s, ctypes.byref(w), base, dX, FAKE, BIG, None)
    names = ("dY", "wq", "aw", "base", "dX")
    size.update(wq=h * o, aw=4 * o)
    spans = {k: (size[k], k == "dX") for k in names}
    assert matmul(**_places(names)) in (-5, -8)
    _overlapping(_places(names), spans, {("dX", "base")}, matmul)


@needs_no_gpu
@pytest.mark.parametrize("xt", [0, 1])
def test_layernorm_outputs_that_overlap_are_refused(lib, xt):
    s, h = 40, 256
    xb = 4 if xt else 2

    def fwd(x, g, b, y, mean, rstd):
        return lib.llmint8_layernorm_forward(x, xt, s, h, g, b, 1, 1e-5, y, mean, rstd, None)
    spans = dict(x=(xb * s * h, False), g=(4 * h, False), b=(4 * h, False),
                 y=(2 * s * h, True), mean=(4 * s, True), rstd=(4 * s, True))
    assert fwd(**_places(spans)) in (-5, -8)
    _overlapping(_places(spans), spans, set() if xt else {("y", "x")}, fwd)
    if not xt:  # in place
        at = _places(spans)
        assert fwd(**dict(at, y=at["x"])) in (-5, -8)

    def bwd(dy, x, g, mean, rstd, dx, dg, db):
        return lib.llmint8_layernorm_backward(dy, x, xt, s, h, g, 1, mean, rstd, dx, dg, db, FAKE,
                                              BIG, None)
    spans = dict(dy=(2 * s * h, False), x=(xb * s * h, False), g=(4 * h, False),
                 mean=(4 * s, False), rstd=(4 * s, False), dx=(xb * s * h, True),
                 dg=(4 * h, True), db=(4 * h, True))
    allowed = {("dx", "x")} | (set() if xt else {("dx", "dy")})
    assert bwd(**_places(spans)) in (-5, -8)
    _overlapping(_places(spans), spans, allowed, bwd)
    at = _places(spans)
    for out, other in allowed:
        assert bwd(**dict(at, **{out: at[other]})) in (-5, -8)


@needs_no_gpu
def test_tensors_inside_the_workspace_are_refused(lib):
    """Its first byte, its last and one in between; a tensor right behind it is
    none of its bytes."""
    s, h, o, n, r = 40, 256, 528, 2, 8
    ws = ctypes.c_void_p(1 << 34)

    def check(names, nbytes, call):
        at = _places(names)
        assert call(**at) in (-5, -8)  # sound, but for the GPU
        for name in names:
            for offset in (0, nbytes // 2 // 256 * 256, nbytes - 256):
                assert call(**dict(at, **{name: ctypes.c_void_p(ws.value + offset)})) == -7, \
                    (name, offset)
            assert call(**dict(at, **{name: ctypes.c_void_p(ws.value + nbytes)})) in (-5, -8)

    def forward(X, ids, base, out, v, a, b, scale, rank):
        ad = binding.llmint8_adapters(h, o, n, r, a, b, scale, rank)
        return lib.llmint8_adapters_forward(X, s, ctypes.byref(ad), ids, base, out, v, ws, BIG,
                                            None)
    size = lib.llmint8_adapters_workspace_size(s, h, o, n, r)
    check(("X", "ids", "base", "out", "v", "a", "b", "scale", "rank"), size, forward)

    def backward(X, dY, ids, v, base, dX, dA, dB, a, b, scale, rank):
        ad = binding.llmint8_adapters(h, o, n, r, a, b, scale, rank)
        return lib.llmint8_adapters_backward(X, dY, s, ctypes.byref(ad), ids, v, base, dX, dA,
                                             dB, ws, BIG, None)
    check(("X", "dY", "ids", "v", "base", "dX", "dA", "dB", "a", "b", "scale", "rank"), size,
          backward)

    def matmul(dY, wq, aw, base, dX):
        w = binding.llmint8_weight(h, o, wq, aw)
        return lib.llmint8_matmul_backward(dY, s, ctypes.byref(w), base, dX, ws, BIG, None)
    check(("dY", "wq", "aw", "base", "dX"), lib.llmint8_matmul_backward_workspace_size(s, h, o),
          matmul)

    def layernorm(dy, x, g, mean, rstd, dx, dg, db):
        return lib.llmint8_layernorm_backward(dy, x, 0, s, h, g, 1, mean, rstd, dx, dg, db, ws,
                                              BIG, None)
    check(("dy", "x", "g", "mean", "rstd", "dx", "dg", "db"),
          lib.llmint8_layernorm_workspace_size(s, h), layernorm)


@needs_no_gpu
def test_clip_refuses_outputs_and_norms_inside_its_table(lib):
    G, table = binding.llmint8_grad, 1 << 34
    size = lib.llmint8_grad_list_size(3)
    lst = binding.llmint8_grad_list(ctypes.c_void_p(table), BIG, 3, 3)

    def init(out):
        grads = (G * 3)(G(FAKE, None, 10, 1), G(ctypes.c_void_p(1 << 24), out, 64, 1),
                        G(None, None, 0, 1))
        return lib.llmint8_grad_list_init(grads, 3, ctypes.byref(lst), None)

    def clip(norm):
        return lib.llmint8_clip_grads(ctypes.byref(lst), 1.0, norm, None)
    for offset in (0, size // 2 // 256 * 256, size - 4):
        assert init(ctypes.c_void_p(table + offset)) == -7
        assert clip(ctypes.c_void_p(table + offset)) == -7
    assert init(ctypes.c_void_p(table - 4)) == -7
    assert init(ctypes.c_void_p(table + size)) in (-5, -8)  # sound, but for the GPU
    assert init(ctypes.c_void_p(table - 256)) in (-5, -8)
    assert clip(ctypes.c_void_p(table + size)) in (-5, -8)
    assert clip(ctypes.c_void_p(table - 4)) in (-5, -8)


def test_address_ranges_of_tensors():
    """The ranges that a clip list's norm is looked up in: merged, in order,
    empty tensors none of them."""
    buf = torch.zeros(64)
    at = buf.data_ptr()
    parts = [buf[32:40], buf[0:4], buf[2:8], buf[8:8], buf[34:36], buf[8:12],
             buf[50:52].to(torch.float16)]
    spans = binding._address_ranges(parts)
    other = parts[-1].data_ptr()
    assert sorted(spans) == spans
    assert [s for s in spans if at <= s[0] < at + 256] == [(at, at + 48), (at + 128, at + 160)]
    assert (other, other + 4) in spans and len(spans) == 3
    for i in range(64):
        inside = i < 12 or 32 <= i < 40
        assert binding._overlaps(spans, buf[i:i + 1]) == inside
        assert binding._overlaps(spans, buf[i:i]) is False
    assert binding._overlaps(spans, buf[12:33]) and not binding._overlaps(spans, buf[12:32])
    assert binding._overlaps(spans, buf)
    assert binding._address_ranges([]) == [] and not binding._overlaps([], buf)


def test_documents_say_how_a_wait_that_ran_out_is_seen():
    """Only a caller's workspace can be asked for its status: the calls that
    can do without one say so."""
    calls = ("llmint8_adapters_forward", "llmint8_adapters_backward", "llmint8_matmul_backward",
             "llmint8_layernorm_backward")
    for name in calls:
        doc = getattr(binding, name).__doc__
        assert "llmint8_read_device_status" in doc and "workspace" in doc, name
