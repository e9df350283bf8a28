"""Cases that measure the fine-tuning and adapter-serving operators: low-rank
adapters beside the int8 projection (forward, backward), the gradient of the
projection's input, layer norm (forward, backward) and gradient clipping.

Every operator is stated twice here besides the library's own calls: `run`
with `own = False` is its plain form (elementary torch operations in 32 bits),
`exact` its definition in 64 bits.
"""
import math

import torch

own = False

# How many low-rank ranks adapter a uses of its r slots: adapters of one server
# are trained at different ranks, odd ones among them.
def _rank(case, a):
    r = case["r"]
    if case["ranks"] == "full":
        return r
    return max(1, r - (a % 3) * (r // 4) - (a % 2))


def _bare_rows(case):
    """Rows of the batch that no adapter serves."""
    if not case["bare"]:
        return 0
    return 1 if case["layout"] == "tokens" else max(1, case["s"] // 8)


def listed():
    return [
        # A decode step of the OPT-175B FFN up-projection: eight requests, seven with an
        # adapter each, one without.
        dict(name="adapters_fwd_decode", op="adapters_fwd", s=8, h=12288, o=49152, n=16, r=16,
             ranks="mixed", layout="tokens", bare=True),
        # Four prompts of different lengths (one without an adapter) through the OPT-13B FFN
        # up-projection in one prefill batch.
        dict(name="adapters_fwd_prefill", op="adapters_fwd", s=4096, h=5120, o=20480, n=3, r=16,
             ranks="full", layout="requests", bare=True),
        # A small fine-tuning batch of odd length on the OPT-6.7B attention projection, two
        # adapters of odd ranks trained side by side.
        dict(name="adapters_bwd_small", op="adapters_bwd", s=517, h=4096, o=4096, n=2, r=8,
             ranks="mixed", layout="requests", bare=False),
        # Fine-tuning at rank 64 on the OPT-13B FFN up-projection.
        dict(name="adapters_bwd_ffn", op="adapters_bwd", s=4096, h=5120, o=20480, n=1, r=64,
             ranks="full", layout="requests", bare=False),
        # The gradient that goes on through the frozen int8 projection: a short odd batch on
        # the OPT-6.7B attention projection, where few tiles of rows exist ...
        dict(name="matmul_bwd_short", op="matmul_bwd", s=131, h=4096, o=4096),
        # ... and a full one on the OPT-13B FFN up-projection.
        dict(name="matmul_bwd_ffn", op="matmul_bwd", s=4096, h=5120, o=20480),
        # The norm before the projection: a decode step at OPT-175B width, a prefill at 13B.
        dict(name="layernorm_fwd_decode", op="layernorm_fwd", s=8, h=12288, x="f16", p="f16"),
        dict(name="layernorm_fwd_prefill", op="layernorm_fwd", s=4093, h=5120, x="f32", p="f16"),
        # Its backward pass on an fp16 stream and at OPT-175B width on an fp32 stream.
        dict(name="layernorm_bwd_f16", op="layernorm_bwd", s=2047, h=4096, x="f16", p="f16"),
        dict(name="layernorm_bwd_f32", op="layernorm_bwd", s=2048, h=12288, x="f32", p="f32"),
        # Gradients of the adapters of every layer of an OPT-6.7B-like model: many small
        # fp32 tensors, some of odd length.
        dict(name="clip_adapters", op="clip", tensors=256, width=4096, r=16, g="f32"),
        # A few large fp16 gradients, as of one whole OPT-13B-like layer.
        dict(name="clip_layer", op="clip", tensors=16, width=5120, r=2560, g="f16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _width(rng, lo, hi):
    """A feature width: any multiple of 16, the projection's own rule."""
    return max(16, _log(rng, lo, hi) // 16 * 16)


def draw(rng):
    op = rng.choice(["adapters_fwd", "adapters_bwd", "matmul_bwd", "layernorm_fwd",
                     "layernorm_bwd", "clip"])
    if op in ("adapters_fwd", "adapters_bwd"):
        # from a decode step to the prefill of a few prompts
        s = _log(rng, 1, 4096)
        h, o = _width(rng, 512, 12288), _width(rng, 512, 20480)
        return dict(op=op, s=s, h=h, o=o, n=rng.choice([1, 2, 3, 5, 8, 16]),
                    r=rng.choice([8, 16, 24, 32, 64]), ranks=rng.choice(["full", "mixed"]),
                    layout="tokens" if s <= 64 and rng.random() < 0.7 else "requests",
                    bare=rng.random() < 0.5 and s >= 2)
    if op == "matmul_bwd":
        return dict(op=op, s=_log(rng, 1, 4096), h=_width(rng, 512, 5120),
                    o=_width(rng, 512, 20480))
    if op in ("layernorm_fwd", "layernorm_bwd"):
        return dict(op=op, s=_log(rng, 1, 4096), h=_width(rng, 256, 12288),
                    x=rng.choice(["f16", "f32"]), p=rng.choice(["f16", "f32"]))
    return dict(op=op, tensors=_log(rng, 2, 400), width=_log(rng, 100, 8192),
                r=_log(rng, 1, 64), g=rng.choice(["f16", "bf16", "f32"]))


DT = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}


def _randn(gen, *shape, std=1.0, dtype=torch.float16):
    return (torch.randn(*shape, generator=gen, device="cuda") * std).to(dtype)


def _activations(gen, s, h):
    """fp16 activations with a few one-sided outlier feature columns."""
    X = torch.randn(s, h, generator=gen, device="cuda")
    cols = torch.randint(0, h, (6,), generator=gen, device="cuda")
    X[:, cols] = 6 + 54 * torch.rand(s, 6, generator=gen, device="cuda")
    return X.half()


def _ids(case, gen):
    """The adapter of each row (-1: none)."""
    s, n = case["s"], case["n"]
    bare = _bare_rows(case)
    if case["layout"] == "tokens":  # one token of each request
        ids = torch.cat([torch.randperm(n, generator=gen, device="cuda")
                         for _ in range((s + n - 1) // n)])[:s]
        if bare:
            at = torch.randint(0, s, (1,), generator=gen, device="cuda")
            ids[at] = -1
    else:  # whole prompts, one after another, of ragged lengths
        cuts = torch.sort(torch.randint(0, s - bare + 1, (n - 1,), generator=gen,
                                        device="cuda")).values
        ids = torch.searchsorted(cuts, torch.arange(s, device="cuda"), right=True)
        ids = torch.where(torch.arange(s, device="cuda") >= s - bare, -1, ids)
    return ids.to(torch.int32)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed * 7919 + 13)
    op = case["op"]
    st = dict(op=op)
    if op in ("adapters_fwd", "adapters_bwd"):
        s, h, o, n, r = (case[k] for k in "shonr")
        st["X"] = _activations(gen, s, h)
        st["A"] = _randn(gen, n, r, h, std=h ** -0.5)
        st["B"] = _randn(gen, n, r, o, std=0.02)
        st["scale"] = 1.0 + torch.rand(n, generator=gen, device="cuda")
        st["ranks"] = torch.tensor([_rank(case, a) for a in range(n)], dtype=torch.int32,
                                   device="cuda")
        st["ids"] = _ids(case, gen)
        st["base"] = _randn(gen, s, o if op == "adapters_fwd" else h)
        st["out"] = torch.empty_like(st["base"])
        if op == "adapters_bwd":
            # the loss's gradient, and what the forward pass kept
            st["dY"] = _randn(gen, s, o, std=1e-2)
            st["v"] = _plain_v(st)
            st["dA"] = torch.empty(n, r, h, device="cuda")
            st["dB"] = torch.empty(n, r, o, device="cuda")
    elif op == "matmul_bwd":
        s, h, o = (case[k] for k in "sho")
        # codes and column scales as the weight preparation leaves them for normal weights
        st["wq"] = (torch.randn(o, h, generator=gen, device="cuda") * 31).round_() \
            .clamp_(-127, 127).to(torch.int8)
        st["aw"] = (0.08 + 0.01 * torch.rand(o, generator=gen, device="cuda")).half().float()
        st["dY"] = _randn(gen, s, o, std=1e-1)
        st["out"] = torch.empty(s, h, dtype=torch.float16, device="cuda")
    elif op in ("layernorm_fwd", "layernorm_bwd"):
        s, h = case["s"], case["h"]
        st["eps"] = 1e-5
        X = _activations(gen, s, h).float() + 0.1 * torch.randn(s, h, generator=gen, device="cuda")
        st["X"] = X.to(DT[case["x"]])
        st["gamma"] = (1 + 0.1 * torch.randn(h, generator=gen, device="cuda")).to(DT[case["p"]])
        st["beta"] = (0.1 * torch.randn(h, generator=gen, device="cuda")).to(DT[case["p"]])
        if op == "layernorm_fwd":
            st["out"] = torch.empty(s, h, dtype=torch.float16, device="cuda")
        else:
            st["dY"] = _randn(gen, s, h, std=1e-1)
            Xd = st["X"].double()
            st["mean"] = Xd.mean(1).float()
            st["rstd"] = (Xd.var(1, unbiased=False) + st["eps"]).rsqrt().float()
            st["dX"] = torch.empty_like(st["X"])
    else:
        shapes = [(case["r"] * case["width"] - (i % 4 == 3) * (i % case["width"]))
                  for i in range(case["tensors"])]
        # gradients of layers of different sizes
        st["grads"] = [_randn(gen, m, std=0.05 * (1 + i % 5), dtype=DT[case["g"]])
                       for i, m in enumerate(shapes)]
        # the clipped gradients lie one behind another in one buffer, 16-byte aligned
        starts, end = [], 0
        for m in shapes:
            starts.append(end)
            end += (m + 7) // 8 * 8
        st["flat"] = torch.zeros(end, dtype=DT[case["g"]], device="cuda")
        st["outs"] = [st["flat"][at:at + m] for at, m in zip(starts, shapes)]
        st["max_norm"] = 1000.0 if seed % 2 else 100.0
    if own:
        _prepare_own(st)
    return st


def _prepare_own(st):
    from mixed_precision_int8_b200 import binding as L
    op = st["op"]
    if op in ("adapters_fwd", "adapters_bwd"):
        s, h = st["X"].shape
        n, r, o = st["B"].shape
        st["adapters"] = L.Adapters(st["A"], st["B"], st["scale"], st["ranks"])
        st["ws"] = L.AdapterWorkspace(s, h, o, n, r)
    elif op == "matmul_bwd":
        st["w"] = L.PreparedWeight(st["wq"], st["aw"])
        st["ws"] = L.BackwardWorkspace(st["dY"].shape[0], st["w"].h, st["w"].o)
    elif op == "layernorm_bwd":
        st["ws"] = L.LayerNormWorkspace(*st["X"].shape)
    elif op == "clip":
        st["list"] = L.GradList(st["grads"], st["outs"])


def _pick(st):
    """[s, n*r]: scale where a column's adapter is the row's and its rank is used, else 0."""
    n, r = st["A"].shape[:2]
    a = torch.arange(n, device="cuda").repeat_interleave(r)
    t = torch.arange(r, device="cuda").repeat(n)
    mine = (st["ids"][:, None] == a[None, :]) & (t < st["ranks"].repeat_interleave(r))[None, :]
    return mine, torch.where(mine, st["scale"].repeat_interleave(r)[None, :], 0.0)


def _plain_v(st):
    """What the forward pass keeps: X . A of each row's own adapter, fp32 [s][r]."""
    n, r, h = st["A"].shape
    mine, _ = _pick(st)
    v = torch.where(mine, st["X"].float() @ st["A"].reshape(n * r, h).float().t(), 0.0)
    return v.reshape(-1, n, r).sum(1).contiguous()


def run(state):
    st = state
    return _run_own(st) if own else _run_plain(st)


def _run_own(st):
    from mixed_precision_int8_b200 import binding as L
    op = st["op"]
    if op == "adapters_fwd":
        return L.llmint8_adapters_forward(st["X"], st["adapters"], st["ids"], base=st["base"],
                                          out=st["out"], workspace=st["ws"])
    if op == "adapters_bwd":
        return L.llmint8_adapters_backward(st["X"], st["dY"], st["adapters"], st["ids"],
                                           v=st["v"], base=st["base"], dX=st["out"],
                                           dA=st["dA"], dB=st["dB"], workspace=st["ws"])
    if op == "matmul_bwd":
        return L.llmint8_matmul_backward(st["dY"], st["w"], out=st["out"], workspace=st["ws"])
    if op == "layernorm_fwd":
        return L.llmint8_layernorm_forward(st["X"], st["gamma"], st["beta"], st["eps"],
                                           out=st["out"])
    if op == "layernorm_bwd":
        return L.llmint8_layernorm_backward(st["dY"], st["X"], st["gamma"], st["mean"],
                                            st["rstd"], dX=st["dX"], workspace=st["ws"])
    norm = L.llmint8_clip_grads(st["list"], st["max_norm"])
    return [norm, st["flat"]]


def _run_plain(st):
    op = st["op"]
    if op in ("adapters_fwd", "adapters_bwd"):
        n, r, h = st["A"].shape
        A = st["A"].reshape(n * r, h).float()
        B = st["B"].reshape(n * r, -1).float()
        mine, scale = _pick(st)
        if op == "adapters_fwd":
            V = torch.where(mine, st["X"].float() @ A.t(), 0.0) * scale
            return (st["base"].float() + V @ B).half()
        dYf = st["dY"].float()
        G = torch.where(mine, dYf @ B.t(), 0.0) * scale
        V = torch.where(mine, st["v"].repeat(1, n), 0.0) * scale
        dX = (st["base"].float() + G @ A).half()
        dA = (G.t() @ st["X"].float()).reshape(st["A"].shape)
        dB = (V.t() @ dYf).reshape(st["B"].shape)
        return dX, dA, dB
    if op == "matmul_bwd":
        W = st["wq"].float() * (st["aw"] / 127.0)[:, None]
        return (st["dY"].float() @ W).half()
    if op == "layernorm_fwd":
        X = st["X"].float()
        mean = X.mean(1)
        xc = X - mean[:, None]
        rstd = 1.0 / torch.sqrt((xc * xc).mean(1) + st["eps"])
        y = xc * rstd[:, None] * st["gamma"].float() + st["beta"].float()
        return y.half(), mean, rstd
    if op == "layernorm_bwd":
        xh = (st["X"].float() - st["mean"][:, None]) * st["rstd"][:, None]
        dY = st["dY"].float()
        g = dY * st["gamma"].float()
        dX = st["rstd"][:, None] * (g - g.mean(1, keepdim=True)
                                    - xh * (g * xh).mean(1, keepdim=True))
        return dX.to(st["X"].dtype), (dY * xh).sum(0), dY.sum(0)
    # many tensors: sums in 64 bits, as the total runs over hundreds of millions of values
    total = torch.stack([(g.float() * g.float()).sum(dtype=torch.float64)
                         for g in st["grads"]]).sum()
    norm = torch.sqrt(total)
    coef = torch.clamp(st["max_norm"] / (norm + 1e-6), max=1.0).float()
    for g, out in zip(st["grads"], st["outs"]):
        out.copy_(g.float() * coef)
    return [norm.float().reshape(1), st["flat"]]


def work(case):
    op = case["op"]
    if op in ("adapters_fwd", "adapters_bwd"):
        s, h, o, n, r = (case[k] for k in "shonr")
        rows = s - _bare_rows(case)
        used = min(n, rows)
        ranks = [_rank(case, a) for a in range(n)]
        mean_rank = sum(ranks) / n
        factors = used * mean_rank * (h + o)
        if op == "adapters_fwd":
            return dict(bytes=int(2 * rows * h + 2 * factors + 4 * s * o),
                        flops=int(2 * rows * mean_rank * (h + o)))
        return dict(bytes=int(2 * rows * (h + o) + 2 * factors + 4 * s * h
                              + 4 * n * r * (h + o) + 4 * rows * mean_rank),
                    flops=int(4 * rows * mean_rank * (h + o)))
    if op == "matmul_bwd":
        s, h, o = (case[k] for k in "sho")
        return dict(bytes=2 * s * (h + o) + h * o + 4 * o, flops=2 * s * h * o)
    if op == "layernorm_fwd":
        s, h = case["s"], case["h"]
        xb, pb = (2 if case["x"] == "f16" else 4), (2 if case["p"] == "f16" else 4)
        return dict(bytes=s * h * (xb + 2) + 2 * h * pb + 8 * s, flops=8 * s * h)
    if op == "layernorm_bwd":
        s, h = case["s"], case["h"]
        xb, pb = (2 if case["x"] == "f16" else 4), (2 if case["p"] == "f16" else 4)
        return dict(bytes=s * h * (2 * xb + 2) + h * (pb + 8) + 8 * s, flops=14 * s * h)
    total = sum(case["r"] * case["width"] - (i % 4 == 3) * (i % case["width"])
                for i in range(case["tensors"]))
    b = 4 if case["g"] == "f32" else 2
    return dict(bytes=2 * b * total, flops=3 * total)


def exact(case, seed):
    """The definitions, in 64 bits."""
    st = prepare(case, seed)
    op = case["op"]
    if op in ("adapters_fwd", "adapters_bwd"):
        ids = st["ids"].tolist()
        X = st["X"].double()
        out = st["base"].double()
        if op == "adapters_bwd":
            dY, dA, dB = (st["dY"].double(), torch.zeros(st["A"].shape, dtype=torch.float64,
                                                         device="cuda"),
                          torch.zeros(st["B"].shape, dtype=torch.float64, device="cuda"))
        for a in sorted(set(ids)):
            if a < 0:
                continue
            rows = torch.tensor([i for i, x in enumerate(ids) if x == a], device="cuda")
            k = _rank(case, a)
            A, B = st["A"][a, :k].double(), st["B"][a, :k].double()
            c = float(st["scale"][a])
            if op == "adapters_fwd":
                out[rows] += c * torch.mm(torch.mm(X[rows], A.T), B)
            else:
                G = torch.mm(dY[rows], B.T)
                out[rows] += c * torch.mm(G, A)
                dA[a, :k] = c * torch.mm(G.T, X[rows])
                dB[a, :k] = c * torch.mm(st["v"][rows, :k].double().T, dY[rows])
        return out if op == "adapters_fwd" else (out, dA, dB)
    if op == "matmul_bwd":
        scaled = st["dY"].double() * (st["aw"].double() / 127)
        return torch.mm(scaled, st["wq"].double())
    if op in ("layernorm_fwd", "layernorm_bwd"):
        X = st["X"].double()
        if op == "layernorm_fwd":
            mean = X.sum(1) / X.shape[1]
            var = ((X - mean[:, None]) ** 2).sum(1) / X.shape[1]
            rstd = (var + st["eps"]) ** -0.5
            y = torch.addcmul(st["beta"].double(), (X - mean[:, None]) * rstd[:, None],
                              st["gamma"].double())
            return y, mean, rstd
        m, q = st["mean"].double()[:, None], st["rstd"].double()[:, None]
        dY, gamma = st["dY"].double(), st["gamma"].double()
        h = X.shape[1]
        c1 = torch.mv(dY, gamma)[:, None] / h
        c2 = torch.mv(dY * (X - m) * q, gamma)[:, None] / h
        return (q * (dY * gamma - c1 - (X - m) * q * c2), ((X - m) * q * dY).sum(0), dY.sum(0))
    norm = math.sqrt(sum(float(torch.dot(g.double(), g.double())) for g in st["grads"]))
    coef = min(1.0, st["max_norm"] / (norm + 1e-6))
    padded = [torch.cat([g.double() * coef, g.new_zeros(-len(g) % 8, dtype=torch.float64)])
              for g in st["grads"]]
    return [torch.tensor([norm], dtype=torch.float64), torch.cat(padded)]
