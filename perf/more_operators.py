"""Cases that measure routing to experts, the rows' way to the experts and back, and products in MXFP4.

Three operators, on row-major matrices (T tokens, E experts, `top` of them for each token):

  route  the experts of each token from its logits x: the `top` largest keys, in falling order, ties
         to the lower expert; the key is x or, with a bias, s + bias (s the softmax or sigmoid of x); a
         logit of -inf is never chosen.  With limited groups the experts lie in equal runs, a run is
         worth the sum of its one or two largest keys, and only the best runs count.  Results: expert
         (-1: none), weight c s or, renormalised, c s / sum of the chosen s; place, the row of each
         (token, expert) pair when the pairs are sorted by expert and token; offsets, where each
         expert's rows start.  With `train` also the gradient of the logits from that of the weights.
  rows   A[place[t][j]] = X[t] (dispatch) and C[t] = sum over j of w[t][j] Y[place[t][j]] (combine), and
         the gradients dY[place[t][j]] = w[t][j] D[t], dw[t][j] = D[t] . Y[place[t][j]], and of dispatch
         the sum of the rows of a token
  mx     rows of activations to MXFP4 (blocks of 32: the power of two two below the largest's, elements
         0 .. 6 rounded to nearest, ties to even) and, by expert, C[r] = GELU(A[r] B_g^T + bias_g) with
         weights in MXFP4: packed nibbles and a scale byte for 32 of them

`run` computes the plain form in elementary torch operations, or, where `own` is true, calls the library.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
GRID = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]  # the magnitudes of a 4-bit element


# ------------------------------------------------------------------------------- cases --

def listed():
    return [
        # the router of one decoded token: sigmoid scores with a balancing bias, four of eight runs
        _case("route_token", "route", T=1, E=256, top=8, score="sigmoid", bias=True, runs=8, best=4,
              of=2, renorm=True, scale=2.5, dtype="f32"),
        # the same router over a long prompt
        _case("route_prompt", "route", T=8191, E=256, top=8, score="sigmoid", bias=True, runs=8,
              best=4, of=2, renorm=True, scale=2.5, dtype="f32"),
        # a small router in training, a padded batch: the last tokens are masked
        _case("route_train_padded", "route", T=1000, E=60, top=4, score="softmax", renorm=True,
              dtype="bf16", pad=0.1, train=True),
        # softmax scores as they are, forward and backward, over a training batch
        _case("route_train", "route", T=16384, E=128, top=8, score="softmax", dtype="f32", train=True),
        # the answers of two experts for a running batch of 16 sequences
        _case("combine_decode", "rows", T=16, top=2, K=2048, E=64, dtype="bf16", part="combine"),
        # a prompt's rows to eight experts each and back
        _case("rows_prompt", "rows", T=8190, top=8, K=2048, E=128, dtype="bf16", part="both"),
        # a training step: both ways, and the gradients of both
        _case("rows_train", "rows", T=4096, top=2, K=4096, E=8, dtype="bf16", part="train"),
        # one decoded token through a wide projection: bound by the weight bytes
        _case("mx_token", "mx", T=1, N=28672, K=8192, dtype="bf16", bias=True),
        # a ragged batch of running sequences
        _case("mx_batch_ragged", "mx", T=37, N=4101, K=4128, dtype="f16", bias=True),
        # 16 tokens, two of 64 experts each: decoding
        _case("mx_experts_decode", "mx", T=16, top=2, N=1024, K=2048, E=64, dtype="bf16", bias=True,
              gelu=True, skew=0.7),
        # a prompt through the first layer of a perceptron, bias and GELU fused
        _case("mx_prompt_gelu", "mx", T=4096, N=4096, K=4096, dtype="bf16", bias=True, gelu=True),
        # prompts through 32 experts of uneven load
        _case("mx_experts_prompt", "mx", T=4096, top=2, N=2048, K=2048, E=32, dtype="bf16", bias=True,
              gelu=True, skew=0.6),
    ]


def _case(name, op, **kw):
    c = {"op": op, "T": 1, "E": 1, "top": 0, "N": 0, "K": 0, "dtype": "bf16", "score": "", "bias": False,
         "runs": 1, "best": 1, "of": 1, "renorm": False, "scale": 1.0, "pad": 0.0, "train": False,
         "part": "", "gelu": False, "skew": 0.5}
    c.update(kw)
    if name:
        c["name"] = name
    return c


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    """A case of the listed ranges: from one token up, sizes of real layers and, one in six, any."""
    op = rng.choice(["route", "route", "rows", "mx", "mx"])
    odd = rng.random() < 1 / 6
    if op == "route":
        while True:
            T, E = _log(rng, 1, 16384), _log(rng, 2, 512)
            if not odd:
                E = max(8, E // 8 * 8)
            if T * E <= 8191 * 256:
                break
        top = min(E, rng.randint(1, 8))
        runs = rng.choice([r for r in (1, 1, 2, 4, 8) if E % r == 0])
        best = rng.randint(-(-top * runs // E), runs)
        score = rng.choice(["softmax", "sigmoid"])
        return _case("", op, T=T, E=E, top=top, score=score, bias=rng.random() < 0.5, runs=runs,
                     best=best, of=rng.choice([1, 2]) if runs > 1 else 1, renorm=rng.random() < 0.5,
                     scale=rng.choice([1.0, 2.5]), dtype=rng.choice(["f32", "bf16", "f16"]),
                     pad=rng.choice([0.0, 0.0, 0.2]), train=rng.random() < 0.5)
    if op == "rows":
        while True:
            T, top, K = _log(rng, 1, 16384), rng.randint(1, 8), _log(rng, 64, 8192)
            if not odd:
                K = max(64, K // 8 * 8)
            if T * top * K <= 4096 * 2 * 4096:
                break
        return _case("", op, T=T, top=top, K=K, E=max(top, _log(rng, 2, 256)),
                     dtype=rng.choice(["bf16", "f16", "f32"]), pad=rng.choice([0.0, 0.0, 0.2]),
                     part=rng.choice(["dispatch", "combine", "both", "train"]),
                     skew=rng.choice([0.0, 0.6, 1.5]))
    while True:
        E = rng.choice([1, _log(rng, 2, 96)])
        T, top = _log(rng, 1, 8192), 0 if E == 1 else rng.randint(1, min(E, 4))
        N, K = _log(rng, 64, 8192), max(1, _log(rng, 64, 8192) // 32) * 32
        if not odd:
            N = N // 8 * 8
        # the listed cases' largest work and largest weights
        if 2.0 * T * max(top, 1) * N * K <= 1.3e11 and E * N * K <= 235e6:
            break
    return _case("", op, T=T, top=top, N=N, K=K, E=E, dtype=rng.choice(["bf16", "f16"]),
                 bias=rng.random() < 0.6, gelu=rng.random() < 0.4, skew=rng.choice([0.0, 0.6, 1.5]))


def _experts(case):
    """Experts of each token (T x top, -1 where a token is padding): a router's choice of uneven
    loads, from the case alone."""
    T, E, top = case["T"], case["E"], case["top"]
    rng = np.random.default_rng([T, E, top, int(1000 * case["skew"])])
    want = case["skew"] * rng.standard_normal(E) + rng.gumbel(size=(T, E))
    e = np.argsort(-want, axis=1)[:, :top]
    e[T - int(case["pad"] * T):] = -1
    return e


def _plan(e, E):
    """Place of each pair (-1: none) and the offsets of the experts, in the pairs' sorted order."""
    flat = e.reshape(-1)
    order = np.argsort(np.where(flat < 0, E, flat), kind="stable")
    place = np.empty(flat.size, dtype=np.int32)
    place[order] = np.arange(flat.size)
    place[flat < 0] = -1
    counts = np.bincount(flat[flat >= 0], minlength=E)
    return place.reshape(e.shape), np.concatenate([[0], np.cumsum(counts)]).astype(np.int64)


def work(case):
    T, E, top, K, N = (case[k] for k in ("T", "E", "top", "K", "N"))
    es = 4 if case["dtype"] == "f32" else 2
    if case["op"] == "route":
        b = T * E * es + 12 * T * top + 8 * (E + 1) + (4 * E if case["bias"] else 0)
        f = 8 * T * E
        if case["train"]:  # the logits count once; the gradients of weights in, of logits out
            b, f = b + 4 * T * top + T * E * es, 2 * f
        return {"bytes": b, "flops": f}
    if case["op"] == "rows":
        live = T - int(case["pad"] * T)
        row, pairs = K * es, live * top
        b = {"dispatch": live + pairs, "combine": pairs + T, "both": live + 2 * pairs + T,
             "train": 3 * live + 5 * pairs + 2 * T}[case["part"]] * row
        return {"bytes": b + 8 * T * top, "flops": (8 if case["part"] == "train" else 2) * pairs * K}
    rows = T * max(top, 1)
    live = 1 if top == 0 else np.unique(_experts(case)).size
    b = 2 * T * K + live * N * (K // 2 + K // 32) + 2 * rows * N + (4 * live * N if case["bias"] else 0)
    return {"bytes": b + (4 * rows + 8 * (E + 1) if top else 0), "flops": 2 * rows * N * K}


# ------------------------------------------------------------------------------ inputs --

def _pack(x):
    """MXFP4 of the rows of x (r x K, fp32): bytes of two nibbles, and scale bytes."""
    r, K = x.shape
    v = x.view(r, K // 32, 32)
    s = (torch.frexp(v.abs().amax(dim=2))[1] + 124).clamp(0, 254)
    a = torch.ldexp(v, (127 - s)[:, :, None])
    q = _nibbles(a).view(r, K // 2, 2)
    return q[:, :, 0] | (q[:, :, 1] << 4), s.to(torch.uint8)


def _nibbles(a):
    """4-bit codes of scaled values: to nearest, ties to the even code, the sign in bit 3."""
    m = a.abs()
    q = (m > 0.25).to(torch.uint8)
    for border, odd_below in ((0.75, True), (1.25, False), (1.75, True), (2.5, False), (3.5, True), (5.0, False)):
        q += (m >= border) if odd_below else (m > border)
    return q | (torch.signbit(a).to(torch.uint8) << 3)


def _inputs(case, seed):
    dev = torch.device("cuda:0")
    gen = torch.Generator(device=dev).manual_seed(seed)
    T, E, top, K, N = (case[k] for k in ("T", "E", "top", "K", "N"))
    dt = DTYPES[case["dtype"]]

    def normal(*shape):
        return torch.randn(*shape, device=dev, generator=gen)

    if case["op"] == "route":
        # trained routers prefer some experts; padding is masked
        x = 1.5 * normal(T, E) + 0.5 * normal(E)
        x[T - int(case["pad"] * T):] = -math.inf
        return {"x": x.to(dt), "bias": 0.1 * normal(E) if case["bias"] else None,
                "dw": normal(T, top) if case["train"] else None}
    st = {}
    if top:
        place, offsets = _plan(_experts(case), E)
        st["place"] = torch.from_numpy(place).to(dev)
        st["offsets"] = torch.from_numpy(offsets).to(dev)
        st["sizes"] = np.diff(offsets).tolist()
    # activations: a few channels far larger than the rest
    x = normal(T, K)
    x *= 1 + 9 * (torch.rand(K, device=dev, generator=gen) < 0.01).float()
    st["X"] = x.to(dt)
    if case["op"] == "rows":
        st["Y"], st["D"] = normal(T * top, K).to(dt), normal(T, K).to(dt)
        w = torch.rand(T, top, device=dev, generator=gen) + 0.1
        st["w"] = w / w.sum(dim=1, keepdim=True)
        return st
    if not top:
        st["place"], st["offsets"], st["sizes"] = None, None, [T]
    st["bias"] = 0.1 * normal(E, N) if case["bias"] else None
    st["B"] = torch.empty(E, N, K // 2, dtype=torch.uint8, device=dev)
    st["sb"] = torch.zeros(E, N, _ceil16(K // 32), dtype=torch.uint8, device=dev)
    for g in range(E):
        for n in range(0, N, 4096):
            w = normal(min(4096, N - n), K) * K ** -0.5
            st["B"][g, n:n + 4096], st["sb"][g, n:n + 4096, :K // 32] = _pack(w)
    return st


def _ceil16(n):
    return (n + 15) // 16 * 16


_handle = None


def _library():
    """The handle a program creates once."""
    global _handle
    import tiled_matrix_multiply_amd as tmm
    if _handle is None:
        _handle = tmm.Gemm(0)
    return tmm, _handle


def prepare(case, seed):
    """The inputs, and the buffers that a program keeps for the results."""
    st = _inputs(case, seed)
    st["case"] = dict(case)
    dev = torch.device("cuda:0")
    T, E, top, K, N = (case[k] for k in ("T", "E", "top", "K", "N"))
    dt = DTYPES[case["dtype"]]
    if case["op"] == "route":
        st["expert"] = torch.empty(T, top, dtype=torch.int32, device=dev)
        st["weight"] = torch.empty(T, top, device=dev)
        st["to"] = torch.empty(T, top, dtype=torch.int32, device=dev)
        st["starts"] = torch.empty(E + 1, dtype=torch.int64, device=dev)
        st["dx"] = torch.empty(T, E, dtype=dt, device=dev) if case["train"] else None
        st["ws"] = None
        if own:
            tmm, _ = _library()
            st["ws"] = torch.empty(tmm.route_workspace_bytes(T, E), dtype=torch.uint8, device=dev)
    elif case["op"] == "rows":
        # rows that no pair has are never written
        st["A"], st["dY"] = (torch.zeros(T * top, K, dtype=dt, device=dev) for _ in range(2))
        st["C"], st["dX"] = (torch.empty(T, K, dtype=dt, device=dev) for _ in range(2))
        st["dw"] = torch.empty(T, top, device=dev)
    else:
        rows = T * max(top, 1)
        st["Q"] = torch.zeros(rows, K // 2, dtype=torch.uint8, device=dev)
        st["s"] = torch.zeros(rows, _ceil16(K // 32), dtype=torch.uint8, device=dev)
        st["C"] = torch.zeros(rows, N, dtype=dt, device=dev)
    if own:
        _library()
    return st


# -------------------------------------------------------------------------------- runs --

def run(st):
    return _run_own(st) if own else _run_plain(st)


def _run_own(st):
    tmm, h = _library()
    c = st["case"]
    T, E, top, K, N = (c[k] for k in ("T", "E", "top", "K", "N"))
    if c["op"] == "route":
        h.route(st["x"], st["expert"], st["weight"], st["to"], st["starts"], tokens=T, experts=E, top=top,
                x_type=c["dtype"], score=c["score"], bias=st["bias"], groups=c["runs"],
                top_groups=c["best"], group_top=c["of"], renorm=c["renorm"], scale=c["scale"],
                workspace=st["ws"])
        out = [st["expert"], st["weight"], st["to"], st["starts"]]
        if c["train"]:
            h.route_grad(st["x"], st["expert"], st["dw"], st["dx"], tokens=T, experts=E, top=top,
                         x_type=c["dtype"], score=c["score"], renorm=c["renorm"], scale=c["scale"])
            out.append(st["dx"])
        return out
    if c["op"] == "rows":
        out, kw = [], {"tokens": T, "top": top, "K": K, "rows": T * top, "dtype": c["dtype"]}
        if c["part"] != "combine":
            h.dispatch_rows(st["X"], st["place"], st["A"], **kw)
            out.append(st["A"])
        if c["part"] != "dispatch":
            h.combine_rows(st["Y"], st["place"], st["C"], weight=st["w"], **kw)
            out.append(st["C"])
        if c["part"] == "train":
            h.combine_rows_grad(st["D"], st["Y"], st["place"], st["w"], st["dY"], st["dw"], **kw)
            h.combine_rows(st["dY"], st["place"], st["dX"], **kw)
            out += [st["dY"], st["dw"], st["dX"]]
        return out
    rows = T * max(top, 1)
    h.quantize_mx(st["X"], st["Q"], st["s"], M=T, K=K, x_type=c["dtype"], place=st["place"],
                  top=max(top, 1), rows=rows, lds=st["s"].shape[1])
    epi = (tmm.GEMM_EPI_BIAS if c["bias"] else 0) | (tmm.GEMM_EPI_GELU if c["gelu"] else 0)
    h.run_grouped_mx(st["Q"], st["s"], st["B"], st["sb"], st["C"], st["offsets"], groups=E, M=rows, N=N, K=K,
                     c_type=c["dtype"], epilogue=epi, bias=st["bias"], ldsa=st["s"].shape[1],
                     ldsb=st["sb"].shape[2])
    return st["C"]


def _run_plain(st):
    return {"route": _plain_route, "rows": _plain_rows, "mx": _plain_mx}[st["case"]["op"]](st)


def _scores(x, kind):
    if kind == "sigmoid":
        return 1 / (1 + torch.exp(-x))
    top = x.amax(dim=1, keepdim=True)
    p = torch.exp(x - torch.where(top == -math.inf, 0.0, top))
    return p / p.sum(dim=1, keepdim=True).clamp_min(1e-300)


def _plain_route(st):
    # in 64 bits: keys next to each other decide
    c = st["case"]
    T, E, top, runs = c["T"], c["E"], c["top"], c["runs"]
    x = st["x"].double()
    s = _scores(x, c["score"])
    off = x == -math.inf
    key = torch.where(off, -math.inf, s + st["bias"].double()) if c["bias"] else x
    if runs > 1:
        worth = key if c["bias"] or c["of"] == 1 else torch.where(off, -math.inf, s)
        best = worth.view(T, runs, E // runs).sort(dim=2, descending=True)[0][:, :, :c["of"]]
        total = torch.where(best[:, :, 0] == -math.inf, -math.inf, torch.where(best == -math.inf, 0.0, best).sum(dim=2))
        rank = total.sort(dim=1, descending=True, stable=True)[1].argsort(dim=1)
        kept = (rank < c["best"]).repeat_interleave(E // runs, dim=1)
        key = torch.where(kept, key, -math.inf)
    v, e = key.sort(dim=1, descending=True, stable=True)
    v, e = v[:, :top], e[:, :top]
    none = v == -math.inf
    w = torch.where(none, 0.0, s.gather(1, e))
    if c["renorm"]:
        w = w / w.sum(dim=1, keepdim=True).clamp_min(1e-300)
    flat = torch.where(none, E, e).flatten()
    ranked, order = flat.sort(stable=True)
    place = torch.empty_like(order)
    place[order] = torch.arange(T * top, device=x.device)
    starts = torch.searchsorted(ranked, torch.arange(E + 1, device=x.device))
    out = [torch.where(none, -1, e).int(), (c["scale"] * w).float(),
           torch.where(none, -1, place.view(T, top)).int(), starts]
    if c["train"]:
        g = torch.where(none, 0.0, c["scale"] * st["dw"].double())
        if c["renorm"]:  # through the quotient to the chosen scores' logarithms
            g = w * (g - (w * g).sum(dim=1, keepdim=True))
        else:
            g = w * g
        dx = torch.zeros_like(x).scatter_add_(1, e, g)  # of the scores' logarithms
        if c["score"] == "sigmoid":
            dx = dx * (1 - s)
        elif not c["renorm"]:
            dx = dx - s * g.sum(dim=1, keepdim=True)
        out.append(dx.to(st["x"].dtype))
    return out


def _plain_rows(st):
    c = st["case"]
    T, top, K, dt = c["T"], c["top"], c["K"], DTYPES[c["dtype"]]
    place = st["place"].long()
    there = (place >= 0)[:, :, None]
    at = place[place >= 0]

    def sorted_rows(v):  # T x top x K to the sorted order
        out = torch.zeros(T * top, K, dtype=dt, device=v.device)
        out[at] = v.to(dt)[place >= 0]
        return out

    def back(y):
        return torch.where(there, y[place.clamp_min(0)].float(), 0.0)

    out = []
    if c["part"] != "combine":
        out.append(sorted_rows(st["X"][:, None, :].expand(T, top, K)))
    if c["part"] != "dispatch":
        out.append((st["w"][:, :, None] * back(st["Y"])).sum(dim=1).to(dt))
    if c["part"] == "train":
        d = st["D"].float()[:, None, :]
        dy = sorted_rows(st["w"][:, :, None] * d)
        out += [dy, (back(st["Y"]) * d).sum(dim=2), back(dy).sum(dim=1).to(dt)]
    return out


def _values(q, s):
    """The fp32 values of packed rows (r x K/2 bytes) and their scale bytes (r x K/32)."""
    grid = torch.tensor(GRID + [-v for v in GRID], device=q.device)
    v = grid[torch.stack([q & 15, q >> 4], dim=2).long()]
    return torch.ldexp(v.view(q.shape[0], -1, 32), s.int()[:, :, None] - 127).view(q.shape[0], -1)


def _gelu(x):
    return 0.5 * x * torch.erfc(x * -(0.5 ** 0.5))


def _plain_mx(st):
    c = st["case"]
    T, K, N = c["T"], c["K"], c["N"]
    a = _values(*_pack(st["X"].float()))
    if st["place"] is not None:
        rows = torch.empty(T * c["top"], K, device=a.device)
        rows[st["place"].long().flatten()] = a.repeat_interleave(c["top"], dim=0)
        a = rows
    outs, r = [], 0
    for g, n in enumerate(st["sizes"]):
        if n:
            y = a[r:r + n] @ _values(st["B"][g], st["sb"][g, :, :K // 32]).t()
            if c["bias"]:
                y = y + st["bias"][g]
            outs.append((_gelu(y) if c["gelu"] else y).to(DTYPES[c["dtype"]]))
        r += n
    return torch.cat(outs)


# ------------------------------------------------------------------------------- exact --

def exact(case, seed):
    """The definitions in 64 bits, from the same inputs."""
    st = _inputs(case, seed)
    return {"route": _exact_route, "rows": _exact_rows, "mx": _exact_mx}[case["op"]](case, st)


def _exact_route(c, st):
    """Choices one by one, and the weights of what was chosen from their logarithms."""
    T, E, top = c["T"], c["E"], c["top"]
    x = st["x"].double()
    dev, inf = x.device, math.inf
    dead = x == -inf
    if c["score"] == "sigmoid":
        ls = torch.nn.functional.logsigmoid(x)
    else:
        ls = x - torch.logsumexp(x, dim=1, keepdim=True)
    ls = torch.where(dead, -inf, ls)
    key = torch.where(dead, -inf, torch.exp(ls) + st["bias"].double()) if c["bias"] else x.clone()
    t = torch.arange(T, device=dev)
    if c["runs"] > 1:
        size = E // c["runs"]
        v = (key if c["bias"] or c["of"] == 1 else torch.exp(ls).masked_fill(dead, -inf)).clone()
        total = torch.full((T, c["runs"]), -inf, dtype=torch.float64, device=dev)
        for i in range(min(c["of"], size)):
            for g in range(c["runs"]):
                m, at = v[:, g * size:(g + 1) * size].max(dim=1)
                total[:, g] = m if i == 0 else total[:, g] + torch.where(m == -inf, 0.0, m)
                v[t, g * size + at] = -inf
        keep = torch.zeros(T, c["runs"], dtype=torch.bool, device=dev)
        for _ in range(c["best"]):
            m = total.amax(dim=1, keepdim=True)
            at = (total == m).to(torch.uint8).argmax(dim=1)
            keep[t, at] = True
            total[t, at] = -inf
        key.masked_fill_(~keep.repeat_interleave(size, dim=1), -inf)
    expert, lw = [], []
    for _ in range(top):
        m = key.amax(dim=1)
        at = (key == m[:, None]).to(torch.uint8).argmax(dim=1)  # the first of them
        expert.append(torch.where(m == -inf, -1, at))
        lw.append(torch.where(m == -inf, -inf, ls[t, at]))
        key[t, at] = -inf
    e, lw = torch.stack(expert, dim=1), torch.stack(lw, dim=1)
    none = e < 0
    if c["renorm"]:
        lw = torch.where(none, -inf, lw - torch.logsumexp(lw, dim=1, keepdim=True))
    w = torch.exp(lw)
    place, starts = _plan(e.cpu().numpy(), E)
    out = [e.int(), c["scale"] * w, torch.from_numpy(place).to(dev), torch.from_numpy(starts).to(dev)]
    if not c["train"]:
        return out
    # d weight_j / d x_e, summed against the weights' gradients
    gw = torch.where(none, 0.0, st["dw"].double() * c["scale"] * w)
    dx = torch.zeros(T, E, dtype=torch.float64, device=dev)
    p = torch.exp(ls)
    slope = 1 - p if c["score"] == "sigmoid" else torch.ones_like(p)
    share = gw.sum(dim=1)
    for j in range(top):
        at = e[:, j].clamp_min(0)
        d = gw[:, j] - (w[:, j] * share if c["renorm"] else 0)
        dx[t, at] += torch.where(none[:, j], 0.0, d * slope[t, at])
    if c["score"] == "softmax" and not c["renorm"]:
        dx -= p * share[:, None]
    return out + [dx]


def _exact_rows(c, st):
    T, top, K = c["T"], c["top"], c["K"]
    dev, dt = st["X"].device, DTYPES[c["dtype"]]
    place, w = st["place"], st["w"].double()
    C, dX = (torch.zeros(T, K, dtype=torch.float64, device=dev) for _ in range(2))
    A, dY = (torch.zeros(T * top, K, dtype=torch.float64, device=dev) for _ in range(2))
    dw = torch.zeros(T, top, dtype=torch.float64, device=dev)
    d = st["D"].double()
    for j in range(top):
        t = torch.nonzero(place[:, j] >= 0).flatten()
        at = place[t, j].long()
        y = st["Y"][at].double()
        A[at] = st["X"][t].double()
        C[t] += w[t, j, None] * y
        dY[at] = w[t, j, None] * d[t]
        dw[t, j] = (d[t] * y).sum(dim=1)
        dX[t] += (w[t, j, None] * d[t]).to(dt).double()  # of the stored gradients
    return {"dispatch": [A], "combine": [C], "both": [A, C], "train": [A, C, dY, dw, dX]}[c["part"]]


def _exact_mx(c, st):
    """The elements by their definition: multiples of a step that grows with the value."""
    f64 = torch.float64
    T, K, N = c["T"], c["K"], c["N"]
    x = st["X"].to(f64).view(T, K // 32, 32)
    big = x.abs().amax(dim=2, keepdim=True)
    scale = torch.exp2(torch.floor(torch.log2(torch.where(big > 0, big, 1.0))) - 2)
    y = x / scale
    step = torch.exp2(torch.floor(torch.log2(y.abs().clamp_min(1.0))) - 1)
    a = ((torch.round(y / step) * step).clamp(-6, 6) * scale).view(T, K)
    out = torch.zeros(T * max(c["top"], 1), N, dtype=f64, device=a.device)
    if st["place"] is not None:
        rows = torch.zeros(T * c["top"], K, dtype=f64, device=a.device)
        for j in range(c["top"]):
            rows[st["place"][:, j].long()] = a
        a = rows
    lo, hi = 0, 0
    for g, n in enumerate(st["sizes"]):
        lo, hi = hi, hi + n
        if n == 0:
            continue
        for n0 in range(0, N, 4096):
            q, s = st["B"][g, n0:n0 + 4096], st["sb"][g, n0:n0 + 4096, :K // 32]
            b = torch.empty(q.shape[0], K, dtype=f64, device=a.device)
            for half in (0, 1):
                code = (q >> (4 * half)) & 15
                m, e = (code & 1).to(f64), (code >> 1) & 3
                v = torch.where(e == 0, 0.5 * m, (1 + 0.5 * m) * torch.exp2(e.to(f64) - 1))
                b[:, half::2] = torch.where(code > 7, -v, v)
            b = (b.view(-1, K // 32, 32) * torch.exp2(s.to(f64) - 127)[:, :, None]).view(-1, K)
            v = torch.mm(a[lo:hi], b.t().contiguous())
            if c["bias"]:
                v += st["bias"][g, n0:n0 + 4096].to(f64)
            out[lo:hi, n0:n0 + 4096] = v * torch.special.ndtr(v) if c["gelu"] else v
    return out
