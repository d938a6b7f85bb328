"""Cases that measure the products grouped by expert and the products in 8-bit integers.

Five operators, on row-major matrices (M rows of tokens, B the weights):

  grouped        C[r] = GELU(A[r] op(B_g) + bias_g) for the rows r of group g, 16-bit types; with
                 the weights' other layout the same call is the data gradient
  grouped_wgrad  dB_g = A_g^T D_g and dbias_g = the sum of D_g's rows
  i8             C = GELU(sa[i] sb[j] (A B)[i][j] + bias[j]) with 8-bit integers A and B
  grouped_i8     the same by group, sb and bias per group
  quantize       s_i = max |x_i| / 127 and the 8-bit integers nearest to x_i / s_i, ties to even

The rows of a group are consecutive; offsets (groups + 1 numbers on the device) say where each
group starts.  `run` computes the plain form in elementary torch operations, or, where `own` is
true, calls the library.
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


# ------------------------------------------------------------------------------- cases --

def listed():
    return [
        # one token's activations on their way into an 8-bit layer
        _case("quantize_token", "quantize", M=1, K=4096, dtype="bf16"),
        # a long prompt's activations of a wide layer
        _case("quantize_prompt", "quantize", M=8191, K=8192, dtype="f16"),
        # one decoded token through a wide projection: bound by the weight bytes
        _case("i8_token", "i8", M=1, N=28672, K=8192, nk=True, dtype="bf16", bias=True),
        # a ragged batch of running sequences, weights stored K x N
        _case("i8_batch_ragged", "i8", M=37, N=4104, K=4112, nk=False, dtype="f16", bias=True),
        # a prompt through the first layer of a perceptron, bias and GELU fused
        _case("i8_prompt_gelu", "i8", M=4096, N=4096, K=4096, nk=True, dtype="bf16", bias=True,
              gelu=True),
        # 32 rows (16 tokens, two experts each) over 64 small experts: decoding
        _case("experts_decode", "grouped", M=32, N=1024, K=2048, groups=64, nk=True,
              dtype="bf16", bias=True, gelu=True, skew=0.7, route=11),
        # 4096 rows over 8 experts of uneven load, the forward pass of training
        _case("experts_forward", "grouped", M=4096, N=4096, K=2048, groups=8, nk=True,
              dtype="bf16", bias=True, skew=0.6, route=12),
        # the data gradient of 8190 rows over 16 experts, some idle: the weights' other layout
        _case("experts_dgrad", "grouped", M=8190, N=2048, K=4096, groups=16, nk=False,
              dtype="f16", skew=0.8, idle=0.15, route=13),
        # the weight gradient of the same kind of layer, in the weights' type
        _case("experts_wgrad", "grouped_wgrad", M=4096, N=4096, K=2048, groups=8, nk=True,
              dtype="bf16", out="bf16", bias=True, skew=0.6, route=12),
        # the largest: weight gradients in fp32 for 16 experts, two of them without a row
        _case("experts_wgrad_long", "grouped_wgrad", M=16383, N=2048, K=4096, groups=16, nk=False,
              dtype="f16", out="f32", skew=0.8, idle=0.15, route=13),
        # decoding through 64 experts in 8 bits
        _case("experts_i8_decode", "grouped_i8", M=32, N=1024, K=2048, groups=64, nk=True,
              dtype="bf16", bias=True, gelu=True, skew=0.7, route=11),
        # prompts through 32 experts in 8 bits
        _case("experts_i8_prompt", "grouped_i8", M=8192, N=2048, K=2048, groups=32, nk=True,
              dtype="bf16", bias=True, gelu=True, skew=0.6, route=14),
    ]


def _case(name, op, **kw):
    c = {"op": op, "M": 1, "N": 0, "K": 1, "groups": 1, "nk": True, "dtype": "bf16", "out": "",
         "bias": False, "gelu": False, "skew": 0.0, "idle": 0.0, "route": 0}
    c.update(kw)
    c["out"] = c["out"] or c["dtype"]
    if name:
        c["name"] = name
    return c


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    """A case of the listed ranges: row counts from one up, widths in multiples of 4, 8 or 16
    (the rows of real weights), one in six of any size at all, loads even to very uneven."""
    op = rng.choice(["quantize", "i8", "i8", "grouped", "grouped", "grouped_wgrad", "grouped_i8"])
    while True:
        odd = rng.random() < 1 / 6
        step = 1 if odd else (16 if op in ("i8", "grouped_i8") else 8)
        hi = 1500 if odd else 8192
        M = _log(rng, 1, 2000 if odd else 16384)
        N = max(step, _log(rng, 64, hi) // step * step)
        K = max(step, _log(rng, 64, hi) // step * step)
        G = 1 if op in ("i8", "quantize") else _log(rng, 1, 96)
        # the listed cases' largest work and largest weights
        if 2.0 * M * N * K <= 2.7e11 and G * N * K <= 134e6:
            break
    return _case("", op, M=M, N=0 if op == "quantize" else N, K=K, groups=G,
                 nk=rng.random() < 0.6, dtype=rng.choice(["bf16", "f16"]),
                 out=rng.choice(["", "f32"]) if op == "grouped_wgrad" else "",
                 bias=op != "quantize" and rng.random() < 0.6,
                 gelu=op not in ("quantize", "grouped_wgrad") and rng.random() < 0.4,
                 skew=rng.choice([0.0, 0.6, 1.5]), idle=rng.choice([0.0, 0.0, 0.3]),
                 route=rng.randrange(1 << 30))


def _sizes(case):
    """Rows of each group: the loads of a router, from the case alone."""
    G, M = case["groups"], case["M"]
    rng = random.Random(case["route"])
    w = [0.0 if rng.random() < case["idle"] else math.exp(case["skew"] * rng.gauss(0, 1))
         for _ in range(G)]
    if not any(w):
        w[rng.randrange(G)] = 1.0
    total, cum, cuts = sum(w), 0.0, [0]
    if M <= 256:  # each row picks its expert
        picks = rng.choices(range(G), weights=w, k=M)
        return [picks.count(g) for g in range(G)]
    for v in w:
        cum += v
        cuts.append(min(M, int(cum / total * M + 0.5)))
    cuts[-1] = M
    return [b - a for a, b in zip(cuts, cuts[1:])]


def work(case):
    M, N, K = case["M"], case["N"], case["K"]
    op = case["op"]
    if op == "quantize":
        return {"bytes": M * K * 2 + M * K + 4 * M, "flops": 2 * M * K}
    G = case["groups"]
    live = sum(1 for s in _sizes(case) if s)  # groups whose weights have to be read
    es = 1 if op in ("i8", "grouped_i8") else 2
    os = 4 if case["out"] == "f32" else 2
    if op == "grouped_wgrad":
        b = M * (N + K) * es + G * N * K * os + (4 * G * N if case["bias"] else 0)
    else:
        b = M * K * es + live * N * K * es + M * N * os
        b += 4 * live * N if case["bias"] else 0
        b += 4 * M + 4 * live * N if es == 1 else 0
    if op != "i8":
        b += 8 * (G + 1)
    return {"bytes": b, "flops": 2 * M * N * K}


# ------------------------------------------------------------------------------ inputs --

def _codes(x):
    """8-bit integers of the rows of x, and their scales."""
    s = (x.abs().amax(dim=-1, keepdim=True) / 127).clamp_min(1e-12)
    return torch.round(x / s).clamp(-127, 127).to(torch.int8), s.squeeze(-1).contiguous()


def _inputs(case, seed):
    dev = torch.device("cuda:0")
    gen = torch.Generator(device=dev).manual_seed(seed)
    M, N, K, G = case["M"], case["N"], case["K"], case["groups"]
    op, dt = case["op"], DTYPES[case["dtype"]]

    def normal(*shape):
        return torch.randn(*shape, device=dev, generator=gen)

    # activations: a few channels far larger than the rest
    x = normal(M, K)
    x *= 1 + 9 * (torch.rand(K, device=dev, generator=gen) < 0.01).float()
    if op == "quantize":
        return {"X": x.to(dt)}
    sizes = _sizes(case) if op != "i8" else [M]
    st = {"sizes": sizes}
    cuts = [0]
    for s in sizes:
        cuts.append(cuts[-1] + s)
    st["offsets"] = torch.tensor(cuts, dtype=torch.int64, device=dev)
    st["bias"] = 0.1 * normal(G, N) if case["bias"] else None
    if op == "grouped_wgrad":
        st["A"], st["D"] = x.to(dt), normal(M, N).to(dt)
        return st
    if op == "grouped":
        st["A"] = x.to(dt)
        b = torch.empty((G, N, K) if case["nk"] else (G, K, N), dtype=dt, device=dev)
        for g in range(G):
            b[g] = (normal(*b.shape[1:]) * K ** -0.5).to(dt)
        st["B"] = b
        return st
    st["A"], st["sa"] = _codes(x)
    b = torch.empty((G, N, K) if case["nk"] else (G, K, N), dtype=torch.int8, device=dev)
    sb = torch.empty(G, N, device=dev)
    for g in range(G):
        q, sb[g] = _codes(normal(N, K) * K ** -0.5)
        b[g] = q if case["nk"] else q.t()
    st["B"], st["sb"] = b, sb
    return st


_handle = None


def _library():
    """The handle a program creates once."""
    global _handle
    import tiled_matrix_multiply_amd as tmm
    if _handle is None:
        _handle = tmm.Gemm(0)
    return tmm, _handle


def prepare(case, seed):
    st = _inputs(case, seed)
    st["case"] = dict(case)
    dev = torch.device("cuda:0")
    M, N, K, G = case["M"], case["N"], case["K"], case["groups"]
    if own:
        if case["op"] == "quantize":
            st["Q"] = torch.empty(M, K, dtype=torch.int8, device=dev)
            st["s"] = torch.empty(M, device=dev)
        elif case["op"] == "grouped_wgrad":
            st["C"] = torch.empty((G, N, K) if case["nk"] else (G, K, N),
                                  dtype=DTYPES[case["out"]], device=dev)
            st["db"] = torch.empty(G, N, device=dev) if case["bias"] else None
        else:
            st["C"] = torch.empty(M, N, dtype=DTYPES[case["out"]], device=dev)
        _library()
    return st


# -------------------------------------------------------------------------------- runs --

def run(st):
    return _run_own(st) if own else _run_plain(st)


def _run_own(st):
    tmm, h = _library()
    c = st["case"]
    op, M, N, K, G = c["op"], c["M"], c["N"], c["K"], c["groups"]
    if op == "quantize":
        h.quantize_rows(st["X"], st["Q"], st["s"], M=M, K=K, x_type=c["dtype"])
        return st["Q"], st["s"]
    if op == "grouped_wgrad":
        h.run_grouped_wgrad(st["A"], st["D"], st["C"], st["offsets"], groups=G, M=M, N=N, K=K,
                            trans_b=c["nk"], a_type=c["dtype"], c_type=c["out"], dbias=st["db"])
        return (st["C"], st["db"]) if c["bias"] else st["C"]
    epi = (tmm.GEMM_EPI_BIAS if c["bias"] else 0) | (tmm.GEMM_EPI_GELU if c["gelu"] else 0)
    if op == "grouped":
        h.run_grouped(st["A"], st["B"], st["C"], st["offsets"], groups=G, M=M, N=N, K=K,
                      trans_b=c["nk"], a_type=c["dtype"], epilogue=epi, bias=st["bias"])
    elif op == "i8":
        h.run_i8(st["A"], st["sa"], st["B"], st["sb"], st["C"], M=M, N=N, K=K, trans_b=c["nk"],
                 c_type=c["out"], epilogue=epi, bias=st["bias"])
    else:
        h.run_grouped_i8(st["A"], st["sa"], st["B"], st["sb"], st["C"], st["offsets"], groups=G,
                         M=M, N=N, K=K, trans_b=c["nk"], c_type=c["out"], epilogue=epi,
                         bias=st["bias"])
    return st["C"]


def _gelu(x):
    return 0.5 * x * torch.erfc(x * -(0.5 ** 0.5))


def _run_plain(st):
    c = st["case"]
    op, nk = c["op"], c["nk"]
    if op == "quantize":
        # in 64 bits: the quotient decides ties
        x = st["X"].double()
        s = (x.abs().amax(dim=1) / 127).float()
        d = torch.where(s > 0, s, torch.ones_like(s)).double()
        return torch.round(x / d[:, None]).to(torch.int8), s
    out_t = DTYPES[c["out"]]
    outs, dbs, r = [], [], 0
    for g, n in enumerate(st["sizes"]):
        rows = slice(r, r + n)
        r += n
        if op == "grouped_wgrad":
            a, d = st["A"][rows].float(), st["D"][rows].float()
            outs.append((d.t() @ a if nk else a.t() @ d).to(out_t))
            if c["bias"]:
                dbs.append(d.sum(dim=0))
            continue
        if n == 0:
            continue
        if op == "grouped":
            a, b = st["A"][rows].float(), st["B"][g].float()
            y = a @ (b.t() if nk else b)
        else:
            # integer sums pass 24 bits: in 64
            a, b = st["A"][rows].double(), st["B"][g].double()
            y = a @ (b.t() if nk else b)
            y = (y.float() * st["sa"][rows, None]) * st["sb"][g]
        if c["bias"]:
            y = y + st["bias"][g]
        outs.append((_gelu(y) if c["gelu"] else y).to(out_t))
    if op == "grouped_wgrad":
        return (torch.stack(outs), torch.stack(dbs)) if c["bias"] else torch.stack(outs)
    return torch.cat(outs)


# ------------------------------------------------------------------------------- exact --

def exact(case, seed):
    """The definitions in 64 bits, from the same inputs."""
    st = _inputs(case, seed)
    f64 = torch.float64
    op, M, N, K, G = case["op"], case["M"], case["N"], case["K"], case["groups"]
    if op == "quantize":
        x = st["X"].to(f64)
        s = torch.maximum(x.amax(dim=1), -x.amin(dim=1)) / 127
        step = s.float().to(f64)  # the codes are defined by the scale as it is stored
        step[step == 0] = 1
        q = x / step[:, None]
        low = torch.floor(q)
        up = (q - low > 0.5) | ((q - low == 0.5) & (low.remainder(2) == 1))
        return (low + up).to(torch.int8), s
    off = [0]
    for n in st["sizes"]:
        off.append(off[-1] + n)
    dev = st["A"].device
    if op == "grouped_wgrad":
        dw = torch.zeros((G, N, K) if case["nk"] else (G, K, N), dtype=f64, device=dev)
        db = torch.zeros(G, N, dtype=f64, device=dev)
        for g in range(G):
            a, d = st["A"][off[g]:off[g + 1]].to(f64), st["D"][off[g]:off[g + 1]].to(f64)
            w = torch.mm(a.t().contiguous(), d)
            dw[g] = w.t() if case["nk"] else w
            db[g] = d.sum(0)
        return (dw, db) if case["bias"] else dw
    y = torch.empty(M, N, dtype=f64, device=dev)
    for g in range(G):
        if off[g] == off[g + 1]:
            continue
        w = st["B"][g].to(f64)
        w = w.t().contiguous() if case["nk"] else w
        x = st["A"][off[g]:off[g + 1]].to(f64)
        if op != "grouped":
            w = w * st["sb"][g].to(f64)[None, :]
            x = x * st["sa"][off[g]:off[g + 1]].to(f64)[:, None]
        v = torch.mm(x, w)
        if case["bias"]:
            v += st["bias"][g].to(f64)
        y[off[g]:off[g + 1]] = v * torch.special.ndtr(v) if case["gelu"] else v
    return y
