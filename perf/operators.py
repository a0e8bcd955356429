"""The expert-layer and microscaled 4-bit operators as plain torch operations, and the cases they are measured on.

T tokens choose k of E experts; a slot is one (token, choice) pair, slots are sorted by (expert, token, choice).
Weights are [E, N, K] (output x input features).  MXFP4: blocks of 32 values along K share a power-of-two scale (one e8m0
byte); a value is one of +-{0, 0.5, 1, 1.5, 2, 3, 4, 6}.  Scale bytes lie in 1024-byte tiles of 128 rows x 256 k.
"""
import math

import numpy as np
import torch

own = False

LEVELS = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ---------------------------------------------------------------- cases
def listed():
    return [
        # one decoding step of a layer with 64 experts
        dict(name="route decode", op="route", T=16, E=64, k=6, score="softmax", renorm=True, f32=False, masked=0.0),
        # a prompt chunk with padding (masked tokens) through a sigmoid router of 256 experts
        dict(name="route prompt", op="route", T=16384, E=256, k=8, score="sigmoid", renorm=True, f32=True, masked=0.03),
        # gate and up products of 8 experts of the MLP that the benchmark uses, 8 tokens decoding
        dict(name="experts bf16 decode", op="grouped", T=8, E=8, k=2, N=14336, K=4096, mx=False, up=True, skew=0.6),
        # down products of the same experts, a prompt of 4096 tokens, the slots already sorted
        dict(name="experts bf16 prompt", op="grouped", T=4096, E=8, k=2, N=4096, K=14336, mx=False, up=False, skew=0.3),
        # many small 4-bit experts, 33 tokens decoding
        dict(name="experts mx decode", op="grouped", T=33, E=128, k=8, N=768, K=2048, mx=True, up=True, skew=0.8),
        # 64 4-bit experts of an odd width, a prompt
        dict(name="experts mx prompt", op="grouped", T=2048, E=64, k=6, N=1408, K=2048, mx=True, up=True, skew=0.5),
        # activations of a small batch to 4 bits and back
        dict(name="mx round trip small", op="mx", rows=37, K=4096, f32=False),
        # a whole projection to 4 bits and back, from its 32-bit master copy
        dict(name="mx round trip weight", op="mx", rows=14336, K=4096, f32=True),
        # one token through a 4-bit gate projection
        dict(name="mx product one token", op="mxgemm", M=1, N=14336, K=4096, xmx=False),
        # a prompt through it with both sides in 4 bits
        dict(name="mx product prompt", op="mxgemm", M=2048, N=14336, K=4096, xmx=True),
        # the sum behind the experts, decoding and prompt
        dict(name="combine decode", op="combine", T=8, k=2, N=4096, masked=0.0),
        dict(name="combine prompt", op="combine", T=8192, k=8, N=4096, masked=0.03),
    ]


def _log(rng, lo, hi, step=1):
    """A multiple of step in [lo, hi], spread over the logarithm."""
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return int(min(hi, max(lo, round(v / step) * step)))


def draw(rng):
    op = rng.choice(["route", "grouped", "grouped", "mx", "mxgemm", "mxgemm", "combine"])
    if op == "route":
        E = _log(rng, 4, 512)
        return dict(op=op, T=_log(rng, 1, 16384), E=E, k=rng.randint(1, min(E, 10)), score=rng.choice(["softmax", "sigmoid"]),
                    renorm=rng.random() < 0.5, f32=rng.random() < 0.5, masked=rng.choice([0.0, 0.1]))
    if op == "grouped":
        E, k = _log(rng, 2, 128), rng.randint(1, 8)
        T, N, K = _log(rng, 1, 4096), _log(rng, 72, 8192), _log(rng, 64, 8192, 64)
        k = min(k, E)
        while T * k * N * K > 1.2e11 or E * N * K > 4.7e8:
            T, N, K = (T + 1) // 2, (N + 1) // 2, max(64, K // 128 * 64)
        return dict(op=op, T=T, E=E, k=k, N=N, K=K, mx=rng.random() < 0.5, up=rng.random() < 0.5, skew=round(rng.uniform(0.0, 1.2), 2))
    if op == "mx":
        return dict(op=op, rows=_log(rng, 1, 8192), K=_log(rng, 64, 7168, 64), f32=rng.random() < 0.5)
    if op == "mxgemm":
        M, N, K = _log(rng, 1, 2048), _log(rng, 40, 14336), _log(rng, 64, 8192, 64)
        return dict(op=op, M=M, N=N, K=K, xmx=rng.random() < 0.5)
    return dict(op=op, T=_log(rng, 1, 8192), k=rng.randint(1, 8), N=_log(rng, 8, 4096, 8), masked=rng.choice([0.0, 0.1]))


def group_sizes(case):
    """Slots of each expert before the seed's permutation: a share falling off as (rank + 1)^-skew."""
    R, E = case["T"] * case["k"], case["E"]
    p = np.arange(1, E + 1, dtype=np.float64) ** -case["skew"]
    edge = np.floor(np.concatenate([[0.0], np.cumsum(p)]) / p.sum() * R + 0.5).astype(np.int64)
    return np.diff(edge)


def work(case):
    op = case["op"]
    if op == "route":
        n = case["T"] * case["E"]
        return {"bytes": n * (4 if case["f32"] else 2) + 16 * case["T"] * case["k"] + 4 * (case["E"] + 1), "flops": 4 * n}
    if op == "grouped":
        R, mats = case["T"] * case["k"], 2 if case["up"] else 1
        active = int((group_sizes(case) > 0).sum())
        weight = mats * case["N"] * case["K"] * (17 / 32 if case["mx"] else 2.0)
        x = (case["T"] if case["up"] else R) * case["K"] * 2 + (4 * R if case["up"] else 0)
        return {"bytes": int(active * weight + x + R * case["N"] * 2 + 4 * (case["E"] + 1)), "flops": 2 * mats * R * case["N"] * case["K"]}
    if op == "mx":
        n = case["rows"] * case["K"]
        return {"bytes": int(n * ((4 if case["f32"] else 2) + 2 * 17 / 32 + 2)), "flops": 4 * n}
    if op == "mxgemm":
        M, N, K = case["M"], case["N"], case["K"]
        return {"bytes": int(2 * M * K + N * K * 17 / 32 + 2 * M * N), "flops": 2 * M * N * K}
    n = case["T"] * case["k"] * case["N"]
    return {"bytes": 2 * n + 2 * case["T"] * case["N"] + 8 * case["T"] * case["k"], "flops": 2 * n}


# ---------------------------------------------------------------- inputs
def _weights(shape, g):
    w = torch.randn(shape, generator=g, device="cuda", dtype=torch.bfloat16) * 0.02
    return w


def _activations(rows, K, g):
    """Unit rows with a few channels that stand out, as behind a normalisation."""
    x = torch.randn(rows, K, generator=g, device="cuda")
    gain = torch.where(torch.rand(K, generator=g, device="cuda") < 0.01, 8.0, 1.0)
    return (x * gain).to(torch.bfloat16)


def _scale_index(rows, K):
    """Byte of row r's block b in the scale tiles of one matrix, and the tiles' size."""
    r = torch.arange(rows, device="cuda")[:, None]
    b = torch.arange(K // 32, device="cuda")[None, :]
    kt = (K + 255) // 256
    at = ((r // 128) * kt + b // 8) * 1024 + (b // 4 % 2) * 512 + (r % 32) * 16 + (r // 32 % 4) * 4 + b % 4
    return at, (rows + 127) // 128 * kt * 1024


def _two_to(s):
    """2^s in fp32 for whole s in [-127, 127], from its bits."""
    return torch.where(s > -127, (s + 127) << 23, 1 << 22).int().view(torch.float32)


def _mx_parts(x):
    """x [batch, rows, K] -> codes (0..15, one a byte), scale exponents; plain quantisation."""
    v = x.float().unflatten(-1, (-1, 32))
    amax = v.abs().amax(-1)
    e = torch.frexp(amax)[1] - 3
    s = torch.where(amax > 0, e, -127).clamp(-127, 127)
    m = (v * _two_to(-s)[..., None]).abs()
    c = ((m > 0.25).to(torch.uint8) + (m >= 0.75) + (m > 1.25) + (m >= 1.75) + (m > 2.5) + (m >= 3.5) + (m > 5.0)).to(torch.uint8)
    return (c + 8 * torch.signbit(v).to(torch.uint8)).flatten(-2), s


def _mx_pack(x):
    """Packed codes and scale tiles of x [batch, rows, K], as the framework holds them."""
    batch, rows, K = x.shape
    c, s = _mx_parts(x)
    at, size = _scale_index(rows, K)
    tiles = torch.zeros(batch, size, dtype=torch.uint8, device=x.device)
    tiles[:, at.flatten()] = (s + 127).to(torch.uint8).flatten(1)
    return c[..., 0::2] | (c[..., 1::2] << 4), tiles


def _mx_values(codes, tiles):
    """fp32 values of packed codes [batch, rows, K/2] and their scale tiles."""
    batch, rows, half = codes.shape
    at, _ = _scale_index(rows, 2 * half)
    s = tiles[:, at].int() - 127
    c = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).long()
    level = torch.tensor(LEVELS + tuple(-v for v in LEVELS), device=codes.device)
    return (level[c].unflatten(-1, (-1, 32)) * _two_to(s)[..., None]).flatten(-2)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    op = case["op"]
    st = dict(case=case)
    if op == "route":
        x = torch.randn(case["T"], case["E"], generator=g, device="cuda") * 1.5
        x += torch.randn(case["E"], generator=g, device="cuda") * 0.5
        if case["masked"]:   # padded tokens: nothing to choose from
            x[torch.rand(case["T"], generator=g, device="cuda") < case["masked"]] = -math.inf
        st["logits"] = x if case["f32"] else x.to(torch.bfloat16)
    elif op == "grouped":
        T, E, k, N, K = (case[n] for n in ("T", "E", "k", "N", "K"))
        sizes = group_sizes(case)[np.random.default_rng(seed).permutation(E)]
        st["offsets"] = torch.tensor(np.concatenate([[0], np.cumsum(sizes)]), dtype=torch.int32, device="cuda")
        st["most"] = int(sizes.max())
        if case["up"]:   # the first products gather their rows from the tokens
            st["X"] = _activations(T, K, g)
            st["rows"] = (torch.randperm(T * k, generator=g, device="cuda") // k).int()
        else:            # the second read the first's outputs
            st["X"] = _activations(T * k, K, g)
            st["rows"] = None
        st["W"] = [_weights((E, N, K), g) for _ in range(2 if case["up"] else 1)]
        if case["mx"]:
            st["W"] = [_mx_pack(w) for w in st["W"]]
    elif op == "mx":
        x = torch.randn(case["rows"], case["K"], generator=g, device="cuda") * 0.02
        x *= torch.exp2(torch.randint(-3, 4, (case["rows"], 1), generator=g, device="cuda").float())
        st["X"] = x if case["f32"] else x.to(torch.bfloat16)
    elif op == "mxgemm":
        st["X"] = _activations(case["M"], case["K"], g)
        st["W"] = _mx_pack(_weights((1, case["N"], case["K"]), g))
    else:
        T, k, N = case["T"], case["k"], case["N"]
        st["Z"] = torch.randn(T * k, N, generator=g, device="cuda", dtype=torch.bfloat16)
        pos = torch.randperm(T * k, generator=g, device="cuda").int().view(T, k)
        w = torch.rand(T, k, generator=g, device="cuda")
        if case["masked"]:   # padded tokens chose nothing
            off = torch.rand(T, 1, generator=g, device="cuda") < case["masked"]
            pos, w = torch.where(off, -1, pos), torch.where(off, 0.0, w)
        st["pos"], st["weights"] = pos.contiguous(), (w / 4).contiguous()
    return st


# ---------------------------------------------------------------- one pass
def run(state):
    return _own(state) if own else _plain(state)


def _own(st):
    import decode_gemm_bf16_b200 as uw
    case = st["case"]
    op = case["op"]
    if op == "route":
        r = uw.uw_route(st["logits"], case["k"], score=case["score"], renorm=case["renorm"])
        return dict(ids=r.ids, weights=r.weights, offsets=r.offsets, rows=r.rows, pos=r.pos)
    if op == "grouped":
        W = [uw.MxMatrix(*w) for w in st["W"]] if case["mx"] else st["W"]
        return uw.uw_gemm_grouped(st["X"], W[0], st["offsets"], rows=st["rows"], up=W[1] if case["up"] else None)
    if op == "mx":
        return uw.uw_mx_dequantize(uw.uw_mx_quantize(st["X"]))
    if op == "mxgemm":
        return uw.uw_mx_gemm(uw.uw_mx_quantize(st["X"]) if case["xmx"] else st["X"], uw.MxMatrix(*st["W"]))
    return uw.uw_combine(st["Z"], st["pos"], st["weights"])


def _plain(st):
    case = st["case"]
    op = case["op"]
    if op == "route":
        return _route(st["logits"].float(), case)
    if op == "grouped":
        X, off = st["X"], st["offsets"].long()
        R, E = case["T"] * case["k"], case["E"]
        slot = torch.arange(R, device=X.device)
        e = torch.searchsorted(off, slot, right=True) - 1
        pad = torch.zeros(E, st["most"], case["K"], device=X.device)
        pad[e, slot - off[e]] = (X if st["rows"] is None else X[st["rows"].long()]).float()
        ys = [torch.bmm(pad, (_mx_values(*w) if case["mx"] else w.float()).transpose(1, 2))[e, slot - off[e]] for w in st["W"]]
        y = ys[0] if not case["up"] else ys[0] / (1 + torch.exp(-ys[0])) * ys[1]
        return y.to(torch.bfloat16)
    if op == "mx":
        c, s = _mx_parts(st["X"])
        level = torch.tensor(LEVELS + tuple(-v for v in LEVELS), device=c.device)
        return (level[c.long()].unflatten(-1, (-1, 32)) * _two_to(s)[..., None]).flatten(-2).to(torch.bfloat16)
    if op == "mxgemm":
        X = st["X"].float()
        if case["xmx"]:
            X = _mx_values(*_mx_pack(X[None]))[0]
        return (X @ _mx_values(*st["W"])[0].T).to(torch.bfloat16)
    z = st["Z"].float()[st["pos"].clamp(min=0).long()]
    w = torch.where(st["pos"] >= 0, st["weights"], 0.0)
    return (z * w[..., None]).sum(1).to(torch.bfloat16)


def _route(x, case):
    T, E, k = case["T"], case["E"], case["k"]
    x = torch.where(x.isnan(), -math.inf, x).clamp(max=torch.finfo(torch.float32).max) + 0.0
    top, ids = torch.sort(x, dim=1, descending=True, stable=True)
    top, ids = top[:, :k], ids[:, :k]
    valid = top > -math.inf
    if case["score"] == "softmax":
        m = top[:, :1].clamp(min=-torch.finfo(torch.float32).max)
        p = torch.exp(top - m)
        total = p.sum(1, keepdim=True) if case["renorm"] else torch.exp(x - m).sum(1, keepdim=True)
        w = p / torch.where(total > 0, total, 1.0)
    else:
        w = 1 / (1 + torch.exp(-top))
        if case["renorm"]:
            total = w.sum(1, keepdim=True)
            w = w / torch.where(total > 0, total, 1.0)
    flat = torch.where(valid, ids, E).flatten()
    order = torch.argsort(flat, stable=True)
    offsets = torch.searchsorted(flat[order], torch.arange(E + 1, device=x.device))
    slot = torch.arange(T * k, device=x.device)
    rows = torch.where(slot < offsets[E], order // k, -1)
    pos = torch.empty_like(slot)
    pos[order] = torch.where(slot < offsets[E], slot, -1)
    return dict(ids=torch.where(valid, ids, -1).int(), weights=torch.where(valid, w, 0.0), offsets=offsets.int(), rows=rows.int(),
                pos=pos.view(T, k).int())


# ---------------------------------------------------------------- in 64 bits
def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "route":
        return _exact_route(st["logits"].double().cpu().numpy(), case)
    if op == "grouped":
        bounds, outs = st["offsets"].tolist(), []
        for e in range(case["E"]):
            rows = slice(bounds[e], bounds[e + 1])
            x = (st["X"][rows] if st["rows"] is None else st["X"][st["rows"][rows].long()]).double()
            w = [_exact_mx(w[0][e], w[1][e]) if case["mx"] else w[e].double() for w in st["W"]]
            y = x @ w[0].T
            outs.append(y * torch.sigmoid(y) * (x @ w[1].T) if case["up"] else y)
        return torch.cat(outs)
    if op == "mx":
        return _exact_round(st["X"].double())
    if op == "mxgemm":
        x = st["X"].double()
        return (_exact_round(x) if case["xmx"] else x) @ _exact_mx(st["W"][0][0], st["W"][1][0]).T
    y = torch.zeros(case["T"], case["N"], dtype=torch.float64, device="cuda")
    for j in range(case["k"]):
        p = st["pos"][:, j].long()
        y += torch.where(p >= 0, st["weights"][:, j].double(), 0.0)[:, None] * st["Z"][p.clamp(min=0)].double()
    return y


def _exact_route(x, case):
    T, E, k = case["T"], case["E"], case["k"]
    ids = np.argsort(-x, axis=1, kind="stable")[:, :k]
    top = np.take_along_axis(x, ids, 1)
    valid = np.isfinite(top)
    with np.errstate(invalid="ignore", divide="ignore", over="ignore"):
        if case["score"] == "softmax":
            s = np.exp(x - x.max(1, keepdims=True))
            w = np.take_along_axis(s, ids, 1)
            w = w / (w.sum(1, keepdims=True) if case["renorm"] else s.sum(1, keepdims=True))
        else:
            w = 1 / (1 + np.exp(-top))
            w = w / (w.sum(1, keepdims=True) if case["renorm"] else 1.0)
    ids = np.where(valid, ids, -1)
    t, j = np.nonzero(valid)
    order = np.lexsort((j, t, ids[t, j]))
    rows = np.full(T * k, -1, np.int32)
    rows[:len(order)] = t[order]
    pos = np.full((T, k), -1, np.int32)
    pos[t[order], j[order]] = np.arange(len(order))
    offsets = np.concatenate([[0], np.cumsum(np.bincount(ids[t, j], minlength=E))])
    return dict(ids=ids.astype(np.int32), weights=np.where(valid, w, 0.0), offsets=offsets.astype(np.int32), rows=rows, pos=pos)


def _exact_power(e):
    """2^e in fp64 for whole e: looked up."""
    return torch.tensor([2.0 ** i for i in range(-160, 161)], dtype=torch.float64, device=e.device)[e.long() + 160]


def _exact_mx(codes, tiles):
    """fp64 values of one matrix from its packed codes and scale tiles."""
    rows, half = codes.shape
    kt = (2 * half + 255) // 256
    s = tiles.view(-1, kt, 2, 32, 4, 4).permute(0, 4, 3, 1, 2, 5).reshape(-1, kt * 8)[:rows, :half // 16]
    c = torch.empty(rows, 2 * half, dtype=torch.int64, device=codes.device)
    c[:, 0::2], c[:, 1::2] = codes & 15, codes >> 4
    mant, expo = c & 1, c >> 1 & 3
    mag = torch.where(expo > 0, (2 + mant) * _exact_power(expo - 2), 0.5 * mant)
    return torch.where(c >= 8, -mag, mag) * _exact_power(s.long() - 127).repeat_interleave(32, 1)


def _exact_round(x):
    """x [rows, K] rounded to MXFP4 and back, in fp64."""
    v = x.view(x.shape[0], -1, 32)
    amax = v.abs().amax(-1, keepdim=True)
    s = torch.where(amax > 0, torch.frexp(amax)[1] - 3, -127).clamp(-127, 127)
    m = v.abs() / _exact_power(s)
    step = torch.where(m < 2, 0.5, torch.where(m < 4, 1.0, 2.0))
    q = (torch.round(m / step) * step).clamp(max=6.0)
    return (torch.sign(v) * q * _exact_power(s)).flatten(-2)
