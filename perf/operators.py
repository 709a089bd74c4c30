"""Cases of the 8-bit and the expert-grouped operators, for timing and comparison.

Five operators, each through the public Python entry points of the package:

* ``quantize_w8``: fp32 weights -> int8 codes (native 16 x 64 tiles) with one scale per output channel;
* ``quantize_tokens``: activations -> int8 codes with one scale per token (row);
* ``linear_w8a8``: y = (sx x d) * (xq q^T), int8 products summed exactly;
* ``grouped_linear``: rows sorted by expert times that expert's 4-bit group-quantized weight;
* ``grouped_linear_w8a8``: the same in int8 with token and channel scales.

``own = False`` computes them in elementary torch operations in fp32; ``own = True``
makes the package's calls.  Weights are laid out once, in ``prepare``, as a program
that serves a model keeps them; the plain forms read the same codes in row-major
order.
"""

import torch

own = False

GROUP = 128  # inputs that share one 4-bit scale

F32, BF16 = "f32", "bf16"
DTYPES = {F32: torch.float32, BF16: torch.bfloat16}


# ----------------------------------------------------------------------------
# cases
# ----------------------------------------------------------------------------

def listed():
    return [
        # loading a checkpoint: the 4B-class FFN matrix, and the largest one of a 70B-class layer
        {"name": "weights 2560x9216", "op": "quantize_w8", "N": 2560, "K": 9216},
        {"name": "weights 28672x8192", "op": "quantize_w8", "N": 28672, "K": 8192},
        # one decoded token of a 27B-class model; a long ragged prefill before a 70B-class down projection
        {"name": "tokens 1x5120", "op": "quantize_tokens", "M": 1, "K": 5120, "x": BF16},
        {"name": "tokens 4099x28672", "op": "quantize_tokens", "M": 4099, "K": 28672, "x": BF16},
        # decode of one token (4B-class up projection): the latency of one call
        {"name": "w8a8 1 row 9216x2560", "op": "linear_w8a8", "M": 1, "N": 9216, "K": 2560, "out": BF16},
        # verifying 12 drafted tokens with a 70B-class gate projection: bound by the weights
        {"name": "w8a8 13 rows 28672x8192", "op": "linear_w8a8", "M": 13, "N": 28672, "K": 8192, "out": BF16},
        # a batch of short prompts with an odd number of rows and outputs, kept in fp32 for a K-split layer
        {"name": "w8a8 333 rows 2561x9216", "op": "linear_w8a8", "M": 333, "N": 2561, "K": 9216, "out": F32},
        # prefill of 4096 tokens through a 27B-class gate projection: bound by the products
        {"name": "w8a8 4096 rows 17408x5120", "op": "linear_w8a8", "M": 4096, "N": 17408, "K": 5120, "out": BF16},
        # decode of 8 sequences, two experts of 64 each: few rows per expert, most experts idle
        {"name": "experts w4 16 rows", "op": "grouped_linear", "tokens": 8, "top": 2, "E": 64, "skew": 0.5,
         "N": 2048, "K": 2560, "scales": F32, "out": BF16},
        # prefill of 4095 tokens, two experts of 8 each, some twice as busy as others
        {"name": "experts w4 8190 rows", "op": "grouped_linear", "tokens": 4095, "top": 2, "E": 8, "skew": 0.5,
         "N": 9216, "K": 2560, "scales": BF16, "out": BF16},
        # a verification step of 24 rows with four experts of 32 each
        {"name": "experts w8a8 96 rows", "op": "grouped_linear_w8a8", "tokens": 24, "top": 4, "E": 32, "skew": 0.7,
         "N": 2560, "K": 1408, "out": F32},
        # prefill of 4096 tokens with two experts of 16 each, the down projection of a 27B-class hidden size
        {"name": "experts w8a8 8192 rows", "op": "grouped_linear_w8a8", "tokens": 4096, "top": 2, "E": 16,
         "skew": 0.5, "N": 5120, "K": 4096, "out": BF16},
    ]


def _log(rng, lo, hi):
    return int(round(lo * (hi / lo) ** rng.random()))


def draw(rng):
    op = rng.choice(["quantize_w8", "quantize_tokens", "linear_w8a8", "linear_w8a8", "grouped_linear", "grouped_linear",
                     "grouped_linear_w8a8", "grouped_linear_w8a8"])
    while True:
        K = GROUP * _log(rng, 1, 224)
        N = _log(rng, 16, 28672)
        M = _log(rng, 1, 8192)
        out = rng.choice([BF16, F32])
        if op == "quantize_w8":
            if 200_000 <= N * K <= 235_000_000:
                return {"op": op, "N": N, "K": K}
        elif op == "quantize_tokens":
            if M * K <= 115_000_000:
                return {"op": op, "M": M, "K": K, "x": rng.choice([BF16, BF16, F32])}
        elif op == "linear_w8a8":
            if 200_000 <= N * K <= 235_000_000 and M * N * K <= 180_000_000_000:
                return {"op": op, "M": M, "N": N, "K": K, "out": out}
        else:
            E, top = _log(rng, 2, 128), rng.choice([1, 2, 4, 8])
            tokens = max(1, M // top)
            # the plain form pads every expert to the busiest one's rows: keep what it computes below the largest case
            if top > E or not 200_000 <= E * N * K <= 300_000_000 or tokens * top * N * K > 170_000_000_000:
                continue
            skew = rng.choice([0.0, 0.5, 1.0])
            if max(_sizes(tokens, top, E, skew)) * E * N * K > 360_000_000_000:
                continue
            c = {"op": op, "tokens": tokens, "top": top, "E": E, "skew": skew, "N": N, "K": K, "out": out}
            if op == "grouped_linear":
                c["scales"] = rng.choice([F32, BF16])
            return c


def _sizes(tokens, top, E, skew):
    """Rows of each expert: tokens * top of them, shared out by a popularity that falls
    as rank^-skew, no expert more than once per token."""
    rows, share = tokens * top, [(e + 1) ** -skew for e in range(E)]
    total = sum(share)
    want = [rows * s / total for s in share]
    size = [min(tokens, int(w)) for w in want]
    order = sorted(range(E), key=lambda e: (-(want[e] - int(want[e])), e))
    left, i = rows - sum(size), 0
    while left:
        e = order[i % E]
        if size[e] < tokens:
            size[e] += 1
            left -= 1
        i += 1
    return size


def _layout(case):
    """Rows of the experts, in an order that is the case's own."""
    return _sizes(case["tokens"], case["top"], case["E"], case["skew"])


def work(case):
    op, N, K = case["op"], case.get("N", 0), case["K"]
    wide = 4 if case.get("out") == F32 else 2
    if op == "quantize_w8":
        return {"bytes": 4 * N * K + N * K + 4 * N, "flops": 2 * N * K}
    if op == "quantize_tokens":
        M = case["M"]
        return {"bytes": (4 if case["x"] == F32 else 2) * M * K + M * K + 4 * M, "flops": 2 * M * K}
    if op == "linear_w8a8":
        M = case["M"]
        return {"bytes": N * K + 4 * N + M * K + 4 * M + wide * M * N, "flops": 2 * M * N * K}
    M, busy = case["tokens"] * case["top"], sum(1 for s in _layout(case) if s)
    if op == "grouped_linear":
        scale = 4 if case["scales"] == F32 else 2
        weights = N * K // 2 + scale * N * (K // GROUP)
        return {"bytes": busy * weights + 2 * M * K + wide * M * N + 4 * (case["E"] + 1), "flops": 2 * M * N * K}
    return {"bytes": busy * (N * K + 4 * N) + M * K + 4 * M + wide * M * N + 4 * (case["E"] + 1),
            "flops": 2 * M * N * K}


# ----------------------------------------------------------------------------
# inputs
# ----------------------------------------------------------------------------

def _codes(W, top):
    """Symmetric round-to-nearest codes and scales along the last axis of W (ties away from zero)."""
    d = W.abs().amax(-1, keepdim=True)
    d = d / torch.full_like(d, float(top))  # by a tensor: a true division, not a product with a reciprocal
    t = W / torch.where(d > 0, d, torch.ones_like(d))
    whole = t.trunc()
    q = whole + ((t - whole).abs() >= 0.5).to(t.dtype) * t.sign()
    return q.clamp_(-top, top).to(torch.int8), d.squeeze(-1)


def _pad_rows(q, rows):
    return q if q.shape[-2] == rows else torch.cat([q, q.new_zeros(q.shape[:-2] + (rows - q.shape[-2], q.shape[-1]))], -2)


def _tiles_w8(q):
    """int8 codes [..., N, K] as 16 x 64 tiles: lane L of a tile holds row L % 16, inputs 16 (L // 16) .. + 15."""
    N, K = q.shape[-2:]
    q = _pad_rows(q, (N + 15) // 16 * 16)
    lead = q.shape[:-2]
    n = len(lead)
    q = q.reshape(lead + (q.shape[-2] // 16, 16, K // 64, 4, 16))
    return q.permute(tuple(range(n)) + (n, n + 2, n + 3, n + 1, n + 4)).reshape(lead + (-1,)).contiguous()


def _tiles_w4(q, d):
    """4-bit codes [N, K] and scales [N, K / 128] as 16 x 128 tiles of nibbles and quads of scales."""
    N, K = q.shape
    rows, G = (N + 15) // 16 * 16, K // GROUP
    GP = (G + 3) // 4 * 4
    u = torch.full((rows, GP * GROUP), 8, dtype=torch.int32, device=q.device)
    u[:N, :K] = q.to(torch.int32) + 8
    u = u.reshape(rows // 16, 16, GP, 4, 4, 8).permute(0, 2, 4, 1, 3, 5)  # tile row, group, quarter, row, word, input
    shift = torch.tensor([16 * (j & 1) + 4 * (j >> 1) for j in range(8)], dtype=torch.int32, device=q.device)
    v = (u << shift).sum(-1, dtype=torch.int32)
    v = (v << 3) | ((v >> 29) & 7)
    s = torch.zeros((rows, GP), dtype=d.dtype, device=d.device)
    s[:N, :G] = d
    s = s.reshape(rows // 16, 16, GP // 4, 4).permute(0, 2, 1, 3)
    return v.contiguous().view(torch.uint8).reshape(-1), s.reshape(-1).contiguous()


def _activations(gen, M, K, dtype, device):
    """N(0, 1) with one channel in a hundred ten times as large, as the inputs of a decoder's
    linears are; in a larger batch one row is a padded token of zeros."""
    x = torch.randn((M, K), generator=gen, device=device)
    x[:, torch.randperm(K, generator=gen, device=device)[: max(1, K // 100)]] *= 10.0
    if M >= 8:
        x[M // 2] = 0.0
    return x.to(dtype)


def prepare(case, seed):
    device = torch.device("cuda", 0)
    gen = torch.Generator(device=device)
    gen.manual_seed(seed)
    op, N, K = case["op"], case.get("N", 0), case["K"]
    s = {"op": op, "N": N, "out": DTYPES.get(case.get("out"))}
    if op == "quantize_w8":
        s["W"] = torch.randn((N, K), generator=gen, device=device).mul_(0.02)
        return s
    if op == "quantize_tokens":
        s["x"] = _activations(gen, case["M"], K, DTYPES[case["x"]], device)
        return s
    if op == "linear_w8a8":
        M = case["M"]
        s["codes"], s["d"] = _codes(torch.randn((N, K), generator=gen, device=device).mul_(0.02), 127)
        s["q"] = _tiles_w8(s["codes"])
        s["xq"], s["sx"] = _codes(_activations(gen, M, K, torch.bfloat16, device).float(), 127)
        return s
    E, M = case["E"], case["tokens"] * case["top"]
    # which expert is how busy differs with the seed; how busy the busiest is does not
    size = torch.tensor(_layout(case), device=device)[torch.randperm(E, generator=gen, device=device)]
    s["offsets"] = torch.cat([size.new_zeros(1), size.cumsum(0)]).to(torch.int32)
    s["most"] = max(_layout(case))
    x = _activations(gen, M, K, torch.bfloat16, device)
    if op == "grouped_linear":
        codes, scales, q, d = [], [], [], []
        for _ in range(E):
            c, t = _codes(torch.randn((N, K // GROUP, GROUP), generator=gen, device=device).mul_(0.02), 7)
            c, t = c.reshape(N, K), t.to(DTYPES[case["scales"]])
            native = _tiles_w4(c, t)
            codes.append(c), scales.append(t), q.append(native[0]), d.append(native[1])
        s["codes"], s["scales"], s["q"], s["d"] = (torch.stack(v) for v in (codes, scales, q, d))
        s["x"] = x
        return s
    codes, d = zip(*(_codes(torch.randn((N, K), generator=gen, device=device).mul_(0.02), 127) for _ in range(E)))
    s["codes"], s["d"] = torch.stack(codes), torch.stack(d)
    s["q"] = _tiles_w8(s["codes"])
    s["xq"], s["sx"] = _codes(x.float(), 127)
    return s


# ----------------------------------------------------------------------------
# one pass
# ----------------------------------------------------------------------------

def _by_expert(x, W, offsets, most):
    """Rows offsets[e] .. offsets[e + 1] - 1 of x (fp32) times W[e] transposed: every expert's rows
    padded to `most` of them, one product over the batch of experts."""
    at = offsets[:-1, None].long() + torch.arange(most, device=x.device)
    here = at < offsets[1:, None]
    rows = x[at.clamp(max=x.shape[0] - 1)] * here[..., None]
    y = torch.bmm(W, rows.transpose(1, 2).contiguous())
    m = torch.arange(x.shape[0], device=x.device)
    e = torch.searchsorted(offsets[1:].long(), m, right=True)
    return y[e, :, m - offsets.long()[e]]


def _plain(s):
    op = s["op"]
    if op == "quantize_w8":
        q, d = _codes(s["W"], 127)
        return _tiles_w8(q), d
    if op == "quantize_tokens":
        return _codes(s["x"].float(), 127)
    if op == "linear_w8a8":
        y = s["xq"].float() @ s["codes"].float().t()
        return (y * s["sx"][:, None] * s["d"]).to(s["out"])
    if op == "grouped_linear":
        c = s["codes"]
        W = (c.reshape(c.shape[0], c.shape[1], -1, GROUP).float() * s["scales"].float()[..., None]).reshape(c.shape)
        return _by_expert(s["x"].float(), W, s["offsets"], s["most"]).to(s["out"])
    y = _by_expert(s["xq"].float() * s["sx"][:, None], s["codes"].float() * s["d"][..., None], s["offsets"], s["most"])
    return y.to(s["out"])


def run(s):
    if not own:
        return _plain(s)
    import bit_group_quantized_w4_amd as w4

    op = s["op"]
    if op == "quantize_w8":
        return w4.quantize_w8(s["W"])
    if op == "quantize_tokens":
        return w4.quantize_tokens(s["x"])
    if op == "linear_w8a8":
        return w4.linear_w8a8(s["xq"], s["sx"], s["q"], s["d"], s["N"], out_dtype=s["out"])
    if op == "grouped_linear":
        return w4.grouped_linear(s["x"], s["offsets"], s["q"], s["d"], s["N"], out_dtype=s["out"])
    return w4.grouped_linear_w8a8(s["xq"], s["sx"], s["offsets"], s["q"], s["d"], s["N"], out_dtype=s["out"])


# ----------------------------------------------------------------------------
# the definitions in 64 bits
# ----------------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    op = s["op"]
    if op in ("quantize_w8", "quantize_tokens"):
        # the scale of a row; its codes are whole numbers with one right value each
        v = s["W"] if op == "quantize_w8" else s["x"]
        return None, v.double().abs().max(dim=1).values / 127.0
    if op == "linear_w8a8":
        left = s["xq"].double() * s["sx"].double()[:, None]
        y = torch.empty((left.shape[0], s["N"]), dtype=torch.float64, device=left.device)
        for n in range(0, s["N"], 4096):
            right = s["codes"][n:n + 4096].double() * s["d"][n:n + 4096].double()[:, None]
            y[:, n:n + 4096] = left @ right.t().contiguous()
        return y
    ends = s["offsets"].tolist()
    left = s["x"].double() if op == "grouped_linear" else s["xq"].double() * s["sx"].double()[:, None]
    y = torch.empty((left.shape[0], s["N"]), dtype=torch.float64, device=left.device)
    for e in range(case["E"]):
        a, b = ends[e], ends[e + 1]
        if a == b:
            continue
        right = s["codes"][e].double()
        if op == "grouped_linear":
            right *= s["scales"][e].double().repeat_interleave(GROUP, dim=1)
        else:
            right *= s["d"][e].double()[:, None]
        y[a:b] = left[a:b] @ right.t().contiguous()
    return y
