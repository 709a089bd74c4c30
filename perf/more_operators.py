"""Cases of the microscaled 4-bit operators and of the way to the experts and back, for timing
and comparison.

Five operators, each through the public Python entry points of the package:

* ``quantize``: weights (``quantize_mx4``) or activations (``quantize_tokens_mx4``) to 4-bit floating
  point (E2M1) with one power-of-two scale (E8M0) per 32 inputs, and back to the values that the
  codes stand for (``dequantize_mx4``, ``dequantize_tokens_mx4``);
* ``linear_mx4``: the product of such activations with such weights;
* ``grouped_linear_mx4``: the same with rows sorted by expert;
* ``dispatch``: tokens sorted by expert (``expert_dispatch``), in training with the gradient;
* ``combine``: the experts' rows weighted and added up token by token (``expert_combine``), in training
  with the gradients of rows and weights.

``own = False`` computes them in elementary torch operations in fp32; ``own = True`` makes the
package's calls.  Weights are laid out once, in ``prepare``, as a program that serves a model keeps
them; the plain forms read the same codes in row-major order.
"""

import torch

own = False

BLOCK = 32  # inputs that share one scale

F32, BF16 = "f32", "bf16"
DTYPES = {F32: torch.float32, BF16: torch.bfloat16}


# ----------------------------------------------------------------------------
# cases
# ----------------------------------------------------------------------------

def listed():
    return [
        # loading a checkpoint: the largest matrix of a 70B-class layer, and what its codes stand for
        {"name": "weights 28672x8192", "op": "quantize", "what": "weights", "M": 28672, "K": 8192, "x": F32},
        # a long ragged prefill before a 70B-class down projection
        {"name": "tokens 4099x28672", "op": "quantize", "what": "tokens", "M": 4099, "K": 28672, "x": BF16},
        # decode of one token (4B-class up projection): the latency of one call
        {"name": "mx4 1 row 9216x2560", "op": "linear_mx4", "M": 1, "N": 9216, "K": 2560, "out": BF16},
        # verifying 12 drafted tokens with a 70B-class gate projection: bound by the weights
        {"name": "mx4 13 rows 28672x8192", "op": "linear_mx4", "M": 13, "N": 28672, "K": 8192, "out": BF16},
        # a batch of short prompts with an odd number of rows and outputs, kept in fp32 for a K-split layer
        {"name": "mx4 333 rows 2561x9216", "op": "linear_mx4", "M": 333, "N": 2561, "K": 9216, "out": F32},
        # prefill of 4096 tokens through a 27B-class gate projection: bound by the products
        {"name": "mx4 4096 rows 17408x5120", "op": "linear_mx4", "M": 4096, "N": 17408, "K": 5120, "out": BF16},
        # decode of 8 sequences, two experts of 64 each: few rows per expert, most experts idle
        {"name": "experts mx4 16 rows", "op": "grouped_linear_mx4", "tokens": 8, "top": 2, "E": 64, "skew": 0.5,
         "N": 2048, "K": 2560, "out": BF16},
        # prefill of 4095 tokens, two experts of 8 each, some twice as busy as others
        {"name": "experts mx4 8190 rows", "op": "grouped_linear_mx4", "tokens": 4095, "top": 2, "E": 8, "skew": 0.5,
         "N": 9216, "K": 2560, "out": BF16},
        # the same decode step's way to the experts and back: the latency of the calls
        {"name": "dispatch 8 tokens", "op": "dispatch", "tokens": 8, "top": 2, "E": 64, "skew": 0.5, "padded": 0,
         "K": 2560, "x": BF16, "train": False},
        # a training step's batch of 4095 tokens with eight experts of 128 each, 256 tokens of it padding
        {"name": "dispatch 4095 tokens, train", "op": "dispatch", "tokens": 4095, "top": 8, "E": 128, "skew": 0.5,
         "padded": 256, "K": 5120, "x": BF16, "train": True},
        {"name": "combine 8 tokens", "op": "combine", "tokens": 8, "top": 2, "E": 64, "skew": 0.5, "padded": 0,
         "K": 2560, "x": BF16, "weights": F32, "train": False},
        {"name": "combine 4095 tokens, train", "op": "combine", "tokens": 4095, "top": 8, "E": 128, "skew": 0.5,
         "padded": 256, "K": 5120, "x": BF16, "weights": F32, "train": True},
    ]


def _log(rng, lo, hi):
    return int(round(lo * (hi / lo) ** rng.random()))


def draw(rng):
    op = rng.choice(["quantize", "quantize", "linear_mx4", "linear_mx4", "linear_mx4", "grouped_linear_mx4",
                     "grouped_linear_mx4", "dispatch", "dispatch", "combine", "combine"])
    while True:
        K = 128 * _log(rng, 1, 224)
        N = _log(rng, 16, 28672)
        M = _log(rng, 1, 8192)
        if op == "quantize":
            what = rng.choice(["weights", "tokens"])
            rows = N if what == "weights" else M
            if rows * K <= (235_000_000 if what == "weights" else 117_000_000):
                return {"op": op, "what": what, "M": rows, "K": K, "x": rng.choice([BF16, F32])}
        elif op == "linear_mx4":
            if 200_000 <= N * K <= 235_000_000 and M * N * K <= 360_000_000_000:
                return {"op": op, "M": M, "N": N, "K": K, "out": rng.choice([BF16, F32])}
        elif op == "grouped_linear_mx4":
            E, top = _log(rng, 2, 128), rng.choice([1, 2, 4, 8])
            tokens, skew = max(1, M // top), rng.choice([0.0, 0.5, 1.0])
            # the plain form pads every expert to the busiest one's rows: keep what it computes below the largest case
            if top > E or not 200_000 <= E * N * K <= 300_000_000 or tokens * top * N * K > 190_000_000_000:
                continue
            if max(_sizes(tokens, top, E, skew)) * E * N * K <= 360_000_000_000:
                return {"op": op, "tokens": tokens, "top": top, "E": E, "skew": skew, "N": N, "K": K,
                        "out": rng.choice([BF16, F32])}
        else:
            E, top = _log(rng, 2, 512), rng.choice([1, 2, 3, 4, 6, 8])
            tokens, K = _log(rng, 1, 32768), _log(rng, 64, 8192)
            x = rng.choice([BF16, BF16, F32])
            if top > E or tokens * top * K * (4 if x == F32 else 2) > 335_000_000:
                continue
            c = {"op": op, "tokens": tokens, "top": top, "E": E, "skew": rng.choice([0.0, 0.5, 1.0]),
                 "padded": rng.choice([0, tokens // 16, tokens // 3]), "K": K, "x": x, "train": rng.random() < 0.5}
            if op == "combine":
                c["weights"] = rng.choice([F32, BF16])
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


def _mx_bytes(rows, K):
    return rows * K // 2 + rows * (K // BLOCK)


def work(case):
    op, K = case["op"], case["K"]
    wide = 4 if case.get("out") == F32 else 2
    if op == "quantize":
        # each value read, its code and its block's scale written, and the bf16 value they stand for
        M = case["M"]
        return {"bytes": (4 if case["x"] == F32 else 2) * M * K + _mx_bytes(M, K) + 2 * M * K, "flops": 2 * M * K}
    if op == "linear_mx4":
        M, N = case["M"], case["N"]
        return {"bytes": _mx_bytes(N, K) + _mx_bytes(M, K) + wide * M * N, "flops": 2 * M * N * K}
    tokens, top, E = case["tokens"], case["top"], case["E"]
    rows = tokens * top
    if op == "grouped_linear_mx4":
        N, busy = case["N"], sum(1 for s in _sizes(tokens, top, E, case["skew"]) if s)
        return {"bytes": busy * _mx_bytes(N, K) + _mx_bytes(rows, K) + wide * rows * N + 4 * (E + 1),
                "flops": 2 * rows * N * K}
    es, real = (4 if case["x"] == F32 else 2), (tokens - case["padded"]) * top
    if op == "dispatch":
        once = es * tokens * K + es * rows * K  # one side read, the other written
        ids = 8 * rows + 4 * (E + 1) + 8 * rows  # the experts read; offsets, places and order written
        back = es * real * K + es * tokens * K if case["train"] else 0
        return {"bytes": once + ids + back, "flops": (real * K if case["train"] else 0)}
    weights = (4 if case["weights"] == F32 else 2) * rows
    forward = es * real * K + weights + 4 * rows + es * tokens * K
    back = es * tokens * K + es * real * K + weights + 4 * rows + es * rows * K + weights if case["train"] else 0
    return {"bytes": forward + back, "flops": (6 if case["train"] else 2) * real * K}


# ----------------------------------------------------------------------------
# inputs
# ----------------------------------------------------------------------------

def _encode(v):
    """Codes [.., K / 2] (the even input in the low four bits) and scales [.., K / 32] of v (fp32 [.., K]):
    a block's scale is 2^(floor(log2 max|v|) - 2), its codes the nearest E2M1 of v / scale, ties to the even
    code, +-6 beyond it.  Ascending codes 0 .. 7 stand for 0, 0.5, 1, 1.5, 2, 3, 4, 6; 8 more for the sign."""
    v = v.reshape(v.shape[:-1] + (v.shape[-1] // BLOCK, BLOCK))
    most = v.abs().amax(-1)
    fine = most < float("inf")
    e = torch.frexp(torch.where(fine, most, torch.ones_like(most)))[1] - 3
    e = torch.where(most > 0, e, torch.full_like(e, -127)).clamp_(-127, 127)
    scale = torch.where(fine, e + 127, torch.full_like(e, 255)).to(torch.uint8)
    # (by two powers of two, each in range)
    a = torch.ldexp(torch.ldexp(v, -(e // 2)[..., None]), (e // 2 - e)[..., None])
    sign = torch.signbit(a)
    a = a.abs()
    code = torch.zeros_like(a, dtype=torch.uint8)
    for tie, even in ((0.25, 0), (0.75, 1), (1.25, 0), (1.75, 1), (2.5, 0), (3.5, 1), (5.0, 0)):
        code += a >= tie if even else a > tie  # a tie goes up where the upper code is the even one
    code += sign.to(torch.uint8) * 8
    code = torch.where(fine[..., None], code, torch.zeros_like(code)).reshape(v.shape[:-2] + (-1,))
    return code[..., 0::2] | (code[..., 1::2] << 4), scale


def _decode(codes, scales, dtype=torch.float32):
    """The values [.., K] that codes and scales stand for."""
    c = torch.stack((codes & 15, codes >> 4), -1).reshape(codes.shape[:-1] + (-1, BLOCK))
    m = (c & 7).to(dtype)
    # 0 and 0.5; then 1 and 1.5 times a power of two
    m = torch.where(m < 2, m * 0.5, (1 + 0.5 * (c & 1).to(dtype)) * (1 << ((c & 7) >> 1).clamp(min=1).to(torch.int32)).to(dtype) * 0.5)
    m = torch.where(c >= 8, -m, m)
    s = scales.to(torch.int32) - 127
    f = torch.ldexp(torch.ones((), dtype=dtype, device=codes.device), s // 2)
    g = torch.ldexp(torch.ones((), dtype=dtype, device=codes.device), s - s // 2)
    f = torch.where(scales == 255, torch.full_like(f, float("nan")), f)
    return (m * f[..., None] * g[..., None]).reshape(codes.shape[:-1] + (-1,))


def _pad_rows(q, rows):
    return q if q.shape[-2] == rows else torch.cat([q, q.new_zeros(q.shape[:-2] + (rows - q.shape[-2], q.shape[-1]))], -2)


def _native(codes, scales):
    """Codes [.., N, K / 2] as tiles of 16 rows x 64 bytes, two for every 256 inputs: lane L of the two holds row
    L % 16, inputs 64 (L // 16) .. + 63, a block of 32 in each.  Scales [.., N, K / 32] as four bytes for each lane
    and 512 inputs, in the order of its blocks.  Zeros past the last row and input."""
    N, lead = codes.shape[-2], codes.shape[:-2]
    rows, n = (N + 15) // 16 * 16, codes.dim() - 2
    pad = torch.nn.functional.pad
    q = _pad_rows(codes, rows)
    q = pad(q, (0, -q.shape[-1] % 128))
    q = q.reshape(lead + (rows // 16, 16, q.shape[-1] // 128, 4, 2, 16))  # row, 256 inputs, quarter, block, byte
    q = q.permute(tuple(range(n)) + (n, n + 2, n + 4, n + 3, n + 1, n + 5)).reshape(lead + (-1,)).contiguous()
    s = _pad_rows(scales, rows)
    s = pad(s, (0, -s.shape[-1] % 16))
    s = s.reshape(lead + (rows // 16, 16, s.shape[-1] // 16, 2, 4, 2))  # row, 512 inputs, half, quarter, block
    s = s.permute(tuple(range(n)) + (n, n + 2, n + 4, n + 1, n + 3, n + 5)).reshape(lead + (-1,)).contiguous()
    return q, s


def _activations(gen, M, K, device):
    """N(0, 1) with one channel in a hundred ten times as large, as the inputs of a decoder's
    linears are; in a larger batch one row is a padded token of zeros."""
    x = torch.randn((M, K), generator=gen, device=device)
    x[:, torch.randperm(K, generator=gen, device=device)[: max(1, K // 100)]] *= 10.0
    if M >= 8:
        x[M // 2] = 0.0
    return x


def _experts(gen, case, device):
    """Each token's experts, int64 [tokens, top]: no expert twice, drawn by a popularity that falls as
    rank^-skew; a padded token's are -1."""
    T, E = case["tokens"], case["E"]
    share = torch.arange(1, E + 1, device=device, dtype=torch.float32).log() * -case["skew"]
    share = share[torch.randperm(E, generator=gen, device=device)]
    noise = torch.rand((T, E), generator=gen, device=device).clamp_(1e-9, 1 - 1e-7)
    ids = (share - (-noise.log()).log()).topk(case["top"], dim=1).indices
    if case["padded"]:
        ids[T - case["padded"]:] = -1
    return ids.contiguous()


def _sorted(ids, E):
    """(offsets [E + 1], place [tokens, top], order [tokens * top]) of the slots sorted by expert, those of
    one expert in their own order; slots of no expert have no row (-1)."""
    flat = ids.reshape(-1)
    key = torch.where((flat >= 0) & (flat < E), flat, torch.full_like(flat, E))
    key, order = torch.sort(key, stable=True)
    offsets = torch.searchsorted(key, torch.arange(E + 1, device=ids.device))
    place = torch.empty_like(order)
    place[order] = torch.arange(order.numel(), device=ids.device)
    none = torch.full_like(order, -1)
    place = torch.where(place < offsets[E], place, none).reshape(ids.shape)
    order = torch.where(key < E, order, none)
    return offsets.to(torch.int32), place.to(torch.int32), order.to(torch.int32)


def prepare(case, seed):
    device = torch.device("cuda", 0)
    gen = torch.Generator(device=device)
    gen.manual_seed(seed)
    op, N, K = case["op"], case.get("N", 0), case["K"]
    s = {"op": op, "N": N, "K": K, "out": DTYPES.get(case.get("out")), "train": case.get("train", False)}
    if op == "quantize":
        s["what"] = case["what"]
        if case["what"] == "weights":
            x = torch.randn((case["M"], K), generator=gen, device=device).mul_(0.02)
        else:
            x = _activations(gen, case["M"], K, device)
        s["x"] = x.to(DTYPES[case["x"]])
        return s
    if op == "linear_mx4":
        s["codes"], s["scales"] = _encode(torch.randn((N, K), generator=gen, device=device).mul_(0.02))
        s["q"], s["s"] = _native(s["codes"], s["scales"])
        s["xq"], s["xs"] = _encode(_activations(gen, case["M"], K, device).bfloat16().float())
        return s
    tokens, top, E = case["tokens"], case["top"], case["E"]
    if op == "grouped_linear_mx4":
        # which expert is how busy differs with the seed; how busy the busiest is does not
        size = torch.tensor(_sizes(tokens, top, E, case["skew"]), device=device)
        s["most"] = int(size.max())
        size = size[torch.randperm(E, generator=gen, device=device)]
        s["offsets"] = torch.cat([size.new_zeros(1), size.cumsum(0)]).to(torch.int32)
        made = [_encode(torch.randn((N, K), generator=gen, device=device).mul_(0.02)) for _ in range(E)]
        s["codes"], s["scales"] = (torch.stack(v) for v in zip(*made))
        s["q"], s["s"] = _native(s["codes"], s["scales"])
        s["xq"], s["xs"] = _encode(_activations(gen, tokens * top, K, device).bfloat16().float())
        return s
    dtype = DTYPES[case["x"]]
    s["E"], s["ids"] = E, _experts(gen, case, device)
    if op == "dispatch":
        s["x"] = _activations(gen, tokens, K, device).to(dtype).requires_grad_(case["train"])
        if case["train"]:
            s["grad"] = torch.randn((tokens * top, K), generator=gen, device=device).to(dtype)
        return s
    # the experts' outputs (rows of no expert hold nothing that may matter) and a router's weights
    s["offsets"], s["place"], s["order"] = _sorted(s["ids"], E)
    y = torch.randn((tokens * top, K), generator=gen, device=device).to(dtype)
    y[int(s["offsets"][E]):] = float("nan")
    w = torch.softmax(torch.randn((tokens, top), generator=gen, device=device), 1).to(DTYPES[case["weights"]])
    s["y"], s["w"] = y.requires_grad_(case["train"]), w.requires_grad_(case["train"])
    if case["train"]:
        s["grad"] = torch.randn((tokens, K), generator=gen, device=device).to(dtype)
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


def _take(x, order, top):
    """Row r is the row of x of slot order[r]; zeros where there is none."""
    rows = x[(order.long() // top).clamp(min=0)]
    return torch.where((order >= 0)[:, None], rows, torch.zeros_like(rows))


def _put(rows, place):
    """[tokens, top, K] in fp32: each slot's row, zeros where it has none."""
    there = (place >= 0)[..., None]
    got = rows.float()[place.long().clamp(min=0)]
    return torch.where(there, got, torch.zeros_like(got))


def _plain(s):
    op = s["op"]
    if op == "quantize":
        return _decode(*_encode(s["x"].float())).to(torch.bfloat16)
    if op == "linear_mx4":
        return (_decode(s["xq"], s["xs"]) @ _decode(s["codes"], s["scales"]).t()).to(s["out"])
    if op == "grouped_linear_mx4":
        return _by_expert(_decode(s["xq"], s["xs"]), _decode(s["codes"], s["scales"]), s["offsets"], s["most"]).to(s["out"])
    if op == "dispatch":
        x, top = s["x"].detach(), s["ids"].shape[1]
        offsets, place, order = _sorted(s["ids"], s["E"])
        out = [offsets, place, order, _take(x, order, top)]
        if s["train"]:
            out.append(_put(s["grad"], place).sum(1).to(x.dtype))
        return out
    y, w, place = s["y"].detach(), s["w"].detach(), s["place"]
    rows = _put(y, place)
    out = [(rows * w.float()[..., None]).sum(1).to(y.dtype)]
    if s["train"]:
        grad = s["grad"].float()
        dy = torch.zeros(y.shape, device=y.device)
        there = place >= 0
        dy[place[there].long()] = (w.float()[..., None] * grad[:, None])[there]
        out += [dy.to(y.dtype), (rows * grad[:, None]).sum(-1).to(w.dtype)]
    return out


def run(s):
    if not own:
        return _plain(s)
    import bit_group_quantized_w4_amd as w4

    op = s["op"]
    if op == "quantize":
        if s["what"] == "weights":
            q, d = w4.quantize_mx4(s["x"])
            return w4.dequantize_mx4(q, d, s["x"].shape[0], s["K"])
        return w4.dequantize_tokens_mx4(*w4.quantize_tokens_mx4(s["x"]))
    if op == "linear_mx4":
        return w4.linear_mx4(s["xq"], s["xs"], s["q"], s["s"], s["N"], out_dtype=s["out"])
    if op == "grouped_linear_mx4":
        return w4.grouped_linear_mx4(s["xq"], s["xs"], s["offsets"], s["q"], s["s"], s["N"], out_dtype=s["out"])
    if op == "dispatch":
        xs, rows = w4.expert_dispatch(s["x"], s["ids"], s["E"])
        out = [rows.offsets, rows.place, rows.order, xs.detach()]
        if s["train"]:
            out.append(torch.autograd.grad(xs, s["x"], s["grad"])[0])
        return out
    y = w4.expert_combine(s["y"], s["w"], w4.ExpertRows(s["offsets"], s["place"], s["order"]))
    out = [y.detach()]
    if s["train"]:
        out += torch.autograd.grad(y, (s["y"], s["w"]), s["grad"])
    return out


# ----------------------------------------------------------------------------
# the definitions in 64 bits
# ----------------------------------------------------------------------------

_GRID = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _values(codes, scales):
    """What codes and scales stand for, by the table of E2M1 and exp2."""
    grid = torch.tensor(_GRID + tuple(-g for g in _GRID), dtype=torch.float64, device=codes.device)
    v = torch.empty(codes.shape[:-1] + (codes.shape[-1], 2), dtype=torch.float64, device=codes.device)
    v[..., 0] = grid[(codes % 16).int()]
    v[..., 1] = grid[torch.div(codes, 16, rounding_mode="floor").int()]
    d = torch.exp2(scales.double() - 127)
    return v.reshape(codes.shape[:-1] + (-1,)) * d.repeat_interleave(BLOCK, dim=-1)


def exact(case, seed):
    s = prepare(case, seed)
    op = s["op"]
    if op == "quantize":
        grid = torch.tensor(_GRID, dtype=torch.float64, device=s["x"].device)
        out = torch.empty(s["x"].shape, dtype=torch.float64, device=s["x"].device)
        for r in range(0, out.shape[0], 512):
            v = s["x"][r:r + 512].double()
            v = v.reshape(v.shape[0], -1, BLOCK)
            most = v.abs().amax(-1, keepdim=True)
            # the power of two at or below the largest member, by comparison with the candidate above it
            e = torch.floor(torch.log2(torch.where(most > 0, most, torch.ones_like(most))))
            e = torch.where(torch.exp2(e) > most, e - 1, e)
            e = torch.where(torch.exp2(e + 1) <= most, e + 1, e)
            d = torch.exp2((e - 2).clamp(-127, 127))
            a = (v / d).abs().clamp(max=6.0)
            up = torch.bucketize(a, grid).clamp(max=7)  # the first member of the grid that is not below
            lo = (up - 1).clamp(min=0)
            below, above = a - grid[lo], grid[up] - a
            near = torch.where((below < above) | ((below == above) & (lo % 2 == 0)), lo, up)
            out[r:r + 512] = (torch.copysign(grid[near], v) * d).reshape(v.shape[0], -1)
        return out
    if op in ("linear_mx4", "grouped_linear_mx4"):
        x = _values(s["xq"], s["xs"])
        y = torch.empty((x.shape[0], s["N"]), dtype=torch.float64, device=x.device)
        if op == "linear_mx4":
            for n in range(0, s["N"], 4096):
                y[:, n:n + 4096] = x @ _values(s["codes"][n:n + 4096], s["scales"][n:n + 4096]).t().contiguous()
            return y
        ends = s["offsets"].tolist()
        for e in range(case["E"]):
            if ends[e] < ends[e + 1]:
                y[ends[e]:ends[e + 1]] = x[ends[e]:ends[e + 1]] @ _values(s["codes"][e], s["scales"][e]).t().contiguous()
        return y
    T, top = s["ids"].shape
    if op == "dispatch":
        x, out = s["x"].detach().double(), [None, None, None]
        ids = s["ids"].reshape(-1)
        slots = torch.cat([torch.nonzero(ids == e).reshape(-1) for e in range(case["E"])])
        xs = torch.zeros((T * top, case["K"]), dtype=torch.float64, device=x.device)
        xs[:slots.numel()] = x[torch.div(slots, top, rounding_mode="floor")]
        out.append(xs)
        if case["train"]:
            g = torch.zeros_like(xs)
            g[slots] = s["grad"][:slots.numel()].double()
            out.append(g.reshape(T, top, -1).sum(1))
        return out
    order = s["order"][s["order"] >= 0].long()
    y, w = s["y"].detach()[:order.numel()].double(), s["w"].detach().double().reshape(-1)[order]
    token = torch.div(order, top, rounding_mode="floor")
    out = [torch.zeros((T, case["K"]), dtype=torch.float64, device=y.device).index_add_(0, token, y * w[:, None])]
    if case["train"]:
        g = s["grad"].double()
        dy = torch.zeros((T * top, case["K"]), dtype=torch.float64, device=y.device)
        dy[:order.numel()] = w[:, None] * g[token]
        dw = torch.zeros(T * top, dtype=torch.float64, device=y.device)
        dw[order] = (y * g[token]).sum(-1)
        out += [dy, dw.reshape(T, top)]
    return out
