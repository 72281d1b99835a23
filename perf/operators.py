"""Measured cases of three operators: rows of microscaled 4-bit floating point (quantised and read
back), their product, and attention with capped scores, distance bias and masks.

Every case can be run in two ways on the same inputs: in a plain form of elementary torch operations
in 32 bits or more (own = False), and through this repository's package (own = True).

4-bit formats.  Elements are e2m1 (0, 0.5, 1, 1.5, 2, 3, 4, 6 and their negatives), two to a byte, the
even column in the low half.  "mxfp4": one power-of-two scale for 32 columns, 2^(floor(log2 amax) - 2),
stored as its exponent + 127.  "nvfp4": one e4m3 scale for 16 columns, amax / (6 r) rounded to nearest
even, with one power of two r for the row, the smallest with amax_row <= 448 * 6 * r.  Block scales are
stored in tiles of 128 rows x 4 blocks, 512 bytes each: row i, block j of a tile at (i % 32) * 16 +
(i // 32) * 4 + j, tiles row-major, zero scales outside the matrix.
"""
import math

import torch

own = False

HEAD = 128


# ---------------------------------------------------------------- cases

def listed():
    return [
        # a prompt's text features on their way into a 4-bit projection: latency
        {"name": "rows of a prompt", "op": "rows", "fmt": "nvfp4", "rows": 32, "cols": 2560, "fp32": False},
        # the normalised activations of one 1024 x 1024 image with its text, before the QKV projection
        {"name": "rows of activations", "op": "rows", "fmt": "nvfp4", "rows": 4128, "cols": 3840, "fp32": False},
        # the fused gate and up weight, packed once when a model is loaded
        {"name": "rows of a weight", "op": "rows", "fmt": "mxfp4", "rows": 20480, "cols": 3840, "fp32": False},
        # an odd batch of the wider inner activations, kept in 32 bits
        {"name": "rows in 32 bits", "op": "rows", "fmt": "mxfp4", "rows": 1037, "cols": 10240, "fp32": True},
        # one row through an output projection: bound by reading the weight
        {"name": "product of one row", "op": "product", "fmt": "nvfp4", "m": 1, "n": 3840, "k": 3840},
        # a prompt's rows through the QKV projection of a text refiner
        {"name": "product of a prompt", "op": "product", "fmt": "mxfp4", "m": 77, "n": 11520, "k": 3840},
        # ragged in every direction: rows, columns and the last block of the inner axis
        {"name": "product, ragged", "op": "product", "fmt": "nvfp4", "m": 1153, "n": 3848, "k": 2592},
        # the gate and up projection of one 1024 x 1024 image with its text
        {"name": "product of an image", "op": "product", "fmt": "nvfp4", "m": 4128, "n": 20480, "k": 3840},
        # single tokens over a long stream kept from earlier, one of two elements shorter
        {"name": "attention of one token", "op": "attention", "batch": 2, "heads": 30, "kv_heads": 30, "q_len": 1,
         "kv_len": 16896, "cap": 0.0, "bias": True, "mask": "lengths"},
        # a causal stream behind a prefix that all may see, shared key heads, capped scores, odd lengths
        {"name": "attention behind a prefix", "op": "attention", "batch": 2, "heads": 30, "kv_heads": 6, "q_len": 1037,
         "kv_len": 1291, "cap": 30.0, "bias": False, "mask": "prefix"},
        # several images and their texts packed into one stream, each with its own
        {"name": "attention of a pack", "op": "attention", "batch": 1, "heads": 30, "kv_heads": 30, "q_len": 4224,
         "kv_len": 4224, "cap": 0.0, "bias": False, "mask": "documents"},
        # the stream of a 2048 x 2048 image with its text, capped scores and a bias that falls with distance
        {"name": "attention of a large image", "op": "attention", "batch": 1, "heads": 30, "kv_heads": 30,
         "q_len": 16896, "kv_len": 16896, "cap": 30.0, "bias": True, "mask": "none"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rows", "product", "attention", "attention"])
    fmt = rng.choice(["mxfp4", "nvfp4"])
    if op == "rows":
        return {"op": op, "fmt": fmt, "rows": _log(rng, 1, 17000), "cols": 32 * _log(rng, 1, 320),
                "fp32": rng.random() < 0.4}
    if op == "product":
        return {"op": op, "fmt": fmt, "m": _log(rng, 1, 4128), "n": 8 * _log(rng, 1, 2560), "k": 32 * _log(rng, 1, 120)}
    mask = rng.choice(["none", "lengths", "prefix", "causal", "documents"])
    kv_heads = rng.choice([1, 2, 3, 5, 6])
    heads = kv_heads * rng.choice([1, 2, 5])
    kv_len = _log(rng, 1, 16896)
    if mask == "documents":
        q_len = kv_len = max(kv_len, 64)
    elif rng.random() < 0.3:
        q_len = min(kv_len, rng.randint(1, 4))
    else:
        q_len = _log(rng, 1, kv_len)
    batch = rng.choice([1, 2, 3])
    if batch * heads * q_len * kv_len > 30 * 16896 ** 2:
        batch = 1
    return {"op": op, "batch": batch, "heads": heads, "kv_heads": kv_heads, "q_len": q_len,
            "kv_len": kv_len, "cap": rng.choice([0.0, 15.0, 30.0, 50.0]), "bias": rng.random() < 0.5, "mask": mask}


def _lengths(case):
    """Keys of each batch element."""
    n, full = case["batch"], case["kv_len"]
    if case["mask"] == "lengths":
        return [full - (b * full) // (2 * n) for b in range(n)]
    return [full] * n


def _prefixes(case):
    return [(case["kv_len"] * (b + 1)) // (2 * case["batch"] + 3) for b in range(case["batch"])]


def _documents(case):
    """Sizes of the packed documents: (image tokens, text tokens) of each.  The images stand first in the
    stream, the texts behind them, and the last few rows are padding that sees nothing."""
    total = case["kv_len"]
    pad = total // 64
    docs = max(1, min(5, total // 400 + 1))
    text = max(1, min(77, total // (8 * docs)))
    image = total - pad - docs * text
    weights = [d + 2 for d in range(docs)]
    sizes = [image * w // sum(weights) for w in weights]
    sizes[-1] += image - sum(sizes)
    return [(s, text) for s in sizes], pad


def _document_ids(case):
    docs, pad = _documents(case)
    ids = [d for d, (image, _) in enumerate(docs) for _ in range(image)]
    ids += [d for d, (_, text) in enumerate(docs) for _ in range(text)]
    return ids + [-1] * pad


def _pairs(case):
    """Pairs of a query and a key that it sees, over the batch, for one head."""
    q = case["q_len"]
    if case["mask"] == "documents":
        return case["batch"] * sum((i + t) ** 2 for i, t in _documents(case)[0])
    total = 0
    for b, n in enumerate(_lengths(case)):
        if case["mask"] in ("prefix", "causal"):
            prefix = min(n, _prefixes(case)[b]) if case["mask"] == "prefix" else 0
            first = n - q + 1  # keys that the first query sees by its place
            total += sum(max(prefix, max(0, first + i)) for i in range(q))
        else:
            total += q * n
    return total


def work(case):
    if case["op"] == "rows":
        n, block = case["rows"] * case["cols"], 32 if case["fmt"] == "mxfp4" else 16
        row = 0 if case["fmt"] == "mxfp4" else 4 * case["rows"]
        # read, stored as codes and scales, and read back into 16-bit values
        return {"bytes": n * (4 if case["fp32"] else 2) + 2 * (n // 2 + n // block + row) + 2 * n, "flops": 4 * n}
    if case["op"] == "product":
        m, n, k = case["m"], case["n"], case["k"]
        block, row = (32, 0) if case["fmt"] == "mxfp4" else (16, 4)
        return {"bytes": (m + n) * (k // 2 + k // block + row) + 2 * m * n, "flops": 2 * m * n * k}
    keys = sum(_lengths(case))
    elements = 2 * case["heads"] * case["batch"] * case["q_len"] + 2 * case["kv_heads"] * keys
    return {"bytes": 2 * HEAD * elements, "flops": 4 * HEAD * case["heads"] * _pairs(case)}


# ---------------------------------------------------------------- 4-bit rows, plain form

def _e2m1_code(v):
    """Codes of v >= 0 to the nearest of 0, 0.5, 1, 1.5, 2, 3, 4, 6; a tie goes to the even code."""
    code = (v > 0.25).to(torch.uint8)
    code += v >= 0.75
    code += v > 1.25
    code += v >= 1.75
    code += v > 2.5
    code += v >= 3.5
    code += v > 5.0
    return code


def _e4m3_near(v):
    """v >= 0 to the nearest e4m3 value, ties to even, at most 448."""
    exponent = torch.frexp(v)[1] - 1
    step = torch.exp2(exponent.clamp(min=-6).double() - 3)
    return (torch.round(v / step) * step).clamp(max=448.0)


def _quantise(fmt, x):
    """Codes [rows, cols] (sign in bit 3), block scales [rows, blocks] and row scales [rows] as the
    numbers they stand for, in 64 bits: whether a value lies above or below a border has to be exact."""
    rows, cols = x.shape
    block = 32 if fmt == "mxfp4" else 16
    parts = x.double().reshape(rows, cols // block, block)
    amax = parts.abs().amax(2)
    if fmt == "mxfp4":
        row = torch.ones(rows, dtype=torch.float64, device=x.device)
        exponent = (torch.frexp(amax)[1] - 3).clamp(-127, 127)
        scale = torch.where(amax > 0, torch.exp2(exponent.double()), torch.ones_like(amax))
    else:
        part, exponent = torch.frexp(amax.amax(1))  # amax = part * 2^exponent; 2688 = 0.65625 * 2^12
        row = torch.exp2((exponent - 12 + (part > 0.65625).int()).clamp(min=-126).double())
        row = torch.where(part > 0, row, torch.ones_like(row))
        scale = _e4m3_near(amax / (6 * row[:, None]))
    unit = scale * row[:, None]
    code = _e2m1_code(parts.abs() / torch.where(unit > 0, unit, torch.full_like(unit, math.inf))[..., None])
    code += 8 * torch.signbit(parts).to(torch.uint8)
    return code.reshape(rows, cols), scale, row


def _tile_scales(fmt, scale):
    """Block scales as bytes in their stored layout."""
    rows, blocks = scale.shape
    if fmt == "mxfp4":
        stored = (torch.frexp(scale)[1] - 1 + 127).to(torch.uint8)
    else:
        stored = scale.to(torch.float8_e4m3fn).view(torch.uint8)
    tiles_r, tiles_b = -(-rows // 128), -(-blocks // 4)
    full = torch.zeros((tiles_r * 128, tiles_b * 4), dtype=torch.uint8, device=scale.device)
    full[:rows, :blocks] = stored
    return full.reshape(tiles_r, 4, 32, tiles_b, 4).permute(0, 3, 2, 1, 4).contiguous().reshape(-1)


def _packed(fmt, x):
    """The 4-bit matrix of x as a user's program keeps it: packed codes, tiled block scales, row scales."""
    code, scale, row = _quantise(fmt, x)
    packed = code[:, 0::2] | (code[:, 1::2] << 4)
    return packed.contiguous(), _tile_scales(fmt, scale), row.float() if fmt == "nvfp4" else None


def _values(fmt, packed, tiled, row):
    """The numbers that a packed matrix stands for, in 32 bits."""
    rows, cols = packed.shape[0], 2 * packed.shape[1]
    block = 32 if fmt == "mxfp4" else 16
    blocks = cols // block
    code = torch.stack((packed & 15, packed >> 4), 2).reshape(rows, cols)
    table = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6], device=packed.device)
    tiles_r, tiles_b = -(-rows // 128), -(-blocks // 4)
    stored = tiled.reshape(tiles_r, tiles_b, 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(tiles_r * 128, tiles_b * 4)
    stored = stored[:rows, :blocks].contiguous()
    if fmt == "mxfp4":
        scale = torch.exp2(stored.float() - 127)
    else:
        scale = stored.view(torch.float8_e4m3fn).float() * row[:, None]
    return (table[code.int()].reshape(rows, blocks, block) * scale[..., None]).reshape(rows, cols)


# ---------------------------------------------------------------- states

def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _rows(g, rows, cols):
    """Activations or weights: normal, each row with its own magnitude, a few columns far larger."""
    x = torch.randn((rows, cols), generator=g, device="cuda")
    x *= torch.exp(0.5 * torch.randn((rows, 1), generator=g, device="cuda"))
    x[:, ::97] *= 8.0
    return x


def prepare(case, seed):
    g = _generator(seed)
    if case["op"] == "rows":
        x = _rows(g, case["rows"], case["cols"])
        return {"case": case, "x": x if case["fp32"] else x.bfloat16()}
    if case["op"] == "product":
        a = _packed(case["fmt"], _rows(g, case["m"], case["k"]))
        b = _packed(case["fmt"], 0.02 * torch.randn((case["n"], case["k"]), generator=g, device="cuda"))
        return {"case": case, "a": a, "b": b}
    batch, heads, kv_heads = case["batch"], case["heads"], case["kv_heads"]
    # queries and keys as a QK-RMSNorm with gains leaves them; scores of a few units
    q = 3.0 * torch.randn((batch, case["q_len"], heads, HEAD), generator=g, device="cuda")
    k = torch.randn((batch, case["kv_len"], kv_heads, HEAD), generator=g, device="cuda")
    v = torch.randn((batch, case["kv_len"], kv_heads, HEAD), generator=g, device="cuda")
    state = {"case": case, "q": q.bfloat16(), "k": k.bfloat16(), "v": v.bfloat16(), "slopes": None, "lengths": None,
             "prefix": None, "documents": None}
    if case["bias"]:
        steps = torch.arange(1, heads + 1, device="cuda", dtype=torch.float32)
        state["slopes"] = torch.exp2(-8.0 * steps / heads)
    if case["mask"] == "lengths":
        state["lengths"] = torch.tensor(_lengths(case), dtype=torch.int32, device="cuda")
    if case["mask"] == "prefix":
        state["prefix"] = torch.tensor(_prefixes(case), dtype=torch.int32, device="cuda")
    if case["mask"] == "documents":
        ids = torch.tensor(_document_ids(case), dtype=torch.int32, device="cuda")
        state["documents"] = ids.expand(batch, -1).contiguous()
    return state


# ---------------------------------------------------------------- one pass

def _attention(case, q, k, v, slopes, lengths, prefix, documents):
    batch, n, heads, _ = q.shape
    m, kv_heads = k.shape[1], k.shape[2]
    group = heads // kv_heads
    # [batch, kv_heads, group * n, m]; the queries of a key head's group side by side
    qs = q.float().reshape(batch, n, kv_heads, group, HEAD).permute(0, 2, 3, 1, 4).reshape(batch, kv_heads, group * n,
                                                                                         HEAD)
    s = torch.matmul(qs * (1.0 / math.sqrt(HEAD)), k.float().permute(0, 2, 3, 1))
    if case["cap"]:
        s.div_(case["cap"]).tanh_().mul_(case["cap"])
    s = s.reshape(batch, heads, n, m)
    keys = torch.arange(m, device=q.device)
    count = torch.full((batch,), m, device=q.device) if lengths is None else lengths.long()
    places = torch.arange(n, device=q.device)[None, :] + (count[:, None] - n)  # [batch, n]
    if slopes is not None:
        distance = (places[:, :, None] - keys).abs().float()
        s.addcmul_(slopes[None, :, None, None], distance[:, None], value=-1.0)
    hidden = (keys >= count[:, None])[:, None, :]
    if case["mask"] in ("prefix", "causal"):
        later = keys > places[:, :, None]
        if prefix is not None:
            later &= (keys >= prefix.long()[:, None])[:, None, :]
        hidden = hidden | later
    if documents is not None:
        hidden = hidden | (documents[:, :, None] != documents[:, None, :]) | (documents < 0)[:, None, :]
    s.masked_fill_(hidden[:, None], -math.inf)
    top = s.amax(3, keepdim=True)
    s.sub_(torch.where(top > -math.inf, top, torch.zeros_like(top))).exp_()
    total = s.sum(3, keepdim=True)
    o = torch.matmul(s.reshape(batch, kv_heads, group * n, m), v.float().permute(0, 2, 1, 3))
    o = o.reshape(batch, heads, n, HEAD) / torch.where(total > 0, total, torch.ones_like(total))
    return o.permute(0, 2, 1, 3).bfloat16()


def run(state):
    case = state["case"]
    if own:
        from stream_diffusion_transformer_b200 import model
        if case["op"] == "rows":
            return model.dequantize_fp4(model.quantize_fp4(state["x"], case["fmt"]))
        if case["op"] == "product":
            return model.gemm_fp4(model.Fp4Matrix(case["fmt"], *state["a"]), model.Fp4Matrix(case["fmt"], *state["b"]))
        return model.attention_masked(state["q"], state["k"], state["v"], softcap=case["cap"], slopes=state["slopes"],
                                      causal=case["mask"] in ("prefix", "causal"), prefix_len=state["prefix"],
                                      kv_len=state["lengths"], q_doc=state["documents"], k_doc=state["documents"])
    if case["op"] == "rows":
        return _values(case["fmt"], *_packed(case["fmt"], state["x"])).bfloat16()
    if case["op"] == "product":
        a, b = _values(case["fmt"], *state["a"]), _values(case["fmt"], *state["b"])
        return torch.matmul(a, b.t()).bfloat16()
    return _attention(case, state["q"], state["k"], state["v"], state["slopes"], state["lengths"], state["prefix"],
                      state["documents"])


# ---------------------------------------------------------------- the definition in 64 bits

def _exact_rows(fmt, x):
    """Each value by the nearest point of its block's grid, written from the formats' definitions."""
    x = x.double()
    rows, cols = x.shape
    grid = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device=x.device)
    # all finite e4m3 values by their bits: 2^(e - 7) (1 + m / 8), or 2^-6 m / 8
    bits = torch.arange(127, device=x.device)
    e, m = (bits >> 3).double(), (bits & 7).double()
    fine = torch.where(e > 0, torch.exp2(e - 7) * (1 + m / 8), torch.exp2(torch.full_like(e, -6.0)) * m / 8)

    def nearest(points, v):
        """Index of the nearest point, the even one of two at the same distance."""
        hi = torch.searchsorted(points, v).clamp(1, len(points) - 1)
        lo = hi - 1
        below, above = v - points[lo], points[hi] - v
        return torch.where((below < above) | ((below == above) & (lo % 2 == 0)), lo, hi)

    out = torch.empty_like(x)
    block = 32 if fmt == "mxfp4" else 16
    for start in range(0, rows, 2048):
        part = x[start:start + 2048]
        blocks = part.reshape(part.shape[0], cols // block, block)
        amax = blocks.abs().amax(2)
        if fmt == "mxfp4":
            unit = torch.exp2((torch.floor(torch.log2(amax)) - 2).clamp(-127, 127))
            # log2 may be rounded across a power of two: 4 unit <= amax < 8 unit
            unit = torch.where((4 * unit > amax) & (unit > 2.0 ** -127), unit / 2, unit)
            unit = torch.where(8 * unit <= amax, unit * 2, unit)
            unit = torch.where(amax > 0, unit, torch.ones_like(unit))
        else:
            top = part.abs().amax(1)
            r = torch.exp2(torch.ceil(torch.log2(top / 2688)).clamp(min=-126))
            r = torch.where((r / 2 * 2688 >= top) & (r > 2.0 ** -126), r / 2, r)
            r = torch.where(r * 2688 < top, r * 2, r)
            r = torch.where(top > 0, r, torch.ones_like(r))
            unit = fine[nearest(fine, amax / (6 * r[:, None]))] * r[:, None]
        safe = torch.where(unit > 0, unit, torch.ones_like(unit))
        index = nearest(grid, blocks.abs() / safe[..., None])
        got = torch.where(unit[..., None] > 0, grid[index] * unit[..., None], torch.zeros_like(blocks))
        out[start:start + 2048] = torch.copysign(got, blocks).reshape(part.shape)
    return out


def _exact_values(fmt, packed, tiled, row):
    rows, width = packed.shape
    block = 32 if fmt == "mxfp4" else 16
    cols = 2 * width
    i = torch.arange(rows, device=packed.device)[:, None]
    j = torch.arange(cols, device=packed.device)[None, :]
    code = (packed[:, :, None].int() >> torch.tensor([0, 4], device=packed.device)) & 15
    code = code.reshape(rows, cols)
    tiles_b = -(-(cols // block) // 4)
    jb = j // block
    byte = tiled[((i // 128) * tiles_b + jb // 4) * 512 + (i % 32) * 16 + (i % 128) // 32 * 4 + jb % 4].long()
    e, m = (code & 7) >> 1, (code & 1).double()
    size = torch.where(e > 0, torch.exp2((e - 1).double()) * (1 + m / 2), m / 2)
    size = torch.where(code >= 8, -size, size)
    if fmt == "mxfp4":
        return size * torch.exp2((byte - 127).double())
    e, m = byte >> 3, (byte & 7).double()
    scale = torch.where(e > 0, torch.exp2((e - 7).double()) * (1 + m / 8), m * 2.0 ** -9)
    return size * scale * row.double()[:, None]


def _exact_attention(state):
    case = state["case"]
    q, k, v = state["q"], state["k"], state["v"]
    batch, n, heads, _ = q.shape
    m, group = k.shape[1], heads // k.shape[2]
    out = torch.zeros((batch, n, heads, HEAD), dtype=torch.float64, device=q.device)
    lengths, prefixes = _lengths(case), _prefixes(case)
    j = torch.arange(m, device=q.device)
    for b in range(batch):
        i = torch.arange(n, device=q.device)[:, None] + lengths[b] - n
        seen = (j < lengths[b]).expand(n, m)
        if case["mask"] == "causal":
            seen = seen & (j <= i)
        elif case["mask"] == "prefix":
            seen = seen & ((j <= i) | (j < prefixes[b]))
        elif case["mask"] == "documents":
            ids = torch.tensor(_document_ids(case), device=q.device)
            seen = (ids[:, None] == ids) & (ids >= 0)
        for h in range(heads):
            s = q[b, :, h].double() @ k[b, :, h // group].double().t() / HEAD ** 0.5
            if case["cap"]:
                s = case["cap"] * torch.tanh(s / case["cap"])
            if case["bias"]:
                s -= state["slopes"][h].double() * (i - j).abs()
            s = torch.where(seen, s, torch.full_like(s, -math.inf))
            p = torch.exp(s - s.amax(1, keepdim=True).clamp(min=-1e300))
            out[b, :, h] = (p @ v[b, :, h // group].double()) / p.sum(1, keepdim=True).clamp(min=1e-300)
    return out


def exact(case, seed):
    state = prepare(case, seed)
    if case["op"] == "rows":
        return _exact_rows(case["fmt"], state["x"])
    if case["op"] == "product":
        return _exact_values(case["fmt"], *state["a"]) @ _exact_values(case["fmt"], *state["b"]).t()
    return _exact_attention(state)
