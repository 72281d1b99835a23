"""Microscaled 4-bit floating point in plain NumPy fp64: the statement that the library's 4-bit rows
and their product are held to.

Elements are e2m1: 0, 0.5, 1, 1.5, 2, 3, 4, 6 and their negatives (code 0..7, sign in bit 3).
  MXFP4  32 columns share X = 2^(floor(log2 amax) - 2), at least 2^-127 (OCP microscaling's conversion);
         a block of zeros takes X = 1.  Stored as the exponent + 127.
  NVFP4  a row has r, the smallest power of two with amax <= 448 * 6 * r, at least 2^-126 (1 for a row
         of zeros); 16 columns share S = e4m3(amax / (6 r)); elements are x / (S r).
Values round to the nearest code, ties to the even one, and saturate at 6.  A block with an infinity or
a NaN takes the NaN scale and zero codes (and does not count for r).
"""
import numpy as np

VALUES = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=np.float64)
# the 127 finite e4m3 values by their code: subnormal m 2^-9, else 2^(e-7) (1 + m/8)
E4M3 = np.array([m * 2.0 ** -9 if e == 0 else 2.0 ** (e - 7) * (1 + m / 8) for e in range(16) for m in range(8)])[:127]
BLOCK = {"mxfp4": 32, "nvfp4": 16}


def nearest_even(points, v):
    """Index of the point nearest to each v >= 0, the even index of two at the same distance; the last
    point for anything past it."""
    mid = (points[1:] + points[:-1]) / 2
    below = np.searchsorted(mid, v, side="left")   # a tie goes down ...
    above = np.searchsorted(mid, v, side="right")  # ... or up
    return np.where(below % 2 == 0, below, above)


def quantize(x, fmt):
    """codes [R, C] (0..15), stored block scales [R, C / block] (uint8), row scales [R] (fp64)."""
    x = np.asarray(x, dtype=np.float64)
    R, C = x.shape
    B = BLOCK[fmt]
    p = x.reshape(R, C // B, B)
    bad = ~np.isfinite(p).all(axis=2)
    p = np.where(bad[..., None], 0.0, p)
    amax = np.abs(p).max(axis=2)
    if fmt == "mxfp4":
        row = np.ones(R)
        e = np.clip(np.frexp(amax)[1] - 1 - 2, -127, 127)
        e = np.where(amax > 0, e, 0)
        stored = (e + 127).astype(np.uint8)
        unit = np.ldexp(1.0, e)
        stored[bad] = 255
    else:
        top = amax.max(axis=1)
        frac, e = np.frexp(top)  # top = frac 2^e, frac in [1/2, 1); 2688 = 0.65625 * 2^12
        row = np.ldexp(1.0, np.maximum(e - 12 + (frac > 0.65625), -126))
        row = np.where(top > 0, row, 1.0)
        stored = nearest_even(E4M3, amax / (6 * row[:, None])).astype(np.uint8)
        unit = E4M3[stored] * row[:, None]
        stored[bad] = 127
    safe = np.where(unit > 0, unit, 1.0)
    code = np.where(unit[..., None] > 0, nearest_even(VALUES, np.abs(p) / safe[..., None]), 0).astype(np.uint8)
    code |= np.where(np.signbit(p) & ~bad[..., None], 8, 0).astype(np.uint8)
    return code.reshape(R, C), stored, row


def dequantize(code, stored, row, fmt):
    """The values, fp64 (NaN where the block's scale is)."""
    R, C = code.shape
    v = np.where(code >= 8, -VALUES[code & 7], VALUES[code & 7])
    if fmt == "mxfp4":
        unit = np.ldexp(1.0, stored.astype(np.int64) - 127)
        unit[stored == 255] = np.nan
    else:
        unit = np.append(E4M3, np.nan)[stored] * np.asarray(row, dtype=np.float64)[:, None]
    return (v.reshape(R, -1, BLOCK[fmt]) * unit[..., None]).reshape(R, C)


def pack_codes(code):
    return (code[:, 0::2] | (code[:, 1::2] << 4)).astype(np.uint8)


def tile_scales(stored):
    """Block scales in the stored layout, written out index by index: tiles of 128 rows x 4 blocks, row i,
    block j of a tile at byte (i % 32) * 16 + (i // 32) * 4 + j; zeros outside the matrix."""
    R, nb = stored.shape
    ty, tx = -(-R // 128), -(-nb // 4)
    out = np.zeros(ty * tx * 512, dtype=np.uint8)
    i, j = np.meshgrid(np.arange(R), np.arange(nb), indexing="ij")
    out[((i // 128) * tx + j // 4) * 512 + (i % 32) * 16 + (i % 128) // 32 * 4 + j % 4] = stored
    return out


def rows_values(x, fmt):
    """What the rows of x stand for after a round trip through the format."""
    return dequantize(*quantize(x, fmt), fmt)


def fp4_linear(h, w, fmt):
    """h [M, K] @ w [N, K]^T with both operands in 4 bits."""
    return rows_values(h, fmt) @ rows_values(w, fmt).T


def block_forward(x, W, prefix, d, angles, c=None, fmt="nvfp4", all=False):
    """The block of zimage_ref.block_forward with the QKV and FFN w1|w3 projections in 4 bits (all=True: the
    output projection and FFN w2 as well); what goes into each is rounded to bf16 first, as the GPU holds it."""
    from . import zimage_ref as ref

    def lin(h, w, four=True):
        return fp4_linear(to_bf16(h), w, fmt) if four else ref.linear(h, w)

    S, D = x.shape
    if c is not None:
        scale_msa, gate_msa, scale_mlp, gate_mlp = ref.adaln(c, W, prefix)
    else:
        scale_msa = scale_mlp = 0.0
        gate_msa = gate_mlp = 1.0
    a, ff = f"{prefix}.attention", f"{prefix}.feed_forward"
    h = ref.rms_norm(x, W(f"{prefix}.attention_norm1.weight")) * (1.0 + scale_msa)
    q, k, v = (lin(h, W(f"{a}.{n}.weight")).reshape(S, d.heads, d.head_dim) for n in ("to_q", "to_k", "to_v"))
    q = ref.apply_rope(ref.rms_norm(q, W(f"{a}.norm_q.weight")), angles)
    k = ref.apply_rope(ref.rms_norm(k, W(f"{a}.norm_k.weight")), angles)
    o = lin(ref.attention(q, k, v).reshape(S, D), W(f"{a}.to_out.weight"), all)
    x1 = x + gate_msa * ref.rms_norm(o, W(f"{prefix}.attention_norm2.weight"))
    h2 = ref.rms_norm(x1, W(f"{prefix}.ffn_norm1.weight")) * (1.0 + scale_mlp)
    u = ref.silu(lin(h2, W(f"{ff}.w1.weight"))) * lin(h2, W(f"{ff}.w3.weight"))
    if u.shape[1] % 32 and all:
        pad = -u.shape[1] % 128  # zero columns, as the library pads them
        f = lin(np.pad(u, ((0, 0), (0, pad))), np.pad(W(f"{ff}.w2.weight"), ((0, 0), (0, pad))))
    else:
        f = lin(u, W(f"{ff}.w2.weight"), all)
    return x1 + gate_mlp * ref.rms_norm(f, W(f"{prefix}.ffn_norm2.weight"))


def block_forward_rows(x, W, prefix, d, angles, c, rows, fmt="nvfp4", all=False):
    """block_forward(x, ...)[rows] for the selected query rows only (keys and values from every row): every step but
    attention is per row, and so are the 4-bit formats.  ffn has to be a multiple of 32 (no padded columns)."""
    from . import zimage_ref as ref

    def lin(h, w, four=True):
        return fp4_linear(to_bf16(h), w, fmt) if four else ref.linear(h, w)

    S, D = x.shape
    n = len(rows)
    if c is not None:
        scale_msa, gate_msa, scale_mlp, gate_mlp = ref.adaln(c, W, prefix)
    else:
        scale_msa = scale_mlp = 0.0
        gate_msa = gate_mlp = 1.0
    a, ff = f"{prefix}.attention", f"{prefix}.feed_forward"
    h = ref.rms_norm(x, W(f"{prefix}.attention_norm1.weight")) * (1.0 + scale_msa)
    q = lin(h[rows], W(f"{a}.to_q.weight")).reshape(n, d.heads, d.head_dim)
    k, v = (lin(h, W(f"{a}.{nm}.weight")).reshape(S, d.heads, d.head_dim) for nm in ("to_k", "to_v"))
    q = ref.apply_rope(ref.rms_norm(q, W(f"{a}.norm_q.weight")), angles[rows])
    k = ref.apply_rope(ref.rms_norm(k, W(f"{a}.norm_k.weight")), angles)
    o = lin(ref.attention(q, k, v).reshape(n, D), W(f"{a}.to_out.weight"), all)
    x1 = x[rows] + gate_msa * ref.rms_norm(o, W(f"{prefix}.attention_norm2.weight"))
    h2 = ref.rms_norm(x1, W(f"{prefix}.ffn_norm1.weight")) * (1.0 + scale_mlp)
    u = ref.silu(lin(h2, W(f"{ff}.w1.weight"))) * lin(h2, W(f"{ff}.w3.weight"))
    f = lin(u, W(f"{ff}.w2.weight"), all)
    return x1 + gate_mlp * ref.rms_norm(f, W(f"{prefix}.ffn_norm2.weight"))


def to_bf16(x):
    """x rounded to bf16 (nearest even), as fp64."""
    u = np.asarray(x, dtype=np.float32).view(np.uint32)
    u = (u + 0x7FFF + ((u >> 16) & 1)) & np.uint32(0xFFFF0000)
    return u.view(np.float32).astype(np.float64)
