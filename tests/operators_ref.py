"""Plain 64-bit references of the block-scaled E4M3 cache and of attention under
a score rule, written from their definitions (numpy and torch on the CPU, no
library code), with the error that each kernel's arithmetic may leave.

Rounding units (half a step relative to the value): bf16 2^-8, f16 2^-11,
f32 2^-24.  What an output element may be off by, with w_j its row's weights:

  scores    delta_j = 2^-24 [ (D + 4) scale sum_d |q_d K_jd| + 4 |s_j| + 8 cap
                              + 4 slope |pos - j| + 16 ]
            (products and sums of D terms in fp32; the scaling, the base-2
            exponent's argument and its approximation; the cap's exponential and
            reciprocal; the bias), which moves the weights by w_j (delta_j +
            sum_i w_i delta_i);
  P         rounded to the operand type before it weights V: u_P w_j;
  sums      (n / 64 + 16) 2^-24 for the fp32 sums over the row's n keys, in tiles;
  output    one rounding: u_out |out|.
So |error| <= sum_j w_j |V_j| (delta_j + sum_i w_i delta_i + u_P + sums) + u_out |out|
(+ a term of the smallest representable step).  E4M3 tensor-core products add
the query's split (2^-17 of the head's largest component, times scale |K_j|_1,
into delta_j) and P's floor (see attention()).
"""
import math

import numpy as np
import torch

U = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
TINY = {torch.float32: 2.0 ** -126, torch.float16: 2.0 ** -24, torch.bfloat16: 2.0 ** -126}

# values of the E4M3 codes 0 .. 126 (code 127 is the NaN), from the format's fields
E4M3 = np.array([(c & 7) * 2.0 ** -9 if c < 8 else (1 + (c & 7) / 8) * 2.0 ** ((c >> 3) - 7)
                 for c in range(127)])


def e4m3_encode(x):
    """Nearest code, ties to the even code, saturating; NaN is 0x7f."""
    x = np.asarray(x, dtype=np.float64)
    mag = np.minimum(np.abs(np.nan_to_num(x, nan=0.0, posinf=1e300, neginf=-1e300)), 448.0)
    hi = np.clip(np.searchsorted(E4M3, mag), 1, 126)
    lo = hi - 1
    below, above = mag - E4M3[lo], E4M3[hi] - mag
    code = np.where(below < above, lo, np.where(above < below, hi, np.where(lo % 2 == 0, lo, hi)))
    code = code.astype(np.uint8) | np.where(np.signbit(x), 0x80, 0).astype(np.uint8)
    return np.where(np.isnan(x), np.uint8(0x7f), code)


def e4m3_decode(codes):
    codes = np.asarray(codes, dtype=np.uint8)
    mag = np.append(E4M3, np.nan)[codes & 0x7f]
    return np.where(codes & 0x80, -mag, mag)


def block_scale(most):
    """The smallest 2^e, -40 <= e <= 80, with most <= 448 * 2^e (2^80 if none)."""
    for e in range(-40, 81):
        if most <= 448.0 * 2.0 ** e:
            return np.float32(2.0 ** e)
    return np.float32(2.0 ** 80)


def append(x, codes, scales, slots):
    """pa_reshape_and_cache_fp8_block for keys or values: x [N, H, D] (float32
    values of the given type), codes uint8 [NB, H, bs, D] and scales float32
    [NB, H], both updated in place."""
    bs = codes.shape[2]
    rows = {}
    for t, s in enumerate(slots):
        if s >= 0:
            rows.setdefault(int(s) // bs, []).append(t)
    for blk, ts in rows.items():
        offs = [int(slots[t]) % bs for t in ts]
        for h in range(x.shape[1]):
            mags = np.abs(x[ts, h].astype(np.float64))
            most = np.nanmax(np.where(np.isnan(mags), 0.0, mags))
            stored = scales[blk, h]
            old = np.float32(0) if 0 in offs or not stored > 0 else stored
            new = max(old, block_scale(most))
            if new > old and 0 not in offs:
                others = [o for o in range(bs) if o not in offs]
                kept = e4m3_decode(codes[blk, h, others]).astype(np.float32) * (old / new)
                codes[blk, h, others] = e4m3_encode(kept)
            with np.errstate(over="ignore", invalid="ignore"):
                codes[blk, h, offs] = e4m3_encode(x[ts, h].astype(np.float32) / new)
            scales[blk, h] = new


def attention(q, key, value, scale, out_dtype, u_p, *, first=None, last=None, pos=None, cap=0.0,
              slopes=None, split=False, floor_values=None):
    """Attention of query rows q [T, Hq, D] over key / value [L, Hkv, D] (float64);
    row t sees positions first[t] .. last[t] (default all).  Returns (out, tol)
    [T, Hq, D] float64: zeros where nothing is seen.

    u_p: the rounding unit of P.  split: E4M3 tensor-core products; then
    floor_values [L, Hkv] is what P is held relative to beside the weight (the
    value scales): P * 2^6 is two E4M3 terms, so an element of P is off by at
    most 2^-8 of itself or by 2^-16 of the largest product w_j floor_values_j."""
    T, Hq, D = q.shape
    L, Hkv = key.shape[0], key.shape[1]
    G = Hq // Hkv
    k = key.repeat_interleave(G, 1).permute(1, 2, 0)              # [Hq, D, L]
    v = value.repeat_interleave(G, 1).permute(1, 0, 2)            # [Hq, L, D]
    j = torch.arange(L, dtype=torch.float64)
    pos = torch.full((T,), float(L - 1), dtype=torch.float64) if pos is None else \
        torch.as_tensor(pos, dtype=torch.float64)
    first = torch.zeros(T) if first is None else torch.as_tensor(first)
    last = torch.full((T,), L - 1) if last is None else torch.as_tensor(last)
    seen = (j[None, :] >= first[:, None]) & (j[None, :] <= last[:, None])          # [T, L]
    any_row = seen.any(0)                       # positions some row sees; others are never read
    k = torch.where(any_row[None, None, :], k, 0.0)
    v = torch.where(any_row[None, :, None], v, 0.0)
    qh = q.permute(1, 0, 2)                                        # [Hq, T, D]
    s = qh @ k * scale
    mag = qh.abs() @ k.abs() * abs(scale)
    if cap:
        s = cap * torch.tanh(s / cap)
    bias = torch.zeros_like(s)
    if slopes is not None:
        bias = slopes.double()[:, None, None] * (pos[:, None] - j).abs()
        s = s - bias
    delta = ((D + 4) * mag + 4 * s.abs() + 8 * cap + 4 * bias.abs() + 16) * 2.0 ** -24
    if split:
        qmax = qh.abs().amax(-1, keepdim=True)
        delta = delta + 2.0 ** -17 * qmax * abs(scale) * k.abs().sum(1, keepdim=True)
    s = s.masked_fill(~seen, -math.inf)
    w = torch.softmax(s, -1).nan_to_num(0.0)
    delta = torch.where(seen, delta, 0.0)
    n = seen.sum(-1)[None, :, None].double()
    rel = delta + (w * delta).sum(-1, keepdim=True) + u_p + (n / 64 + 16) * 2.0 ** -24
    out = w @ v
    tol = (w * rel) @ v.abs() + U[out_dtype] * out.abs() + TINY[out_dtype]
    if split:
        vs = torch.ones(L, Hkv, dtype=torch.float64) if floor_values is None else floor_values
        vs = vs.repeat_interleave(G, 1).t()[:, None, :]            # [Hq, 1, L]
        top = (w * vs).amax(-1, keepdim=True)                      # the largest product
        codes = (v / vs.transpose(1, 2)).abs()
        tol = tol + 2.0 ** -16 * top * (seen.double() @ codes)
    return out.permute(1, 0, 2), tol.permute(1, 0, 2)


def limits(L, pos, window=0, key_start=0, prefix=0):
    """First and last position that the query at `pos` of L tokens sees."""
    first = max(0, key_start)
    if window:
        first = max(first, pos - window + 1)
    return first, max(pos, min(prefix, L) - 1)


def gather(cache, table, L, scales=None):
    """Positions 0 .. L - 1 of a sequence [L, Hkv, D] in float64 (and the scale of
    each position and head), from a cache on the CPU."""
    bs = cache.shape[2]
    at = torch.arange(L)
    blk = table[at // bs].long()
    x = cache[blk, :, at % bs]
    if scales is None:
        return x.double()
    x = torch.from_numpy(e4m3_decode(x.view(torch.uint8).numpy()))
    s = scales[blk].double().clamp(2.0 ** -40, 2.0 ** 80)      # as pa_decode_fp8_block reads them
    return x * s[:, :, None], s


def worst(got, out, tol):
    """The largest error in units of what each element may be off by; infinite where
    the result is not finite."""
    got = got.detach().cpu().double()
    ratio = (got - out).abs() / tol.clamp(min=1e-300)
    return float(torch.where(torch.isfinite(got), ratio, math.inf).max())
