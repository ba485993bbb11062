"""Attention over a paged 8-bit cache in 64 bits, for contexts of many thousand keys, with tolerances that a tail of small
weights cannot hide in (imported by the cache tests)."""
import torch

E4M3 = torch.float8_e4m3fn


def values(codes, scales, table, length, T):
    """[H][length][D] of one side: codes [N][H][T][D] uint8, scales [N][H], table row of one request (linear)."""
    ids = torch.as_tensor(table[:-(-length // T)], dtype=torch.long, device=codes.device)
    x = codes[ids].view(E4M3).double() * scales[ids].double()[..., None, None]
    return x.permute(1, 0, 2, 3).reshape(codes.shape[1], -1, codes.shape[3])[:, :length]


def attention(q, k, v, dtype, scale=None, seen=None):
    """q [rows][Hq][D], k, v [H][n][D] in 64 bits, seen bool [rows][n] or None. The outputs and how far a call may be off,
    element by element:
      u = eps / 2 of the result, its rounding to dtype; 2^-25 where it is below f16's normal range, whose step is 2^-24;
      2^-11 of each probability: it enters as a value of 11 significant bits;
      2^-30 of the row's largest one for each key: the step at which small ones end (half of 2^-20, the largest is kept at 2^9
      or more); 2^17 keys can add up 2^-13 of the largest value so, below u;
      the scores, as products of D terms of 2 D roundings at 2^-23 and 2^-22 of the exponent's argument;
      the sums: a few thousand additions in turn in 32 bits, whose errors of 2^-24 do not all point one way: 2^-15."""
    rows, Hq, D = q.shape
    H, n = k.shape[:2]
    scale = D ** -0.5 if scale is None else scale
    u = torch.finfo(dtype).eps / 2
    qh = q.double().reshape(rows, H, Hq // H, D).permute(1, 0, 2, 3).reshape(H, -1, D)
    s = qh @ k.transpose(1, 2) * scale
    if seen is not None:
        s = s.masked_fill(~seen[None, :, None].expand(H, rows, Hq // H, n).reshape(H, -1, n), -torch.inf)
    p = torch.softmax(s, -1)
    off = (qh.abs() @ k.abs().amax(1)[..., None])[..., 0] * abs(scale) * 2 * D * 2.0 ** -23
    off = off + s.masked_fill(s == -torch.inf, 0).abs().amax(-1) * 2.0 ** -22
    o, reach = p @ v, p @ v.abs()
    tol = (u * o.abs() + (2.0 ** -11 + 2.0 ** -15 + 2 * off[..., None]) * reach
           + 2.0 ** -30 * p.amax(-1, keepdim=True) * v.abs().sum(1, keepdim=True) + 2.0 ** -25)
    back = lambda t: t.reshape(H, rows, Hq // H, D).permute(1, 0, 2, 3).reshape(rows, Hq, D)   # noqa: E731
    return back(o), back(tol)
