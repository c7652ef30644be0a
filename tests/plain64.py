"""Plain 64-bit forms of whole-prompt and tree attention, with the bound each
result is held to.

A result is out[d] = sum_u w_u v_u[d] with w = softmax(s).  Counted against it:
 - its own rounding to the output type: h_o |out|, h = eps / 2 of the type;
 - each weight's rounding to the type it is multiplied in (the output's type;
   f16 with an fp8 cache): h_p sum w |v|; an f16 weight below 2^-14 has the
   absolute error 2^-25 instead, relative to a sum of at least 1:
   n 2^-25 max |v| over n keys;
 - the scores' fp32 sums: d terms, each within d 2^-24 sum |q k| scale; with
   the inputs here (|q| of about 2, |k| of about 1, d <= 128, scale
   1 / sqrt(d)) below 2^-12.9 in ln units, in the numerator and in the sum:
   2^-11.9 sum w |v|;
 - the exponential, within 2^-13.5 (a polynomial for 2^f or the hardware's), in
   the numerator and the sum: 2^-12.5 sum w |v|.
The last two are below 2^-11 sum w |v| together.
"""
import torch

HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}


def attend(q, k, v, seen, scale):
    """(out, sum of w |v|) in float64 of q [T, h, d], k / v [N, kv, d] and
    seen [T, N]; rows that see nothing are zero."""
    G = q.shape[1] // k.shape[1]
    q, k, v = q.double(), k.double(), v.double()
    k, v = (x.masked_fill(~seen.any(0)[:, None, None], 0.0) for x in (k, v))
    k, v = (x.repeat_interleave(G, 1) for x in (k, v))
    s = torch.einsum("thd,nhd->htn", q, k) * scale
    s = s.masked_fill(~seen[None], float("-inf"))
    w = torch.softmax(s, -1).masked_fill(~seen[None], 0.0)
    w = torch.where(seen.any(-1)[None, :, None], w, torch.zeros_like(w))
    return torch.einsum("htn,nhd->thd", w, v), torch.einsum("htn,nhd->thd", w, v.abs())


def check(got, ref, mag, n_keys, v_max, weight_type, what):
    h_o, h_p = HALF_STEP[got.dtype], HALF_STEP[weight_type]
    tol = h_o * ref.abs() + (h_p + 2.0 ** -11) * (1 + h_o) * mag
    if weight_type == torch.float16:
        tol = tol + n_keys * 2.0 ** -25 * v_max
    if got.dtype == torch.float16:  # results below f16's normal range
        tol = tol + 2.0 ** -25
    err = (got.double() - ref).abs()
    assert torch.isfinite(got).all(), f"{what}: not finite"
    worst = (err - tol).max().item() if err.numel() else -1.0
    assert worst <= 0, f"{what}: {int((err > tol).sum())} of {err.numel()} values out of " \
                       f"tolerance, the worst by {worst:.3e}; largest error {err.max().item():.3e}"


def causal(n, device):
    at = torch.arange(n, device=device)
    return at[None, :] <= at[:, None]
