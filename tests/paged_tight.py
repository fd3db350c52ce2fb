"""Bounds on attention outputs that shrink with the outputs, for random values.

The 64-bit result of a row is sum_j w_j v_j, w its softmax weights. For values that are independent and of
zero mean, and weights that differ (all tests that use this file draw such), a sum of errors e_j w_j v_j with |e_j| <= u
stays below 8 u S, S = sqrt(sum_j w_j^2 v_j^2), but for a chance of 2 exp(-32) (Hoeffding), and
always below u A, A = sum_j w_j |v_j|. What a kernel's result may be off by:

  u_o |out|              the output's own rounding, u_o half a step of its type
  min(8 S, A) u_p        the weights' rounding before the value product: u_p = u_o for one 16-bit
                         term (more than 16 query rows per KV head), u_o^2 for two
  min(8 S, A) dw         a weight's own error: its logit's, d products summed in fp32, each
                         addition off by 2^-23 of sum_c |q_c k_c| (twice: the denominator has it too),
                         and 2^-21 for the constants, the argument and the exponential, relative to 1 + |z|
  (n/16 + 64) 2^-23 6 S  n/16 additions of fp32 products; a partial sum of such values stays below 6 S
  (n/64 + 64) 2^-24 |out|   the denominator's additions

fp16 weights, scaled so that the largest is at least 2^7, stop at 2^-25: 2^-32 of the largest each.
The root mean square of the error over N outputs of a head: a rounding of at most u is uniform at worst,
u / sqrt(3), and independent between outputs; 5 / sqrt(2 N) for the sample.
"""
import numpy as np
import torch

from paged_util import DT


class Rows:
    """Rows q [R, d] of one KV head over k, v [n, d], where see [R, n] (bool, or None: all).
    rows_per_head: query rows per KV head that the call has room for."""

    def __init__(self, q, k, v, see, scale, dtype, rows_per_head):
        n, d = k.shape
        z = scale * (q @ k.T)
        if see is not None:
            z = np.where(see, z, -np.inf)
        m = z.max(1, keepdims=True)
        self.empty = np.isneginf(m[:, 0])
        m = np.where(np.isneginf(m), 0.0, m)
        p = np.exp(z - m)
        l = p.sum(1, keepdims=True)
        self.w = p / np.where(l == 0, 1.0, l)
        self.v, self.n, self.dtype = v, n, dtype
        self.out = self.w @ v
        with np.errstate(divide="ignore"):
            self.lse = (m + np.log(l))[:, 0]
        uo = torch.finfo(DT[dtype]).eps / 2
        up = uo if rows_per_head > 16 else uo * uo
        self.up = up
        zabs = np.abs(np.where(np.isneginf(z), 0.0, z)).max(1, keepdims=True)
        dl = (d + 2) * 2.0 ** -23 * scale * (np.abs(q) @ np.abs(k).T).max(1, keepdims=True)
        dw = 2 * (dl + 2.0 ** -21 * (1 + zabs))
        S = np.sqrt((self.w ** 2) @ (v ** 2))
        A = self.w @ np.abs(v)
        ref = np.abs(self.out)
        den = (n / 64 + 64) * 2.0 ** -24
        acc = (n / 16 + 64) * 2.0 ** -23 * 6
        sub = 2.0 ** -32 * np.abs(v).sum(0)[None] / np.where(l == 0, 1.0, l) if dtype == "fp16" else 0.0
        tiny = torch.finfo(DT[dtype]).smallest_normal * torch.finfo(DT[dtype]).eps
        self.tol = (1 + 2 * uo) * (uo * ref + np.minimum(8 * S, A) * (up + dw) + acc * S + (den + dw) * ref + sub) + tiny
        rms = lambda x: float(np.sqrt(np.mean(np.square(x))))
        big = 5 / np.sqrt(2 * self.out.size)
        self.rms = (1 + big) * np.sqrt((uo * rms(ref)) ** 2 / 3 + (up * rms(S)) ** 2 / 3) + \
            rms((dw + acc) * S) + rms((den + dw) * ref) + rms(sub) + tiny
        self.lse_tol = (dl + 2.0 ** -21 * (1 + zabs))[:, 0] + den + \
            2.0 ** -22 * np.abs(np.where(np.isfinite(self.lse), self.lse, 0.0))

    def problem(self, out, lse=None):
        """What is wrong with a result, or None."""
        err = np.abs(out - self.out)
        if not (err <= self.tol).all():
            at = np.argwhere(~(err <= self.tol))
            return f"{len(at)} outputs off, the first at {at[0].tolist()}: {out[tuple(at[0])]} for {self.out[tuple(at[0])]}"
        got = float(np.sqrt(np.mean(err ** 2)))
        if not got <= self.rms:
            return f"rms of the error {got}, allowed {self.rms}"
        if lse is not None:
            if not np.array_equal(np.isneginf(lse), self.empty):
                return "rows that see nothing"
            at = ~self.empty
            if not (np.abs(lse[at] - self.lse[at]) <= self.lse_tol[at]).all():
                return f"lse off by {np.abs(lse[at] - self.lse[at]).max()}"
        return None

    def rounded(self, w=None, v=None):
        """The result with 16-bit weights where the kernels have them, rounded to the output's type."""
        t = DT[self.dtype]
        w = self.w if w is None else w
        if self.up == torch.finfo(t).eps / 2:
            top = np.maximum(self.w.max(1, keepdims=True), 1e-300)
            w = torch.from_numpy(w / top * 128).to(t).double().numpy() / 128 * top
        return torch.from_numpy(w @ (self.v if v is None else v)).to(t).double().numpy()
