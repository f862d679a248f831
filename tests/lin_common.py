"""The definition of linear attention with one decay per head in 64 bits, and the error bounds that the
kernels of include/kda_lin.h have to keep.

With w_tj = e^(g_(j+1) + .. + g_t), an output is scale (sum_j w_tj (q_t . k_j) v_j + w_t (S0^T q_t)) and a state
sum_j w_Tj k_j v_j^T + w_T S0. Let A be the same sum of magnitudes. Each term of it, up to the output's own
rounding, is rounded
 - in its decay: e^x is off by 2^-22 of itself and by |x| 2^-24 where x is rounded; a factor matters down to
   e^-104 (below, it is 0 in fp32), so all the factors of a term together by (104 + 2 n / 16) 2^-24 + (n / 16) 2^-22
   at most when one is taken per 16 tokens (a longer step takes fewer), and in the products with k and v by 3 2^-24;
 - in its sums, each at most 2^-24 of A: over d_k channels, 64 tokens, one more for each step of 16 tokens and
   one for each of up to 64 segments.
With bf16 inputs the decayed scores and the state that q reads are held in bf16 where they are multiplied, one
number for bf16 outputs (2^-8 of each term, once), two for fp32 ones (2^-16); the decayed values in 24 bits
(2^-24). Single tokens: no such rounding, one step.
"""

import numpy as np
import torch

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def e32(n, d_k):
    steps = n / 16 + 1
    return (104 + 2 * steps + 4 * steps + 3 + d_k + 64 + steps + 64) * 2.0 ** -24


def definition(q, k, v, g, S0, scale):
    """One sequence, 64 bits on the CPU: q, k [T, Hk, d_k], v [T, H, d_v], g [T, H], S0 [H, d_k, d_v] or None.
    Returns (o, A_o, state, A_state), the A being the sums of magnitudes."""
    H = v.shape[1]
    rep = H // q.shape[1]
    q, k = (np.repeat(x.double().cpu().numpy(), rep, 1) for x in (q, k))
    v, a = v.double().cpu().numpy(), np.exp(g.double().cpu().numpy())
    T, _, dk = q.shape
    S = np.zeros((H, dk, v.shape[2])) if S0 is None else S0.double().cpu().numpy().copy()
    A = np.abs(S)
    o, ao = np.zeros(v.shape), np.zeros(v.shape)
    for t in range(T):
        S = a[t][:, None, None] * S + k[t][:, :, None] * v[t][:, None, :]
        A = a[t][:, None, None] * A + np.abs(k[t][:, :, None] * v[t][:, None, :])
        o[t] = np.einsum("hi,hij->hj", q[t], S) * scale
        ao[t] = np.einsum("hi,hij->hj", np.abs(q[t]), A) * abs(scale)
    return o, ao, S, A


def check(name, got, ref, A, e, bf16_out=False):
    """|got - ref| <= e A, and half a step of a bf16 output."""
    got = got.double().cpu().numpy()
    lim = e * A + 2.0 ** -120
    if bf16_out:
        lim = lim + 2.0 ** -8 * (np.abs(ref) + lim)
    assert np.isfinite(got).all(), f"{name}: not finite"
    worst = float((np.abs(got - ref) / lim).max()) if ref.size else 0.0
    print(f"  {name}: worst error / bound = {worst:.3f}", flush=True)
    assert worst <= 1.0, f"{name}: {worst:.3f} of its bound"


def offsets(lens, device="cuda"):
    return torch.tensor([0] + list(np.cumsum(lens)), dtype=torch.int32, device=device)


class Inputs:
    """Seeded inputs on the GPU. decay: "tokens" [T, H] or "heads" [H]."""

    def __init__(self, seed, lens, H, Hk, dk, dv, dt, decay="tokens", rate=0.3, spare=0):
        r = np.random.default_rng(seed)
        T = sum(lens) + spare

        def t(x):
            return torch.from_numpy(np.asarray(x, np.float32)).cuda()

        self.lens, self.cu, self.T = list(lens), offsets(lens), T
        self.q = t(r.standard_normal((T, Hk, dk))).to(DT[dt])
        self.k = t(r.standard_normal((T, Hk, dk)) / np.sqrt(dk)).to(DT[dt])
        self.v = t(r.standard_normal((T, H, dv))).to(DT[dt])
        rates = rate * np.exp(r.uniform(np.log(0.01), 0, H))
        self.g = t(-rates) if decay == "heads" else t(-rates * np.log1p(np.exp(r.standard_normal((T, H)))))
        self.s0 = t(0.3 * r.standard_normal((len(lens), H, dk, dv)))
        self.dt = dt

    def args(self):
        return self.q, self.k, self.v, self.g, self.cu

    def tokens(self, g=None):
        """g as [T, H]."""
        g = self.g if g is None else g
        return g.expand(self.T, g.shape[-1])

    def reference(self, S0, scale):
        """[(o, A_o, state, A_state)] of every sequence."""
        out, at = [], 0
        g = self.tokens()
        for n, L in enumerate(self.lens):
            i = slice(at, at + L)
            out.append(definition(self.q[i], self.k[i], self.v[i], g[i], None if S0 is None else S0[n], scale))
            at += L
        return out

    def bound(self, L, dk, bf16_out):
        return e32(L, dk) + (0.0 if self.dt == "f32" else 2.0 ** -8 if bf16_out else 2.0 ** -16)

    def check(self, o, state, S0, scale, what=""):
        at = 0
        for n, (L, (ro, ao, rs, as_)) in enumerate(zip(self.lens, self.reference(S0, scale))):
            dk = self.q.shape[2]
            half = o.dtype == torch.bfloat16
            check(f"{what} o {n} ({L})", o[at:at + L], ro, ao, self.bound(L, dk, half), half)
            if state is not None:
                check(f"{what} state {n} ({L})", state[n], rs, as_, e32(L, dk))
            at += L
