"""Plain 64-bit forms of the attention operators and of the e4m3 cache, for the
tests of include/kda_attn.h, and the error bounds that the kernels have to keep.

Error bound of an attention output element, from the arithmetic:
 - a score is an fp32 sum of d_k products: off by at most (d_k + 4) 2^-24 of
   scale sum |q||k| (the 4: scaling, the cache's scale, the reference's
   subtraction, the product with log2 e). With S the row's largest scale
   sum |q||k| and |ref| at most as large, a weight is off by a factor of at most
   1 + e_s, e_s = 2 (d_k + 4) 2^-24 S + 2^-22 (the exponential itself);
 - with bf16 inputs the weight rounds to bf16: 2^-8;
 - sums of n terms in fp32: n 2^-24, and 2^-21 for joining pieces and dividing.
The weights enter above and below, so with A = sum w|v| / sum w:
   |error| <= A (2 e_s + [bf16] 2^-8 + 2 n 2^-24 + 2^-21) + [bf16 output] 2^-8 |o|
and a bf16 output's own half step. Denormal outputs round by 2^-134 at most.
"""

import numpy as np
import torch

INF = float("inf")


def attend(q, k, v, sees, scale):
    """One head in 64 bits: (o, A, S, n) with A, S and n as above. Unseen tokens take no part,
    whatever they hold."""
    q, k, v = (x.double() for x in (q, k, v))
    o = torch.zeros((q.shape[0], v.shape[1]), dtype=torch.float64)
    A, S, n = torch.zeros_like(o), torch.zeros(q.shape[0], dtype=torch.float64), sees.sum(1)
    for i in range(q.shape[0]):
        at = sees[i].nonzero()[:, 0]
        if at.numel() == 0:
            continue
        x = k[at] @ q[i] * scale
        w = torch.exp(x - x.max())
        o[i] = (w @ v[at]) / w.sum()
        A[i] = (w @ v[at].abs()) / w.sum()
        S[i] = (abs(scale) * (k[at].abs() @ q[i].abs())).max()
    return o, A, S, n


def bound(o, A, S, n, d_k, bf16_in, bf16_out):
    e = 2 * (d_k + 4) * 2.0 ** -24 * S + 2.0 ** -22
    rel = 2 * e + (2.0 ** -8 if bf16_in else 0.0) + 2 * n * 2.0 ** -24 + 2.0 ** -21
    return A * rel[:, None] + (2.0 ** -8 * (o.abs() + A * rel[:, None]) if bf16_out else 0.0) + 2.0 ** -134


def check(name, got, ref, limit):
    got = got.double().cpu()
    fine = torch.isfinite(ref)
    assert torch.equal(torch.isfinite(got), fine), f"{name}: infinities or NaN in other places"
    d = (got - ref).abs()[fine]
    worst = float((d / limit[fine]).max()) if d.numel() else 0.0
    print(f"  {name}: worst error / bound = {worst:.3f}", flush=True)
    assert worst <= 1.0, f"{name}: {worst:.3f} of its bound"


def prompt_reference(q, k, v, lens, scale, bf16_in, bf16_out):
    """(o, bound) of causal attention in each of the packed sequences, on the CPU."""
    q, k, v = q.cpu(), k.cpu(), v.cpu()
    T, H, d_k = q.shape
    G = H // k.shape[1]
    o = torch.zeros((T, H, v.shape[2]), dtype=torch.float64)
    lim = torch.ones_like(o)
    at = 0
    for L in lens:
        sees = torch.ones((L, L), dtype=torch.bool).tril()
        for h in range(H):
            r = attend(q[at:at + L, h], k[at:at + L, h // G], v[at:at + L, h // G], sees, scale)
            o[at:at + L, h] = r[0]
            lim[at:at + L, h] = bound(*r, d_k, bf16_in, bf16_out)
        at += L
    return o, lim


# ---- the paged cache


def round_e4m3(x):
    """The e4m3 number nearest to each x (|x| <= 448), ties to the even one, by arithmetic."""
    mag = np.abs(x)
    power = np.maximum(np.floor(np.log2(np.where(mag > 0, mag, 1.0))), -6)
    step = np.exp2(power - 3)
    return np.rint(x / step) * step


def to_codes(x):
    """[..., d] in 64 bits: (values of the codes, exponents)."""
    x = np.asarray(x, np.float64)
    fine = np.isfinite(x)
    top = np.where(fine, np.abs(x), 0).max(-1)
    e = np.full(top.shape, -127, np.int64)
    for i in np.ndindex(top.shape):
        while top[i] > 448 * 2.0 ** int(e[i]):
            e[i] += 1
    codes = np.where(fine, round_e4m3(np.where(fine, x, 0) * np.exp2(-e.astype(np.float64))[..., None]), np.nan)
    return codes, e


class Cache:
    """A paged cache on the GPU and its contents in 64 bits on the CPU. Everything that no sequence
    holds is NaN (byte 0xFF of every element and exponent)."""

    def __init__(self, lens, Hk, d_k, d_v, page, kv, seed=0, spare=2, max_pages=None, device="cuda"):
        self.dt = {"f32": torch.float32, "bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn}[kv]
        self.kv, self.page, self.Hk = kv, page, Hk
        need = [-(-n // page) for n in lens]
        pages = sum(need) + spare
        order = np.random.default_rng(seed).permutation(pages).astype(np.int32)
        table = np.full((len(lens), max_pages or max(1, max(need))), -1, np.int32)
        at = 0
        for n, c in enumerate(need):
            table[n, :c] = order[at:at + c]
            at += c
        self.host_table, self.host_lens = table, list(lens)
        self.table = torch.from_numpy(table).to(device)
        self.lens = torch.tensor(list(lens), dtype=torch.int32, device=device)

        def full(*shape):
            size = torch.empty(0, dtype=self.dt).element_size()
            return torch.full(shape[:-1] + (shape[-1] * size,), 0xFF, dtype=torch.uint8, device=device).view(self.dt)

        self.k, self.v = full(pages, Hk, page, d_k), full(pages, Hk, page, d_v)
        self.k_exp = self.v_exp = None
        if kv == "e4m3":
            self.k_exp, self.v_exp = (torch.full((pages, Hk, page), 0xFF, dtype=torch.uint8, device=device) for _ in "kv")

    def args(self):
        return self.lens, self.table, self.k, self.v

    def exps(self):
        return dict(k_exp=self.k_exp, v_exp=self.v_exp)

    def place(self, n, pos):
        pos = np.asarray(pos)
        return self.host_table[n, pos // self.page], pos % self.page

    def put(self, n, k, v):
        """All tokens of sequence n, by torch: k, v [len, Hk, d] on the CPU."""
        page, off = (torch.from_numpy(np.asarray(x)).long() for x in self.place(n, np.arange(k.shape[0])))
        for c, x in (("k", k), ("v", v)):
            cache = getattr(self, c)
            dev = cache.device
            if self.kv == "e4m3":
                codes, e = to_codes(x.double().numpy())
                cache.view(torch.uint8)[page.to(dev), :, off.to(dev)] = torch.from_numpy(codes).float().to(
                    torch.float8_e4m3fn).view(torch.uint8).to(dev)
                getattr(self, c + "_exp")[page.to(dev), :, off.to(dev)] = torch.from_numpy(e + 127).to(torch.uint8).to(dev)
            else:
                cache[page.to(dev), :, off.to(dev)] = x.to(self.dt).to(dev)

    def values(self, n, count):
        """The first `count` tokens of sequence n as the cache holds them, 64 bits on the CPU."""
        page, off = (torch.from_numpy(np.asarray(x)).long() for x in self.place(n, np.arange(count)))
        out = []
        for c in ("k", "v"):
            cache = getattr(self, c).cpu()
            if self.kv == "e4m3":
                x = cache.view(torch.uint8)[page, :, off].view(torch.float8_e4m3fn).double()
                x = x * torch.exp2(getattr(self, c + "_exp").cpu()[page, :, off].double() - 127)[..., None]
            else:
                x = cache[page, :, off].double()
            out.append(x)
        return out


def cache_reference(q, cache, new, masks, scale, bf16_in, bf16_out):
    """(o, bound) of attention of the new tokens (the last new[n] of each sequence) over the cache."""
    q = q.cpu()
    T, H, d_k = q.shape
    G = H // cache.Hk
    o = torch.zeros((T, H, cache.v.shape[3]), dtype=torch.float64)
    lim = torch.ones_like(o)
    at = 0
    for n, L in enumerate(new):
        if L == 0:
            continue
        total = cache.host_lens[n]
        k, v = cache.values(n, total)
        ctx = total - L
        sees = torch.zeros((L, total), dtype=torch.bool)
        for i in range(L):
            for p in range(total):
                b = p - ctx
                sees[i, p] = b < 0 or (b <= i if masks is None else b < 64 and bool((masks[at + i] >> b) & 1))
        for h in range(H):
            r = attend(q[at:at + L, h], k[:, h // G], v[:, h // G], sees, scale)
            o[at:at + L, h] = r[0]
            lim[at:at + L, h] = bound(*r, d_k, bf16_in, bf16_out)
        at += L
    return o, lim


def tree_masks(new, seed):
    """A random tree over each sequence's new tokens: a token sees itself and its ancestors."""
    r = np.random.default_rng(seed)
    rows = []
    for n in new:
        seen = []
        for i in range(n):
            p = int(r.integers(-1, i)) if i else -1
            seen.append((1 << i) | (seen[p] if p >= 0 else 0))
        rows += seen
    return rows


def mask_tensor(rows, device="cuda"):
    return torch.from_numpy(np.array(rows, np.uint64).view(np.int64)).to(device)


def offsets(lens, device="cuda"):
    return torch.tensor([0] + list(np.cumsum(lens)), dtype=torch.int32, device=device)


def normal(seed, *shape):
    return torch.from_numpy(np.random.default_rng(seed).standard_normal(shape).astype(np.float32))
