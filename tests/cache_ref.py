"""Plain 64-bit CPU forms of the paged 4-bit history cache, for the tests:
quantisation, the page layout, the plan as a walk over the sequences, and the
attention token by token from the mask's definition."""
import numpy as np
import torch


def f32(x):
    return x.float().double()


def quantise(x):
    """bf16 [..., d] -> codes (int64), step, minimum (float64 [...])."""
    x = x.double()
    fine = torch.isfinite(x).all(-1)
    m = x.min(-1).values
    span = f32(x.max(-1).values - m)
    step = f32(span / 15).bfloat16().double()
    fine &= torch.isfinite(step)
    step = torch.where(step < 2.0 ** -126, torch.zeros_like(step), step)
    inv = torch.where(step > 0, f32(1 / step), torch.zeros_like(step))
    code = torch.round(f32(f32(x - m[..., None]) * inv[..., None])).clamp(0, 15)
    code = torch.where(fine[..., None], code, torch.zeros_like(code))
    nan = torch.full_like(m, float("nan"))
    return code.nan_to_num().long(), torch.where(fine, step, nan), torch.where(fine, m, nan)


def values(x):
    c, s, m = quantise(x)
    return m[..., None] + s[..., None] * c


def bf16_once(x):
    """float64 rounded to bf16 once, ties to even (torch goes through fp32)."""
    x = x.double().numpy()
    e = np.maximum(np.frexp(x)[1], -125)
    return torch.from_numpy(np.ldexp(np.rint(np.ldexp(x, 8 - e)), e - 8))


def offsets(H, d, ps):
    """Byte offsets within a page of (head, token, dim): K byte, K shift, V byte,
    V shift; and of the (step, minimum) pairs of K and V."""
    h = np.arange(H)[:, None, None]
    r = np.arange(ps)[None, :, None]
    e = np.arange(d)[None, None, :]
    base = h * ps * (d + 8)
    n = (e % 8) // 2 + 4 * (e % 2)
    kb = base + r * (d // 2) + e // 8 * 4 + n // 2
    ks = (n % 2) * 4 + 0 * r
    vb = base + ps * (d // 2) + (e // 2) * ps + r // 4 * 4 + np.array([0, 2, 1, 3])[r % 4]
    vs = (e % 2) * 4 + 0 * r
    kp = (base + ps * d + 4 * r)[..., 0]
    return kb, np.broadcast_to(ks, (1, ps, d)), vb, np.broadcast_to(vs, (1, ps, d)), kp, kp + 4 * ps


def unpack(pages, ps, d):
    """uint8 [P, H, ps * (d + 8)] -> K and V values, float64 [P, ps, H, d]."""
    P, H, n = pages.shape
    flat = pages.cpu().numpy().reshape(P, H * n)
    kb, ks, vb, vs, kp, vp = offsets(H, d, ps)
    res = []
    for byte, shift, par in ((kb, ks, kp), (vb, vs, vp)):
        code = (flat[:, byte] >> shift) & 15
        raw = np.stack([flat[:, par + i] for i in range(4)], -1)
        sm = torch.from_numpy(np.ascontiguousarray(raw)).view(torch.bfloat16).double().numpy()
        res.append(torch.from_numpy((sm[..., 1:] + sm[..., :1] * code).transpose(0, 2, 1, 3)))
    return res


def pack(pages, ps, slots, k, v):
    """Write the quantised rows k, v ([T, H, d] bf16) into a uint8 pages tensor."""
    P, H, n = pages.shape
    d = n // ps - 8
    flat = pages.numpy().reshape(P, H * n)
    kb, ks, vb, vs, kp, vp = offsets(H, d, ps)
    for x, byte, shift, par in ((k, kb, ks, kp), (v, vb, vs, vp)):
        code, s, m = quantise(x)
        sm = torch.stack([s, m], -1).bfloat16().contiguous().view(torch.uint8).numpy()
        for t, slot in enumerate(slots.tolist()):
            if slot < 0:
                continue
            p, r = divmod(slot, ps)
            for sh in (0, 4):
                at = np.broadcast_to(shift, byte.shape)[:, r] == sh
                b = byte[:, r][at]
                flat[p, b] = (flat[p, b] & (0xF0 >> sh)) | (code[t].numpy()[at] << sh)
            for i in range(4):
                flat[p, par[:, r] + i] = sm[t, :, i]
    return torch.from_numpy(flat.reshape(P, H, n))


class Tables:
    """A cache's tables on the host."""

    def __init__(self, lengths, block_table, free, num_pages, ps):
        self.lengths = [int(x) for x in lengths]
        self.bt = [list(map(int, r)) for r in block_table]
        self.stack = [int(x) for x in free]
        self.count = len(self.stack)
        self.stack += [0] * (num_pages - self.count)
        self.P, self.ps = num_pages, ps

    def plan(self, rows, cand, release, total):
        ps = self.ps
        up = lambda n: -(-n // ps)  # noqa: E731
        for b, gone in enumerate(release):
            if gone:
                for j in range(up(self.lengths[b])):
                    self.stack[self.count] = self.bt[b][j]
                    self.count += 1
                self.lengths[b] = 0
        slots = [-1] * total
        t = 0
        for b, (n, c) in enumerate(zip(rows, cand)):
            for r in range(n - c):
                pos = self.lengths[b] + r
                if pos % ps == 0:
                    self.count -= 1
                    self.bt[b][pos // ps] = self.stack[self.count]
                slots[t + r] = self.bt[b][pos // ps] * ps + pos % ps
            self.lengths[b] += n - c
            t += n
        return slots


def silu(x):
    return x / (1 + torch.exp(-x))


def attend(q, k, v, rows, cand, lengths, pages, *, K1, K2e, alpha, N):
    """The rows' attention and a bound of the kernels' error.  q, k, v [T, H, d];
    pages[b] = (codes, step, minimum) of K and V, token by token.

    Bound, with P = SiLU(x), h = x / 2 and u = 2^-8 bf16's relative half step:
      u |out|            the result in bf16
      u sum |P| s c      P s in bf16 or f16, the matrix product's operand
      2^-10 sum |h| |v|  tanh's instruction (relative error below 2^-10.9)
      1.1 dx |v|         x in fp32: sums of d products of q c in d / 16 matrix
                         steps, each off by 2^-22 of the sum (SiLU' <= 1.1); c
                         taken as 31, the most a code with an offset of 16 is
      fp32 sums over n keys: n / 16 steps of P s c (c as 31), and of P m."""
    out = torch.zeros(q.shape, dtype=torch.float64)
    tol = torch.zeros(q.shape, dtype=torch.float64)
    q, k, v = q.double(), k.double(), v.double()
    d = q.shape[2]
    t = 0
    for b, (n, c) in enumerate(zip(rows, cand)):
        L = lengths[b]
        (kc, ks, km), (vc, vs, vm) = pages[b]
        K, V = kc * ks[..., None] + km[..., None], vc * vs[..., None] + vm[..., None]
        j = torch.arange(L)
        for r in range(n):
            if r < n - c:
                i = L - (n - c) + r
                see = (j <= i) & ((i - j < K1) | (j < K2e))
            else:
                see = (L - j < K1) | (j < K2e)
            x = alpha * torch.einsum("hd,jhd->jh", q[t + r], K[see])
            P = silu(x)
            o = torch.einsum("jh,jhd->hd", P, V[see])
            steps = int(see.sum()) / 16 + 12
            dx = abs(alpha) * (31 * ks[see] + km[see].abs()) * q[t + r].abs().sum(-1) * \
                (d / 16 + 2) * 2.0 ** -22
            e = torch.einsum("jh,jhd->hd", P.abs() * vs[see], vc[see].double()) * 2.0 ** -8
            e += torch.einsum("jh,jhd->hd", x.abs() * 2.0 ** -11 + 1.1 * dx, V[see].abs())
            e += ((P.abs() * (31 * vs[see] + vm[see].abs())).sum(0) * steps * 2.0 ** -22)[:, None]
            if r >= n - c:
                x = alpha * (q[t + r] * k[t + r]).sum(-1)
                o = o + silu(x)[:, None] * v[t + r]
                e += (x.abs()[:, None] * v[t + r].abs() + 1e-3) * 2.0 ** -18
            out[t + r] = o / N
            tol[t + r] = e / N + o.abs() / N * 2.0 ** -8 + 1e-30
        t += n
    return out, tol
