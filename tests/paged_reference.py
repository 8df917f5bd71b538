"""The rotary positions and the paged cache from their definitions, in float64
on the CPU, one row and head after another.  Test infrastructure only."""
import math

import torch

F64 = torch.float64


def frequencies(rot, base=10000.0, factor=1.0, low=0.0, high=0.0, train_len=0.0, **_):
    out = []
    for i in range(rot // 2):
        f = base ** (-2.0 * i / rot)
        s = 0.0
        if high > low:
            s = min(1.0, max(0.0, (train_len * f / (2 * math.pi) - low) / (high - low)))
        out.append(f * (s + (1.0 - s) / factor))
    return out


def turn(x, p, spec, backward=False):
    """x [..., T, d] at the positions p [T]; spec: the arguments of tc.Rotary."""
    rot, inter, gain = spec["rot"], spec.get("interleaved", False), spec.get("gain", 1.0)
    x = x.to(F64)
    y = x.clone()
    for i, f in enumerate(frequencies(**spec)):
        a, b = (2 * i, 2 * i + 1) if inter else (i, i + rot // 2)
        ang = p.to(F64) * f
        c, s = gain * torch.cos(ang), gain * torch.sin(ang) * (-1.0 if backward else 1.0)
        y[..., a] = x[..., a] * c - x[..., b] * s
        y[..., b] = x[..., a] * s + x[..., b] * c
    return y


class Cache:
    """One cache on the CPU: pages as they are stored (their dtype), the rest in
    float64 / int64."""

    def __init__(self, k, v, table, lens, clocks, mass, pos, A=None, lam=None, eta=None):
        self.k, self.v, self.mass, self.pos = k.clone(), v.clone(), mass.to(F64), pos.to(torch.int64)
        self.table, self.lens, self.clocks = table, lens.tolist(), clocks.tolist()
        self.A = None if A is None else A.to(F64)
        self.lam, self.eta = (None, None) if lam is None else (lam.to(F64), eta.to(F64))
        self.page, self.H, self.d = k.shape[2], k.shape[1], k.shape[3]
        # sums of |terms| behind A, for error bounds
        self.A_abs = None if A is None else self.A.abs()

    def at(self, b, slots):
        s = torch.as_tensor(slots, dtype=torch.int64)
        return self.table[b][s // self.page].long(), s % self.page

    def append(self, k, v, spec=None, q=None, counts=None, mass=None):
        q_out = None if q is None else torch.zeros(q.shape, dtype=F64)
        for b, n in enumerate(self.lens):
            t = 0 if n < 0 else k.shape[2] if counts is None else int(counts[b])
            if t == 0:
                continue
            p = self.clocks[b] + torch.arange(t)
            pg, sl = self.at(b, n + torch.arange(t))
            new = k[b, :, :t] if spec is None else turn(k[b, :, :t], p, spec)
            self.k[pg, :, sl] = new.transpose(0, 1).to(self.k.dtype)
            self.v[pg, :, sl] = v[b, :, :t].transpose(0, 1)
            self.mass[pg, :, sl] = 0.0 if mass is None else mass[b, :, :t].transpose(0, 1).to(F64)
            self.pos[pg, :, sl] = p[:, None].expand(-1, self.H)
            if q is not None:
                q_out[b, :, :t] = q[b, :, :t].to(F64) if spec is None else turn(q[b, :, :t], p, spec)
            self.lens[b] += t
            self.clocks[b] += t
        return q_out

    def evict(self, budget, recent):
        for b, n in enumerate(self.lens):
            if n <= budget:
                continue
            pg, sl = self.at(b, range(n))
            for h in range(self.H):
                w = self.mass[pg, h, sl].tolist()
                z = self.pos[pg, h, sl].tolist()
                heavy = lambda x: (1, 0.0) if math.isnan(x) else (0, x)  # noqa: E731
                gone = sorted(range(n), key=lambda j: (z[j] >= self.clocks[b] - recent, heavy(w[j]), z[j], j))[:n - budget]
                if self.A is not None:
                    for j in gone:
                        kv = torch.outer(self.k[pg[j], h, sl[j]].to(F64), self.v[pg[j], h, sl[j]].to(F64)) * self.eta[h]
                        self.A[b, h] = self.lam[h] * self.A[b, h] + kv
                        self.A_abs[b, h] = self.lam[h].abs() * self.A_abs[b, h] + kv.abs()
                left = set(gone)
                free = sorted(j for j in gone if j < budget)
                tail = [j for j in range(budget, n) if j not in left]
                for to, fr in zip(free, tail):
                    for x in (self.k, self.v, self.mass, self.pos):
                        x[pg[to], h, sl[to]] = x[pg[fr], h, sl[fr]]
            self.lens[b] = budget

    def attend(self, q, g=None, accumulate=False, bad_pages=()):
        """y [B,Hq,d] float64 (rows of negative length zero) and a bound on a
        float32 computation's error; see attend_bound."""
        B, Hq, d = q.shape
        G = Hq // self.H
        y, tol = torch.zeros(B, Hq, d, dtype=F64), torch.zeros(B, Hq, d, dtype=F64)
        for b, n in enumerate(self.lens):
            if n < 0:
                continue
            slots = [j for j in range(n) if int(self.table[b][j // self.page]) not in bad_pages]
            pg, sl = self.at(b, slots)
            for h in range(self.H):
                qq = q[b, h * G:(h + 1) * G].to(F64)
                o, e = torch.zeros(G, d, dtype=F64), torch.zeros(G, d, dtype=F64)
                if slots:
                    kk, vv = self.k[pg, h, sl].to(F64), self.v[pg, h, sl].to(F64)
                    p = torch.softmax(qq @ kk.T / math.sqrt(d), -1)
                    o = p @ vv
                    # a score of d products and sums, then scaled: each step
                    # off by 2^-23 at most of the sum of magnitudes; exp turns
                    # an error of x into a factor 1 + x, in p and in the sum
                    ds = ((qq.abs() @ kk.abs().T) / math.sqrt(d)).amax(-1, keepdim=True) * (d + 4) * 2.0 ** -23
                    e = (2 * ds + (len(slots) + 64) * 2.0 ** -23 + 2.0 ** -16) * (p @ vv.abs())
                    if accumulate:
                        self.mass[pg, h, sl] += p.sum(0)
                if g is not None:
                    gate = torch.sigmoid(g[h * G:(h + 1) * G].to(F64))[:, None]
                    o = o + gate * (qq @ self.A[b, h])
                    e = e + gate * (qq.abs() @ self.A_abs[b, h]) * (d + 8) * 2.0 ** -22
                y[b, h * G:(h + 1) * G], tol[b, h * G:(h + 1) * G] = o, e
        return y, tol
