"""What each pair's accumulated weight grows by in one attention, and how far a
float32 computation of it may be off.  Test infrastructure only."""
import math

import torch

F64 = torch.float64


def weights(cpu, q):
    """cpu: a paged_reference.Cache, q [B,Hq,d].  Growth of cpu.mass, its bound
    (both shaped as mass), and where there is a pair.

    A score is d products and their sum, scaled: off by (d + 4) 2^-23 of the sum
    of its terms' magnitudes at most (each step rounds or truncates by 2^-23 of
    what it has).  exp turns an error of its argument into a factor, in the weight
    and in the sum it is divided by; the exponential itself, rescaling and the sum
    over n pairs add (n + 64) 2^-23.  The sum over the heads and onto the old
    weight rounds by 2^-24 of the result, G + 1 times."""
    B, Hq, d = q.shape
    G = Hq // cpu.H
    grow, tol = torch.zeros_like(cpu.mass), torch.zeros_like(cpu.mass)
    held = torch.zeros_like(cpu.mass, dtype=torch.bool)
    for b, n in enumerate(cpu.lens):
        if n <= 0:
            continue
        pg, sl = cpu.at(b, range(n))
        for h in range(cpu.H):
            qq, kk = q[b, h * G:(h + 1) * G].to(F64), cpu.k[pg, h, sl].to(F64)
            p = torch.softmax(qq @ kk.T / math.sqrt(d), -1)
            ds = ((qq.abs() @ kk.abs().T) / math.sqrt(d)).amax(-1, keepdim=True) * (d + 4) * 2.0 ** -23
            g = p.sum(0)
            held[pg, h, sl] = True
            grow[pg, h, sl] = g
            tol[pg, h, sl] = (p * (2 * ds + (n + 64) * 2.0 ** -23)).sum(0) + (G + 1) * 2.0 ** -24 * (cpu.mass[pg, h, sl].abs() + g)
    return grow, tol, held
