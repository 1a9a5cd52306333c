"""The losses on X·Wᵀ and their gradients in 64 bits, and how far a float32
computation of them may be off.

Tolerances count roundings.  u = 2^-23 bounds one operation of the matrix
cores and of the vector units (a whole step, as not every one of them rounds
to nearest); a matrix instruction sums 16 products, so a term of a sum of n
passes through at most n/16 + 16 roundings.  A float32 operand is split into
three planes: six times the additions, and what the split and the products
left out miss is below 8·2^-24 of the product of the magnitudes.  A rounding
to a type is off by half a step, finfo(type).eps / 2.
"""

from __future__ import annotations

import torch

U = 2.0 ** -23


def depth(n, dtype):
    return (6 if dtype == torch.float32 else 1) * (n / 16 + 1) + 16


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def teacher_probabilities(logits, temperature):
    """q (0 where there is no entry) and which rows have one."""
    t = logits.double()
    kept = t > float("-inf")
    some = kept.any(dim=1)
    high = torch.where(some, t.amax(dim=1), 0.0)[:, None]
    e = torch.where(kept, torch.exp((t - high) / temperature), 0.0)
    return e / torch.where(some, e.sum(dim=1), 1.0)[:, None], kept, some


class Reference:
    """target: (T,), or ids and logits (T, K) of a teacher."""

    def __init__(self, X, W, target=None, ignore_index=-100, ids=None, logits=None, temperature=1.0):
        self.X, self.W = X.double(), W.double()
        self.dtype, self.tau = X.dtype, temperature
        T, D = X.shape
        V = W.shape[0]
        if target is not None:
            self.counts = target != ignore_index
        else:
            q, kept, self.counts = teacher_probabilities(logits, temperature)
        self.Xc = torch.where(self.counts[:, None], self.X, 0.0)  # rows that do not count may hold anything
        z = (self.X @ self.W.t()) / temperature
        size = (self.Xc.abs() @ self.W.abs().t()) / temperature
        self.z, self.lse = z, torch.logsumexp(z, dim=1)
        off = depth(D, self.dtype) * U * size + 4 * U * z.abs()
        if self.dtype == torch.float32:
            off += 8 * 2.0 ** -24 * size
        self.z_off = off
        # exponentials of arguments up to the spread of a row, and a sum of V through 64 in a lane, the groups of
        # columns 64 apart and two exchanges
        spread = (z.amax(dim=1) - z.amin(dim=1)).clamp(max=200.0)
        self.lse_off = off.amax(dim=1) + (2 * spread + 96 + V / 2048 + 4 * self.lse.abs()) * U
        self.wanted = torch.zeros_like(z)
        if target is not None:
            r = torch.nonzero(self.counts)[:, 0]
            self.wanted[r, target[r]] = 1.0
            zt = (self.wanted * z).sum(dim=1)
            self.loss = torch.where(self.counts, self.lse - zt, 0.0)
            self.loss_off = self.lse_off + (self.wanted * off).sum(dim=1) + (self.lse.abs() + zt.abs()) * U
        else:
            safe = torch.where(kept, ids, 0)
            self.wanted.scatter_add_(1, safe, q)
            self.student = torch.where(kept, z.gather(1, safe), 0.0)
            self.student_off = torch.where(kept, off.gather(1, safe), 0.0)
            log_q = torch.where(q > 0, torch.log(torch.where(q > 0, q, 1.0)), 0.0)
            term = torch.where(kept, log_q - (self.student - self.lse[:, None]), 0.0)
            self.loss = temperature ** 2 * (q * term).sum(dim=1)
            large = torch.where(kept & (q > 0), log_q.abs() + self.student.abs() + self.lse.abs()[:, None], 0.0).amax(dim=1)
            K = ids.shape[1]
            self.loss_off = temperature ** 2 * (self.lse_off + self.student_off.amax(dim=1)
                                                + (K + 32 + large) * U * large)
            # a probability of the teacher is off by the rounding of its exponent's argument and of its sum
            self.wanted_off = (2 * large + K + 32)[:, None] * U * self.wanted

    def check_rows(self, loss, lse, student=None):
        c = self.counts
        assert bool(torch.isfinite(lse[c]).all())
        worst = ((lse.double() - self.lse).abs() / self.lse_off)[c]
        assert worst.numel() == 0 or float(worst.max()) <= 1, f"lse off by {float(worst.max())} of its tolerance"
        assert bool((loss[~c] == 0).all())
        worst = ((loss.double() - self.loss).abs() / self.loss_off)[c]
        assert worst.numel() == 0 or float(worst.max()) <= 1, f"loss off by {float(worst.max())} of its tolerance"
        if student is not None:
            bad = (student.double() - self.student).abs()[c] > self.student_off[c]
            assert not bool(bad.any())

    def gradients(self, grad):
        """dX, dW and how far each may be off, for g_t = grad[t] (64 bits)."""
        T, V = self.z.shape
        dt = self.dtype
        c = torch.where(self.counts, grad * self.tau, 0.0)[:, None]
        zs = torch.where(self.counts[:, None], self.z - self.lse[:, None], -1e9)
        p = torch.exp(zs)
        g = c * (p - self.wanted)
        rel = torch.where(self.counts[:, None], self.z_off + self.lse_off[:, None] + (zs.abs() * 4 + 8) * U, 0.0)
        off = c.abs() * (p * torch.expm1(rel.clamp(max=1.0)) + 4 * U * self.wanted)
        if hasattr(self, "wanted_off"):
            off += c.abs() * torch.where(self.counts[:, None], self.wanted_off, 0.0)
        off += half_step(dt) * g.abs()
        if dt == torch.float16:
            off += c.abs() * 2.0 ** -39  # below the least fp16 of the scaled gradient
        w, x = self.W, self.Xc
        dX, dW = g @ w, g.t() @ x
        plane = 8 * 2.0 ** -24 if dt == torch.float32 else 0.0
        gs = g.abs() + off
        # at most 64 partial sums of the vocabulary and as many pieces are added besides
        dX_off = off @ w.abs() + ((depth(V, dt) + 130) * U + plane) * (gs @ w.abs())
        dW_off = off.t() @ x.abs() + (depth(T, dt) * U + plane) * (gs.t() @ x.abs())
        least = torch.finfo(dt).tiny * torch.finfo(dt).eps  # the least subnormal number
        dX_off += half_step(dt) * (dX.abs() + dX_off) + least
        dW_off += half_step(dt) * (dW.abs() + dW_off) + least
        if dt == torch.float16:  # rows scaled by their power of two relative to the largest
            dW_off += 2.0 ** -25 * grad.abs().max() * self.tau * 2 * gs.div(c.abs().clamp(min=1e-300)).sum(dim=0)[:, None]
        return dX, dX_off, dW, dW_off

    def check_gradients(self, grad, dX=None, dW=None):
        want_x, off_x, want_w, off_w = self.gradients(grad)
        if dX is not None:
            self.within("dX", dX, want_x, off_x)
            assert bool((dX[~self.counts] == 0).all())
        if dW is not None:
            self.within("dW", dW, want_w, off_w)

    @staticmethod
    def within(name, got, want, off):
        assert bool(torch.isfinite(got).all()), f"{name} is not finite"
        d = (got.double() - want).abs()
        over = d > off
        if bool(over.any()):
            at = torch.nonzero(over)[0].tolist()
            raise AssertionError(f"{name}{at}: {float(got[tuple(at)])} for {float(want[tuple(at)])}, tolerance "
                                 f"{float(off[tuple(at)])}; {int(over.sum())} of {over.numel()} are over theirs")
