"""Plain 64-bit forms of the dense cross attention, its gradients and the
8-bit checkpoints on CPU tensors, with the error bounds the tests use, each
derived from the arithmetic of the kernels:

u = 2^-24 is fp32's rounding, r half a step of the token type (2^-8 for bf16;
0 stands for fp32, whose own rounding is among the u terms).

* A score is a d-term fp32 dot product of exact products, scaled:
  |ds_ij| <= e_s = (d + 8) u scale sum_k |q_k k_k|, plus 2^-20 for the
  subtraction, base change and exp of the weight (each a few u of |s - m|,
  and 2^-22 for the exponential): weights are off by a factor 1 +- e_w with
  e_w = 2 e_s + 2^-20 + 4 u |s - m|_max.
* Sums over n terms go through tiles of at most 128 and a running sum of the
  tiles: (128 + n / 64 + 16) u =: e_n of the sum of magnitudes.
* With bf16 the weights p and the score gradients ds enter the second product
  rounded to bf16: one more r each.
"""
import math

import torch

U = 2.0 ** -24


def rounding(dtype):
    return torch.finfo(dtype).eps / 2 if dtype != torch.float32 else 0.0


def _en(n):
    return (128 + n / 64 + 16) * U


def lens_of(k_len, B, Nk):
    if k_len is None:
        return [Nk] * B
    return [min(max(int(x), 0), Nk) for x in k_len]


def forward(q, k, v, scale, k_len=None):
    """O, lse and their bounds, all float64 [B, Hq, Nq, (d)]."""
    r = rounding(q.dtype)
    q64, k64, v64 = (t.detach().cpu().double() for t in (q, k, v))
    B, Hq, Nq, d = q64.shape
    G = Hq // k64.shape[1]
    O = torch.zeros(B, Hq, Nq, d, dtype=torch.float64)
    lse = torch.full((B, Hq, Nq), -math.inf, dtype=torch.float64)
    tO, tl = torch.zeros_like(O), torch.zeros(B, Hq, Nq, dtype=torch.float64)
    for b, n in enumerate(lens_of(k_len, B, k64.shape[2])):
        for h in range(Hq if n else 0):
            qq, kk, vv = q64[b, h], k64[b, h // G, :n], v64[b, h // G, :n]
            s = scale * (qq @ kk.T)
            e_s = ((d + 8) * U * scale * (qq.abs() @ kk.abs().T)).amax(1)
            span = (s.amax(1) - s.amin(1)) + s.abs().amax(1)
            e_w = 2 * e_s + 2.0 ** -20 + 4 * U * span
            m = s.amax(1, keepdim=True)
            p = torch.exp(s - m)
            l = p.sum(1)
            O[b, h] = (p @ vv) / l[:, None]
            lse[b, h] = m[:, 0] + torch.log(l)
            mag = (p @ vv.abs()) / l[:, None]
            tO[b, h] = ((r + 2 * U) * O[b, h].abs()
                        + mag * (r + 2 * e_w + 2 * _en(n) + 2.0 ** -20)[:, None])
            tl[b, h] = e_w + _en(n) + 4 * U * lse[b, h].abs() + 2.0 ** -20
    return O, lse, tO, tl


def backward(do, q, k, v, o, lse, scale, k_len=None):
    """(dQ, dK, dV) and their bounds, float64.  q and o may be float64 already
    (the values of a checkpoint); the rounding is k's type's."""
    r = rounding(k.dtype)
    do64, q64, k64, v64, o64, lse64 = (t.detach().cpu().double() for t in (do, q, k, v, o, lse))
    B, Hq, Nq, d = q64.shape
    G = Hq // k64.shape[1]
    dQ, dK, dV = torch.zeros_like(q64), torch.zeros_like(k64), torch.zeros_like(k64)
    tQ, tK, tV = torch.zeros_like(q64), torch.zeros_like(k64), torch.zeros_like(k64)
    for b, n in enumerate(lens_of(k_len, B, k64.shape[2])):
        for h in range(Hq if n else 0):
            qq, gg, oo = q64[b, h], do64[b, h], o64[b, h]
            kk, vv = k64[b, h // G, :n], v64[b, h // G, :n]
            s = scale * (qq @ kk.T)
            e_s = (d + 8) * U * scale * (qq.abs() @ kk.abs().T)
            e_w = 2 * e_s + 2.0 ** -20 + 4 * U * (s.abs() + lse64[b, h].abs()[:, None])
            p = torch.exp(s - lse64[b, h][:, None])
            dp, delta = gg @ vv.T, (gg * oo).sum(1, keepdim=True)
            ds = p * (dp - delta)
            e_dp = (d + 8) * U * (gg.abs() @ vv.abs().T + (gg * oo).abs().sum(1, keepdim=True))
            e_p = p * (r + e_w)                       # error of a weight entering dV
            e_ds = ds.abs() * (r + e_w + 4 * U) + p * (1 + r) * e_dp
            dQ[b, h] = scale * (ds @ kk)
            tQ[b, h] = scale * (e_ds + _en(n) * ds.abs()) @ kk.abs()
            dK[b, h // G, :n] += scale * (ds.T @ qq)
            tK[b, h // G, :n] += scale * (e_ds + _en(Nq * G) * ds.abs()).T @ qq.abs()
            dV[b, h // G, :n] += p.T @ gg
            tV[b, h // G, :n] += (e_p + _en(Nq * G) * p).T @ gg.abs()
    f = r + 4 * U
    return (dQ, dK, dV), (tQ * 1.01 + f * dQ.abs() + 1e-30, tK * 1.01 + f * dK.abs() + 1e-30,
                          tV * 1.01 + f * dV.abs() + 1e-30)


def pack(x):
    """Codes (int64) and exponent bytes of a checkpoint, group by group."""
    g = x.detach().cpu().double().unflatten(-1, (-1, 32))
    top = g.abs().amax(-1, keepdim=True)
    bad = ~torch.isfinite(g).all(-1, keepdim=True)
    top = torch.where(bad, torch.zeros_like(top), top)
    e = torch.full(top.shape, -127.0, dtype=torch.float64)
    for _ in range(256):      # the smallest e that keeps every quotient within 127
        over = (torch.round(torch.ldexp(top, -e)) > 127) & (e < 121)
        if not over.any():
            break
        e = torch.where(over, e + 1, e)
    codes = torch.round(torch.ldexp(torch.where(bad, torch.zeros_like(g), g), -e)).clamp(-127, 127)
    exps = torch.where(bad, torch.full_like(e, 255), e + 127)
    return codes.flatten(-2).long(), exps.squeeze(-1).long()


def unpack(codes, exps):
    e = exps.cpu().double()
    step = torch.ldexp(torch.ones_like(e), e - 127)
    step = torch.where(e == 255, torch.full_like(e, math.nan), step)
    return codes.cpu().double() * step.repeat_interleave(32, -1)
