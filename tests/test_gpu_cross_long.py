"""Cross attention at video length against the 64-bit forms: long sums of equal terms, whose
rounding errors do not cancel, and the forward and backward passes of 75,600 queries."""
import pytest
import torch

import cross_oracle as co
from test_gpu_cross import _csa, _klen, _within

pytestmark = pytest.mark.gpu

BF, FP = torch.bfloat16, torch.float32
VIDEO = 75600
HEADS = 150           # more than the GPU has multiprocessors: long sums are not cut
CHECKED = (0, 75, 149)


def _randn(seed, *shape):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed))


@pytest.mark.parametrize("dtype", [FP, BF])
def test_equal_terms_over_many_queries(dtype):
    """dV and dK as sums over 75,600 equal queries (O = 0, so that ds = p dO.v): one chain of
    fp32 additions is off by up to 1e-3."""
    d, Nk = 64, 64
    q = (0.2 * _randn(1, 1, 1, 1, d).abs()).to(dtype).cuda().expand(1, 1, VIDEO, d).contiguous()
    q = q.expand(1, HEADS, VIDEO, d)
    k = (0.2 * _randn(2, 1, HEADS, Nk, d).abs()).to(dtype).cuda()
    one = torch.ones(1, 1, 1, 1, dtype=dtype, device="cuda")
    v = one.expand(1, HEADS, 1, d).contiguous().expand(1, HEADS, Nk, d).contiguous()
    do = one.expand(1, 1, VIDEO, d).contiguous().expand(1, HEADS, VIDEO, d)
    O = torch.zeros(1, 1, VIDEO, d, dtype=dtype, device="cuda").expand(1, HEADS, VIDEO, d)
    lse = _csa().svgear_cross_attend(q, k, v, 0.125)[1]
    got = _csa().svgear_cross_attend_backward(do, q, k, v, O, lse, 0.125, check_status=True)
    for h in CHECKED:
        at = [t[:, h:h + 1] for t in (do, q, k, v, O, lse)]
        want, tol = co.backward(*at, 0.125)
        for g, w, t, name in zip(got, want, tol, ("dQ", "dK", "dV")):
            _within(g[:, h:h + 1], w, t, "%s, head %d" % (name, h))


@pytest.mark.parametrize("dtype", [FP, BF])
def test_equal_terms_over_many_keys(dtype):
    """O, lse and dQ as sums over 75,600 keys that the heads share, all but the first equal."""
    d, Nq = 64, 33
    q = _randn(3, 1, HEADS, Nq, d).abs().to(dtype).cuda()
    k = (0.2 * _randn(4, 1, 1, 1, d).abs()).to(dtype).cuda().expand(1, 1, VIDEO, d).contiguous()
    k[:, :, 0] *= 2
    v = torch.ones(1, 1, VIDEO, d, dtype=dtype, device="cuda")
    O, lse = _csa().svgear_cross_attend(q, k, v, 0.125, check_status=True)
    do, zero = torch.ones_like(q), torch.zeros_like(q)
    dq = _csa().svgear_cross_attend_backward(do, q, k, v, zero, lse, 0.125, check_status=True)[0]
    for h in CHECKED:
        at = slice(h, h + 1)
        wO, wl, tO, tl = co.forward(q[:, at], k, v, 0.125)
        _within(lse[:, at], wl, tl, "lse, head %d" % h)
        _within(O[:, at], wO, tO, "O, head %d" % h)
        want, tol = co.backward(do[:, at], q[:, at], k, v, zero[:, at], lse[:, at], 0.125)
        _within(dq[:, at], want[0], tol[0], "dQ, head %d" % h)


@pytest.mark.parametrize("dtype", [FP, BF])
def test_video_tokens_over_a_prompt(dtype):
    """Forward, backward and backward from checkpoints of 75,600 strided queries, two heads
    sharing the keys of a padded prompt."""
    csa, d, lens, scale = _csa(), 128, [500], 128 ** -0.5
    q, do = (_randn(s, 1, VIDEO, 2, d).to(dtype).cuda().transpose(1, 2) for s in (5, 6))
    k, v = (_randn(s, 1, 1, 512, d).to(dtype).cuda() for s in (7, 8))
    O, lse = csa.svgear_cross_attend(q, k, v, scale, k_len=_klen(lens), check_status=True)
    wO, wl, tO, tl = co.forward(q, k, v, scale, lens)
    _within(lse, wl, tl, "lse")
    _within(O, wO, tO, "O")
    got = csa.svgear_cross_attend_backward(do, q, k, v, O, lse, scale, k_len=_klen(lens),
                                           check_status=True)
    want, tol = co.backward(do, q, k, v, O, lse, scale, lens)
    for g, w, t, name in zip(got, want, tol, ("dQ", "dK", "dV")):
        _within(g, w, t, name)
    qc, oc = csa.svgear_checkpoint_save(q), csa.svgear_checkpoint_save(O)
    got = csa.svgear_cross_attend_backward_ckpt(do, qc, k, v, oc, lse, scale, k_len=_klen(lens),
                                                check_status=True)
    want, tol = co.backward(do, co.unpack(qc.codes, qc.exps), k, v, co.unpack(oc.codes, oc.exps),
                            lse, scale, lens)
    for g, w, t, name in zip(got, want, tol, ("dQ", "dK", "dV")):
        _within(g, w, t, name + " from checkpoints")
