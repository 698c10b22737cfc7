"""Dense cross attention (forward, backward) and the 8-bit activation
checkpoints on the GPU against their 64-bit forms (cross_oracle.py)."""
import math

import pytest
import torch

import cross_oracle as co

pytestmark = pytest.mark.gpu

BF, FP = torch.bfloat16, torch.float32


def _csa():
    import clustered_sparse_attention_b200 as csa
    return csa


def _tokens(g, B, H, N, d, dtype, layout="head", gain=1.0):
    shape = (B, H, N, d) if layout == "head" else (B, N, H, d)
    x = (torch.randn(shape, generator=g) * gain).to(dtype).cuda()
    return x if layout == "head" else x.transpose(1, 2)


def _inputs(seed, B, Hq, Hkv, Nq, Nk, d, dtype, layout="head", gain=1.0):
    g = torch.Generator().manual_seed(seed)
    q = _tokens(g, B, Hq, Nq, d, dtype, layout, gain)
    k = _tokens(g, B, Hkv, Nk, d, dtype, layout, gain)
    v = _tokens(g, B, Hkv, Nk, d, dtype, layout)
    do = _tokens(g, B, Hq, Nq, d, dtype, layout)
    return q, k, v, do


def _within(got, want, tol, what):
    got = got.detach().cpu().double()
    assert got.shape == want.shape, what
    same = got == want               # infinities among them
    bad = ~((got - want).abs() <= tol) & ~same
    assert not bad.any(), "%s: %d of %d off, worst %.3g of its bound" % (
        what, int(bad.sum()), bad.numel(),
        float(((got - want).abs() / tol)[bad].nan_to_num(math.inf).max()))


def _klen(lens):
    return None if lens is None else torch.tensor(lens, dtype=torch.int32, device="cuda")


def _check_forward(q, k, v, lens, scale, **kw):
    O, lse = _csa().svgear_cross_attend(q, k, v, scale, k_len=_klen(lens), check_status=True, **kw)
    torch.cuda.synchronize()
    wO, wl, tO, tl = co.forward(q, k, v, scale, lens)
    _within(lse, wl, tl, "lse")
    _within(O, wO, tO, "O")
    return O, lse


def _check_backward(do, q, k, v, O, lse, lens, scale):
    got = _csa().svgear_cross_attend_backward(do, q, k, v, O, lse, scale, k_len=_klen(lens),
                                              check_status=True)
    torch.cuda.synchronize()
    want, tol = co.backward(do, q, k, v, O, lse, scale, lens)
    for g, w, t, name in zip(got, want, tol, ("dQ", "dK", "dV")):
        _within(g, w, t, name)
    for b, n in enumerate(co.lens_of(lens, k.shape[0], k.shape[2])):
        assert not got[1][b, :, n:].any() and not got[2][b, :, n:].any()
        if n == 0:
            assert not got[0][b].any()
    return got


SHAPES = [
    # B, Hq, Hkv, Nq, Nk, lens
    (1, 1, 1, 1, 1, None),
    (1, 3, 3, 1, 77, None),
    (2, 2, 2, 5, 128, [128, 1]),
    (1, 2, 2, 128, 129, None),
    (3, 4, 2, 127, 127, [127, 64, 0]),
    (2, 6, 2, 129, 300, [65, 300]),
    (1, 2, 1, 257, 512, None),
    (1, 4, 1, 383, 255, [254]),
    (2, 2, 2, 64, 64, [63, 64]),
    (1, 1, 1, 700, 641, [640]),
]


@pytest.mark.parametrize("layout", ["head", "token"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dtype", [FP, BF])
@pytest.mark.parametrize("shape", SHAPES)
def test_forward_and_backward(shape, dtype, d, layout):
    B, Hq, Hkv, Nq, Nk, lens = shape
    q, k, v, do = _inputs(1, B, Hq, Hkv, Nq, Nk, d, dtype, layout)
    O, lse = _check_forward(q, k, v, lens, d ** -0.5)
    if layout == "token":
        assert O.stride() == q.stride()
    _check_backward(do, q, k, v, O, lse, lens, d ** -0.5)


@pytest.mark.parametrize("dtype", [FP, BF])
@pytest.mark.parametrize("Nq,Nk,lens", [(1, 5000, None), (3, 20011, [20011, 9]), (77, 12345, [0, 12288]),
                                        (130, 4097, [4097, 2049])])
def test_few_queries_over_many_keys(Nq, Nk, lens, dtype):
    B = 1 if lens is None else 2
    q, k, v, do = _inputs(2, B, 2, 1, Nq, Nk, 128, dtype)
    O, lse = _check_forward(q, k, v, lens, 0.1)
    _check_backward(do, q, k, v, O, lse, lens, 0.1)


@pytest.mark.parametrize("dtype", [FP, BF])
def test_many_queries_over_few_keys(dtype):
    q, k, v, do = _inputs(3, 2, 4, 2, 4001, 77, 64, dtype)
    O, lse = _check_forward(q, k, v, [77, 13], 0.125)
    _check_backward(do, q, k, v, O, lse, [77, 13], 0.125)


@pytest.mark.parametrize("layout", ["head", "token"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Nk,lens", [(512, [512, 0, 449]), (513, [513, 0, 512]), (64, [64, 1, 0]), (65, [65, 64, 0])])
def test_fp32_gradients_either_side_of_the_key_limit(Nk, lens, d, layout):
    """fp32 dQ comes from the dK/dV kernel's parts up to 512 keys, from its own kernel past that."""
    q, k, v, do = _inputs(17, 3, 4, 2, 133, Nk, d, FP, layout)
    O, lse = _check_forward(q, k, v, lens, d ** -0.5)
    _check_backward(do, q, k, v, O, lse, lens, d ** -0.5)


@pytest.mark.parametrize("dtype", [FP, BF])
@pytest.mark.parametrize("d", [64, 128])
def test_peaked_scores(dtype, d):
    """Scores of some hundreds: the running maximum moves, most weights vanish."""
    q, k, v, do = _inputs(4, 1, 2, 2, 200, 700, d, dtype, gain=6.0)
    k = k * torch.linspace(0.05, 1.5, 700, device="cuda").to(dtype)[None, None, :, None]
    O, lse = _check_forward(q, k, v, None, 0.5)
    _check_backward(do, q, k, v, O, lse, None, 0.5)


@pytest.mark.parametrize("dtype", [FP, BF])
@pytest.mark.parametrize("fill", [float("nan"), float("inf"), -float("inf"), "lowest"])
def test_padded_rows_may_hold_anything(dtype, fill):
    lens = [70, 0, 130]
    q, k, v, do = _inputs(5, 3, 2, 2, 150, 200, 128, dtype)
    fill = torch.finfo(dtype).min if fill == "lowest" else fill
    kp, vp = k.clone(), v.clone()
    for b, n in enumerate(lens):
        kp[b, :, n:] = fill
        vp[b, :, n:] = fill
    csa, kl = _csa(), _klen(lens)
    O, lse = csa.svgear_cross_attend(q, k, v, k_len=kl)
    Op, lsep = csa.svgear_cross_attend(q, kp, vp, k_len=kl)
    assert torch.equal(O, Op) and torch.equal(lse, lsep)
    assert not O[1].any() and bool((lse[1] == -math.inf).all())
    a = csa.svgear_cross_attend_backward(do, q, k, v, O, lse, k_len=kl)
    b = csa.svgear_cross_attend_backward(do, q, kp, vp, O, lse, k_len=kl)
    for x, y in zip(a, b):
        assert torch.equal(x, y) and bool(torch.isfinite(x).all())


@pytest.mark.parametrize("dtype", [FP, BF])
def test_lengths_outside_the_tensor_are_clamped(dtype):
    q, k, v, do = _inputs(6, 2, 2, 2, 40, 100, 64, dtype)
    O, lse = _check_forward(q, k, v, [1 << 30, -5], 0.2)
    _check_backward(do, q, k, v, O, lse, [1 << 30, -5], 0.2)


@pytest.mark.parametrize("dtype", [FP, BF])
def test_not_a_number_stays_in_its_row(dtype):
    q, k, v, _ = _inputs(7, 1, 2, 2, 300, 140, 128, dtype)
    want, wl, tO, tl = co.forward(q, k, v, 0.1)
    q[0, 1, 200, 3] = float("nan")
    O, lse = _csa().svgear_cross_attend(q, k, v, 0.1)
    assert bool(torch.isnan(O[0, 1, 200]).all()) and bool(torch.isnan(lse[0, 1, 200]))
    keep = torch.ones(1, 2, 300, dtype=torch.bool)
    keep[0, 1, 200] = False
    _within(O.cpu()[keep], want[keep], tO[keep], "O")
    _within(lse.cpu()[keep], wl[keep], tl[keep], "lse")


@pytest.mark.parametrize("dtype", [FP, BF])
def test_strided_and_broadcast_inputs(dtype):
    """q, k, v as slices of one packed projection, k and v of one prompt
    broadcast over the batch, O and lse written into given buffers with a
    guard around them."""
    B, H, N, d = 2, 3, 150, 64
    g = torch.Generator().manual_seed(8)
    packed = torch.randn(B, N, 3, H, d, generator=g).to(dtype).cuda()
    q = packed[:, :, 0].transpose(1, 2)
    kv = torch.randn(1, 1, 90, 2, d, generator=g).to(dtype).cuda()
    k = kv[:, :, :, 0].expand(B, H, 90, d)
    v = kv[:, :, :, 1].expand(B, H, 90, d)
    do = torch.randn(B, H, N, d, generator=g).to(dtype).cuda()
    buf = torch.full((B, N + 2, H, 2 * d), 7.0, dtype=dtype, device="cuda")
    O = buf[:, 1:-1, :, :d].transpose(1, 2)
    out, lse = _check_forward(q, k, v, [90, 31], 0.1, O=O)
    assert out.data_ptr() == O.data_ptr()
    guard = torch.ones_like(buf, dtype=torch.bool)
    guard[:, 1:-1, :, :d] = False
    assert bool((buf[guard] == 7).all())
    _check_backward(do, q, k, v, O, lse, [90, 31], 0.1)


@pytest.mark.parametrize("dtype", [FP, BF])
def test_equal_calls_give_equal_bits(dtype):
    q, k, v, do = _inputs(9, 2, 8, 2, 1000, 333, 128, dtype)
    csa, kl = _csa(), _klen([333, 100])

    def run():
        O, lse = csa.svgear_cross_attend(q, k, v, k_len=kl)
        return (O, lse) + csa.svgear_cross_attend_backward(do, q, k, v, O, lse, k_len=kl)

    first = run()
    for _ in range(3):
        for a, b in zip(first, run()):
            assert torch.equal(a, b)


@pytest.mark.parametrize("dtype", [FP, BF])
def test_gradients_match_differences(dtype):
    """Central differences of the 64-bit loss at the kernel's own inputs."""
    q, k, v, do = _inputs(10, 1, 2, 1, 20, 33, 64, dtype)
    csa, scale = _csa(), 0.125
    O, lse = csa.svgear_cross_attend(q, k, v, scale)
    grads = csa.svgear_cross_attend_backward(do, q, k, v, O, lse, scale)
    # the saved O is rounded to the token type: the gradient with it, and its
    # distance from the one with the exact O, |ds| += p |do| |o| r
    o64, lse64, tO, tl = co.forward(q, k, v, scale)
    want, tol = co.backward(do, q, k, v, O, lse, scale)
    exact, _ = co.backward(do, q, k, v, o64, lse64, scale)
    host = [t.detach().cpu().double() for t in (q, k, v)]
    do64 = do.cpu().double()
    g = torch.Generator().manual_seed(11)
    h = 1e-4
    for i in range(3):
        for _ in range(6):
            dirn = torch.randn(host[i].shape, generator=g, dtype=torch.float64)
            up, down = list(host), list(host)
            up[i], down[i] = host[i] + h * dirn, host[i] - h * dirn
            diff = sum(s * float((co.forward(*x, scale)[0] * do64).sum())
                       for s, x in ((1, up), (-1, down))) / (2 * h)
            slack = float((dirn.abs() * (tol[i] + (want[i] - exact[i]).abs())).sum())
            got = float((grads[i].cpu().double() * dirn).sum())
            assert abs(got - diff) <= slack + 1e-5 * (1 + abs(diff))


@pytest.mark.parametrize("dtype", [FP, BF])
def test_graph_replay_and_side_stream(dtype):
    q, k, v, do = _inputs(12, 2, 4, 2, 300, 200, 128, dtype)
    csa, kl = _csa(), _klen([200, 77])

    def run():
        O, lse = csa.svgear_cross_attend(q, k, v, k_len=kl)
        return (O, lse) + csa.svgear_cross_attend_backward(do, q, k, v, O, lse, k_len=kl)

    want = [t.clone() for t in run()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = run()
    side.synchronize()
    for a, b in zip(want, other):
        assert torch.equal(a, b)
    graphs = []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = run()
        graphs.append((graph, out))
    for graph, out in graphs + graphs[::-1]:
        for t in out:
            t.fill_(3)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(want, out):
            assert torch.equal(a, b)
    # new lengths and values in the captured buffers
    kl.copy_(torch.tensor([3, 0], dtype=torch.int32))
    q.mul_(0.5)
    graphs[0][0].replay()
    torch.cuda.synchronize()
    for a, b in zip(graphs[0][1], run()):
        assert torch.equal(a, b)


def test_two_calls_at_once():
    """Two streams, both kernels of either call resident together or in turn."""
    csa = _csa()
    sets = [_inputs(20 + i, 1, 8, 8, 3000, 300, 128, BF) for i in range(2)]
    want = []
    for q, k, v, do in sets:
        O, lse = csa.svgear_cross_attend(q, k, v)
        want.append((O, lse) + csa.svgear_cross_attend_backward(do, q, k, v, O, lse))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(5):
        got = []
        for s, (q, k, v, do) in zip(streams, sets):
            with torch.cuda.stream(s):
                O, lse = csa.svgear_cross_attend(q, k, v)
                got.append((O, lse) + csa.svgear_cross_attend_backward(do, q, k, v, O, lse))
        torch.cuda.synchronize()
        for a, b in zip(want, got):
            for x, y in zip(a, b):
                assert torch.equal(x, y)


@pytest.mark.parametrize("dtype", [FP, BF])
def test_offsets_past_32_bits(dtype):
    """Rows of k, v, q and o far apart in one buffer: element offsets past 2^31."""
    row, N, d = 1 << 16, 33000, 64                       # 2.16e9 elements
    buf = torch.empty(N * row, dtype=dtype, device="cuda")
    g = torch.Generator().manual_seed(14)
    far = [buf.as_strided((1, 2, N, d), (0, d, row, 1), 2 * d * i) for i in range(4)]
    for t in far:
        t.copy_(torch.randn(1, 2, N, d, generator=g).to(dtype))
    q, k, v, O = far
    few = q[:, :, -3:]
    o1, l1 = _csa().svgear_cross_attend(few, k, v, 0.1)
    w, wl, tO, tl = co.forward(few, k, v, 0.1)
    _within(o1, w, tO, "O")
    _within(l1, wl, tl, "lse")
    kk, vv = k[:, :, -70:], v[:, :, -70:]
    lse = _csa().svgear_cross_attend(q, kk, vv, 0.1, O=O)[1]
    dense = [t.contiguous() for t in (q, kk, vv)]
    o2, lse2 = _csa().svgear_cross_attend(*dense, 0.1)
    assert torch.equal(O, o2) and torch.equal(lse, lse2)
    do = dense[0] * 0.5
    got = _csa().svgear_cross_attend_backward(do, q, kk, vv, O, lse, 0.1)
    want = _csa().svgear_cross_attend_backward(do, *dense, o2, lse2, 0.1)
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    c = _csa().svgear_checkpoint_save(q)
    assert torch.equal(c.codes, _csa().svgear_checkpoint_save(dense[0]).codes)


@pytest.mark.parametrize("dtype", [FP, BF])
def test_many_batches_and_heads(dtype):
    """More batches than lanes or CTAs, most of them without keys."""
    B, Hq, Hkv, Nq, Nk, d = 700, 2, 1, 3, 40, 64
    q, k, v, do = _inputs(15, B, Hq, Hkv, Nq, Nk, d, dtype)
    lens = [(7 * b) % 41 if b % 3 == 0 else 0 for b in range(B)]
    O, lse = _check_forward(q, k, v, lens, 0.2)
    _check_backward(do, q, k, v, O, lse, lens, 0.2)


def test_arguments_by_name_and_given_outputs():
    csa = _csa()
    q, k, v, do = _inputs(16, 1, 2, 2, 140, 60, 64, BF)
    want = csa.svgear_cross_attend(q, k, v)
    lse = torch.full((1, 2, 140), 9.0, device="cuda")
    O, got = csa.svgear_cross_attend(Q=q, K=k, V=v, lse=lse)
    assert got is lse and torch.equal(O, want[0]) and torch.equal(lse, want[1])
    c = csa.svgear_checkpoint_save(X=q)
    assert torch.equal(csa.svgear_checkpoint_load(c=c), csa.svgear_checkpoint_load(c))
    a = csa.svgear_cross_attend_backward(dO=do, Q=q, K=k, V=v, O=O, lse=lse)
    b = csa.svgear_cross_attend_backward(do, q, k, v, O, lse)
    for x, y in zip(a, b):
        assert torch.equal(x, y)


def test_binding_refusals_on_the_gpu():
    csa = _csa()
    q, k, v, do = _inputs(13, 2, 4, 2, 10, 12, 64, BF)
    O, lse = csa.svgear_cross_attend(q, k, v)
    with pytest.raises(ValueError, match="V must"):
        csa.svgear_cross_attend(q, k, v[:, :, :5])
    with pytest.raises(ValueError, match="K must"):
        csa.svgear_cross_attend(q, k[:1], v[:1])
    with pytest.raises(ValueError, match="K must"):
        csa.svgear_cross_attend(q, k.float(), v)
    with pytest.raises(ValueError, match="contiguous"):
        csa.svgear_cross_attend(q.transpose(2, 3), k, v)
    with pytest.raises(ValueError, match="k_len"):
        csa.svgear_cross_attend(q, k, v, k_len=torch.tensor([1, 2], device="cuda"))
    with pytest.raises(ValueError, match="k_len"):
        csa.svgear_cross_attend(q, k, v, k_len=torch.tensor([1, 2], dtype=torch.int32))
    with pytest.raises(ValueError, match="lse"):
        csa.svgear_cross_attend_backward(do, q, k, v, O, lse.double())
    with pytest.raises(ValueError, match="dO"):
        csa.svgear_cross_attend_backward(do[:, :2], q, k, v, O, lse)
    with pytest.raises(TypeError):
        csa.svgear_cross_attend(q.half(), k.half(), v.half())
    with pytest.raises(csa.SvgearError, match="invalid"):
        csa.svgear_cross_attend(q, k, v, scale=-1.0)
    with pytest.raises(csa.SvgearError):
        csa.svgear_cross_attend(q, k[:, :1].expand(2, 3, 12, 64), v[:, :1].expand(2, 3, 12, 64))
    with pytest.raises(csa.SvgearError, match="invalid"):      # O's heads overlap
        csa.svgear_cross_attend(q, k, v, O=O[:, :1].expand(2, 4, 10, 64))
    with pytest.raises(csa.SvgearError):                       # rows not on 16 bytes
        csa.svgear_cross_attend(q, k, torch.zeros(2, 2, 12, 65, dtype=BF, device="cuda")[..., :64])
    with pytest.raises(ValueError, match="Qc"):
        csa.svgear_cross_attend_backward_ckpt(do, csa.svgear_checkpoint_save(q.float()), k, v,
                                              csa.svgear_checkpoint_save(O), lse)


# ---------------------------------------------------------------------------
# Checkpoints
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("layout", ["head", "token"])
@pytest.mark.parametrize("dtype", [FP, BF])
@pytest.mark.parametrize("B,H,N,d", [(1, 1, 1, 64), (2, 3, 37, 128), (1, 5, 1001, 64), (3, 1, 2, 128)])
def test_checkpoint_round_trip(B, H, N, d, dtype, layout):
    csa = _csa()
    g = torch.Generator().manual_seed(30)
    shape = (B, H, N, d) if layout == "head" else (B, N, H, d)
    x = torch.randn(shape, generator=g) * torch.exp(20 * torch.randn(shape[:-1] + (1,), generator=g))
    x = x.clamp(-3e38, 3e38).to(dtype).cuda()
    x = x if layout == "head" else x.transpose(1, 2)
    c = csa.svgear_checkpoint_save(x)
    codes, exps = co.pack(x)
    assert torch.equal(c.codes.cpu().long(), codes) and torch.equal(c.exps.cpu().long(), exps)
    y = csa.svgear_checkpoint_load(c)
    assert y.dtype == dtype and torch.equal(y.cpu().double(), co.unpack(codes, exps))
    if layout == "token":
        out = torch.zeros(B, N, H, 2 * d, dtype=dtype, device="cuda")
        csa.svgear_checkpoint_load(c, out=out[..., :d].transpose(1, 2))
        assert torch.equal(out[..., :d].transpose(1, 2), y) and not out[..., d:].any()


@pytest.mark.parametrize("dtype", [FP, BF])
def test_checkpoint_special_values(dtype):
    csa = _csa()
    x = torch.zeros(1, 1, 12, 64, dtype=dtype, device="cuda")
    x[0, 0, 0] = 1.9921875                               # 127.5 steps
    x[0, 0, 1, :32] = torch.finfo(dtype).max
    x[0, 0, 1, 32:] = -torch.finfo(dtype).max
    x[0, 0, 2, 5] = float("inf")
    x[0, 0, 3, 40] = float("nan")
    x[0, 0, 4] = torch.finfo(dtype).tiny                 # smallest normal number
    x[0, 0, 5] = torch.finfo(dtype).tiny / 4             # below it
    x[0, 0, 6, 0] = 2.0 ** -120
    x[0, 0, 7, 0] = 127.5 * 2.0 ** -127
    x[0, 0, 8] = -0.0
    x[0, 0, 9] = torch.arange(64) - 31.5
    codes, exps = co.pack(x)
    c = csa.svgear_checkpoint_save(x)
    assert torch.equal(c.codes.cpu().long(), codes) and torch.equal(c.exps.cpu().long(), exps)
    y = csa.svgear_checkpoint_load(c).cpu().double()
    want = co.unpack(codes, exps)
    assert torch.equal(y.isnan(), want.isnan())
    assert bool((y == want)[~want.isnan()].all())


@pytest.mark.parametrize("dtype", [FP, BF])
@pytest.mark.parametrize("shape", [(1, 1, 1, 1, 1, None), (2, 4, 2, 129, 300, [300, 65]),
                                   (1, 2, 2, 1000, 77, [0]), (3, 2, 1, 260, 130, [1, 130, 128])])
@pytest.mark.parametrize("d", [64, 128])
def test_backward_from_checkpoints(shape, dtype, d):
    csa = _csa()
    B, Hq, Hkv, Nq, Nk, lens = shape
    q, k, v, do = _inputs(40, B, Hq, Hkv, Nq, Nk, d, dtype, "token")
    O, lse = csa.svgear_cross_attend(q, k, v, k_len=_klen(lens))
    qc, oc = csa.svgear_checkpoint_save(q), csa.svgear_checkpoint_save(O)
    got = csa.svgear_cross_attend_backward_ckpt(do, qc, k, v, oc, lse, k_len=_klen(lens),
                                                check_status=True)
    want, tol = co.backward(do, co.unpack(qc.codes, qc.exps), k, v, co.unpack(oc.codes, oc.exps),
                            lse, d ** -0.5, lens)
    for g, w, t, name in zip(got, want, tol, ("dQ", "dK", "dV")):
        _within(g, w, t, name)
    assert got[0].stride() == do.stride()


@pytest.mark.parametrize("dtype", [FP, BF])
@pytest.mark.parametrize("gain", [1.0, 2.0])
def test_checkpoint_gradients_beside_those_of_the_saved_tensors(dtype, gain):
    """How far holding q and o in 8 bits moves the gradients, element by element: with
    |q~ - q| <= h_q and |o~ - o| <= h_o (half a step of their groups),
      |s~ - s| <= b = scale h_q.|k|,  |p~ - p| <= p (e^b - 1),  |D~ - D| <= c = |do|.h_o,
      |ds~ - ds| <= w = p e^b c + p (e^b - 1) |do.v - D|,
      |dq~ - dq| <= scale sum_j w |k|,  |dk~ - dk| <= scale sum_i (w |q~| + |ds| h_q),
      |dv~ - dv| <= sum_i p (e^b - 1) |do|,
    beside the bounds of the kernels' own arithmetic."""
    csa, d, scale = _csa(), 64, 0.125
    q, k, v, do = _inputs(44, 1, 2, 2, 130, 90, d, dtype, gain=gain)
    O, lse = csa.svgear_cross_attend(q, k, v, scale)
    qc, oc = csa.svgear_checkpoint_save(q), csa.svgear_checkpoint_save(O)
    got = csa.svgear_cross_attend_backward_ckpt(do, qc, k, v, oc, lse, scale)
    qh, oh = co.unpack(qc.codes, qc.exps), co.unpack(oc.codes, oc.exps)
    _, tol = co.backward(do, qh, k, v, oh, lse, scale)
    want, _ = co.backward(do, q, k, v, O, lse, scale)
    q64, k64, v64, do64, o64, l64 = (t.cpu().double() for t in (q, k, v, do, O, lse))
    hq, ho = (torch.exp2(c.exps.cpu().double() - 128).repeat_interleave(32, -1) for c in (qc, oc))
    assert bool(((qh - q64).abs() <= hq).all()) and bool(((oh - o64).abs() <= ho).all())
    p = torch.exp(scale * q64 @ k64.mT - l64[..., None])
    g = do64 @ v64.mT - (do64 * o64).sum(-1, keepdim=True)
    grow = torch.expm1(scale * hq @ k64.abs().mT)
    c = (do64.abs() * ho).sum(-1, keepdim=True)
    w = p * (1 + grow) * c + p * grow * g.abs()
    moved = (scale * w @ k64.abs(),
             scale * (w.mT @ qh.abs() + (p * g).abs().mT @ hq),
             (p * grow).mT @ do64.abs())
    for x, y, a, b, name in zip(got, want, tol, moved, ("dQ", "dK", "dV")):
        _within(x, y, a + b, name)


@pytest.mark.parametrize("dtype", [FP, BF])
def test_checkpoints_captured_and_replayed(dtype):
    csa = _csa()
    q, k, v, do = _inputs(41, 2, 4, 2, 201, 140, 128, dtype)
    kl = _klen([140, 64])
    O, lse = csa.svgear_cross_attend(q, k, v, k_len=kl)

    def run():
        qc, oc = csa.svgear_checkpoint_save(q), csa.svgear_checkpoint_save(O)
        return (csa.svgear_checkpoint_load(qc),) + csa.svgear_cross_attend_backward_ckpt(
            do, qc, k, v, oc, lse, k_len=kl)

    run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = run()
    for gain in (1.0, 0.25):        # new values in the captured buffers
        do.mul_(gain)
        q.mul_(gain)
        want = run()
        for t in out:
            t.fill_(3)
        graph.replay()
        torch.cuda.synchronize()
        for x, y in zip(out, want):
            assert torch.equal(x, y)


@pytest.mark.parametrize("dtype", [FP, BF])
def test_status_words_of_a_used_workspace_are_cleared(dtype, monkeypatch):
    csa = _csa()
    from clustered_sparse_attention_b200 import _lib
    q, k, v, do = _inputs(42, 1, 2, 2, 40, 70, 64, dtype)
    plain = _lib._cross_workspace

    def dirty(op, dims, device):
        ws, n = plain(op, dims, device)
        return ws.fill_(255), n

    monkeypatch.setattr(_lib, "_cross_workspace", dirty)
    O, lse = csa.svgear_cross_attend(q, k, v, check_status=True)
    got = csa.svgear_cross_attend_backward(do, q, k, v, O, lse, check_status=True)
    c = csa.svgear_checkpoint_save(q), csa.svgear_checkpoint_save(O)
    held = csa.svgear_cross_attend_backward_ckpt(do, c[0], k, v, c[1], lse, check_status=True)
    want, tol = co.backward(do, q, k, v, O, lse, 64 ** -0.5, None)
    for g, w, t, name in zip(got, want, tol, ("dQ", "dK", "dV")):
        _within(g, w, t, name)
    assert all(bool(torch.isfinite(x).all()) for x in held)


@pytest.mark.parametrize("dtype", [FP, BF])
@pytest.mark.parametrize("B,H", [(0, 3), (2, 0)])
def test_no_batch_or_no_head(B, H, dtype):
    csa = _csa()
    q = torch.zeros(B, H, 5, 64, dtype=dtype, device="cuda")
    k = torch.zeros(B, H, 9, 64, dtype=dtype, device="cuda")
    O, lse = csa.svgear_cross_attend(q, k, k)
    grads = csa.svgear_cross_attend_backward(q, q, k, k, O, lse)
    c = csa.svgear_checkpoint_save(q)
    grads += csa.svgear_cross_attend_backward_ckpt(q, c, k, k, c, lse)
    assert O.shape == q.shape and lse.shape == q.shape[:3]
    assert [tuple(x.shape) for x in grads] == [tuple(x.shape) for x in (q, k, k)] * 2
    assert csa.svgear_checkpoint_load(c).shape == q.shape
    torch.cuda.synchronize()


@pytest.mark.parametrize("dtype", [FP, BF])
def test_keys_as_values_and_queries(dtype):
    """The same tensor in every place it may take."""
    csa = _csa()
    x, _, _, do = _inputs(43, 2, 3, 3, 150, 150, 64, dtype)
    O, lse = _check_forward(x, x, x, [150, 31], 0.125)
    _check_backward(do, x, x, x, O, lse, [150, 31], 0.125)


def test_a_training_step_beside_the_clustered_layer():
    """The operators as a block uses them: clustered self-attention, its output
    as the queries of a cross attention to padded prompts, activations held in
    8 bits, gradients from them; each against its 64-bit form."""
    csa = _csa()
    from clustered_sparse_attention_b200 import synth
    from helpers import to_torch
    w = synth.custom_workload("cross_block", H=2, frames=1, grid_h=24, grid_w=32, d=128,
                              dtype="bf16", Cq=8, Ck=24, iters=3, density=0.3, n_centres=16,
                              sigma=0.5, index=77)
    dev = [to_torch(synth.layer_tensor(w, n), w.dtype) for n in ("q", "k", "v")]
    x = csa.layer(*dev, w.Cq, w.Ck, w.iters, w.density, w.scale)["O"]
    _, k, v, do = _inputs(50, 1, 2, 2, w.N, 100, 128, BF)
    O, lse = _check_forward(x, k, v, [81], w.scale)
    xc, oc = csa.svgear_checkpoint_save(x), csa.svgear_checkpoint_save(O)
    got = csa.svgear_cross_attend_backward_ckpt(do, xc, k, v, oc, lse, w.scale, k_len=_klen([81]))
    want, tol = co.backward(do, co.unpack(xc.codes, xc.exps), k, v, co.unpack(oc.codes, oc.exps),
                            lse, w.scale, [81])
    for g, wv, t, name in zip(got, want, tol, ("dQ", "dK", "dV")):
        _within(g, wv, t, name)
