"""Host-side checks of the cross attention and checkpoint entry points (no
call below reaches the GPU), and of the tests' 64-bit forms against
differences."""
import ctypes
import inspect
import os
import re

import pytest
import torch

import cross_oracle as co
import cross_protocol


@pytest.fixture(scope="module")
def lib():
    from clustered_sparse_attention_b200 import build
    build.build()
    from clustered_sparse_attention_b200 import _lib
    return _lib


FAKE = 1 << 20      # never dereferenced: validation fails first
BIG = ctypes.c_size_t(1 << 42)


def _tok(m, N=100, H=4, d=128, data=FAKE, sb=None, sh=None, sn=None):
    sn = d if sn is None else sn
    sh = N * sn if sh is None else sh
    return m.Tokens(data, H * sh if sb is None else sb, sh, sn)


def _fwd(m, dims=None, Q=None, K=None, V=None, O=None, lse=FAKE, scale=0.1, ws=FAKE, n=BIG):
    dims = m.CrossDims(2, 4, 4, 100, 100, 128, m.BF16) if dims is None else dims
    t = _tok(m)
    return m.lib().svgear_cross_attend(Q or t, K or t, V or t, dims, None, scale, O or t, lse, ws,
                                       n, None)


def test_forward_refusals(lib):
    m = lib
    bad, uns = m.ERR_INVALID_ARG, m.ERR_UNSUPPORTED
    D = m.CrossDims
    for dims, want in ((D(2, 4, 3, 100, 100, 128, 1), bad),      # Hkv does not divide Hq
                       (D(2, 4, 0, 100, 100, 128, 1), bad),
                       (D(2, 4, 4, 0, 100, 128, 1), bad),
                       (D(2, 4, 4, 100, 0, 128, 1), bad),
                       (D(-1, 4, 4, 100, 100, 128, 1), bad),
                       (D(2, 4, 4, 100, 100, 96, 1), uns),
                       (D(2, 4, 4, 100, 100, 128, 2), uns),
                       (D(2, 40000, 40000, 100, 100, 128, 1), uns),
                       (D(2, 1024, 1024, 1 << 20, 100, 128, 1), uns)):
        assert _fwd(m, dims) == want
        assert m.lib().svgear_cross_workspace_bytes(m.CROSS_FORWARD, dims) == 0
    assert _fwd(m, Q=_tok(m, data=None)) == bad
    assert _fwd(m, Q=_tok(m, data=FAKE + 8)) == bad              # alignment
    assert _fwd(m, K=_tok(m, sn=132)) == bad                     # 264-byte rows
    assert _fwd(m, V=_tok(m, sn=-128)) == bad
    assert _fwd(m, V=_tok(m, sn=0)) == bad
    assert _fwd(m, V=_tok(m, sh=1 << 40)) == bad
    assert _fwd(m, O=_tok(m, sn=64)) == bad                      # rows overlap
    assert _fwd(m, O=_tok(m, sh=0)) == bad                       # heads overlap
    assert _fwd(m, O=_tok(m, sh=128, sn=256)) == bad             # 4 heads of 128 in 256
    assert _fwd(m, lse=None) == bad
    assert _fwd(m, ws=None) == bad
    for scale in (0.0, -0.1, float("inf"), float("nan"), 3e38):
        assert _fwd(m, scale=scale) == bad
    assert _fwd(m, n=ctypes.c_size_t(64)) == m.ERR_WORKSPACE
    assert m.lib().svgear_cross_workspace_bytes(9, D(2, 4, 4, 100, 100, 128, 1)) == 0


def test_backward_refusals(lib):
    m = lib
    L, dims, t = m.lib(), m.CrossDims(2, 4, 4, 100, 100, 128, m.BF16), _tok(m)

    def call(dims=dims, dO=t, dQ=t, dK=t, dV=t, O=t, lse=FAKE, scale=0.1, n=BIG):
        return L.svgear_cross_attend_backward(dO, t, t, t, O, lse, dims, None, scale, dQ, dK, dV,
                                              FAKE, n, None)

    def held(qc=FAKE, qe=FAKE, oc=FAKE, oe=FAKE, n=BIG):
        return L.svgear_cross_attend_backward_ckpt(t, qc, qe, t, t, oc, oe, FAKE, dims, None, 0.1, t,
                                                   t, t, FAKE, n, None)

    for kw in (dict(dO=_tok(m, data=None)), dict(dQ=_tok(m, sh=0)), dict(dK=_tok(m, sb=0)),
               dict(dV=_tok(m, sn=64)), dict(O=_tok(m, data=FAKE + 2)), dict(lse=None),
               dict(scale=0.0)):
        assert call(**kw) == m.ERR_INVALID_ARG, kw
    for kw in (dict(qc=None), dict(qe=None), dict(oc=None), dict(oe=None), dict(qc=FAKE + 8)):
        assert held(**kw) == m.ERR_INVALID_ARG, kw
    small = ctypes.c_size_t(L.svgear_cross_workspace_bytes(m.CROSS_BACKWARD, dims))
    assert held(n=small) == m.ERR_WORKSPACE
    assert call(n=ctypes.c_size_t(small.value - 1)) == m.ERR_WORKSPACE
    assert call(dims=m.CrossDims(2, 4, 4, 100, 100, 80, m.BF16)) == m.ERR_UNSUPPORTED


@pytest.mark.parametrize("Nq,Nk", [(1, (1 << 31) - 1), (1, (1 << 31) - 1023), ((1 << 31) - 1, 1)])
def test_lengths_whose_tiles_pass_32_bits_are_refused(lib, Nq, Nk):
    m = lib
    dims = m.CrossDims(1, 1, 1, Nq, Nk, 64, m.BF16)
    t = _tok(m, N=1, H=1, d=64, sn=8)
    assert m.lib().svgear_cross_workspace_bytes(m.CROSS_FORWARD, dims) == 0
    assert _fwd(m, dims, t, t, t, t) == m.ERR_UNSUPPORTED
    dims.Nq, dims.Nk = min(Nq, (1 << 31) - 1024), min(Nk, (1 << 31) - 1024)
    assert m.lib().svgear_cross_workspace_bytes(m.CROSS_FORWARD, dims) > 0


@pytest.mark.parametrize("lse,k_len,ws", [(2, 0, 0), (0, 1, 0), (0, 2, 0), (0, 0, 4), (0, 0, 8)])
def test_misaligned_buffers_are_refused(lib, lse, k_len, ws):
    """Byte offsets of lse, k_len and the workspace that a load or store would fault on."""
    m, t = lib, _tok(lib)
    L, dims = m.lib(), m.CrossDims(2, 4, 4, 100, 100, 128, m.BF16)
    lse, k_len, ws = FAKE + lse, FAKE + k_len if k_len else None, FAKE + ws
    assert L.svgear_cross_attend(t, t, t, dims, k_len, 0.1, t, lse, ws, BIG, None) == m.ERR_INVALID_ARG
    assert L.svgear_cross_attend_backward(t, t, t, t, t, lse, dims, k_len, 0.1, t, t, t, ws, BIG,
                                          None) == m.ERR_INVALID_ARG
    assert L.svgear_cross_attend_backward_ckpt(t, FAKE, FAKE, t, t, FAKE, FAKE, lse, dims, k_len, 0.1,
                                               t, t, t, ws, BIG, None) == m.ERR_INVALID_ARG


def test_checkpoint_refusals(lib):
    m = lib
    L, dims, t = m.lib(), m.Dims(2, 4, 100, 128, m.BF16), _tok(m)
    assert L.svgear_checkpoint_save(t, dims, None, FAKE, None) == m.ERR_INVALID_ARG
    assert L.svgear_checkpoint_save(t, dims, FAKE + 4, FAKE, None) == m.ERR_INVALID_ARG
    assert L.svgear_checkpoint_save(_tok(m, sn=4), dims, FAKE, FAKE, None) == m.ERR_INVALID_ARG
    assert L.svgear_checkpoint_load(FAKE, FAKE, dims, _tok(m, sn=64), None) == m.ERR_INVALID_ARG
    assert L.svgear_checkpoint_load(FAKE, None, dims, t, None) == m.ERR_INVALID_ARG
    assert L.svgear_checkpoint_save(t, m.Dims(2, 4, 100, 32, m.BF16), FAKE, FAKE,
                                    None) == m.ERR_UNSUPPORTED
    assert L.svgear_checkpoint_save(t, m.Dims(2, 4, 0, 128, m.BF16), FAKE, FAKE,
                                    None) == m.ERR_INVALID_ARG


def test_nothing_to_do(lib):
    m = lib
    t = _tok(m, data=None)
    for dims in (m.CrossDims(0, 4, 4, 10, 10, 64, m.F32), m.CrossDims(2, 0, 0, 10, 10, 64, m.BF16)):
        assert _fwd(m, dims, t, t, t, t, lse=None) == m.OK
        assert m.lib().svgear_cross_attend_backward(t, t, t, t, t, None, dims, None, 0.1, t, t, t,
                                                    FAKE, BIG, None) == m.OK
    assert m.lib().svgear_checkpoint_save(t, m.Dims(0, 4, 10, 64, m.F32), None, None, None) == m.OK


def test_binding_refuses_before_any_call():
    import clustered_sparse_attention_b200 as csa
    q = torch.zeros(1, 2, 4, 64)
    with pytest.raises(ValueError, match="CUDA tensor"):
        csa.svgear_cross_attend(q, q, q)
    with pytest.raises(ValueError, match="CUDA tensor"):
        csa.svgear_checkpoint_save(q)
    with pytest.raises(ValueError, match="Checkpoint"):
        csa.svgear_checkpoint_load(csa.Checkpoint(torch.zeros(1, 2, 4, 64, dtype=torch.int8),
                                                  torch.zeros(1, 2, 4, 2, dtype=torch.uint8),
                                                  torch.float32))


@pytest.mark.parametrize("fn", ["svgear_cross_attend", "svgear_cross_attend_backward",
                                "svgear_cross_attend_backward_ckpt", "svgear_checkpoint_save",
                                "svgear_checkpoint_load"])
def test_calls_run_on_their_tensors_device(fn, monkeypatch):
    """Whichever way the arguments come, with another device than theirs current."""
    import clustered_sparse_attention_b200 as csa
    from clustered_sparse_attention_b200 import _lib

    class Reached(Exception):
        pass

    class Tensor:                       # as much of one as is looked at before the call
        is_cuda, device, dtype = True, torch.device("cuda", 1), torch.bfloat16
        shape = torch.Size((1, 2, 4, 64))

        def stride(self):
            raise Reached

        dim = stride

    entered = []

    class Device:
        def __init__(self, d):
            self.d = d

        def __enter__(self):
            entered.append(self.d)

        def __exit__(self, *exc):
            return False

    monkeypatch.setattr(_lib.torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(_lib.torch.cuda, "device", Device)
    call = getattr(csa, fn)
    t = Tensor()
    tensor = csa.Checkpoint(t, t, t.dtype) if fn == "svgear_checkpoint_load" else t
    names = list(inspect.signature(call).parameters)
    needed = {n: t for n in names if n in ("dO", "Q", "K", "V", "O", "lse", "Qc", "Oc")}
    needed[names[0]] = tensor
    last = dict(reversed(list(needed.items())))         # the first argument at the end
    optional = {n: None for n in names if n in ("scale", "k_len", "out")}
    for args, kw in (((tensor,), {n: x for n, x in needed.items() if n != names[0]}),
                     ((), needed), ((), {**optional, **last})):
        entered.clear()
        with pytest.raises(Reached):
            call(*args, **kw)
        assert entered == [t.device]
        Tensor.device = torch.device("cuda", 0)         # the current one: nothing to switch
        with pytest.raises(Reached):
            call(*args, **kw)
        assert entered == [torch.device("cuda", 1)]
        Tensor.device = torch.device("cuda", 1)


def test_current_stream_without_the_private_function(monkeypatch):
    from types import SimpleNamespace
    from clustered_sparse_attention_b200 import _lib
    dev = torch.device("cuda", 3)
    monkeypatch.setattr(_lib, "_current_raw_stream", None)
    monkeypatch.setattr(_lib.torch.cuda, "current_stream",
                        lambda d: SimpleNamespace(cuda_stream=1000 + d.index))
    assert _lib._raw_stream(dev) == 1003


def test_oracle_gradients_match_differences():
    g = torch.Generator().manual_seed(3)
    q = torch.randn(2, 4, 3, 8, generator=g, dtype=torch.float64)
    k, v = (torch.randn(2, 2, 5, 8, generator=g, dtype=torch.float64) for _ in range(2))
    do = torch.randn(2, 4, 3, 8, generator=g, dtype=torch.float64)
    k_len, scale = [5, 3], 0.4

    def loss(q, k, v):
        return float((co.forward(q, k, v, scale, k_len)[0] * do).sum())

    o, lse, _, _ = co.forward(q, k, v, scale, k_len)
    grads, _ = co.backward(do, q, k, v, o, lse, scale, k_len)
    h = 1e-5
    for i, t in enumerate((q, k, v)):
        flat = t.view(-1)
        for j in range(0, flat.numel(), 7):
            x = float(flat[j])
            flat[j] = x + h
            up = loss(q, k, v)
            flat[j] = x - h
            down = loss(q, k, v)
            flat[j] = x
            # central difference: h^2 / 6 |f'''| (a few units here) + eps / h
            assert abs((up - down) / (2 * h) - float(grads[i].view(-1)[j])) <= 1e-7


def test_oracle_pack_rule():
    x = torch.zeros(1, 1, 7, 32)
    x[0, 0, 0, 0] = 1.0                          # 64 steps of 2^-6
    x[0, 0, 1, 0] = 127.5 / 64                   # rounds to 128: one step up
    x[0, 0, 2, 0] = 127.25 / 64
    x[0, 0, 4, 3] = float("inf")
    x[0, 0, 5] = 3e38
    x[0, 0, 6] = -torch.finfo(torch.float32).max  # saturates
    codes, exps = co.pack(x)
    assert exps[0, 0, :, 0].tolist() == [121, 122, 121, 0, 255, 248, 248]
    assert codes[0, 0, :, 0].tolist() == [64, 64, 127, 0, 0, 113, -127]
    assert torch.isnan(co.unpack(codes, exps)[0, 0, 4]).all()


@pytest.mark.parametrize("iterations", [1, 2, 3, 7])
def test_dkv_barriers_never_lap(iterations):
    """However its roles are delayed, the dK/dV kernel's waits end: a wait that a second
    completion could overtake would look open again and run into its time limit."""
    src = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                       "clustered_sparse_attention_b200", "csrc", "cross_bwd_sm100.cu")
    with open(src) as f:
        m = re.search(r"uint64_t s_issued(\[(\d+)\])?;", f.read())
    assert cross_protocol.stuck_states(iterations, int(m.group(2) or 1)) == []
    if iterations > 1:
        assert cross_protocol.stuck_states(iterations, 1)   # the model sees the fault


TMEM_ACCESS = re.compile(r"\b(tmem_ld\d+|tmem_st\d+|mask_columns<|mma_\w+<|issue_s\(\);|issue_dp\(\);)")


def unfenced_accesses(source):
    """Accesses to tensor memory (products, loads, stores) that follow a barrier wait of the
    same thread without tcgen05.fence::after_thread_sync in between: line numbers."""
    waited, bad = False, []
    for n, line in enumerate(source.splitlines(), 1):
        line = line.split("//")[0]
        if "auto issue_" in line:       # a lambda: its calls are looked at, not its body
            waited = False
        if "fence_after_sync()" in line:
            waited = False
        if "poll_bar(" in line or "drain_bar(" in line:
            waited = True
        if waited and TMEM_ACCESS.search(line):
            bad.append(n)
    return bad


@pytest.mark.parametrize("name", ["cross_sm100.cu", "cross_bwd_sm100.cu"])
def test_tensor_memory_is_fenced_after_every_wait(name):
    """A barrier orders tensor-memory accesses of two threads only together with the fence
    behind the wait."""
    src = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                       "clustered_sparse_attention_b200", "csrc", name)
    with open(src) as f:
        text = f.read()
    assert text.count("poll_bar(") > 10 and unfenced_accesses(text) == []
    # the scan sees the fault: without the first fence behind a wait
    at = text.index("fence_after_sync()", text.index("poll_bar("))
    assert unfenced_accesses(text[:at] + text[at + len("fence_after_sync()"):])


def test_checkpoint_error_bound():
    """|error| <= 2^(e-1), at most 1/127 of the group's largest magnitude for e > -127; 2^-128
    at e = -127, where it may be all of a value; 2^e where codes saturate."""
    g = torch.Generator().manual_seed(6)
    x = torch.randn(1, 1, 4000, 32, generator=g, dtype=torch.float64)
    x = x * torch.exp2(torch.randint(-140, 126, (1, 1, 4000, 1), generator=g).double())
    x[0, 0, 0] = torch.finfo(torch.float32).max
    x[0, 0, 1] = 2.0 ** -130
    x[0, 0, 2] = 0.4 * 2.0 ** -126
    x = x.float().double()
    codes, exps = co.pack(x)
    e = exps[..., :1].double() - 127
    err = (co.unpack(codes, exps) - x).abs().amax(-1, keepdim=True)
    top = x.abs().amax(-1, keepdim=True)
    assert bool((err <= torch.exp2(e - 1) + (e == 121) * torch.exp2(e - 1)).all())
    low = e == -127
    assert bool((err <= top / 127)[~low].all()) and bool((err[low] <= 2.0 ** -128).all())
    assert bool(low[0, 0, 1:3].all()) and not codes[0, 0, 1].any()      # 2^-130: all of it lost
    assert err[0, 0, 2] > 0.2 * top[0, 0, 2]
    # exact in bf16 too: every loaded value is a bf16 number
    y = co.unpack(codes, exps)
    assert torch.equal(y.to(torch.bfloat16).double(), y)
