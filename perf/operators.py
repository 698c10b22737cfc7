"""Cases, plain forms and exact values of the dense operators around the
clustered layer: cross attention to an encoder's states (forward, backward)
and activation checkpoints in 8 bits (saved and loaded, and read by the cross
attention's backward pass).

Definitions, with G = Hq / Hkv query heads sharing key/value head h // G and
keys j < k_len[b] only:

  cross                s_ij = scale q_i.k_j,  lse_i = log sum_j e^{s_ij},
                       o_i = sum_j e^{s_ij - lse_i} v_j;
                       no key: o_i = 0, lse_i = -inf
  backward             p_ij = e^{s_ij - lse_i},  D_i = do_i.o_i,
                       ds_ij = p_ij (do_i.v_j - D_i),
                       dq_i = scale sum_j ds_ij k_j,
                       dk_j = scale sum_i ds_ij q_i,  dv_j = sum_i p_ij do_i
                       (sums over the sharing heads too; 0 for keys past k_len)
  checkpoint           groups of 32 elements share a power of two 2^e, the
                       smallest (e >= -127) with every |round(x / 2^e)| <= 127;
                       element codes are those rounded quotients (half to even).
                       e stops at 121, where codes saturate at 127, so that what
                       a finite value loads as is finite
  checkpoint_backward  backward with q and o held as such codes
"""
import math

import torch

own = False

GROUP = 32      # elements sharing one exponent


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------
def _case(name, op, dtype, layout, B, Hq, Hkv, Nq, Nk, d, lens=""):
    c = {"op": op, "dtype": dtype, "layout": layout, "B": B, "Hq": Hq, "Hkv": Hkv, "Nq": Nq,
         "Nk": Nk, "d": d, "lens": lens}
    return dict(c, name=name) if name else c


def listed():
    return [
        # one query token against one prompt's 512 text states: latency only
        _case("cross_token", "cross", "bf16", "head", 1, 40, 40, 1, 512, 128),
        # one latent frame (45 x 80) of three requests whose prompts differ in
        # length, one of them empty; q, k, v straight from their projections
        _case("cross_prompts", "cross", "bf16", "token", 3, 40, 40, 3600, 512, 128, "512,77,0"),
        # the Wan 720p layer's video tokens against the text states
        _case("cross_wan720p", "cross", "bf16", "head", 1, 40, 40, 75600, 512, 128),
        # the other direction: 77 text tokens reading the HunyuanVideo tokens
        _case("cross_text_reads_video", "cross", "bf16", "head", 1, 24, 24, 77, 118800, 128),
        # fp32 tokens, four query heads per key/value head, odd lengths
        _case("cross_fp32_shared", "cross", "fp32", "head", 2, 16, 4, 1023, 331, 64, "331,129"),
        # training on a short clip: shared heads, two prompts
        _case("backward_clip", "backward", "bf16", "token", 2, 32, 8, 1285, 333, 64, "333,77"),
        # training at the Wan 720p length
        _case("backward_wan720p", "backward", "bf16", "head", 1, 40, 40, 75600, 512, 128),
        # fp32 gradients
        _case("backward_fp32", "backward", "fp32", "head", 1, 8, 8, 2049, 257, 128),
        # one latent frame's activation saved and loaded again
        _case("checkpoint_frame", "checkpoint", "bf16", "token", 1, 40, 40, 3600, 0, 128),
        # a whole layer's activation saved and loaded again
        _case("checkpoint_wan720p", "checkpoint", "bf16", "head", 1, 40, 40, 75600, 0, 128),
        # gradients of a frame from 8-bit q and o, two prompts
        _case("checkpoint_backward_frame", "checkpoint_backward", "bf16", "head", 2, 40, 40, 3600,
              512, 128, "512,129"),
        # gradients at the HunyuanVideo length from 8-bit q and o
        _case("checkpoint_backward_hunyuan", "checkpoint_backward", "bf16", "head", 1, 24, 24,
              118800, 256, 128),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["cross", "cross", "backward", "checkpoint", "checkpoint_backward"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "fp32"])
    layout = rng.choice(["head", "token"])
    d = rng.choice([64, 128])
    B = rng.choice([1, 1, 2, 3, 4])
    Hkv = rng.randint(1, 24)
    G = rng.choice([1, 1, 1, 2, 4, 5])
    Nq = _log_int(rng, 1, 75600)
    Nk = _log_int(rng, 1, 1024)
    if op == "cross" and rng.random() < 0.3:    # few queries over many keys
        Nq, Nk = _log_int(rng, 1, 300), _log_int(rng, 1024, 118800)
    if op == "checkpoint":
        Hkv, G, Nk = Hkv * G, 1, 0
    lens = ""
    if B > 1 and Nk and rng.random() < 0.7:
        lens = ",".join(str(rng.choice([Nk, rng.randint(0, Nk), rng.randint(0, min(Nk, 200))]))
                        for _ in range(B))
    # keep the work (fp32 has no tensor cores to run on) and the bytes below
    # the largest listed cases'
    flops, nbytes = (4e11, 2e9) if dtype == "bf16" else (2e10, 1e9)
    while Nq > 1:
        w = work(_case("", op, dtype, layout, B, Hkv * G, Hkv, Nq, Nk, d))
        if w["flops"] <= flops and w["bytes"] <= nbytes:
            break
        Nq = (Nq * 2) // 3
    while Nk > 1:
        w = work(_case("", op, dtype, layout, B, Hkv * G, Hkv, Nq, Nk, d))
        if w["flops"] <= flops and w["bytes"] <= nbytes:
            break
        Nk = (Nk * 2) // 3
    if lens:
        lens = ",".join(str(min(int(x), Nk)) for x in lens.split(","))
    return _case("", op, dtype, layout, B, Hkv * G, Hkv, Nq, Nk, d, lens)


def _lens(case):
    return [int(x) for x in case["lens"].split(",")] if case["lens"] else [case["Nk"]] * case["B"]


def work(case):
    es = 2 if case["dtype"] == "bf16" else 4
    q = case["B"] * case["Hq"] * case["Nq"] * case["d"]             # elements of q, o, ...
    kv_read = case["Hkv"] * case["d"] * sum(_lens(case))            # valid elements of k (and v)
    kv_all = case["B"] * case["Hkv"] * case["Nk"] * case["d"]
    pairs = case["Hq"] * case["Nq"] * sum(_lens(case))
    lse = 4 * case["B"] * case["Hq"] * case["Nq"]
    held = q + q // GROUP                                           # bytes of 8-bit codes
    op = case["op"]
    if op == "cross":
        return {"bytes": es * (2 * q + 2 * kv_read) + lse, "flops": 4 * pairs * case["d"]}
    if op == "backward":
        return {"bytes": es * (4 * q + 2 * kv_read + 2 * kv_all) + lse,
                "flops": 10 * pairs * case["d"]}
    if op == "checkpoint":
        return {"bytes": 2 * es * q + 2 * held, "flops": 4 * q}
    return {"bytes": es * (2 * q + 2 * kv_read + 2 * kv_all) + 2 * held + lse,
            "flops": 10 * pairs * case["d"]}


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------
def _normed(x, gain):
    return x * torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6) * gain


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed))
    dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
    B, Hq, Hkv, Nq, Nk, d = (case[k] for k in ("B", "Hq", "Hkv", "Nq", "Nk", "d"))

    def tokens(H, N, kind):
        shape = (B, H, N, d) if case["layout"] == "head" else (B, N, H, d)
        x = torch.randn(shape, device=dev, generator=g)
        if kind == "normed":        # q and k pass a normalisation with a learned gain
            x = _normed(x, 0.5 + torch.rand(d, device=dev, generator=g))
        elif kind == "small":       # an incoming gradient
            x = x * 0.02
        x = x.to(dt)
        return x if case["layout"] == "head" else x.transpose(1, 2)

    st = {"case": case, "scale": d ** -0.5}
    op = case["op"]
    if op == "checkpoint":
        st["x"] = tokens(Hq, Nq, "plain")
        return st
    q, k, v = tokens(Hq, Nq, "normed"), tokens(Hkv, Nk, "normed"), tokens(Hkv, Nk, "plain")
    st["k_len"] = None
    if case["lens"]:
        st["k_len"] = torch.tensor(_lens(case), dtype=torch.int32, device=dev)
        for b, n in enumerate(_lens(case)):     # whatever a padded buffer holds
            k[b, :, n:] *= 100
            v[b, :, n:] *= 100
    st.update(q=q, k=k, v=v)
    if op == "cross":
        return st
    st["do"] = tokens(Hq, Nq, "small")
    o, st["lse"] = _plain_cross(q, k, v, st["k_len"], st["scale"])
    if case["layout"] == "token":
        o = o.transpose(1, 2).contiguous().transpose(1, 2)
    if op == "backward":
        st["o"] = o
        return st
    st["q_held"], st["o_held"] = _plain_save(q), _plain_save(o)
    del st["q"]
    if own:
        import clustered_sparse_attention_b200 as csa
        st["q_held"] = csa.Checkpoint(*st["q_held"], dt)
        st["o_held"] = csa.Checkpoint(*st["o_held"], dt)
    return st


# ---------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------
def run(state):
    op = state["case"]["op"]
    if own:
        return _run_own(state, op)
    if op == "cross":
        return _plain_cross(state["q"], state["k"], state["v"], state["k_len"], state["scale"])
    if op == "checkpoint":
        return _plain_load(_plain_save(state["x"])).to(state["x"].dtype)
    if op == "backward":
        q, o = state["q"].float(), state["o"].float()
    else:
        q, o = _plain_load(state["q_held"]), _plain_load(state["o_held"])
    return _plain_backward(state["do"], q, state["k"], state["v"], o, state["lse"],
                           state["k_len"], state["scale"])


def _run_own(state, op):
    import clustered_sparse_attention_b200 as csa
    if op == "cross":
        return csa.svgear_cross_attend(state["q"], state["k"], state["v"], state["scale"],
                                       k_len=state["k_len"])
    if op == "checkpoint":
        return csa.svgear_checkpoint_load(csa.svgear_checkpoint_save(state["x"]))
    if op == "backward":
        return csa.svgear_cross_attend_backward(state["do"], state["q"], state["k"], state["v"],
                                                state["o"], state["lse"], state["scale"],
                                                k_len=state["k_len"])
    return csa.svgear_cross_attend_backward_ckpt(state["do"], state["q_held"], state["k"],
                                                 state["v"], state["o_held"], state["lse"],
                                                 state["scale"], k_len=state["k_len"])


# ---------------------------------------------------------------------------
# Plain forms: elementary torch operations in 32 bits, rounded once at the end
# ---------------------------------------------------------------------------
def _valid(k, k_len):
    """[B, 1, Nk] truth values of the keys that take part, or None for all."""
    if k_len is None:
        return None
    return (torch.arange(k.shape[2], device=k.device) < k_len[:, None])[:, None]


def _clean(x, valid):
    x = x.float()
    return x if valid is None else torch.where(valid[..., None], x, torch.zeros_like(x))


def _grouped(x, Hkv):
    """[B, Hq, N, d] -> [B, Hkv, G * N, d]: the heads that share keys in one."""
    B, Hq, N, d = x.shape
    return x.reshape(B, Hkv, (Hq // Hkv) * N, d)


def _plain_cross(q, k, v, k_len, scale):
    B, Hq, Nq, d = q.shape
    valid = _valid(k, k_len)
    s = _grouped(q.float(), k.shape[1]) @ _clean(k, valid).transpose(2, 3)
    s *= scale
    if valid is not None:
        s.masked_fill_(~valid[:, :, None], -math.inf)
    m = s.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    p = s.sub_(m).exp_()
    total = p.sum(-1, keepdim=True)
    o = (p @ _clean(v, valid)) / torch.where(total == 0, torch.ones_like(total), total)
    lse = m + torch.log(total)
    return o.reshape(B, Hq, Nq, d).to(q.dtype), lse.reshape(B, Hq, Nq)


def _plain_backward(do, q, k, v, o, lse, k_len, scale):
    B, Hq, Nq, d = q.shape
    Hkv = k.shape[1]
    valid = _valid(k, k_len)
    kf, vf = _clean(k, valid), _clean(v, valid)
    qf, dof = _grouped(q, Hkv), _grouped(do.float(), Hkv)
    delta = (dof * _grouped(o, Hkv)).sum(-1, keepdim=True)
    p = qf @ kf.transpose(2, 3)
    p *= scale
    p -= lse.reshape(B, Hkv, -1, 1)
    if valid is not None:
        p.masked_fill_(~valid[:, :, None], -math.inf)
    p.exp_()
    dv = p.transpose(2, 3) @ dof
    ds = dof @ vf.transpose(2, 3)
    ds -= delta
    ds *= p
    if valid is not None:
        ds.masked_fill_(~valid[:, :, None], 0.0)
    dq = (ds @ kf) * scale
    dk = (ds.transpose(2, 3) @ qf) * scale
    dt = k.dtype
    return dq.reshape(B, Hq, Nq, d).to(dt), dk.to(dt), dv.to(dt)


def _pow2(e):
    """2^e in fp32 from its bits, -127 <= e <= 127 (powf need not be exact)."""
    bits = torch.where(e == -127, torch.full_like(e, 1 << 22), (e + 127) << 23)
    return bits.to(torch.int32).view(torch.float32)


def _plain_save(x):
    """Codes int8 [B, H, N, d] and biased exponents uint8 [B, H, N, d / 32]."""
    B, H, N, d = x.shape
    g = x.float().reshape(B, H, N, d // GROUP, GROUP)
    amax = g.abs().amax(-1, keepdim=True)
    finite = torch.isfinite(amax)
    e = torch.frexp(torch.where(finite, amax, torch.zeros_like(amax)))[1] - 7
    e = torch.clamp(e, min=-127)
    e = torch.where(amax * _pow2(-e) >= 127.5, e + 1, e).clamp(max=121)
    e = torch.where(amax == 0, torch.full_like(e, -127), e)
    codes = torch.round(torch.where(finite, g, torch.zeros_like(g)) * _pow2(-e)).clamp(-127, 127)
    exps = torch.where(finite, e + 127, torch.full_like(e, 255))
    return codes.to(torch.int8).reshape(B, H, N, d), exps.to(torch.uint8).squeeze(-1)


def _plain_load(held):
    codes, exps = held
    B, H, N, d = codes.shape
    e = exps.to(torch.int32)[..., None]
    step = torch.where(e == 255, torch.full_like(e, math.nan, dtype=torch.float32),
                       _pow2(torch.clamp(e, max=254) - 127))
    x = codes.reshape(B, H, N, d // GROUP, GROUP) * step
    return x.reshape(B, H, N, d)


# ---------------------------------------------------------------------------
# From the definitions, in 64 bits, one (batch, key/value head) at a time
# ---------------------------------------------------------------------------
def _step64(e):
    """2^e in 64 bits from its bits (whole e in any type; pow need not be exact)."""
    return ((e.to(torch.int64) + 1023) << 52).view(torch.float64)


def _held64(held):
    codes, exps = held if isinstance(held, tuple) else (held.codes, held.exps)
    step = _step64(exps.to(torch.int64) - 127)
    return codes.double() * step.repeat_interleave(GROUP, dim=-1)


def exact(case, seed):
    st = prepare(case, seed)
    op, scale = case["op"], st["scale"]
    if op == "checkpoint":
        x = st["x"].double().unflatten(-1, (-1, GROUP))
        top = x.abs().amax(-1, keepdim=True)
        e = torch.full_like(top, -127, dtype=torch.int64)
        for bit in (128, 64, 32, 16, 8, 4, 2, 1):   # the largest step that is too small, plus one
            more = e + bit
            e = torch.where(torch.round(top / _step64(more - 1)) > 127, more, e)
        e = torch.clamp(e, max=121)
        return (torch.clamp(torch.round(x / _step64(e)), -127, 127) * _step64(e)).flatten(-2)
    G = case["Hq"] // case["Hkv"]
    shape = (case["B"], case["Hq"], case["Nq"])
    kvshape = (case["B"], case["Hkv"], case["Nk"], case["d"])
    dev = st["k"].device
    if op == "cross":
        o = torch.zeros(shape + (case["d"],), dtype=torch.float64, device=dev)
        lse = torch.full(shape, -math.inf, dtype=torch.float64, device=dev)
        for b, n in enumerate(_lens(case)):
            for h in range(case["Hq"] if n else 0):
                kk, vv = st["k"][b, h // G, :n].double(), st["v"][b, h // G, :n].double()
                for r in range(0, case["Nq"], 16384):
                    rows = slice(r, r + 16384)
                    s = scale * torch.mm(st["q"][b, h, rows].double(), kk.T)
                    lse[b, h, rows] = torch.logsumexp(s, 1)
                    o[b, h, rows] = torch.mm(torch.softmax(s, 1), vv)
        return o, lse
    q = st["q"].double() if op == "backward" else _held64(st["q_held"])
    o = st["o"].double() if op == "backward" else _held64(st["o_held"])
    dq = torch.zeros_like(q)
    dk, dv = (torch.zeros(kvshape, dtype=torch.float64, device=dev) for _ in range(2))
    for b, n in enumerate(_lens(case)):
        for h in range(case["Hq"] if n else 0):
            kk, vv = st["k"][b, h // G, :n].double(), st["v"][b, h // G, :n].double()
            for r in range(0, case["Nq"], 16384):
                rows = slice(r, r + 16384)
                qq, gg = q[b, h, rows], st["do"][b, h, rows].double()
                w = torch.exp(scale * torch.mm(qq, kk.T) - st["lse"][b, h, rows, None].double())
                ds = w * (torch.mm(gg, vv.T) - torch.linalg.vecdot(gg, o[b, h, rows])[:, None])
                dq[b, h, rows] = scale * torch.mm(ds, kk)
                dk[b, h // G, :n] += scale * torch.mm(ds.T, qq)
                dv[b, h // G, :n] += torch.mm(w.T, gg)
    return dq, dk, dv
