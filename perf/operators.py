"""The query/key preparation, cache and 8-bit attention operators as measured cases.

Four operators, each a call of ``programmable_block_sparse_b200``:

* ``prep``   -- per-head RMS norm of queries and keys with the position
  rotation in the same pass (``flexattn_qk_norm_rope``);
* ``prep_bwd`` -- its gradients (``flexattn_qk_norm_rope_backward``);
* ``append`` -- new keys and values into a paged cache, keys normed and rotated
  on the way, e4m3 pools with one scale per block of tokens and head, or bf16
  pools (``flexattn_cache_append``);
* ``attend`` -- attention over the e4m3 cache (``flexattn_forward_fp8``).

``own`` False computes the same results in elementary torch operations.
"""

import math

import torch

own = False

E4M3 = torch.float8_e4m3fn
E4M3_MAX = 448.0


# --------------------------------------------------------------------------
# cases
# --------------------------------------------------------------------------
def listed():
    return [
        # one decode step of 32 sequences, 32/8 heads: a launch-bound call
        dict(name="prep_step_b32", op="prep", B=32, N=1, Hq=32, Hkv=8, D=128, rot=128, inter=False, dtype="bf16",
             norm=True, fused=True),
        # prompts / training batch of the grouped-head configuration (2 x 16384 tokens)
        dict(name="prep_16384", op="prep", B=2, N=16384, Hq=32, Hkv=8, D=128, rot=128, inter=False, dtype="bf16",
             norm=True, fused=True),
        # odd length, fp32, partial interleaved rotation
        dict(name="prep_odd_f32", op="prep", B=3, N=2047, Hq=16, Hkv=16, D=64, rot=32, inter=True, dtype="fp32",
             norm=True, fused=False),
        # gradients of the training batch
        dict(name="prep_bwd_16384", op="prep_bwd", B=2, N=16384, Hq=32, Hkv=8, D=128, rot=128, inter=False,
             dtype="bf16", norm=True, fused=False),
        # gradients of a short odd batch, head dim 80
        dict(name="prep_bwd_odd", op="prep_bwd", B=1, N=333, Hq=16, Hkv=4, D=80, rot=80, inter=False, dtype="bf16",
             norm=True, fused=False),
        # one decode step: one token for each of 32 sequences, queries in the same launch
        dict(name="append_step_b32", op="append", B=32, N=1, Hq=32, Hkv=8, D=128, rot=128, inter=False, page=64,
             block=64, start=4096, ragged=True, pool="e4m3", norm=True),
        # a ragged prompt chunk into the e4m3 pages
        dict(name="append_prompt", op="append", B=8, N=2048, Hq=0, Hkv=8, D=128, rot=128, inter=False, page=64,
             block=64, start=1000, ragged=True, pool="e4m3", norm=True),
        # a packed prompt into bf16 pages
        dict(name="append_bf16_8192", op="append", B=1, N=8191, Hq=0, Hkv=8, D=64, rot=64, inter=False, page=16,
             block=16, start=5, ragged=False, pool="bf16", norm=False),
        # the decode configuration: 32 sequences of 4k..32k keys, one query
        dict(name="attend_b32_32k", op="attend", B=32, Hq=32, Hkv=8, L=1, D=128, lo=4096, hi=32768, page=64, block=64,
             mask="causal", window=0, cap=0.0),
        # a single long sequence: the latency of one step
        dict(name="attend_b1_32k", op="attend", B=1, Hq=32, Hkv=8, L=1, D=128, lo=32768, hi=32768, page=64, block=64,
             mask="causal", window=0, cap=0.0),
        # four drafted tokens, window and soft cap, head dim 64, small pages, short ragged sequences
        # (one shorter than the drafted tokens leaves rows without a key)
        dict(name="attend_draft_cap", op="attend", B=17, Hq=16, Hkv=4, L=4, D=64, lo=1, hi=4099, page=16, block=16,
             mask="sliding_window", window=1024, cap=50.0),
        # a prompt chunk against its cached history
        dict(name="attend_chunk_1024", op="attend", B=2, Hq=32, Hkv=8, L=1024, D=128, lo=5000, hi=8192, page=64,
             block=64, mask="causal", window=0, cap=0.0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["prep", "prep_bwd", "append", "attend", "attend"])
    Hkv = rng.choice([1, 2, 4, 8])
    G = rng.choice([1, 2, 3, 4, 8])
    if op in ("prep", "prep_bwd"):
        D = rng.choice([64, 80, 96, 128])
        rot = rng.choice([D, D, D // 2])
        B = rng.randint(1, 16)
        return dict(op=op, B=B, N=max(1, _log(rng, 1, 16384) // B), Hq=Hkv * G, Hkv=Hkv, D=D, rot=rot,
                    inter=rng.random() < 0.4, dtype=rng.choice(["bf16", "bf16", "fp32"]), norm=rng.random() < 0.8,
                    fused=rng.random() < 0.5)
    page = rng.choice([16, 32, 64, 128])
    block = rng.choice([b for b in (1, 8, 16, 32, 64, 128) if b <= page])
    D = rng.choice([64, 128])
    if op == "append":
        B = rng.randint(1, 32)
        return dict(op=op, B=B, N=max(1, _log(rng, 1, 8192) // B), Hq=rng.choice([0, Hkv * G]), Hkv=Hkv, D=D,
                    rot=rng.choice([D, D // 2]), inter=rng.random() < 0.4, page=page, block=block,
                    start=_log(rng, 1, 4096) - 1, ragged=rng.random() < 0.6,
                    pool=rng.choice(["e4m3", "e4m3", "bf16"]), norm=rng.random() < 0.6)
    L = rng.choice([1, 1, 2, 4, 7, 16, 33, 200])
    B = rng.randint(1, 2) if L > 16 else rng.randint(1, 24)
    hi = _log(rng, 300, 8192 if L > 16 else 16384)
    mask = rng.choice(["causal", "causal", "sliding_window"])
    return dict(op=op, B=B, Hq=Hkv * G, Hkv=Hkv, L=L, D=D, lo=max(1, hi // rng.randint(1, 6)), hi=hi, page=page,
                block=block, mask=mask, window=rng.randint(16, 1024) if mask == "sliding_window" else 0,
                cap=rng.choice([0.0, 0.0, 30.0]))


# --------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------
def _rope_inputs(rot, dev):
    i = torch.arange(rot // 2, dtype=torch.float64, device=dev)
    return (10000.0 ** (-2.0 * i / rot)).float()


def _pages_for(c, lens, g, dev):
    """A page table whose pages are shuffled over the pool."""
    per_seq = -(-int(lens) // c["page"])
    total = c["B"] * per_seq
    ids = torch.randperm(total, generator=g, device=dev).to(torch.int32)
    return ids.reshape(c["B"], per_seq).contiguous(), total


def _pow2_scale(amax):
    """2^ceil(log2(amax / 448)), at least 2^-126; 0 where amax is 0."""
    m, e = torch.frexp(amax)  # amax = m 2^e, m in [0.5, 1): amax <= 448 * 2^(e - 9) when m <= 0.875
    e = torch.where(m <= 0.875, e - 9, e - 8).clamp(min=-126)
    return torch.where(amax > 0, torch.ldexp(torch.ones_like(amax), e), torch.zeros_like(amax))


def _quantised_pool(pages, c, g, dev):
    """Random e4m3 pool (pages, Hkv, page, D) with its scales (pages, Hkv, page / block)."""
    codes = torch.empty((pages, c["Hkv"], c["page"], c["D"]), dtype=E4M3, device=dev)
    scale = torch.empty((pages, c["Hkv"], c["page"] // c["block"]), dtype=torch.float32, device=dev)
    step = max(1, (1 << 26) // (c["Hkv"] * c["page"] * c["D"]))
    for p in range(0, pages, step):
        n = min(step, pages - p)
        x = torch.randn((n, c["Hkv"], c["page"] // c["block"], c["block"], c["D"]), generator=g, device=dev)
        s = _pow2_scale(x.abs().amax((-1, -2)))
        codes[p:p + n] = (x / s[..., None, None]).to(E4M3).reshape(n, c["Hkv"], c["page"], c["D"])
        scale[p:p + n] = s
    return codes, scale


def prepare(case, seed):
    c, dev = dict(case), "cuda"
    g = torch.Generator(dev).manual_seed(int(seed))

    def randn(*shape, dtype=torch.bfloat16):
        return torch.randn(shape, generator=g, device=dev, dtype=torch.float32).to(dtype)

    s = {"case": c}
    if c["op"] in ("prep", "prep_bwd"):
        dt = torch.bfloat16 if c["dtype"] == "bf16" else torch.float32
        B, N, Hq, Hkv, D = c["B"], c["N"], c["Hq"], c["Hkv"], c["D"]
        if c["fused"]:  # slices of one projection's output (B, N, heads, D)
            qkv = randn(B, N, Hq + 2 * Hkv, D, dtype=dt).transpose(1, 2)
            s["q"], s["k"] = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv]
        else:
            s["q"], s["k"] = randn(B, Hq, N, D, dtype=dt), randn(B, Hkv, N, D, dtype=dt)
        s["qw"], s["kw"] = 1 + 0.1 * randn(D, dtype=torch.float32), 1 + 0.1 * randn(D, dtype=torch.float32)
        s["inv_freq"] = _rope_inputs(c["rot"], dev)
        # each row of the batch is a stretch of a longer text
        first = torch.randint(0, 100000, (B, 1), generator=g, device=dev)
        s["pos"] = (first + torch.arange(N, device=dev)).to(torch.int32).contiguous()
        if c["op"] == "prep_bwd":
            s["dq"], s["dk"] = randn(B, Hq, N, D, dtype=dt), randn(B, Hkv, N, D, dtype=dt)
    elif c["op"] == "append":
        B, N, Hkv, D = c["B"], c["N"], c["Hkv"], c["D"]
        qkv = randn(B, N, c["Hq"] + 2 * Hkv, D).transpose(1, 2)
        s["q"] = qkv[:, :c["Hq"]] if c["Hq"] else None
        s["k"], s["v"] = qkv[:, c["Hq"]:c["Hq"] + Hkv], qkv[:, c["Hq"] + Hkv:]
        s["kw"], s["qw"] = 1 + 0.1 * randn(D, dtype=torch.float32), 1 + 0.1 * randn(D, dtype=torch.float32)
        s["inv_freq"] = _rope_inputs(c["rot"], dev)
        if c["ragged"]:
            s["cache_len"] = torch.randint(0, c["start"] + 1, (B,), generator=g, device=dev).to(torch.int32)
            s["new_len"] = torch.randint((N + 1) // 2, N + 1, (B,), generator=g, device=dev).to(torch.int32)
        else:
            s["cache_len"] = torch.full((B,), c["start"], dtype=torch.int32, device=dev)
            s["new_len"] = torch.full((B,), N, dtype=torch.int32, device=dev)
        s["table"], pages = _pages_for(c, c["start"] + N, g, dev)
        if c["pool"] == "e4m3":
            s["kp"], s["ks"] = _quantised_pool(pages, c, g, dev)
            s["vp"], s["vs"] = _quantised_pool(pages, c, g, dev)
        else:
            s["kp"], s["vp"] = randn(pages, Hkv, c["page"], D), randn(pages, Hkv, c["page"], D)
            s["ks"] = s["vs"] = None
    else:
        B = c["B"]
        s["q"] = randn(B, c["Hq"], c["L"], c["D"])
        s["kv_len"] = torch.randint(c["lo"], c["hi"] + 1, (B,), generator=g, device=dev).to(torch.int32)
        s["table"], pages = _pages_for(c, c["hi"], g, dev)
        s["kp"], s["ks"] = _quantised_pool(pages, c, g, dev)
        s["vp"], s["vs"] = _quantised_pool(pages, c, g, dev)
        s["mask"] = dict(kind=c["mask"], kv_len=s["kv_len"])
        if c["mask"] == "sliding_window":
            s["mask"].update(window=c["window"], n_sink=4)
        s["score"] = dict(kind="softcap", cap=c["cap"]) if c["cap"] > 0 else None
        if own:  # the plan of a step: the block mask of these lengths, which every layer of the model shares
            import programmable_block_sparse_b200 as fa
            s["bm"] = fa.flexattn_build_block_mask(s["mask"], B, 1, c["L"], s["table"].shape[1] * c["page"], 128, 128)
    return s


# --------------------------------------------------------------------------
# plain forms
# --------------------------------------------------------------------------
def _cos_sin(pos, inv_freq):
    ang = pos.double()[..., None] * inv_freq.double()
    return ang.cos().float(), ang.sin().float()


def _split(x, rot, inter):
    h = rot // 2
    return (x[..., 0:rot:2], x[..., 1:rot:2]) if inter else (x[..., :h], x[..., h:rot])


def _rotate(x, cos, sin, rot, inter):
    a, b = _split(x, rot, inter)
    ra, rb = a * cos - b * sin, b * cos + a * sin
    turned = torch.stack((ra, rb), -1).flatten(-2) if inter else torch.cat((ra, rb), -1)
    return torch.cat((turned, x[..., rot:]), -1)


def _norm_rotate(x, w, c, cos, sin):
    x = x.float()
    if c["norm"]:
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6) * w
    return _rotate(x, cos, sin, c["rot"], c["inter"])


def _norm_rotate_grad(x, dy, w, c, cos, sin):
    x, dy = x.float(), dy.float()
    g = _rotate(dy, cos, -sin, c["rot"], c["inter"])
    if not c["norm"]:
        return g, None
    r = torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6)
    dw = (g * x * r).double().sum((0, 1, 2)).float()
    gw = g * w
    return r * (gw - x * r.square() * (gw * x).mean(-1, keepdim=True)), dw


def _append_plain(new, pool, scale, s, c):
    """new (B, Hkv, N, D) fp32 into the pages that its tokens touch."""
    B, N, page, block, D = c["B"], c["N"], c["page"], c["block"], c["D"]
    start, count = s["cache_len"].long(), s["new_len"].long()
    nb = (N + block - 2) // block + 1
    j = torch.arange(nb, device=new.device)
    last = torch.clamp(start + count - 1, min=0) // block
    blk = torch.minimum((start // block)[:, None] + j, last[:, None])  # (B, nb); repeats name one block twice
    blk = torch.maximum(blk, torch.minimum(start // block, last)[:, None])
    slot = blk[..., None] * block + torch.arange(block, device=new.device)  # (B, nb, block)
    n = slot - start[:, None, None]
    is_new, is_old = (n >= 0) & (n < count[:, None, None]), n < 0
    pg = s["table"].long().gather(1, torch.clamp(blk * block // page, max=s["table"].shape[1] - 1))
    ib = blk % (page // block)
    vals = new.permute(0, 2, 1, 3)[torch.arange(B, device=new.device)[:, None, None], n.clamp(0, N - 1)]
    vals = vals.permute(0, 1, 3, 2, 4)  # (B, nb, Hkv, block, D)
    view = pool.view(pool.shape[0], pool.shape[1], page // block, block, D)
    m_new, m_old = is_new[:, :, None, :, None], is_old[:, :, None, :, None]
    if scale is None:
        view[pg, :, ib] = torch.where(m_new, vals.to(pool.dtype), view[pg, :, ib])
        return
    codes = view.view(torch.uint8)[pg, :, ib].view(E4M3).float()
    s_old = scale[pg, :, ib]  # (B, nb, Hkv)
    fresh = _pow2_scale(torch.where(m_new, vals, 0.0).abs().amax((-1, -2)))
    had = is_old.any(-1)[:, :, None]
    s_new = torch.where(had, torch.maximum(s_old, fresh), fresh)
    s_new = torch.where(is_new.any(-1)[:, :, None], s_new, s_old)
    inv = torch.where(s_new > 0, 1.0 / s_new, 0.0)[..., None, None]
    old = torch.where((s_new > s_old)[..., None, None] & m_old, codes * (s_old[..., None, None] * inv), codes)
    out = torch.where(m_new, vals * inv, old).to(E4M3)
    view.view(torch.uint8)[pg, :, ib] = out.view(torch.uint8)
    scale[pg, :, ib] = s_new


def _dense(pool, scale, table, c):
    x = pool.view(torch.uint8)[table.long()].view(E4M3).float()  # (B, P, Hkv, page, D)
    x = x * scale[table.long()].repeat_interleave(c["block"], -1)[..., None]
    return x.permute(0, 2, 1, 3, 4).flatten(2, 3)  # (B, Hkv, S, D)


def _visible(c, kv_len, S, dev):
    q = torch.arange(c["L"], device=dev)[None, :, None] + (kv_len.long()[:, None, None] - c["L"])
    kv = torch.arange(S, device=dev)[None, None, :]
    m = (kv <= q) & (kv < kv_len[:, None, None])
    if c["mask"] == "sliding_window":
        m = m & ((q - kv < c["window"]) | (kv < 4))
    return m  # (B, L, S)


def _attend_plain(s, c):
    B, Hq, Hkv, L, D = c["B"], c["Hq"], c["Hkv"], c["L"], c["D"]
    G = Hq // Hkv
    k = _dense(s["kp"], s["ks"], s["table"], c)
    q = s["q"].float().reshape(B, Hkv, G * L, D)
    x = torch.matmul(q, k.transpose(-1, -2)) * (1.0 / math.sqrt(D))
    del k
    if c["cap"] > 0:
        x = c["cap"] * torch.tanh(x / c["cap"])
    vis = _visible(c, s["kv_len"], x.shape[-1], x.device)[:, None, None]
    x = x.reshape(B, Hkv, G, L, -1).masked_fill(~vis, -math.inf)
    top = x.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    p = torch.exp(x - top)
    del x
    total = p.sum(-1, keepdim=True)
    v = _dense(s["vp"], s["vs"], s["table"], c)
    out = torch.matmul(p.reshape(B, Hkv, G * L, -1), v).reshape(B, Hkv, G, L, D)
    out = torch.where(total > 0, out / total, 0.0).reshape(B, Hq, L, D).to(torch.bfloat16)
    lse = (top + torch.log(total)).reshape(B, Hq, L)
    return out, lse


def _run_plain(s):
    c = s["case"]
    if c["op"] == "prep":
        cos, sin = (t[:, None] for t in _cos_sin(s["pos"], s["inv_freq"]))
        return tuple(_norm_rotate(s[x], s[x + "w"], c, cos, sin).to(s[x].dtype) for x in "qk")
    if c["op"] == "prep_bwd":
        cos, sin = (t[:, None] for t in _cos_sin(s["pos"], s["inv_freq"]))
        (dq, dqw), (dk, dkw) = (_norm_rotate_grad(s[x], s["d" + x], s[x + "w"], c, cos, sin) for x in "qk")
        return dq.to(s["q"].dtype), dk.to(s["k"].dtype), dqw, dkw
    if c["op"] == "append":
        pos = s["cache_len"][:, None] + torch.arange(c["N"], device=s["k"].device)
        cos, sin = (t[:, None] for t in _cos_sin(pos, s["inv_freq"]))
        _append_plain(_norm_rotate(s["k"], s["kw"], c, cos, sin), s["kp"], s["ks"], s, c)
        _append_plain(s["v"].float(), s["vp"], s["vs"], s, c)
        q = None if s["q"] is None else _norm_rotate(s["q"], s["qw"], c, cos, sin).to(s["q"].dtype)
        return q, s["kp"], s["vp"], s["ks"], s["vs"]
    return _attend_plain(s, c)


# --------------------------------------------------------------------------
# the framework's calls
# --------------------------------------------------------------------------
def _run_own(s):
    import programmable_block_sparse_b200 as fa
    c = s["case"]
    if c["op"] == "attend":
        return fa.flexattn_forward_fp8(
            s["q"], s["kp"], s["vp"], s["bm"], quant={"k_scale": s["ks"], "v_scale": s["vs"],
                                                      "scale_block": c["block"]},
            score_mod=s["score"], mask_mod=s["mask"], enable_gqa=c["Hq"] != c["Hkv"],
            paged={"page_table": s["table"], "page_size": c["page"]})
    q_norm = {"weight": s["qw"], "eps": 1e-6} if c["norm"] else None
    k_norm = {"weight": s["kw"], "eps": 1e-6} if c["norm"] else None
    rope = {"inv_freq": s["inv_freq"], "interleaved": c["inter"]}
    if c["op"] == "append":
        cache = {"k": s["kp"], "v": s["vp"], "cache_len": s["cache_len"], "new_len": s["new_len"],
                 "page_table": s["table"]}
        if c["pool"] == "e4m3":
            cache.update(k_scale=s["ks"], v_scale=s["vs"], scale_block=c["block"])
        q = fa.flexattn_cache_append(s["k"], s["v"], cache, k_norm=k_norm, rope=rope, q=s["q"], q_norm=q_norm)
        return q, s["kp"], s["vp"], s["ks"], s["vs"]
    rope["pos"] = s["pos"]
    if c["op"] == "prep":
        return fa.flexattn_qk_norm_rope(s["q"], s["k"], q_norm=q_norm, k_norm=k_norm, rope=rope)
    return fa.flexattn_qk_norm_rope_backward(s["q"], s["k"], s["dq"], s["dk"], q_norm=q_norm, k_norm=k_norm, rope=rope)


def run(state):
    return _run_own(state) if own else _run_plain(state)


# --------------------------------------------------------------------------
# work and the definition in 64 bits
# --------------------------------------------------------------------------
def work(case):
    c = case
    if c["op"] in ("prep", "prep_bwd"):
        el = 2 if c["dtype"] == "bf16" else 4
        elems = c["B"] * c["N"] * (c["Hq"] + c["Hkv"]) * c["D"]
        if c["op"] == "prep":
            return {"bytes": 2 * el * elems + 4 * c["B"] * c["N"], "flops": 8 * elems}
        streams = 3 if c["norm"] else 2
        return {"bytes": streams * el * elems + 4 * c["B"] * c["N"], "flops": 16 * elems}
    if c["op"] == "append":
        toks = c["B"] * c["N"] * (0.75 if c["ragged"] else 1.0)
        el = 1 if c["pool"] == "e4m3" else 2
        scales = 8.0 * toks * c["Hkv"] / c["block"] if el == 1 else 0.0
        return {"bytes": toks * c["D"] * (c["Hkv"] * 2 * (2 + el)) + scales + 4.0 * c["B"] * c["N"] * c["Hq"] * c["D"],
                "flops": 8.0 * toks * c["D"] * (2 * c["Hkv"] + c["Hq"])}
    mean = 0.5 * (c["lo"] + c["hi"])
    keys = mean if c["mask"] == "causal" else min(mean, c["window"] + c["L"] + 4)
    per_query = keys if c["L"] <= 16 else min(mean - c["L"] / 2, c["window"] + 4 if c["window"] else mean)
    return {"bytes": c["B"] * (c["Hkv"] * keys * (2 * c["D"] + 8.0 / c["block"]) + 4.0 * c["Hq"] * c["L"] * (c["D"] + 1)),
            "flops": 4.0 * c["B"] * c["Hq"] * c["L"] * max(per_query, 1) * c["D"]}


def _exact_rows(x, w, pos, inv_freq, c):
    """(H, N, D) rows of one sequence, as complex pairs turned by e^{i pos f}."""
    y = x.double()
    if c["norm"]:
        y = y / torch.sqrt((y * y).sum(-1, keepdim=True) / c["D"] + 1e-6) * w.double()
    h, y = c["rot"] // 2, y.clone()
    first = slice(0, c["rot"], 2) if c["inter"] else slice(0, h)
    second = slice(1, c["rot"], 2) if c["inter"] else slice(h, c["rot"])
    ang = pos.double()[:, None] * inv_freq.double()[None, :]
    z = torch.complex(y[..., first], y[..., second]) * torch.polar(torch.ones_like(ang), ang)
    y[..., first], y[..., second] = z.real, z.imag
    return y


def _exact_grad(x, dy, w, pos, inv_freq, c):
    """Row gradients through the Jacobian of the norm; dw in 64 bits."""
    bare = dict(c, norm=False)
    g = _exact_rows(dy, w, -pos, inv_freq, bare)
    if not c["norm"]:
        return g, None
    x, w = x.double(), w.double()
    r = 1.0 / torch.sqrt((x * x).sum(-1, keepdim=True) / c["D"] + 1e-6)
    xhat, u = x * r, g * w
    return r * (u - xhat * (xhat * u).sum(-1, keepdim=True) / c["D"]), (g * xhat).sum((0, 1))


def _exact_append(rows, pool, scale, table, start, count, c):
    """One sequence's rows (Hkv, count, D) in 64 bits into the pool, block by block."""
    if scale is None:
        slot = torch.arange(start, start + count, device=rows.device)
        pool[table[slot // c["page"]].long(), :, slot % c["page"]] = rows.permute(1, 0, 2)
        return
    block = c["block"]
    first, last = start // block, (start + count - 1) // block
    for j in range(first, last + 1) if count else ():
        a, b = max(j * block, start), min((j + 1) * block, start + count)
        pg, at = int(table[j * block // c["page"]]), j * block % c["page"]
        new = rows[:, a - start:b - start]
        amax = new.abs().amax((1, 2))
        s = torch.where(amax > 0, 2.0 ** torch.ceil(torch.log2(amax / E4M3_MAX)), 0.0)
        if a > j * block:
            had = scale[pg, :, at // block].double()
            s = torch.maximum(s, had)
            old = pool[pg, :, at:at + a - j * block]
            pool[pg, :, at:at + a - j * block] = (old * (had / s)[:, None, None]).float().to(E4M3).double()
        scale[pg, :, at // block] = s
        pool[pg, :, at + a - j * block:at + b - j * block] = torch.where(
            s[:, None, None] > 0, new / s[:, None, None], 0.0).float().to(E4M3).double()


def exact(case, seed):
    c, s = dict(case), prepare(case, seed)
    if c["op"] in ("prep", "prep_bwd"):
        outs = []
        for x in "qk":
            per = [(_exact_grad(s[x][b], s["d" + x][b], s[x + "w"], s["pos"][b], s["inv_freq"], c)
                    if c["op"] == "prep_bwd" else (_exact_rows(s[x][b], s[x + "w"], s["pos"][b], s["inv_freq"], c), None))
                   for b in range(c["B"])]
            outs.append((torch.stack([p[0] for p in per]), None if per[0][1] is None else sum(p[1] for p in per)))
        return (outs[0][0], outs[1][0]) + ((outs[0][1], outs[1][1]) if c["op"] == "prep_bwd" else ())
    if c["op"] == "append":
        if c["B"] * c["N"] // c["block"] > 20000:
            return None  # block by block this takes too long
        kp, vp = s["kp"].double(), s["vp"].double()
        ks, vs = (None, None) if s["ks"] is None else (s["ks"].double(), s["vs"].double())
        q = None if s["q"] is None else []
        start, count = s["cache_len"].tolist(), s["new_len"].tolist()
        for b in range(c["B"]):
            pos = start[b] + torch.arange(c["N"], device="cuda")
            k = _exact_rows(s["k"][b], s["kw"], pos, s["inv_freq"], c)[:, :count[b]]
            table = s["table"][b].cpu() if ks is not None else s["table"][b]
            _exact_append(k, kp, ks, table, start[b], count[b], c)
            _exact_append(s["v"][b, :, :count[b]].double(), vp, vs, table, start[b], count[b], c)
            if q is not None:
                q.append(_exact_rows(s["q"][b], s["qw"], pos, s["inv_freq"], c))
        return None if q is None else torch.stack(q), kp, vp, ks, vs
    outs, lses = [], []
    G = c["Hq"] // c["Hkv"]
    for b, n in enumerate(s["kv_len"].tolist()):
        pages = s["table"][b].long()
        k, v = ((p.view(torch.uint8)[pages].view(E4M3).double() * sc[pages].double().repeat_interleave(
            c["block"], -1)[..., None]).transpose(0, 1).reshape(c["Hkv"], -1, c["D"])[:, :n]
            for p, sc in ((s["kp"], s["ks"]), (s["vp"], s["vs"])))
        at = torch.arange(n - c["L"], n, device="cuda")[:, None]
        kv = torch.arange(n, device="cuda")[None, :]
        see = kv <= at
        if c["mask"] == "sliding_window":
            see &= (at - kv < c["window"]) | (kv < 4)
        out, lse = [], []
        for h in range(c["Hq"]):
            x = s["q"][b, h].double() @ k[h // G].T / math.sqrt(c["D"])
            if c["cap"] > 0:
                x = c["cap"] * torch.tanh(x / c["cap"])
            x = torch.where(see, x, -math.inf)
            z = torch.logsumexp(x, -1)
            out.append(torch.where(z > -math.inf, 1.0, 0.0)[:, None] * (
                torch.exp(x - torch.where(z > -math.inf, z, 0.0)[:, None]) @ v[h // G]))
            lse.append(z)
        outs.append(torch.stack(out))
        lses.append(torch.stack(lse))
    return torch.stack(outs), torch.stack(lses)
