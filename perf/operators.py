"""Cases of the layer operators around the 4-bit products: what they compute, in plain
torch, and the calls a program makes of them.

    epilogue   y = residual + act(x . W~^T + bias), W~ packed as include/qmm.h lays it out
    store      keys and values of new tokens into a paged 4-bit cache, and read back
    load       rows of the cache, decoded
    attend     attention of each sequence's last tokens over its pages of the cache

`own` False computes every case with elementary torch operations on the packed bytes; `own`
True makes the library's calls on the same bytes.
"""
import math
import random

import torch

own = False


# ------------------------------------------------------------------------ cases

def listed():
    return [
        # LLaMA-7B output projection, one token, added onto the residual stream
        dict(name="epilogue_m1_4096", op="epilogue", M=1, N=4096, K=4096, mode="sym", group=128,
             dtype="f16", bias=False, act="none", residual=True),
        # LLaMA-7B down projection, a batch of 16 tokens
        dict(name="epilogue_m16_down", op="epilogue", M=16, N=4096, K=11008, mode="asym", group=128,
             dtype="f16", bias=False, act="none", residual=True),
        # LLaMA-70B fused QKV projection with a bias, 64 tokens, bf16
        dict(name="epilogue_m64_qkv_bf16", op="epilogue", M=64, N=10240, K=8192, mode="asym",
             group=128, dtype="bf16", bias=True, act="none", residual=False),
        # an ungated feed-forward layer of a prompt: bias and GELU
        dict(name="epilogue_m1024_gelu", op="epilogue", M=1024, N=11008, K=4096, mode="sym",
             group=128, dtype="f16", bias=True, act="gelu", residual=False),
        # one decode step of eight sequences, 70B heads
        dict(name="store_step8", op="store", tokens=8, heads=8, dim=128, page=64, mode="sym",
             group=-1, dtype="bf16"),
        # the prompt of a 7B model, 32 heads, asymmetric groups of 64
        dict(name="store_prompt", op="store", tokens=8191, heads=32, dim=128, page=64, mode="asym",
             group=64, dtype="f16"),
        # a short prefix of a small model read back
        dict(name="load_prefix", op="load", tokens=333, heads=4, dim=64, page=16, mode="asym",
             group=32, dtype="f16"),
        # long prefixes read back for a dense product
        dict(name="load_long", op="load", tokens=16384, heads=32, dim=128, page=32, mode="sym",
             group=128, dtype="bf16"),
        # one sequence, a short cache, a head of keys per query head: latency
        dict(name="attend_one_short", op="attend", batch=1, ctx=517, queries=1, heads=32, kv=32,
             dim=128, page=16, mode="sym", group=-1, dtype="f16", window=0),
        # decode of a ragged batch, 70B heads
        dict(name="attend_batch32", op="attend", batch=32, ctx=4096, queries=1, heads=64, kv=8,
             dim=128, page=64, mode="asym", group=32, dtype="bf16", window=0),
        # decode of long sequences, larger than L2
        dict(name="attend_long", op="attend", batch=16, ctx=32768, queries=1, heads=64, kv=8,
             dim=128, page=64, mode="sym", group=-1, dtype="bf16", window=0),
        # a chunk of a prompt behind a cached prefix
        dict(name="attend_chunk", op="attend", batch=2, ctx=6000, queries=2048, heads=32, kv=8,
             dim=128, page=64, mode="sym", group=-1, dtype="f16", window=0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["epilogue", "epilogue", "store", "load", "attend", "attend", "attend"])
    dtype = rng.choice(["f16", "bf16"])
    if op == "epilogue":
        mode = rng.choice(["sym", "asym", "lut"])
        group = rng.choice([-1, 32, 64, 128])
        K, N = 128 * _log(rng, 4, 86), 16 * _log(rng, 8, 640)
        M = min(_log(rng, 1, 1024), 46_000_000_000 // (N * K))
        return dict(op=op, M=M, N=N, K=K, mode=mode,
                    group=group, dtype=dtype, bias=rng.random() < 0.5,
                    act=rng.choice(["none", "relu", "gelu", "gelu_tanh", "silu"]),
                    residual=rng.random() < 0.5)
    dim = rng.choice([64, 128, 128, 256])
    mode = rng.choice(["sym", "asym"])
    group = rng.choice([g for g in (-1, 32, 64, 128) if g <= dim])
    page = rng.choice([16, 32, 64, 128])
    if op in ("store", "load"):
        heads = rng.choice([1, 2, 4, 5, 8, 16, 32])
        tokens = min(_log(rng, 1, 8192), 33_000_000 // (heads * dim))
        return dict(op=op, tokens=tokens, heads=heads, dim=dim, page=page, mode=mode, group=group, dtype=dtype)
    kv = rng.choice([1, 2, 4, 8])
    heads = kv * rng.choice([1, 2, 3, 4, 7, 8])
    queries = rng.choice([1, 1, 1, _log(rng, 2, 16), _log(rng, 16, 1024)])
    ctx = max(queries, _log(rng, 1, 16384))
    # no more work than the longest listed case: tokens of cache, and pairs of a chunk
    batch = min(_log(rng, 1, 64), max(1, 300_000_000 // (ctx * kv * dim)),
                max(1, (1 << 21) // (queries * ctx)))
    return dict(op=op, batch=batch, ctx=ctx, queries=queries, heads=heads, kv=kv, dim=dim, page=page,
                mode=mode, group=group, dtype=dtype,
                window=rng.choice([0, 0, 0, max(1, ctx // 3)]))


def _lens(case):
    """Ragged sequence lengths (the first is the longest) and query counts of an attend case."""
    rng = random.Random("lens %(batch)d %(ctx)d %(queries)d" % case)
    lens, nq = [case["ctx"]], [case["queries"]]
    for _ in range(case["batch"] - 1):
        n = rng.randint(max(1, case["ctx"] // 3), case["ctx"])
        lens.append(n)
        nq.append(min(n, case["queries"] if case["queries"] == 1
                      else rng.randint(max(1, case["queries"] // 2), case["queries"])))
    return lens, nq


def _groups(case):
    return 1 if case["group"] == -1 else case["dim"] // case["group"]


def _tile_bytes(dim, G, mode):
    return 16 * dim + (64 if mode == "sym" else 128) * G


def work(case):
    op = case["op"]
    if op == "epilogue":
        M, N, K = case["M"], case["N"], case["K"]
        G = 1 if case["group"] == -1 else K // case["group"]
        b = N * K // 2 + N * G * (4 if case["mode"] == "asym" else 2) + 2 * M * K + 2 * M * N
        b += (2 * N if case["bias"] else 0) + (2 * M * N if case["residual"] else 0)
        return {"bytes": b, "flops": 2 * M * N * K}
    G, D = _groups(case), case["dim"]
    per_token = _tile_bytes(D, G, case["mode"]) / 16           # K and V of one head
    if op == "store":      # k and v read, the cache written; the cache read, k and v written back
        rows = case["tokens"] * case["heads"]
        return {"bytes": int(rows * (8 * D + 2 * per_token) + 4 * case["tokens"]), "flops": 8 * rows * D}
    if op == "load":
        rows = case["tokens"] * case["heads"]
        return {"bytes": int(rows * (4 * D + per_token) + 4 * case["tokens"]), "flops": 4 * rows * D}
    lens, nq = _lens(case)
    w = case["window"]
    keys = pairs = 0
    for n, m in zip(lens, nq):
        first = 0 if not w else max(0, n - m - w + 1)
        keys += n - first
        for i in range(m):
            pos = n - m + i
            pairs += min(pos + 1, w) if w else pos + 1
    b = keys * case["kv"] * per_token + 4 * sum(nq) * case["heads"] * D
    return {"bytes": int(b), "flops": 4 * D * case["heads"] * pairs}


# ---------------------------------------------------------------------- inputs

def _dtype(case):
    return torch.float16 if case["dtype"] == "f16" else torch.bfloat16


def _page_list(case, pages_needed, gen):
    """The pages a cache of some spare pages hands out, in no order."""
    total = pages_needed + max(2, pages_needed // 8)
    return total, torch.randperm(total, generator=gen, device="cuda")[:pages_needed].to(torch.int32)


def _random_cache(case, heads, pages, gen):
    """A cache as a program finds it: codes of roughly normal values, scales of their spread."""
    D, G, mode, page = case["dim"], _groups(case), case["mode"], case["page"]
    T = _tile_bytes(D, G, mode)
    cache = torch.empty(pages, heads, page // 16, T, dtype=torch.uint8, device="cuda")
    step = max(1, (1 << 27) // (heads * (page // 16) * 16 * D * 2))
    for p0 in range(0, pages, step):
        c = cache[p0:p0 + step]
        n = c.shape[0]
        x = torch.randn(n, heads, page // 16, 16 * D * 2, generator=gen, device="cuda") * 2.5
        code = (x.round_().clamp_(-7, 7) + 8).to(torch.uint8)
        c[..., :16 * D] = code[..., 0::2] | (code[..., 1::2] << 4)
        s = torch.rand(n, heads, page // 16, 32 * G, generator=gen, device="cuda") * 0.3 + 0.25
        if mode == "asym":
            z = torch.randint(5, 11, s.shape, generator=gen, device="cuda").float()
            s = torch.stack([s, z], -1).flatten(-2)
        c[..., 16 * D:] = s.half().view(torch.uint8)
    return cache


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    st = dict(case=case)
    if own:
        import weight_only_quantized_int4_b200 as lib
        st["lib"] = lib
    dt = _dtype(case)
    if case["op"] == "epilogue":
        M, N, K, mode = case["M"], case["N"], case["K"], case["mode"]
        G = 1 if case["group"] == -1 else K // case["group"]
        st["qweight"] = torch.randint(0, 256, (N * K // 2,), dtype=torch.uint8, device="cuda",
                                      generator=gen)
        st["scales"] = ((torch.rand(N * G, device="cuda", generator=gen) + 0.5) *
                        (0.03 if mode == "lut" else 0.004)).half().view(torch.int16)
        st["zl"] = None
        if mode == "asym":
            st["zl"] = torch.randint(5, 11, (N * G,), device="cuda", generator=gen).half().view(torch.int16)
        elif mode == "lut":
            v = torch.erfinv((torch.arange(16, device="cuda") + 0.5) / 8 - 1)
            st["zl"] = (v / v.abs().max()).half().view(torch.int16)
        st["x"] = torch.randn(M, K, device="cuda", generator=gen).to(dt)
        st["bias"] = torch.randn(N, device="cuda", generator=gen).to(dt) if case["bias"] else None
        st["residual"] = torch.randn(M, N, device="cuda", generator=gen).to(dt) if case["residual"] else None
        if own:
            st["ws"] = st["lib"].workspace(M, N, K, mode, 4, case["group"])
        return st
    if case["op"] in ("store", "load"):
        T, H, D, page = case["tokens"], case["heads"], case["dim"], case["page"]
        pages, mine = _page_list(case, (T + page - 1) // page, gen)
        pos = torch.arange(T, device="cuda")
        st["slots"] = (mine[pos // page].long() * page + pos % page).to(torch.int32)
        if case["op"] == "load":
            st["cache"] = _random_cache(case, H, pages, gen)
            return st
        st["cache"] = torch.zeros(pages, H, page // 16, _tile_bytes(D, _groups(case), case["mode"]),
                                  dtype=torch.uint8, device="cuda")
        # keys and values are slices of the fused projection's rows; keys carry a few large channels
        qkv = torch.randn(T, 3, H, D, device="cuda", generator=gen)
        qkv[:, 1] *= 1 + 4 * (torch.rand(H, D, device="cuda", generator=gen) < 0.05)
        st["qkv"] = qkv.to(dt)
        return st
    lens, nq = _lens(case)
    page, D, B = case["page"], case["dim"], case["batch"]
    need = [(n + page - 1) // page for n in lens]
    pages, mine = _page_list(case, sum(need), gen)
    st["cache"] = _random_cache(case, case["kv"], pages, gen)
    table = torch.zeros(B, max(need), dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = mine[at:at + n]
        at += n
    st["table"] = table
    st["lens_host"], st["nq_host"] = lens, nq
    st["lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
    cu = [0]
    for m in nq:
        cu.append(cu[-1] + m)
    st["cu"] = torch.tensor(cu, dtype=torch.int32, device="cuda")
    st["q"] = torch.randn(cu[-1], case["heads"], D, device="cuda", generator=gen).to(dt)
    st["scale"] = 1.0 / math.sqrt(D)
    if own:
        st["ws"] = st["lib"].kv_workspace(B, max(nq), case["heads"], case["kv"], D)
    return st


# ------------------------------------------------------------------ plain forms

def _act(v, act):
    if act == "relu":
        return v.clamp(min=0)
    if act == "gelu":
        return 0.5 * v * (1 + torch.erf(v / math.sqrt(2.0)))
    if act == "gelu_tanh":
        return 0.5 * v * (1 + torch.tanh(math.sqrt(2 / math.pi) * (v + 0.044715 * v * v * v)))
    if act == "silu":
        return v / (1 + torch.exp(-v))
    return v


def _plain_weights(st):
    """W~ [N, K] in fp32 from the packed bytes: blocks of 16 rows, chunks of 64 columns, lane
    4g + t, word j (16 columns), nibble."""
    c = st["case"]
    N, K, mode = c["N"], c["K"], c["mode"]
    b = st["qweight"].view(N // 16, K // 64, 8, 4, 4, 4)            # block, chunk, g, t, j, byte
    nib = torch.stack([b & 15, b >> 4], -1).flatten(-2)             # ..., j, nibble 0..7
    # pair p = h + 2 (c / 2), member c % 2: SYM/ASYM nibbles p + 4 (c % 2), LUT 2 p + c % 2
    if mode == "lut":
        v = nib.view(N // 16, K // 64, 8, 4, 4, 2, 2, 2).permute(0, 6, 2, 1, 4, 3, 5, 7)
    else:
        v = nib.view(N // 16, K // 64, 8, 4, 4, 2, 2, 2).permute(0, 7, 2, 1, 4, 3, 6, 5)
    code = v.reshape(N, K)                                          # row 8 h + g; column 64 ch + 16 j + 4 t + c
    G = 1 if c["group"] == -1 else K // c["group"]

    def rows(t):                                                    # [N/16][G][16], slot 2 (r % 8) + r / 8
        return t.view(torch.float16).view(N // 16, G, 8, 2).permute(0, 3, 2, 1).reshape(N, G, 1).float()

    if mode == "lut":
        w = st["zl"].view(torch.float16).float()[code.long()]
    else:
        w = code.float()
    w = w.view(N, G, K // G)
    if mode == "sym":
        w = w - 8
    elif mode == "asym":
        w = w - rows(st["zl"])
    return (w * rows(st["scales"])).view(N, K)


def _plain_epilogue(st):
    c = st["case"]
    v = st["x"].float() @ _plain_weights(st).t()
    if st["bias"] is not None:
        v = v + st["bias"].float()
    v = _act(v, c["act"])
    if st["residual"] is not None:
        v = v + st["residual"].float()
    return v.to(_dtype(c))


def _swizzle_k(D, device):
    """Position, among a key row's 32-bit words, of natural word n (dims 8n .. 8n + 7), for
    tokens of even and odd place."""
    n = torch.arange(D // 8, device=device)
    w, t = n // 4, n % 4
    if D == 64:
        pos = 2 * t + w
        return torch.stack([pos, pos])
    even = 4 * (t + 4 * (w // 4)) + w % 4
    odd = even if D == 128 else even ^ 16
    return torch.stack([even, odd])


def _swizzle_v(D, device):
    """The same for a value row, per token of a tile."""
    n = torch.arange(D // 8, device=device)
    tok = torch.arange(16, device=device)[:, None]
    per = D // 64                                                   # words per piece (a lane's dims)
    flip = {64: 0 * tok, 128: 4 * ((tok >> 1) & 1), 256: 2 * (tok & 3)}[D]
    return ((n // per) ^ flip) * per + n % per


def _plain_quantize(x, G, mode):
    """(codes, scale, zero) of x [..., D]; quotients next to a rounding border in 64 bits."""
    g = x.unflatten(-1, (G, -1))
    if mode == "sym":
        s = (g.abs().amax(-1, keepdim=True).double() / 7).float()
    else:
        lo, hi = g.amin(-1, keepdim=True).clamp(max=0), g.amax(-1, keepdim=True).clamp(min=0)
        s = ((hi - lo).double() / 15).float()
    s = s.clamp(max=4096).half()
    d = torch.where(s > 0, s, torch.ones_like(s)).double()
    z = torch.full_like(s, 8) if mode == "sym" else torch.round(-lo.double() / d).clamp(0, 15)
    live = s > 0
    if mode == "asym":
        z = torch.where(live, z, torch.zeros_like(z))
    q = (torch.round(g.double() / d) + z).clamp(0, 15)
    q = torch.where(live, q, z.to(q.dtype).expand_as(q))
    return q.flatten(-2).to(torch.uint8), s.squeeze(-1), z.half().squeeze(-1)


def _rows_of(slots, page):
    s = slots.long()
    return s // page, s % page // 16, s % 16


def _plain_store(st):
    c = st["case"]
    D, G, mode, H = c["dim"], _groups(c), c["mode"], c["heads"]
    cache, (pg, tile, tok) = st["cache"], _rows_of(st["slots"], c["page"])
    heads = torch.arange(H, device="cuda")
    for which in (0, 1):
        q, s, z = _plain_quantize(st["qkv"][:, 1 + which].float(), G, mode)
        words = (q[..., 0::2] | (q[..., 1::2] << 4)).unflatten(-1, (-1, 4))     # [T, H, D/8, 4]
        pos = _swizzle_k(D, "cuda")[tok % 2] if which == 0 else _swizzle_v(D, "cuda")[tok]
        base = which * 8 * D + tok[:, None] * (D // 2)
        at = (base[:, :, None] + 4 * pos[:, :, None] + torch.arange(4, device="cuda")).view(-1, 1, D // 2)
        index = (pg[:, None, None], heads[None, :, None], tile[:, None, None])
        cache[(*index, at)] = words.flatten(-2)
        par = s if mode == "sym" else torch.stack([s, z], -1).flatten(-2)
        pb = par.contiguous().view(torch.uint8)
        n = pb.shape[-1]
        at = 16 * D + which * 16 * n + tok[:, None, None] * n + torch.arange(n, device="cuda")
        cache[(*index, at)] = pb


def _plain_rows(cache, slots, case, heads):
    """K~ and V~ [T, heads, D] in fp32 of the given slots."""
    D, G, mode = case["dim"], _groups(case), case["mode"]
    pg, tile, tok = _rows_of(slots, case["page"])
    rec = cache[pg, :, tile]                                                    # [T, heads, bytes]
    out = []
    for which in (0, 1):
        codes = rec[..., which * 8 * D:(which + 1) * 8 * D].unflatten(-1, (16, D // 8, 4))
        idx = torch.arange(len(tok), device=cache.device)
        row = codes[idx, :, tok]                                                # [T, heads, D/8, 4]
        pos = _swizzle_k(D, cache.device)[tok % 2] if which == 0 else _swizzle_v(D, cache.device)[tok]
        row = torch.gather(row, 2, pos[:, None, :, None].expand_as(row)).flatten(-2)
        q = torch.stack([row & 15, row >> 4], -1).flatten(-2).float()
        n = 2 * G if mode == "sym" else 4 * G
        par = rec[..., 16 * D + which * 16 * n:16 * D + (which + 1) * 16 * n].unflatten(-1, (16, n))
        par = par[idx, :, tok].contiguous().view(torch.float16).float()
        if mode == "sym":
            s, z = par, 8.0
        else:
            s, z = par[..., 0::2], par[..., 1::2].unsqueeze(-1)
        out.append(((q.unflatten(-1, (G, -1)) - z) * s.unsqueeze(-1)).flatten(-2))
    return out


def _plain_attend(st):
    c = st["case"]
    H, KV, D, page = c["heads"], c["kv"], c["dim"], c["page"]
    outs, row = [], 0
    for b, (n, m) in enumerate(zip(st["lens_host"], st["nq_host"])):
        first = 0 if not c["window"] else max(0, n - m - c["window"] + 1)
        t = torch.arange(first, n, device="cuda")
        slots = st["table"][b].long()[t // page] * page + t % page
        qpos = torch.arange(n - m, n, device="cuda")
        k, v = _plain_rows(st["cache"], slots, c, KV)
        step = max(1, (1 << 27) // max(1, (n - first) * H))
        for i in range(0, m, step):
            qi = st["q"][row + i:row + min(m, i + step)].float()
            l = torch.einsum("mkgd,tkd->kgmt", qi.unflatten(1, (KV, H // KV)), k) * st["scale"]
            p = qpos[i:i + step, None]
            seen = t[None] <= p
            if c["window"]:
                seen = seen & (t[None] > p - c["window"])
            l = l.masked_fill(~seen, -math.inf)
            e = torch.exp(l - l.amax(-1, keepdim=True))
            o = torch.einsum("kgmt,tkd->mkgd", e, v) / e.sum(-1).permute(2, 0, 1)[..., None]
            outs.append(o.flatten(1, 2).to(_dtype(c)))
        row += m
    return torch.cat(outs)


def run(st):
    c = st["case"]
    op = c["op"]
    if not own:
        if op == "epilogue":
            return _plain_epilogue(st)
        if op == "attend":
            return _plain_attend(st)
        if op == "store":
            _plain_store(st)
        k, v = _plain_rows(st["cache"], st["slots"], c, c["heads"])
        return k.to(_dtype(c)), v.to(_dtype(c))
    lib = st["lib"]
    if op == "epilogue":
        return lib.qmm_epilogue(st["x"], st["qweight"], st["scales"], st["zl"], c["N"], c["K"], c["mode"],
                                4, c["group"], bias=st["bias"], act=c["act"], residual=st["residual"],
                                ws=st["ws"])
    fmt = dict(mode=c["mode"], group=c["group"])
    if op == "attend":
        return lib.kv_attend(st["q"], st["cache"], st["table"], st["lens"], cu_q=st["cu"],
                             max_q=c["queries"], scale=st["scale"], window=c["window"], ws=st["ws"], **fmt)
    if op == "store":
        lib.kv_store(st["qkv"][:, 1], st["qkv"][:, 2], st["slots"], st["cache"], **fmt)
    return lib.kv_load(st["cache"], st["slots"], c["dim"], dtype=_dtype(c), **fmt)


# ----------------------------------------------------- from the definition, 64 bits

def _exact_weights(st):
    """Each weight by the place of its nibble in the packed bytes."""
    c = st["case"]
    N, K, mode = c["N"], c["K"], c["mode"]
    byte, shift = torch.zeros(16, 64, dtype=torch.long), torch.zeros(16, 64, dtype=torch.long)
    for r in range(16):
        for k in range(64):
            g, h = r % 8, r // 8
            j, t, cc = k // 16, (k % 16) // 4, k % 4
            p = h + 2 * (cc // 2)
            nib = 2 * p + cc % 2 if mode == "lut" else p + 4 * (cc % 2)
            byte[r, k] = 16 * (4 * g + t) + 4 * j + nib // 2
            shift[r, k] = 4 * (nib % 2)
    raw = st["qweight"].view(N // 16, K // 64, 512)
    code = (raw[:, :, byte.cuda()] >> shift.cuda().to(torch.uint8)) & 15        # [N/16, K/64, 16, 64]
    code = code.permute(0, 2, 1, 3).reshape(N, K)
    L = K if c["group"] == -1 else c["group"]
    n = torch.arange(N, device="cuda")[:, None]
    k = torch.arange(K, device="cuda")[None]
    at = ((n // 16) * (K // L) + k // L) * 16 + 2 * (n % 8) + n % 16 // 8
    s = st["scales"].view(torch.float16)[at].double()
    if mode == "sym":
        return (code.double() - 8) * s
    if mode == "asym":
        return (code.double() - st["zl"].view(torch.float16)[at].double()) * s
    return st["zl"].view(torch.float16)[code.int()].double() * s


def _exact_store(st):
    """What the cache stands for after the call: each group's stored scale and zero, each code."""
    c = st["case"]
    G, out = _groups(c), []
    for which in (1, 2):
        x = st["qkv"][:, which].double().unflatten(-1, (G, -1))
        if c["mode"] == "sym":
            span = x.abs().max(-1, keepdim=True).values / 7
            lo = None
        else:
            lo = torch.minimum(x.min(-1, keepdim=True).values, torch.zeros((), dtype=x.dtype, device="cuda"))
            hi = torch.maximum(x.max(-1, keepdim=True).values, torch.zeros((), dtype=x.dtype, device="cuda"))
            span = (hi - lo) / 15
        s = torch.minimum(span, torch.full_like(span, 4096.0)).float().half().double()
        ok = s != 0
        r = torch.where(ok, s, torch.ones_like(s))
        if c["mode"] == "sym":
            steps = torch.round(x / r).clamp(-8, 7)
        else:
            z = torch.round(-lo / r).clamp(0, 15)
            steps = (torch.round(x / r) + z).clamp(0, 15) - z
        out.append(torch.where(ok, steps * s, torch.zeros_like(steps)).flatten(-2))
    return tuple(out)


def _exact_rows(cache, slots, c, heads, chunk=None):
    """K~ and V~ by the byte of every value."""
    D, G, mode = c["dim"], _groups(c), c["mode"]
    T = _tile_bytes(D, G, mode)
    d = torch.arange(D, device="cuda")
    word = d // 8
    flat = cache.view(-1)
    sl = slots.long()[:, None, None]
    h = torch.arange(heads, device="cuda")[None, :, None]
    base = ((sl // c["page"] * heads + h) * (c["page"] // 16) + sl % c["page"] // 16) * T
    tok = sl % 16
    # keys: the words of a row go by lane (n % 4) first; values: in pieces of D / 16 bytes
    lane, blk = word % 4, word // 4
    if D == 64:
        kw = lane * 2 + blk + 0 * tok
    else:
        piece = lane + 4 * (blk // 4)
        if D == 256:
            piece = piece ^ (4 * (tok % 2))
        kw = piece * 4 + blk % 4 + 0 * tok
    piece = d // (D // 8)
    if D == 128:
        piece = piece ^ (tok // 2 % 2 * 4)
    elif D == 256:
        piece = piece ^ (tok % 4 * 2)
    vw = piece * (D // 64) + d % (D // 8) // 8 + 0 * tok
    per = 2 if mode == "sym" else 4
    out = []
    for which, w in ((0, kw), (1, vw)):
        at = base + which * 8 * D + tok * (D // 2) + 4 * w + d % 8 // 2
        q = (flat[at] >> (4 * (d % 2)).to(torch.uint8)) & 15
        pa = base + 16 * D + which * 16 * per * G + (tok * G + d // (D // G)) * per

        def half(a):
            bits = flat[a].int() | (flat[a + 1].int() << 8)
            return bits.to(torch.int16).view(torch.float16).double()

        z = 8.0 if mode == "sym" else half(pa + 2)
        out.append((q.double() - z) * half(pa))
    return out


def _exact_attend(st):
    c = st["case"]
    H, KV, page = c["heads"], c["kv"], c["page"]
    per = H // KV
    out = torch.zeros(st["q"].shape, dtype=torch.float64, device="cuda")
    row = 0
    for b, (n, m) in enumerate(zip(st["lens_host"], st["nq_host"])):
        first = max(0, n - m - c["window"] + 1) if c["window"] else 0
        t = torch.arange(first, n, device="cuda")
        slots = st["table"][b].long()[t // page] * page + t % page
        ks, vs = [], []
        for a in range(0, len(t), 4096):
            k, v = _exact_rows(st["cache"], slots[a:a + 4096], c, KV)
            ks.append(k)
            vs.append(v)
        k, v = torch.cat(ks), torch.cat(vs)
        q = st["q"][row:row + m].double()
        for h in range(H):
            logit = st["scale"] * (q[:, h] @ k[:, h // per].t())
            ahead = t[None, :] - torch.arange(n - m, n, device="cuda")[:, None]
            hide = ahead > 0
            if c["window"]:
                hide |= ahead <= -c["window"]
            logit[hide] = -math.inf
            out[row:row + m, h] = torch.softmax(logit, -1) @ v[:, h // per]
        row += m
    return out


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "epilogue":
        v = st["x"].double() @ _exact_weights(st).t()
        if st["bias"] is not None:
            v += st["bias"].double()
        a = case["act"]
        if a == "relu":
            v = torch.where(v > 0, v, torch.zeros_like(v))
        elif a == "gelu":
            v = v * torch.special.ndtr(v)
        elif a == "gelu_tanh":
            v = v * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (v + 0.044715 * v ** 3))
        elif a == "silu":
            v = v * torch.sigmoid(v)
        return v if st["residual"] is None else v + st["residual"].double()
    if case["op"] == "store":
        return _exact_store(st)
    if case["op"] == "load":
        parts = [_exact_rows(st["cache"], st["slots"][a:a + 2048], case, case["heads"])
                 for a in range(0, case["tokens"], 2048)]
        return tuple(torch.cat([p[i] for p in parts]) for i in (0, 1))
    return _exact_attend(st)
