"""The multi-token and cache-management operators, as measured work.

Four operators around the packed cache of one attention layer:

* chunk:   attention of several new tokens per sequence (drafted tokens to verify, a tree of
           drafts, a chunk of a prompt) over the packed cache and over each other;
* append:  each sequence branches off a parent (a fork) and takes the tokens it accepted,
           quantizing the groups that leave the window;
* fork:    branches sequences: shared pages in a paged cache, copies in an unpaged one;
* compact: gathers a page pool's used pages at one end, then at the other.

``run`` computes each in plain torch operations, or, with ``own`` set, through the package.
"""
import math

import torch

own = False

GROUP_BITS = ((4, 2), (4, 4), (8, 4), (2, 2))     # key and value bits the caches are built with


# ---- cases -------------------------------------------------------------------
def _chunk(name, B, Hq, Hkv, dk, L, T, kb=4, vb=2, g=64, window=128, ret=0, ragged=0, tree=0, paged=0):
    return dict(op="chunk", name=name, B=B, Hq=Hq, Hkv=Hkv, dk=dk, dv=128, L=L, T=T, kb=kb, vb=vb, gk=g, gv=g,
                window=window, ret=ret, ragged=ragged, tree=tree, paged=paged)


def _append(name, B, Hkv, L, T, kb=4, vb=2, g=64, window=128, ret=0, pick=0):
    return dict(op="append", name=name, B=B, Hq=4 * Hkv, Hkv=Hkv, dk=128, dv=128, L=L, T=T, kb=kb, vb=vb, gk=g,
                gv=g, window=window, ret=ret, ragged=1, pick=pick, paged=0)


def _fork(name, B, Hkv, L, paged, dk=128, kb=4, vb=2, g=64, window=128, ret=0):
    return dict(op="fork", name=name, B=B, Hq=4 * Hkv, Hkv=Hkv, dk=dk, dv=128, L=L, kb=kb, vb=vb, gk=g, gv=g,
                window=window, ret=ret, ragged=1, paged=paged)


def _compact(name, B, Hkv, L, kb=4, vb=2, g=64, window=128):
    return dict(op="compact", name=name, B=B, Hq=4 * Hkv, Hkv=Hkv, dk=128, dv=128, L=L, kb=kb, vb=vb, gk=g, gv=g,
                window=window, ret=0, ragged=1, paged=1)


def listed():
    return [
        # one head, 512 cached tokens, one new token: the latency of a call
        _chunk("chunk-one-token", 1, 1, 1, 128, 512, 1, g=32, window=64),
        # a serving batch with four drafted tokens each, lengths that differ, a paged cache
        _chunk("chunk-draft4-4k", 8, 32, 8, 128, 4096, 4, ragged=1, paged=1),
        # thin keys, five drafted tokens (an odd number), lengths that differ
        _chunk("chunk-draft5-thin-16k", 16, 32, 8, 32, 16384, 5, g=32, window=64, ragged=1),
        # the long-context case with a tree of eight drafted tokens and retained older tokens
        _chunk("chunk-tree8-32k", 32, 32, 8, 128, 32768, 8, ret=1, tree=1),
        # a chunk of one prompt over its own 8k prefix, 4-bit keys and values, odd sizes
        _chunk("chunk-prompt333-8k", 1, 32, 8, 128, 8191, 333, kb=4, vb=4),
        # chunked prefill: 1024 tokens of each of eight prompts over 16k
        _chunk("chunk-prompt1024-16k", 8, 32, 8, 128, 16384, 1024, ragged=1),
        # branches of short sequences take up to four accepted tokens, picked from a tree
        _append("append-accepted-4", 8, 8, 600, 4, ret=1, pick=1),
        # branches of 32 sequences take up to 500 prompt tokens: eight groups leave the window
        _append("append-prompt-500", 32, 8, 700, 500),
        # beam search on a paged cache: 16 beams branch, their pages are shared
        _fork("fork-paged-16k", 16, 8, 16384, 1, ret=1),
        # branches of an unpaged cache: 16 copies of up to 8k tokens
        _fork("fork-copy-8k", 16, 8, 8192, 0),
        # a small pool, fragmented by sequences that ended
        _compact("compact-2k", 8, 8, 2048),
        # the long-context pool: about 0.5 GB of used pages, moved to one end and back
        _compact("compact-32k", 32, 8, 32768),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["chunk", "chunk", "chunk", "append", "fork", "compact"])
    kb, vb = rng.choice(GROUP_BITS)
    g = rng.choice([32, 64]) if (kb, vb) in ((4, 2), (2, 2), (8, 4)) else 64
    window = rng.choice([0, 64, 100, 128])
    ret = rng.randint(0, 1)
    if op == "chunk":
        Hkv = rng.choice([1, 2, 8])
        Hq = Hkv * rng.choice([1, 4, 4, 8])
        dk = rng.choice([32, 64, 128, 128, 128])
        tree = rng.randint(0, 1)
        T = _log_int(rng, 1, 64 if tree else 1024)
        L = _log_int(rng, 64, 32768)
        B = _log_int(rng, 1, 32)
        while B > 1 and (B * Hq * T * (L + T) > 2.0e9 or B * Hkv * L > 4.0e6):
            B -= 1
        while T > 1 and B * Hq * T * (L + T) > 2.0e9:
            T = T * 3 // 4
        return _chunk("", B, Hq, Hkv, dk, L, T, kb, vb, g, window, ret, rng.randint(0, 1), tree, rng.randint(0, 1))
    if op == "append":
        return _append("", _log_int(rng, 1, 32), rng.choice([1, 2, 8]), _log_int(rng, 64, 2048),
                       _log_int(rng, 1, 500), kb, vb, g, window, ret, rng.randint(0, 1))
    if op == "fork":
        paged = rng.randint(0, 1)
        return _fork("", _log_int(rng, 1, 16), rng.choice([1, 2, 8]), _log_int(rng, 64, 16384 if paged else 8192),
                     paged, rng.choice([32, 64, 128]), kb, vb, g, window, ret)
    return _compact("", _log_int(rng, 2, 32), rng.choice([1, 2, 8]), _log_int(rng, 512, 32768), kb, vb, g, window)


# ---- sizes that follow from a case --------------------------------------------
def _generator(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed * 7919 + 13)
    return gen


def _spread(n, top, low, seed, on):
    """n whole numbers in [low, top], the largest among them; all `top` when not `on`."""
    if not on or n == 0:
        return [top] * n
    out = []
    x = seed * 2654435761 % (1 << 32)
    for _ in range(n):
        x = (x * 1664525 + 1013904223) % (1 << 32)
        out.append(low + (x >> 8) % (top - low + 1))
    out[seed % n] = top
    return out


def _lengths(case):
    """Cached tokens of each sequence: part of the case, like its batch, so no seed changes them."""
    L = case["L"]
    return _spread(case["B"], L, max(1, L * 3 // 4), L + case["B"], case["ragged"])


def _counts(case):
    """New tokens of each sequence: T for all, or 0..T when lengths differ."""
    T = case["T"]
    return _spread(case["B"], T, 0 if T < 64 else T // 2, T + case["B"] + 5, case["ragged"])


def _prefix(case, L):
    return max(L - case["window"], 0) // case["gk"] * case["gk"]


def _retained(Q):
    """One position per octave of age: p < Q with p a multiple of 2^floor(log2(Q - p))."""
    out, step = [], 1
    while step <= Q:
        out.append((Q - step) // step * step)
        step *= 2
    return sorted(out)


def _config(case, slots, max_context, n_pages=0):
    return dict(batch=slots, n_q_heads=case["Hq"], n_kv_heads=case["Hkv"], d_k=case["dk"], d_v=case["dv"],
                k_bits=case["kb"], v_bits=case["vb"], group_k=case["gk"], group_v=case["gv"],
                window=case["window"], log_retain=case["ret"], max_context=max_context,
                paged=case["paged"], n_pages=n_pages)


def _capacity(case):
    return case["L"] + case.get("T", 0) + 64


# ---- inputs -------------------------------------------------------------------
def _tokens(case, gen, batch, n):
    """Keys with per-channel outliers and means, plain values: fp16 [batch][Hkv][n][d]."""
    H, dk, dv = case["Hkv"], case["dk"], case["dv"]
    u = torch.rand((H, 1, dk), generator=gen, device="cuda")
    sigma = torch.exp(math.log(0.5) + u * math.log(16.0))
    mu = torch.randn((H, 1, dk), generator=gen, device="cuda") * math.sqrt(2.0)
    if dk < 128:                       # thin keys: about the spread of a 128-channel key's projection
        sigma, mu = sigma.sqrt(), mu * 0.5
    k = torch.empty((batch, H, n, dk), dtype=torch.float16, device="cuda")
    v = torch.empty((batch, H, n, dv), dtype=torch.float16, device="cuda")
    for b in range(batch):
        k[b] = (torch.randn((H, n, dk), generator=gen, device="cuda") * sigma + mu).half()
        v[b] = torch.randn((H, n, dv), generator=gen, device="cuda").half()
    return k, v, sigma, mu


def _tree(T, seed):
    """A random draft tree: token j sees itself and its ancestors.  bool [T][T]."""
    sees = torch.zeros((T, T), dtype=torch.bool)
    x = seed * 40503 + 1
    for j in range(T):
        x = (x * 1664525 + 1013904223) % (1 << 32)
        if j:
            parent = max(0, j - 1 - (x >> 8) % 3)
            sees[j] = sees[parent]
        sees[j, j] = True
    return sees


def _mask_words(sees, B):
    T = sees.shape[0]
    words = torch.zeros((T, (T + 31) // 32), dtype=torch.int64)
    for j in range(T):
        words[:, j // 32] |= sees[:, j].long() << (j % 32)
    words = torch.where(words >= 1 << 31, words - (1 << 32), words).to(torch.int32)
    return words.expand(B, -1, -1).contiguous().cuda()


def _inputs(case, seed):
    """Everything that the seed decides, before any cache is built."""
    gen = _generator(case, seed)
    lens = _lengths(case)
    x = dict(lens=lens)
    x["k"], x["v"], sigma, mu = _tokens(case, gen, case["B"], case["L"])
    if case["op"] in ("chunk", "append"):
        B, H, T, dk, dv = case["B"], case["Hkv"], case["T"], case["dk"], case["dv"]
        x["k_new"] = (torch.randn((B, H, T, dk), generator=gen, device="cuda") * sigma + mu).half()
        x["v_new"] = torch.randn((B, H, T, dv), generator=gen, device="cuda").half()
        x["counts"] = _counts(case)
    if case["op"] == "chunk":
        x["q"] = torch.randn((case["B"], case["Hq"], case["T"], case["dk"]), generator=gen, device="cuda").half()
        x["sees"] = _tree(case["T"], seed) if case["tree"] else None
    if case["op"] == "append" and case["pick"]:
        # the accepted tokens of sequence b: counts[b] rows of the T drafted ones, in any order
        x["pick"] = torch.rand((case["B"], case["T"]), generator=gen, device="cuda").argsort(1).to(torch.int32)
    return x


# ---- the plain cache: codes of whole groups, their scales and zeros, fp16 rows ---
def _minmax(x, bits, dim):
    """Groupwise asymmetric codes of fp16 x: one rounding at a time in 32 bits."""
    mn, mx = x.amin(dim, keepdim=True).float(), x.amax(dim, keepdim=True).float()
    top = torch.full_like(mx, float(2 ** bits - 1))     # a tensor: by a number torch multiplies with 1 / top
    s = ((mx - mn) / top).half()
    s = torch.where(s == 0, torch.zeros_like(s), s)
    z = (mn + 0.0).half()
    c = torch.round((x.float() - z.float()) / s.float()).clamp(0.0, float(2 ** bits - 1))
    c = torch.where(s == 0, torch.zeros_like(c), c)
    return c.to(torch.uint8), s, z


def _quant_keys(case, k):
    H, n, dk = k.shape
    c, s, z = _minmax(k.view(H, n // case["gk"], case["gk"], dk), case["kb"], 2)
    return c.view(H, n, dk), s[:, :, 0], z[:, :, 0]


def _quant_values(case, v):
    H, n, dv = v.shape
    c, s, z = _minmax(v.view(H, n, dv // case["gv"], case["gv"]), case["vb"], 3)
    return c.view(H, n, dv), s[..., 0], z[..., 0]


def _plain_sequence(case, k, v, L):
    """One sequence's cache from its first L tokens, k and v [Hkv][>= L][d]."""
    Q = _prefix(case, L)
    ret = _retained(Q) if case["ret"] else []
    kc, ks, kz = _quant_keys(case, k[:, :Q])
    vc, vs, vz = _quant_values(case, v[:, :Q])
    return dict(L=L, Q=Q, ret=ret, kc=kc, ks=ks, kz=kz, vc=vc, vs=vs, vz=vz, wk=k[:, Q:L].clone(),
                wv=v[:, Q:L].clone(), rk=k[:, ret].clone(), rv=v[:, ret].clone())


def _words(codes, bits):
    """Codes packed least significant first into 32-bit words of a row."""
    per = 32 // bits
    c = codes.view(codes.shape[:-1] + (codes.shape[-1] // per, per)).long()
    w = torch.zeros(c.shape[:-1], dtype=torch.long, device=c.device)
    for i in range(per):
        w = w + (c[..., i] << (i * bits))
    return torch.where(w >= 1 << 31, w - (1 << 32), w).to(torch.int32)


def _key_block_order(dk, bits):
    """Channel and kind (0 scale, 1 zero) at each position of a key group's block."""
    P = 32 // bits
    W, H = dk // P, P // 2
    where = [0] * (2 * dk)
    for w in range(W):
        at = (w % (W // 4)) * 4 + w // (W // 4) if W % 4 == 0 else w
        for kind in range(2):
            for i in range(H):
                where[at * 2 * P + kind * P + 2 * i] = (w * P + i) + kind * dk
                where[at * 2 * P + kind * P + 2 * i + 1] = (w * P + i + H) + kind * dk
    return where


def _key_block(case, s, z):
    order = torch.tensor(_key_block_order(case["dk"], case["kb"]), device=s.device)
    return torch.cat([s, z], dim=-1)[..., order]


def _plain_buffers(case, slots, max_context, n_pages=0):
    """Zeroed packed buffers in the cache's layout: per slot, or a pool of pages."""
    H, dk, dv, gk = case["Hkv"], case["dk"], case["dv"], case["gk"]
    groups = -(-max_context // gk)
    cap = case["window"] + gk

    def z(shape, dt):
        return torch.zeros(shape, dtype=dt, device="cuda")
    lead, glead = ((n_pages, H, gk), (n_pages, H)) if case["paged"] else ((slots, H, groups * gk), (slots, H, groups))
    buf = dict(kcode=z(lead + (dk * case["kb"] // 32,), torch.int32), ksz=z(glead + (2 * dk,), torch.float16),
               vcode=z(lead + (dv * case["vb"] // 32,), torch.int32),
               vsz=z(lead + (dv // case["gv"], 2), torch.float16),
               win_k=z((slots, H, cap, dk), torch.float16), win_v=z((slots, H, cap, dv), torch.float16),
               ret_k=z((slots, H, 32, dk), torch.float16), ret_v=z((slots, H, 32, dv), torch.float16))
    if case["paged"]:
        buf["block_table"] = z((slots, groups), torch.int32)
    return buf


def _store_groups(case, buf, b, g0, k, v, pages=None):
    """Quantizes k, v [Hkv][n * gk][d] into groups g0.. of slot b (or into `pages`)."""
    gk, H = case["gk"], case["Hkv"]
    n = k.shape[1] // gk
    if n == 0:
        return
    kc, ks, kz = _quant_keys(case, k)
    vc, vs, vz = _quant_values(case, v)
    rows = dict(kcode=_words(kc, case["kb"]), vcode=_words(vc, case["vb"]), vsz=torch.stack([vs, vz], -1))
    block = _key_block(case, ks, kz)
    if pages is None:
        for name, r in rows.items():
            buf[name][b, :, g0 * gk:(g0 + n) * gk] = r
        buf["ksz"][b, :, g0:g0 + n] = block
    else:
        for name, r in rows.items():
            buf[name][pages] = r.reshape((H, n, gk) + r.shape[2:]).transpose(0, 1)
        buf["ksz"][pages] = block.transpose(0, 1)


def _plain_prefill(case, buf, b, k, v, L, pages=None):
    Q = _prefix(case, L)
    cap = case["window"] + case["gk"]
    _store_groups(case, buf, b, 0, k[:, :Q], v[:, :Q], pages)
    slots = [p % cap for p in range(Q, L)]
    buf["win_k"][b][:, slots] = k[:, Q:L]
    buf["win_v"][b][:, slots] = v[:, Q:L]
    ret = _retained(Q) if case["ret"] else []
    buf["ret_k"][b][:, :len(ret)] = k[:, ret]
    buf["ret_v"][b][:, :len(ret)] = v[:, ret]


def _pages_of(case, lens):
    """The pages a fresh pool hands out, in order, to sequences of these lengths."""
    out, at = [], 0
    for L in lens:
        n = _prefix(case, L) // case["gk"]
        out.append(list(range(at, at + n)))
        at += n
    return out, at


def _pool_size(case, lens):
    # compaction: room for every used page at either end; forks share pages
    used = _pages_of(case, lens)[1]
    return max(1, 2 * used + 3 if case["op"] == "compact" else used + 8)


def _ended(case):
    """Sequences whose pages are freed before the pool is compacted: every other one."""
    return list(range(0, case["B"], 2)) if case["B"] > 1 else []


# ---- prepare ------------------------------------------------------------------
def prepare(case, seed):
    x = _inputs(case, seed)
    B, op = case["B"], case["op"]
    state = dict(case=case, **x)
    cap = _capacity(case)
    slots = 2 * B if op in ("append", "fork") else B
    n_pages = _pool_size(case, x["lens"]) if case["paged"] else 0
    if op == "chunk":
        state["out"] = torch.zeros((B, case["Hq"], case["T"], case["dv"]), dtype=torch.float16, device="cuda")
    if own:
        from mixed_precision_quantized_pack_b200 import kvq
        cache = kvq.KVCache(_config(case, slots, cap, n_pages), device="cuda")
        for b in range(B):
            cache.prefill_sequence(b, x["k"][b][:, :x["lens"][b]].contiguous(),
                                   x["v"][b][:, :x["lens"][b]].contiguous())
        if op == "compact":
            for b in _ended(case):
                cache.release(b)
        state["cache"] = cache
        if op == "chunk" and x["sees"] is not None:
            state["mask"] = _mask_words(x["sees"], B)
        if op == "append":             # rows of the branches behind rows of the parents
            state["k_all"] = torch.cat([torch.zeros_like(x["k_new"]), x["k_new"]])
            state["v_all"] = torch.cat([torch.zeros_like(x["v_new"]), x["v_new"]])
            if case["pick"]:
                state["pick_all"] = torch.cat([torch.zeros_like(x["pick"]), x["pick"]])
    elif op == "chunk":
        state["seqs"] = [_plain_sequence(case, x["k"][b], x["v"][b], x["lens"][b]) for b in range(B)]
        if x["sees"] is not None:
            state["sees"] = x["sees"].cuda()
    else:
        buf = _plain_buffers(case, slots, cap, n_pages)
        pages, _ = _pages_of(case, x["lens"])
        for b in range(B):
            pg = torch.tensor(pages[b], dtype=torch.long, device="cuda") if case["paged"] else None
            _plain_prefill(case, buf, b, x["k"][b], x["v"][b], x["lens"][b], pg)
            if case["paged"] and pages[b]:
                buf["block_table"][b, :len(pages[b])] = pg.int()
        state["buf"] = buf
        if op == "compact":
            ended = set(_ended(case))
            state["held"] = [[] if b in ended else pages[b] for b in range(B)]
            state["n_pages"] = n_pages
    del state["k"], state["v"]
    return state


# ---- run: the plain forms -------------------------------------------------------
def _plain_chunk(state):
    case, out = state["case"], state["out"]
    H, T, n_rep = case["Hkv"], case["T"], case["Hq"] // case["Hkv"]
    for b, s in enumerate(state["seqs"]):
        n = state["counts"][b]
        if n == 0:
            continue
        Q, gk = s["Q"], case["gk"]
        K = (s["kc"].float().view(H, Q // gk, gk, -1) * s["ks"].float()[:, :, None] +
             s["kz"].float()[:, :, None]).view(H, Q, -1)
        V = (s["vc"].float().view(H, Q, -1, case["gv"]) * s["vs"].float()[..., None] +
             s["vz"].float()[..., None]).view(H, Q, -1)
        if s["ret"]:
            K[:, s["ret"]] = s["rk"].float()
            V[:, s["ret"]] = s["rv"].float()
        K = torch.cat([K, s["wk"].float(), state["k_new"][b][:, :n].float()], 1)
        V = torch.cat([V, s["wv"].float(), state["v_new"][b][:, :n].float()], 1)
        q = state["q"][b].view(H, n_rep, T, -1)[:, :, :n].float()
        sc = torch.matmul(q.reshape(H, n_rep * n, -1), K.transpose(1, 2)).view(H, n_rep, n, -1)
        sc *= 1.0 / math.sqrt(case["dk"])
        sees = state["sees"][:n, :n] if state["sees"] is not None else \
            torch.ones((n, n), dtype=torch.bool, device="cuda").tril()
        sc[..., -n:].masked_fill_(~sees, float("-inf"))
        sc -= sc.amax(-1, keepdim=True)
        sc.exp_()
        den = sc.sum(-1, keepdim=True)
        o = torch.matmul(sc.view(H, n_rep * n, -1), V).view(H, n_rep, n, -1) / den
        out[b].view(H, n_rep, T, -1)[:, :, :n] = o.half()
    return out


def _plain_fork(state):
    """Slot B + b becomes a copy of slot b: groups (unpaged) or table entries, live fp16 rows."""
    case, buf = state["case"], state["buf"]
    B, gk, cap = case["B"], case["gk"], case["window"] + case["gk"]
    for b, L in enumerate(state["lens"]):
        Q = _prefix(case, L)
        if case["paged"]:
            buf["block_table"][B + b, :Q // gk] = buf["block_table"][b, :Q // gk]
        else:
            for name in ("kcode", "vcode", "vsz"):
                buf[name][B + b, :, :Q] = buf[name][b, :, :Q]
            buf["ksz"][B + b, :, :Q // gk] = buf["ksz"][b, :, :Q // gk]
        first, n = Q % cap, L - Q        # the live slots of the window's ring
        for name in ("win_k", "win_v"):
            head = min(n, cap - first)
            buf[name][B + b, :, first:first + head] = buf[name][b, :, first:first + head]
            buf[name][B + b, :, :n - head] = buf[name][b, :, :n - head]
        if case["ret"]:
            n_ret = Q.bit_length()
            for name in ("ret_k", "ret_v"):
                buf[name][B + b, :, :n_ret] = buf[name][b, :, :n_ret]


def _plain_append(state):
    case, buf = state["case"], state["buf"]
    B, gk, cap = case["B"], case["gk"], case["window"] + case["gk"]
    for b, (L, n) in enumerate(zip(state["lens"], state["counts"])):
        if n == 0:
            continue
        Q, Q2 = _prefix(case, L), _prefix(case, L + n)
        kn, vn = state["k_new"][b], state["v_new"][b]
        if case["pick"]:
            rows = state["pick"][b, :n].long()
            kn, vn = kn[:, rows], vn[:, rows]
        live = torch.arange(Q, L, device="cuda") % cap
        k = torch.cat([buf["win_k"][B + b][:, live], kn[:, :n]], 1)      # tokens Q .. L + n - 1
        v = torch.cat([buf["win_v"][B + b][:, live], vn[:, :n]], 1)
        if Q2 > Q:
            _store_groups(case, buf, B + b, Q // gk, k[:, :Q2 - Q], v[:, :Q2 - Q])
            if case["ret"]:
                old, new = _retained(Q), _retained(Q2)
                for name, src in (("ret_k", k), ("ret_v", v)):
                    rows = [buf[name][B + b][:, old.index(p)] if p < Q else src[:, p - Q] for p in new]
                    buf[name][B + b, :, :len(new)] = torch.stack(rows, 1)
        first = max(L, Q2)                 # new tokens that stay in the window
        slots = torch.arange(first, L + n, device="cuda") % cap
        buf["win_k"][B + b][:, slots] = k[:, first - Q:]
        buf["win_v"][B + b][:, slots] = v[:, first - Q:]


def _plain_compact(state):
    """Used pages to the high end of the pool, then to its low end: the i-th lowest page outside
    the end moves to the i-th lowest free page inside it."""
    buf, n_pages = state["buf"], state["n_pages"]
    for high in (True, False):
        used = sorted(p for row in state["held"] for p in row)
        lo = n_pages - len(used) if high else 0
        target = range(lo, lo + len(used))
        taken = set(used)
        src = [p for p in used if p not in target]
        dst = [p for p in target if p not in taken]
        to = dict(zip(src, dst))
        if src:
            s = torch.tensor(src, device="cuda")
            t = torch.tensor(dst, device="cuda")
            for name in ("kcode", "ksz", "vcode", "vsz"):
                buf[name][t] = buf[name][s]
        state["held"] = [[to.get(p, p) for p in row] for row in state["held"]]
        for b, row in enumerate(state["held"]):
            if row:
                buf["block_table"][b, :len(row)] = torch.tensor(row, dtype=torch.int32, device="cuda")


def _state_outputs(state, view):
    """The caches' buffers after a pass: packed words and fp16 rows of the branches; for a pool,
    the end the pages ended at.  Words are compared as whole numbers: a bit-exact contract."""
    case = state["case"]
    B = case["B"]
    if case["op"] == "compact":
        used = sum(_prefix(case, L) // case["gk"] for b, L in enumerate(state["lens"]) if b not in _ended(case))
        out = {n: view(n)[:used] for n in ("kcode", "ksz", "vcode", "vsz")}
        # table entries of the sequences that still hold pages (those that ended have none)
        for b, L in enumerate(state["lens"]):
            if b not in _ended(case):
                out["table%d" % b] = view("block_table")[b, :_prefix(case, L) // case["gk"]]
        return out
    names = ["win_k", "win_v"] + (["ret_k", "ret_v"] if case["ret"] else [])
    names += ["block_table"] if case["paged"] else ["kcode", "ksz", "vcode", "vsz"]
    return {n: view(n)[B:] for n in names}


def run(state):
    case = state["case"]
    op, B = case["op"], case["B"]
    if own:
        cache = state["cache"]
        if op == "chunk":
            return cache.chunk_attention(state["q"], state["k_new"], state["v_new"], counts=state["counts"],
                                         mask=state.get("mask"), out=state["out"])
        if op == "compact":
            cache.compact("high")
            cache.compact("low")
        else:
            cache.fork(range(B), range(B, 2 * B))
            if op == "append":
                cache.append_tokens(state["k_all"], state["v_all"], counts=[0] * B + state["counts"],
                                    index=state.get("pick_all"))
        return _state_outputs(state, cache.view)
    if op == "chunk":
        return _plain_chunk(state)
    if op == "compact":
        _plain_compact(state)
    else:
        _plain_fork(state)
        if op == "append":
            _plain_append(state)
    return _state_outputs(state, state["buf"].__getitem__)


# ---- exact: from the definition, in 64 bits --------------------------------------
def _decoded(x, bits, dim):
    """What the quantizer keeps of fp16 x, in 64 bits: codes from its 32-bit steps, each a
    64-bit operation rounded once (the quotient of 32-bit numbers rounds the same either way)."""
    x = x.double()
    lo, hi = x.amin(dim, keepdim=True), x.amax(dim, keepdim=True)
    top = 2.0 ** bits - 1.0
    scale = ((hi - lo).float().double() / top).float().half().double()
    steps = ((x - lo).float().double() / torch.where(scale == 0, torch.ones_like(scale), scale)).float().double()
    code = torch.where(scale == 0, torch.zeros_like(x), steps.round().clamp(0.0, top))
    return code * scale + lo, scale, lo, (hi - lo) / top


def _exact_chunk(case, seed):
    x = _inputs(case, seed)
    B, Hq, H, T, gk, gv = case["B"], case["Hq"], case["Hkv"], case["T"], case["gk"], case["gv"]
    if B * Hq * T * (case["L"] + T) > 6.0e9:
        return None
    n_rep = Hq // H
    out = torch.zeros((B, Hq, T, case["dv"]), dtype=torch.float64, device="cuda")
    for b in range(B):
        L, n = x["lens"][b], x["counts"][b]
        if n == 0:
            continue
        Q = _prefix(case, L)
        may = x["sees"][:n, :n].cuda() if x["sees"] is not None else \
            torch.arange(n, device="cuda")[:, None] >= torch.arange(n, device="cuda")[None, :]
        for h in range(H):
            k, v = x["k"][b, h, :L].double(), x["v"][b, h, :L].double()
            if Q:
                kq = _decoded(x["k"][b, h, :Q].view(-1, gk, case["dk"]), case["kb"], 1)[0].view(Q, -1)
                vq = _decoded(x["v"][b, h, :Q].view(Q, -1, gv), case["vb"], 2)[0].view(Q, -1)
                keep = torch.zeros(Q, 1, dtype=torch.bool, device="cuda")
                if case["ret"]:
                    keep[_retained(Q)] = True
                k[:Q] = torch.where(keep, k[:Q], kq)
                v[:Q] = torch.where(keep, v[:Q], vq)
            k = torch.cat([k, x["k_new"][b, h, :n].double()])
            v = torch.cat([v, x["v_new"][b, h, :n].double()])
            for r in range(n_rep):
                hq = h * n_rep + r
                logits = x["q"][b, hq, :n].double() @ k.T / math.sqrt(case["dk"])
                logits[:, L:] = torch.where(may, logits[:, L:], torch.full_like(logits[:, L:], -math.inf))
                p = torch.softmax(logits, -1)
                out[b, hq, :n] = p @ v
    return out


def _exact_append(case, seed):
    """The scales that the cache holds, unrounded; the rest has no such value."""
    x = _inputs(case, seed)
    names = ["win_k", "win_v"] + (["ret_k", "ret_v"] if case["ret"] else []) + ["kcode", "ksz", "vcode", "vsz"]
    out = dict.fromkeys(names)
    B, H, gk, gv = case["B"], case["Hkv"], case["gk"], case["gv"]
    groups = -(-_capacity(case) // gk)
    ksz = torch.zeros((B, H, groups, 2 * case["dk"]), dtype=torch.float64, device="cuda")
    vsz = torch.zeros((B, H, groups * gk, case["dv"] // gv, 2), dtype=torch.float64, device="cuda")
    order = torch.tensor(_key_block_order(case["dk"], case["kb"]), device="cuda")
    for b in range(B):
        L, n = x["lens"][b], x["counts"][b]
        rows = x["pick"][b, :n].long() if case["pick"] else torch.arange(n, device="cuda")
        Q = _prefix(case, L + n)
        if Q == 0:
            continue
        k = torch.cat([x["k"][b][:, :L], x["k_new"][b][:, rows]], 1)[:, :Q]
        v = torch.cat([x["v"][b][:, :L], x["v_new"][b][:, rows]], 1)[:, :Q]
        _, _, z, s = _decoded(k.reshape(H, Q // gk, gk, -1), case["kb"], 2)
        ksz[b, :, :Q // gk] = torch.cat([s, z], -1)[:, :, 0][..., order]
        _, _, z, s = _decoded(v.reshape(H, Q, -1, gv), case["vb"], 3)
        vsz[b, :, :Q] = torch.cat([s, z], -1)
    out["ksz"], out["vsz"] = ksz, vsz
    return out


def exact(case, seed):
    if case["op"] == "chunk":
        return _exact_chunk(case, seed)
    if case["op"] == "append":
        return _exact_append(case, seed)
    return None                       # forks and compactions move bits


# ---- what a pass cannot do without ------------------------------------------------
def _group_bytes(case):
    """One key group of one head: codes, scales and zeros of its keys and values."""
    gk, dk, dv = case["gk"], case["dk"], case["dv"]
    return gk * (dk * case["kb"] + dv * case["vb"]) // 8 + dk * 4 + gk * (dv // case["gv"]) * 4


def work(case):
    H, d2 = case["Hkv"], case["dk"] + case["dv"]
    lens = _lengths(case)
    if case["op"] == "compact":
        used = sum(_prefix(case, L) // case["gk"] for b, L in enumerate(lens) if b not in _ended(case))
        return {"bytes": 4 * used * (H * _group_bytes(case) + 8), "flops": 0}
    nbytes = flops = 0
    for b, L in enumerate(lens):
        Q = _prefix(case, L)
        groups, fp16 = Q // case["gk"], L - Q + (Q.bit_length() if case["ret"] else 0)
        if case["op"] == "chunk":
            n = _counts(case)[b]
            if n == 0:
                continue
            nbytes += H * (groups * _group_bytes(case) + (fp16 + n) * d2 * 2) + case["Hq"] * n * d2 * 2
            flops += 2 * d2 * case["Hq"] * (n * L + n * (n + 1) // 2)
            continue
        moved = H * fp16 * d2 * 2 + (groups * 4 if case["paged"] else H * groups * _group_bytes(case))
        nbytes += 2 * moved
        if case["op"] == "append":
            n = _counts(case)[b]
            Q2 = _prefix(case, L + n)
            more = (Q2 - Q) // case["gk"]
            old = max(0, min(L, Q2) - Q)                  # window tokens read again to be quantized
            stay = L + n - max(L, Q2)
            nbytes += H * ((n + stay + old) * d2 * 2 + more * _group_bytes(case))
            flops += 8 * H * (Q2 - Q) * d2
    return {"bytes": nbytes, "flops": flops}
