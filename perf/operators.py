"""Measured cases of the position, packed-attention and cache operators.

rope     rotary positions with up to three axes (time, height, width), in grid
         order, fused with the fractal flattening, or at given positions
packed   attention over packed sequences of different lengths, grouped heads,
         causal or not; forward alone or forward and backward
paged    attention of one new token per sequence over a paged key-value cache
append   writing new key and value rows into the pages of such a cache

`run` computes them in elementary torch operations, or through the package's
entry points when `own` is set.  `exact` is the definition in float64.
"""
import math

import torch

own = False

DEV = "cuda"
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


# --------------------------------------------------------------------------
# cases
# --------------------------------------------------------------------------
def listed():
    return [
        # q and k of the 720p-like video latent (40 heads, 20 x 48 x 80 tokens), rotated by frame,
        # row and column and laid out in flattened order for the mask build and the attention
        {"name": "rope_720p_flatten", "op": "rope", "dtype": "bf16", "heads": 40, "heads_kv": 40,
         "D": 128, "T": 20, "H": 48, "W": 80, "pairs": "22,21,21", "layout": "adjacent",
         "source": "grid", "back": False, "theta": 10000.0, "offset": 0.0},
        # gradients of q and k of the 8,192-token video training step, flattened order back to grid order
        {"name": "rope_small_back", "op": "rope", "dtype": "bf16", "heads": 24, "heads_kv": 24,
         "D": 128, "T": 8, "H": 32, "W": 32, "pairs": "22,21,21", "layout": "adjacent",
         "source": "grid", "back": True, "theta": 10000.0, "offset": 0.0},
        # packed text prompts with given positions on three axes, grouped heads, part of the head
        # rotated: the smallest call, where latency counts
        {"name": "rope_text", "op": "rope", "dtype": "fp16", "heads": 24, "heads_kv": 8,
         "D": 64, "T": 333, "H": 1, "W": 1, "pairs": "8,8,8", "layout": "halves",
         "source": "pos", "back": False, "theta": 10000.0, "offset": 1000.0},
        # one decoding step of 64 sequences: one row each
        {"name": "append_token", "op": "append", "heads_kv": 8, "D": 128, "page": 16,
         "starts": ",".join(str(37 * i % 1500) for i in range(64)), "lens": ",".join(["1"] * 64)},
        # prompts of different lengths, some behind a cached prefix
        {"name": "append_prompt", "op": "append", "heads_kv": 8, "D": 128, "page": 64,
         "starts": "0,130,0,0,4097,0", "lens": "8192,3001,77,1,2500,2611"},
        # one user, a short context: latency
        {"name": "paged_one", "op": "paged", "heads": 24, "heads_kv": 8, "D": 128, "page": 16,
         "lens": "1531"},
        # a serving batch with ragged contexts, an empty one among them
        {"name": "paged_batch", "op": "paged", "heads": 40, "heads_kv": 8, "D": 128, "page": 64,
         "lens": ",".join(str(1 + (i * i * 131 + 977 * i) % 8192) for i in range(62)) + ",0,8192"},
        # few users with very long contexts
        {"name": "paged_long", "op": "paged", "heads": 12, "heads_kv": 4, "D": 64, "page": 128,
         "lens": "262144,131071,200001"},
        # short text prompts: latency
        {"name": "packed_text", "op": "packed", "heads": 24, "heads_kv": 8, "D": 64,
         "lens_q": "77,1,200,33", "lens_k": "", "causal": True, "back": False},
        # long prompts of a batch, causal, grouped heads
        {"name": "packed_prompt", "op": "packed", "heads": 40, "heads_kv": 8, "D": 128,
         "lens_q": "8192,5003,1200,2000", "lens_k": "", "causal": True, "back": False},
        # a causal training step on packed clips
        {"name": "packed_train", "op": "packed", "heads": 24, "heads_kv": 8, "D": 128,
         "lens_q": "4096,2500,1,997,598", "lens_k": "", "causal": True, "back": True},
        # training the cross attention of video tokens to the text of each clip, one prompt empty
        {"name": "packed_cross_train", "op": "packed", "heads": 24, "heads_kv": 24, "D": 128,
         "lens_q": "4096,3000,1096", "lens_k": "512,77,0", "causal": False,
         "back": True},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _texts(values):
    return ",".join(str(int(v)) for v in values)


def _ints(text):
    return [int(v) for v in text.split(",")] if text else []


def draw(rng):
    op = rng.choice(["rope", "rope", "append", "paged", "paged", "packed", "packed", "packed"])
    if op == "rope":
        D = rng.choice([64, 128])
        heads = rng.choice([2, 12, 24, 40])
        grouped = rng.choice([1, 1, 2])
        dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
        if dtype == "fp32":
            heads = min(heads, 12)
        layout = rng.choice(["adjacent", "adjacent", "halves"])
        if layout == "halves":
            total = rng.choice([D // 2, D // 4])
        else:
            total = rng.choice([D // 2, D // 2, rng.randrange(3, D // 2 + 1)])
        a = rng.randrange(1, total - 1)
        b = rng.randrange(1, total - a) if total - a > 1 else 1
        pairs = [a, b, total - a - b]
        source = rng.choice(["grid", "grid", "pos"])
        if source == "grid":
            grid = (_log_int(rng, 1, 20), 8 * rng.randrange(1, 7), 8 * rng.randrange(1, 11))
        else:
            grid = (_log_int(rng, 1, 30000), 1, 1)
        return {"op": op, "dtype": dtype, "heads": heads, "heads_kv": heads // grouped, "D": D,
                "T": grid[0], "H": grid[1], "W": grid[2], "pairs": _texts(pairs), "layout": layout,
                "source": source, "back": rng.random() < 0.4,
                "theta": rng.choice([10000.0, 500000.0]),
                "offset": rng.choice([0.0, float(rng.randrange(1, 100000))])}
    if op == "append":
        n = _log_int(rng, 1, 64)
        most = 1 if rng.random() < 0.4 else 20000 // n
        return {"op": op, "heads_kv": rng.choice([1, 2, 4, 8, 12]), "D": rng.choice([64, 128]),
                "page": rng.choice([16, 32, 64, 128]),
                "starts": _texts(rng.randrange(0, 3000) for _ in range(n)),
                "lens": _texts(_log_int(rng, 1, max(1, most)) for _ in range(n))}
    if op == "paged":
        heads_kv = rng.choice([1, 2, 4, 8])
        n = _log_int(rng, 1, 64)
        most = max(2, min(200000, 560000 // (n * heads_kv) * 4))
        return {"op": op, "heads": heads_kv * rng.choice([1, 2, 3, 5, 8, 16]), "heads_kv": heads_kv,
                "D": rng.choice([64, 128]), "page": rng.choice([16, 32, 64, 128]),
                "lens": _texts(_log_int(rng, 1, most) for _ in range(n))}
    heads_kv = rng.choice([2, 8, 12])
    back = rng.random() < 0.5
    n = rng.randrange(1, 7)
    most = max(2, (5000 if back else 9000) // n)
    lens_q = [_log_int(rng, 1, most) for _ in range(n)]
    causal = rng.random() < 0.6
    same = rng.random() < 0.5
    if same:
        lens_k = []
    elif causal:  # new tokens behind a cached context
        lens_k = [q + _log_int(rng, 1, 4000) for q in lens_q]
    else:
        lens_k = [_log_int(rng, 1, 600) for _ in range(n)]
    return {"op": op, "heads": heads_kv * rng.choice([1, 2, 3]) if heads_kv < 12 else 12,
            "heads_kv": heads_kv, "D": rng.choice([64, 128]), "lens_q": _texts(lens_q),
            "lens_k": _texts(lens_k), "causal": causal, "back": back}


# --------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------
def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed) * 7919 + 13)
    return g


def _normal(g, shape, dtype):
    return torch.randn(shape, generator=g, device=DEV, dtype=torch.float32).to(dtype)


def _package():
    from adaptive_block_sparse_fractal_b200 import nabla
    return nabla


def _offsets(lens):
    out = [0]
    for n in lens:
        out.append(out[-1] + n)
    return out


def _cache(case, lens, g, fill):
    """A page pool and the table of the pages of every sequence, in shuffled order."""
    page, hkv, D = case["page"], case["heads_kv"], case["D"]
    need = [-(-n // page) for n in lens]
    width = max(1, max(need))
    pages = sum(need) + 3
    order = torch.randperm(pages, generator=g, device=DEV).to(torch.int32)
    table = torch.zeros((len(lens), width), dtype=torch.int32, device=DEV)
    at = 0
    for s, n in enumerate(need):
        table[s, :n] = order[at:at + n]
        at += n
    shape = (pages, page, hkv, D)
    if fill:
        kc = torch.empty(shape, dtype=torch.bfloat16, device=DEV)
        vc = torch.empty(shape, dtype=torch.bfloat16, device=DEV)
        kc.normal_(generator=g)
        vc.normal_(generator=g)
    else:
        kc = torch.zeros(shape, dtype=torch.bfloat16, device=DEV)
        vc = torch.zeros(shape, dtype=torch.bfloat16, device=DEV)
    return kc, vc, table


def prepare(case, seed):
    g = _gen(seed)
    st = {"case": case}
    D = case["D"]
    if case["op"] == "rope":
        dt = DTYPES[case["dtype"]]
        N = case["T"] * case["H"] * case["W"]
        hq, hk = case["heads"], case["heads_kv"]
        if case["source"] == "pos":  # views of one fused projection, token-major
            qk = _normal(g, (N, hq + hk, D), dt)
            st["q"] = qk[:, :hq].permute(1, 0, 2)
            st["k"] = qk[:, hq:].permute(1, 0, 2)
            step = torch.randint(0, 3, (N, 3), generator=g, device=DEV)
            st["pos"] = step.cumsum(0).to(torch.int32)
        else:  # heads in front of the tokens
            st["q"] = _normal(g, (hq, N, D), dt)
            st["k"] = _normal(g, (hk, N, D), dt)
            st["pos"] = None
        if own:
            nb = _package()
            st["params"] = nb.rope_params_of(
                _ints(case["pairs"]), theta=case["theta"], offset=(case["offset"], 0.0, 0.0),
                layout=nb.ROPE_ADJACENT if case["layout"] == "adjacent" else nb.ROPE_HALVES,
                inverse=case["back"])
        return st
    if case["op"] == "append":
        starts, lens = _ints(case["starts"]), _ints(case["lens"])
        cu = _offsets(lens)
        st["kc"], st["vc"], st["table"] = _cache(case, [a + n for a, n in zip(starts, lens)], g, False)
        kv = _normal(g, (cu[-1], 2 * case["heads_kv"], D), torch.bfloat16)
        st["k"], st["v"] = kv[:, :case["heads_kv"]], kv[:, case["heads_kv"]:]
        st["starts"] = torch.tensor(starts, dtype=torch.int32, device=DEV)
        st["cu"] = torch.tensor(cu, dtype=torch.int32, device=DEV)
        if own:
            st["ws"] = _package().cache_workspace(DEV)
        return st
    if case["op"] == "paged":
        lens = _ints(case["lens"])
        st["kc"], st["vc"], st["table"] = _cache(case, lens, g, True)
        st["q"] = _normal(g, (len(lens), case["heads"], D), torch.bfloat16)
        st["lens"] = torch.tensor(lens, dtype=torch.int32, device=DEV)
        st["host_lens"] = lens
        if own:
            st["ws"] = _package().paged_workspace(st["q"], st["kc"])
        return st
    lens_q = _ints(case["lens_q"])
    lens_k = _ints(case["lens_k"]) or lens_q
    cq, ck = _offsets(lens_q), _offsets(lens_k)
    hq, hk = case["heads"], case["heads_kv"]
    if case["lens_k"]:
        st["q"] = _normal(g, (cq[-1], hq, D), torch.bfloat16)
        kv = _normal(g, (ck[-1], 2 * hk, D), torch.bfloat16)
        st["k"], st["v"] = kv[:, :hk], kv[:, hk:]
    else:  # views of one fused projection
        qkv = _normal(g, (cq[-1], hq + 2 * hk, D), torch.bfloat16)
        st["q"], st["k"], st["v"] = qkv[:, :hq], qkv[:, hq:hq + hk], qkv[:, hq + hk:]
    if case["back"]:
        st["dout"] = _normal(g, (cq[-1], hq, D), torch.bfloat16)
    st["host_q"], st["host_k"] = cq, ck
    st["cu_q"] = torch.tensor(cq, dtype=torch.int32, device=DEV)
    st["cu_k"] = torch.tensor(ck, dtype=torch.int32, device=DEV) if case["lens_k"] else st["cu_q"]
    if own:
        st["ws"] = _package().packed_workspace(st["q"], st["k"], len(lens_q), back=case["back"])
    return st


# --------------------------------------------------------------------------
# plain forms
# --------------------------------------------------------------------------
def _flat_index(T, H, W, P=8):
    """n[token in grid order] = its place in flattened order."""
    t = torch.arange(T, device=DEV).view(T, 1, 1)
    y = torch.arange(H, device=DEV).view(1, H, 1)
    x = torch.arange(W, device=DEV).view(1, 1, W)
    n = ((t * (H // P) + y // P) * (W // P) + x // P) * P * P + (y % P) * P + x % P
    return n.reshape(-1)


def _rope_angles(case, pos):
    """[N, total pairs] angles in float64."""
    pairs = _ints(case["pairs"])
    if pos is None:
        T, H, W = case["T"], case["H"], case["W"]
        grid = torch.meshgrid(torch.arange(T, device=DEV), torch.arange(H, device=DEV),
                              torch.arange(W, device=DEV), indexing="ij")
        pos = torch.stack([c.reshape(-1) for c in grid], 1)
    shift = (case["offset"], 0.0, 0.0)
    cols = []
    for a, n in enumerate(pairs):
        i = torch.arange(n, device=DEV, dtype=torch.float64)
        cols.append((pos[:, a].double() + shift[a])[:, None] * case["theta"] ** (-i / n)[None])
    return torch.cat(cols, 1)


def _rope_plain(st):
    case = st["case"]
    R = sum(_ints(case["pairs"]))
    ang = _rope_angles(case, st["pos"])
    c, s = ang.cos().float(), ang.sin().float()
    if case["back"]:
        s = -s
    order = None if case["source"] == "pos" else _flat_index(case["T"], case["H"], case["W"])
    out = []
    for x in (st["q"], st["k"]):
        y = torch.empty(x.shape, dtype=x.dtype, device=DEV)
        for h in range(x.shape[0]):
            z = x[h].float()
            if order is not None and case["back"]:
                z = z[order]  # the gradient comes in flattened order
            w = z.clone()
            if case["layout"] == "adjacent":
                a, b = z[:, 0:2 * R:2], z[:, 1:2 * R:2]
                w[:, 0:2 * R:2] = a * c - b * s
                w[:, 1:2 * R:2] = b * c + a * s
            else:
                a, b = z[:, :R], z[:, R:2 * R]
                w[:, :R] = a * c - b * s
                w[:, R:2 * R] = b * c + a * s
            if order is not None and not case["back"]:
                y[h, order] = w.to(x.dtype)
            else:
                y[h] = w.to(x.dtype)
        out.append(y)
    return out


def _append_plain(st):
    page = st["case"]["page"]
    cu, starts, table = st["cu"].long(), st["starts"].long(), st["table"].long()
    tok = torch.arange(st["k"].shape[0], device=DEV)
    seq = torch.searchsorted(cu, tok, right=True) - 1
    p = starts[seq] + tok - cu[seq]
    rows = table[seq, p // page]
    st["kc"][rows, p % page] = st["k"]
    st["vc"][rows, p % page] = st["v"]
    return st["kc"], st["vc"]


def _paged_plain(st):
    q = st["q"]
    n, hq, D = q.shape
    hk = st["kc"].shape[2]
    page = st["kc"].shape[1]
    o = torch.zeros((n, hq, D), dtype=q.dtype, device=DEV)
    lse = torch.full((n, hq), -math.inf, device=DEV)
    for s, L in enumerate(st["host_lens"]):
        if L == 0:
            continue
        rows = st["table"][s, :-(-L // page)].long()
        for h in range(hk):
            k = st["kc"][rows, :, h].reshape(-1, D)[:L].float()
            v = st["vc"][rows, :, h].reshape(-1, D)[:L].float()
            g = slice(h * hq // hk, (h + 1) * hq // hk)
            x = (q[s, g].float() @ k.T) * D ** -0.5
            m = x.amax(1, keepdim=True)
            e = (x - m).exp()
            t = e.sum(1, keepdim=True)
            o[s, g] = (e @ v / t).to(q.dtype)
            lse[s, g] = (m + t.log())[:, 0]
    return o, lse


def _packed_plain(st):
    case = st["case"]
    q, k, v = st["q"], st["k"], st["v"]
    hq, D = q.shape[1:]
    G = hq // k.shape[1]
    sc = D ** -0.5
    o = torch.zeros(q.shape, dtype=q.dtype, device=DEV)
    lse = torch.full((hq, q.shape[0]), -math.inf, device=DEV)
    back = case["back"]
    if back:
        dq = torch.zeros(q.shape, dtype=q.dtype, device=DEV)
        dk = torch.zeros(k.shape, dtype=torch.float32, device=DEV)
        dv = torch.zeros(v.shape, dtype=torch.float32, device=DEV)
    for a, b, c, d in zip(st["host_q"], st["host_q"][1:], st["host_k"], st["host_k"][1:]):
        Lq, Lk = b - a, d - c
        if Lq == 0 or Lk == 0:
            continue
        hide = None
        if case["causal"]:
            i = torch.arange(Lq, device=DEV)[:, None]
            j = torch.arange(Lk, device=DEV)[None]
            hide = j > i + (Lk - Lq)
        for h in range(hq):
            qs, ks, vs = q[a:b, h].float(), k[c:d, h // G].float(), v[c:d, h // G].float()
            x = (qs @ ks.T) * sc
            if hide is not None:
                x.masked_fill_(hide, -math.inf)
            m = x.amax(1, keepdim=True)
            m = torch.where(m == -math.inf, torch.zeros_like(m), m)
            e = (x - m).exp()
            t = e.sum(1, keepdim=True)
            p = e / torch.where(t == 0, torch.ones_like(t), t)
            y = p @ vs
            o[a:b, h] = y.to(q.dtype)
            lse[h, a:b] = (m + t.log())[:, 0]
            if back:
                g = st["dout"][a:b, h].float()
                dv[c:d, h // G] += p.T @ g
                dp = g @ vs.T
                ds = p * (dp - (g * y).sum(1, keepdim=True))
                dq[a:b, h] = (ds @ ks * sc).to(q.dtype)
                dk[c:d, h // G] += ds.T @ qs * sc
    if back:
        return o, lse, dq, dk.to(k.dtype), dv.to(v.dtype)
    return o, lse


# --------------------------------------------------------------------------
# the framework's calls
# --------------------------------------------------------------------------
def _rope_own(st):
    nb, case = _package(), st["case"]
    if case["source"] == "pos":
        return nb.rope(st["params"], st["q"], st["k"], pos=st["pos"])
    grid = (case["T"], case["H"], case["W"])
    return nb.rope(st["params"], st["q"], st["k"], grid=grid, flat_in=case["back"],
                   flat_out=not case["back"])


def _append_own(st):
    _package().cache_append(st["k"], st["v"], st["kc"], st["vc"], st["table"], st["starts"],
                            cu=st["cu"], ws=st["ws"])
    return st["kc"], st["vc"]


def _paged_own(st):
    return _package().attn_paged(st["q"], st["kc"], st["vc"], st["table"], st["lens"], ws=st["ws"])


def _packed_own(st):
    nb, case = _package(), st["case"]
    q, k, v = st["q"], st["k"], st["v"]
    o, lse = nb.attn_packed_fwd(q, k, v, st["cu_q"], st["cu_k"], causal=case["causal"], ws=st["ws"])
    if not case["back"]:
        return o, lse
    dq, dk, dv = nb.attn_packed_bwd(q, k, v, o, st["dout"], lse, st["cu_q"], st["cu_k"],
                                    causal=case["causal"], ws=st["ws"])
    return o, lse, dq, dk, dv


def run(st):
    op = st["case"]["op"]
    if own:
        return {"rope": _rope_own, "append": _append_own, "paged": _paged_own,
                "packed": _packed_own}[op](st)
    return {"rope": _rope_plain, "append": _append_plain, "paged": _paged_plain,
            "packed": _packed_plain}[op](st)


# --------------------------------------------------------------------------
# what a pass cannot do without
# --------------------------------------------------------------------------
def _pairs_kept(case):
    lens_q = _ints(case["lens_q"])
    lens_k = _ints(case["lens_k"]) or lens_q
    total = 0
    for a, b in zip(lens_q, lens_k):
        if not case["causal"]:
            total += a * b
        else:  # row i keeps b - a + i + 1 keys, where that is positive
            first = max(0, a - b)
            total += sum((b - a + first + 1, b)) * (a - first) // 2 if a > first else 0
    return total, sum(lens_q), sum(lens_k)


def work(case):
    D = case["D"]
    if case["op"] == "rope":
        N = case["T"] * case["H"] * case["W"]
        size = 4 if case["dtype"] == "fp32" else 2
        heads = case["heads"] + case["heads_kv"]
        R = sum(_ints(case["pairs"]))
        return {"bytes": 2 * heads * N * D * size + (12 * N if case["source"] == "pos" else 0),
                "flops": 6 * R * heads * N}
    if case["op"] == "append":
        lens = _ints(case["lens"])
        rows = sum(lens)
        pages = sum(-(-n // case["page"]) for n in lens)
        return {"bytes": 2 * 2 * 2 * rows * case["heads_kv"] * D + 4 * (pages + 2 * len(lens) + 1),
                "flops": 0}
    if case["op"] == "paged":
        lens = _ints(case["lens"])
        pages = sum(-(-n // case["page"]) for n in lens)
        return {"bytes": 2 * 2 * sum(lens) * case["heads_kv"] * D
                + len(lens) * case["heads"] * (4 * D + 4) + 4 * (pages + len(lens)),
                "flops": 4 * sum(lens) * case["heads"] * D}
    kept, nq, nk = _pairs_kept(case)
    n = len(_ints(case["lens_q"]))
    rows_q, rows_k = nq * case["heads"], nk * case["heads_kv"]
    size = 2 * (2 * rows_q * D + 2 * rows_k * D) + 4 * rows_q + 8 * (n + 1)
    flops = 4 * kept * case["heads"] * D
    if case["back"]:
        size += 2 * (2 * rows_q * D + 2 * rows_k * D)  # dout in; dq, dk, dv out
        flops += 10 * kept * case["heads"] * D
    return {"bytes": size, "flops": flops}


# --------------------------------------------------------------------------
# definitions in float64
# --------------------------------------------------------------------------
def _rope_exact(case, st):
    """Rotation as a product of complex numbers, one head at a time."""
    total = sum(_ints(case["pairs"]))
    N = case["T"] * case["H"] * case["W"]
    tok = torch.arange(N, device=DEV)
    if st["pos"] is not None:
        coords = [st["pos"][:, a].double() for a in range(3)]
    else:
        coords = [(tok // (case["H"] * case["W"])).double(),
                  (tok // case["W"] % case["H"]).double(), (tok % case["W"]).double()]
    coords[0] = coords[0] + case["offset"]
    turn = torch.empty((N, total), dtype=torch.complex128, device=DEV)
    at = 0
    for a, n in enumerate(_ints(case["pairs"])):
        for i in range(n):
            phi = coords[a] * math.exp(-math.log(case["theta"]) * i / n)
            turn[:, at] = torch.polar(torch.ones_like(phi), -phi if case["back"] else phi)
            at += 1
    place = None
    if st["pos"] is None:
        v = torch.arange(N, device=DEV).view(case["T"], case["H"] // 8, 8, case["W"] // 8, 8)
        place = v.permute(0, 1, 3, 2, 4).reshape(-1)  # flattened order: the grid token at each place
    out = []
    for x in (st["q"], st["k"]):
        y = torch.empty(x.shape, dtype=torch.float64, device=DEV)
        for h in range(x.shape[0]):
            z = x[h].double()
            if place is not None and case["back"]:
                grid = torch.empty_like(z)
                grid[place] = z
                z = grid
            if case["layout"] == "adjacent":
                first = list(range(0, 2 * total, 2))
                second = list(range(1, 2 * total, 2))
            else:
                first, second = list(range(total)), list(range(total, 2 * total))
            r = torch.complex(z[:, first], z[:, second]) * turn
            z[:, first], z[:, second] = r.real, r.imag
            if place is not None and not case["back"]:
                z = z[place]
            y[h] = z
        out.append(y)
    return out


def _append_exact(case, st):
    kc, vc = st["kc"].double(), st["vc"].double()
    table = st["table"].tolist()
    at = 0
    for s, (p0, n) in enumerate(zip(_ints(case["starts"]), _ints(case["lens"]))):
        p = p0
        while p < p0 + n:
            page, off = divmod(p, case["page"])
            m = min(case["page"] - off, p0 + n - p)
            for cache, rows in ((kc, st["k"]), (vc, st["v"])):
                cache[table[s][page], off:off + m] = rows[at:at + m].double()
            p += m
            at += m
    return kc, vc


def _softmax_parts(x):
    """exp(x - max) and its logarithmic sum along the last axis; rows of -inf give zeros and -inf."""
    top = x.detach().amax(-1, keepdim=True).clamp_min(torch.finfo(torch.float64).min)
    e = torch.exp(x - top)
    z = e.sum(-1, keepdim=True)
    return e / z.clamp_min(1e-300), (top + torch.log(z)).squeeze(-1)


def _paged_exact(case, st):
    q = st["q"].double()
    n, hq, D = q.shape
    hk = case["heads_kv"]
    o, lse = torch.zeros_like(q), torch.full((n, hq), -math.inf, dtype=torch.float64, device=DEV)
    for s, L in enumerate(_ints(case["lens"])):
        if L:
            j = torch.arange(L, device=DEV)
            slot = st["table"][s].long()[j // case["page"]] * case["page"] + j % case["page"]
            for h in range(hk):
                keys = st["kc"].view(-1, hk, D)[slot, h].double()
                vals = st["vc"].view(-1, hk, D)[slot, h].double()
                for r in range(h * (hq // hk), (h + 1) * (hq // hk)):
                    p, z = _softmax_parts(torch.mv(keys, q[s, r]) / math.sqrt(D))
                    o[s, r] = torch.mv(vals.T, p)
                    lse[s, r] = z
    return o, lse


def _packed_exact(case, st):
    """The definition in float64; its gradients by differentiation of that definition."""
    lens_q = _ints(case["lens_q"])
    lens_k = _ints(case["lens_k"]) or lens_q
    hq, hk, D = case["heads"], case["heads_kv"], case["D"]
    G = hq // hk
    q, k, v = (st[n].double() for n in ("q", "k", "v"))
    o = torch.zeros_like(q)
    lse = torch.full((hq, q.shape[0]), -math.inf, dtype=torch.float64, device=DEV)
    grads = [torch.zeros_like(t) for t in (q, k, v)]
    a = c = 0
    for Lq, Lk in zip(lens_q, lens_k):
        b, d = a + Lq, c + Lk
        for h in range(hk if Lq and Lk else 0):
            keys = k[c:d, h].clone().requires_grad_(case["back"])
            vals = v[c:d, h].clone().requires_grad_(case["back"])
            for r in range(h * G, (h + 1) * G):
                rows = q[a:b, r].clone().requires_grad_(case["back"])
                x = rows.matmul(keys.t()) / math.sqrt(D)
                if case["causal"]:
                    keep = torch.ones(Lq, Lk, dtype=torch.bool, device=DEV).tril(Lk - Lq)
                    x = torch.where(keep, x, torch.full_like(x, -math.inf))
                p, z = _softmax_parts(x)
                y = p.matmul(vals)
                o[a:b, r] = y.detach()
                lse[r, a:b] = z.detach()
                if case["back"]:
                    part = torch.autograd.grad(y, (rows, keys, vals), st["dout"][a:b, r].double())
                    grads[0][a:b, r] = part[0]
                    grads[1][c:d, h] += part[1]
                    grads[2][c:d, h] += part[2]
                del x, p, z, y
        a, c = b, d
    if case["back"]:
        return [o, lse] + grads
    return o, lse


def exact(case, seed):
    st = prepare(case, seed)
    return {"rope": _rope_exact, "append": _append_exact, "paged": _paged_exact,
            "packed": _packed_exact}[case["op"]](case, st)
