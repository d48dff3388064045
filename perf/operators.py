"""What the training and rotary operators are measured on.

Two families, as a chunk-wise video model calls them around its attention layer:

  rope      rotary positions with three axes (time, height, width) over the frames of a
            chunk or of the key cache, with the RMS norm of queries and keys that precedes
            it, read from strided projections and written through cache slots; and its
            gradient (projections and norm weight).
  attn_bwd  the gradient of block-sparse attention: queries and keys of the current chunk
            and, on request, of the key and value cache, with the probabilities recomputed
            from the saved log-normaliser.

`run` computes a case in plain torch operations (32 bits, angles in 64), or, where `own` is
true, through the framework's public entry points.  `exact` is the definition in 64 bits.
"""
from __future__ import annotations

import math
from types import SimpleNamespace

import torch

own = False

DEV = "cuda"
BASE = 10000.0        # frequency base of the rotary positions
EPS = 1e-6            # added to the mean square in the norm


# --------------------------------------------------------------------------- cases
def _rope(name, bwd, H, d, frames, height, width, norm, halves, strided, slots, pos0):
    return dict(name=name, op="rope", bwd=bwd, H=H, d=d, frames=frames, height=height,
                width=width, norm=norm, halves=halves, strided=strided, slots=slots, pos0=pos0)


def _attn(name, H, d, T, block, fc, hist, sink, kf, kb, kc, cache_grad):
    return dict(name=name, op="attn_bwd", H=H, d=d, T=T, block=block, fc=fc, hist=hist,
                sink=sink, kf=kf, kb=kb, kc=kc, cache_grad=cache_grad)


def listed():
    return [
        # one token of a small model: nothing but latency
        _rope("rope_token", False, 2, 64, 1, 1, 1, "head", False, False, 0, 41),
        # queries of a 480p chunk (3 latent frames of 30 x 52), read from the fused QKV
        # projection, norm over the whole token
        _rope("rope_480p_q", False, 12, 128, 3, 30, 52, "row", False, True, 0, 18),
        # a rolling cache's keys (3 sinks + 21 frames) rotated to new positions on their way
        # out of their slots, no norm
        _rope("rope_cache_24", False, 12, 128, 24, 30, 52, "none", False, False, 27, 100000),
        # gradient for the same queries: projection and norm weight
        _rope("rope_bwd_480p_q", True, 12, 128, 3, 30, 52, "row", False, True, 0, 18),
        # gradient, odd grid, few heads, small head dimension, per-head norm, half pairing,
        # through slots
        _rope("rope_bwd_odd", True, 5, 64, 4, 17, 23, "head", True, False, 6, 3),
        # the smallest attention call of the workloads
        _attn("attn_bwd_tiny", 2, 64, 256, 64, 1, 4, 0, 2, 2, 0, True),
        # odd sizes: ragged last blocks, an odd number of query blocks, sinks, d = 64
        _attn("attn_bwd_odd", 5, 64, 391, 64, 2, 5, 1, 3, 3, 0, True),
        # the first chunk at 80 % sparsity: no history, sparse current chunk
        _attn("attn_bwd_chunk1_80", 12, 128, 1560, 64, 3, 0, 0, 1, 1, 15, False),
        # a 480p chunk trained against a detached cache
        _attn("attn_bwd_480p", 12, 128, 1560, 64, 3, 18, 0, 6, 12, 0, False),
        # the same with gradients into the cache's keys and values
        _attn("attn_bwd_480p_cache", 12, 128, 1560, 64, 3, 18, 0, 6, 12, 0, True),
        # rolling cache: 3 dense sink frames and 21 history frames
        _attn("attn_bwd_rolling", 12, 128, 1560, 64, 3, 21, 3, 4, 6, 0, True),
        # a large model: 40 heads, 42 history frames, blocks of 128
        _attn("attn_bwd_large", 40, 128, 1560, 128, 3, 42, 0, 8, 5, 0, True),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    if rng.random() < 0.4:
        d = rng.choice([64, 128])
        H = _log_int(rng, 1, 40)
        frames = _log_int(rng, 1, 48)
        height, width = _log_int(rng, 1, 60), _log_int(rng, 1, 104)
        while frames * height * width * H * d > 24 * 1560 * 1536:
            if frames > 1:
                frames = (frames + 1) // 2
            else:
                H = (H + 1) // 2
        slots = frames + rng.randint(0, 5) if rng.random() < 0.5 else 0
        return _rope(None, rng.random() < 0.5, H, d, frames, height, width,
                     rng.choice(["none", "head", "row"]), rng.random() < 0.5,
                     rng.random() < 0.5, slots, _log_int(rng, 1, 10 ** 6))
    d, block = rng.choice([64, 128]), rng.choice([64, 128])
    H, T, fc = _log_int(rng, 1, 40), _log_int(rng, 1, 2048), rng.randint(1, 4)
    hist, sink = rng.choice([0, 1, 3, 7, 12, 18, 24]), rng.randint(0, 3)
    nb = -(-T // block)
    kf, kb = rng.randint(1, 8), _log_int(rng, 1, nb)
    kc = rng.randint(1, fc * nb) if rng.random() < 0.3 else 0
    case = _attn(None, H, d, T, block, fc, hist, sink, kf, kb, kc, rng.random() < 0.5)
    limit = _pairs(listed()[-1])[0]
    while _pairs(case)[0] > limit:
        case["H"] = (case["H"] + 1) // 2
    return case


def _shape(case):
    nslots = case["hist"] + case["sink"] + (2 if case["hist"] + case["sink"] else 0)
    return SimpleNamespace(H=case["H"], d=case["d"], T=case["T"], block=case["block"],
                           n_cur_frames=case["fc"], n_hist=case["hist"], n_sink=case["sink"],
                           n_slots=nslots, k_f=case["kf"], k_b=case["kb"],
                           scale=1.0 / math.sqrt(case["d"]), k_c=case["kc"])


def _counts(case):
    """(blocks per frame, query blocks, frames kept, blocks kept per frame, current blocks)"""
    nb = -(-case["T"] // case["block"])
    kf = min(case["kf"], case["hist"])
    return nb, case["fc"] * nb, kf, min(case["kb"], nb) if kf else 0, min(case["kc"], case["fc"] * nb)


def _pairs(case):
    """(query, key) pairs of the call, and those whose keys are the current chunk's (a
    selected block counted at its average length)."""
    nb, _, kf, kb, kc = _counts(case)
    ncur = case["fc"] * case["T"]
    avg = case["T"] / nb
    cur = kc * avg if kc else ncur
    keys = cur + case["sink"] * case["T"] + kf * kb * avg
    return int(case["H"] * ncur * keys), int(case["H"] * ncur * cur)


def work(case):
    if case["op"] == "rope":
        n = case["frames"] * case["height"] * case["width"] * case["H"] * case["d"]
        if not case["bwd"]:
            # projection in, rotated out
            return {"bytes": 4 * n, "flops": (10 if case["norm"] != "none" else 4) * n}
        # gradient in, gradient out, and the projection where the norm needs it
        return {"bytes": (6 if case["norm"] != "none" else 4) * n,
                "flops": (18 if case["norm"] != "none" else 4) * n}
    pairs, pairs_cur = _pairs(case)
    d, ncur = case["d"], case["fc"] * case["T"]
    row = 2 * case["H"] * d
    cached = (case["hist"] + case["sink"]) * case["T"]
    grad = pairs if case["cache_grad"] else pairs_cur
    # scores, dP and dQ over all pairs; dK and dV over the keys that want a gradient
    flops = 6 * d * pairs + 4 * d * grad
    # q, k, v, out, dout in, dq, dk, dv out; the cache's k, v in and, on request, dk, dv out
    nbytes = 8 * ncur * row + 2 * cached * row + (2 * cached * row if case["cache_grad"] else 0)
    return {"bytes": nbytes + 4 * case["H"] * ncur, "flops": flops}


# --------------------------------------------------------------------------- inputs
def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _normal(g, *shape, std=1.0):
    return torch.randn(*shape, generator=g, device=DEV) * std


def _axes(d):
    """Channel pairs per axis (time, height, width): a third of the head each, the rest to
    time."""
    third = d // 6
    return d // 2 - 2 * third, third, third


def prepare(case, seed):
    st = _prepare_rope(case, seed) if case["op"] == "rope" else _prepare_attn(case, seed)
    st["case"] = case
    return st


def _prepare_rope(case, seed):
    g = _gen(seed)
    H, d, F, T = case["H"], case["d"], case["frames"], case["height"] * case["width"]
    n_slots = case["slots"] or F
    pick = torch.randperm(n_slots, generator=torch.Generator().manual_seed(seed))[:F].tolist()
    slots = pick if case["slots"] else None
    parts = 3 if case["strided"] else 1
    # a projection's output: channels of unequal size
    qkv = (_normal(g, n_slots, T, parts, H, d) * (0.5 + torch.rand(H, d, generator=g, device=DEV))
           ).to(torch.bfloat16)
    st = dict(slots=slots, x=qkv[:, :, 0], weight=None, dweight=None, workspace=None, rope=None,
              pos=[case["pos0"] + f for f in range(F)])
    if case["norm"] != "none":
        st["weight"] = 1.0 + _normal(g, d if case["norm"] == "head" else H * d, std=0.2)
    if case["bwd"]:
        st["dout"] = _normal(g, F, T, H, d).to(torch.bfloat16)
        st["dx"] = torch.zeros_like(qkv)[:, :, 0] if case["strided"] else torch.zeros_like(qkv[:, :, 0])
        if st["weight"] is not None:
            st["dweight"] = torch.empty_like(st["weight"])
    else:
        st["out"] = torch.empty(F, T, H, d, dtype=torch.bfloat16, device=DEV)
    if own:
        import block_sparse_attention_46_b200 as lf
        st["rope"] = lf.make_rope(H=H, d=d, n_frames=F, height=case["height"],
                                  width=case["width"], pairs=_axes(d), halves=case["halves"],
                                  norm=None if case["norm"] == "none" else case["norm"],
                                  base=BASE, eps=EPS)
        if case["bwd"]:
            st["workspace"] = torch.empty(max(lf.lf_rope_backward_workspace_size(st["rope"]), 256),
                                          dtype=torch.uint8, device=DEV)
    return st


def _topk_sorted(scores, k):
    return scores.topk(k, dim=-1).indices.sort(dim=-1).values


def _block_means(x, T, block):
    """[frames * T, H, d] -> [H, frames, blocks, d] in 32 bits."""
    H, d = x.shape[1:]
    nb = -(-T // block)
    xf = x.view(-1, T, H, d).float()
    pad = nb * block - T
    if pad:
        xf = torch.cat([xf, xf.new_zeros(xf.shape[0], pad, H, d)], 1)
    s = xf.view(-1, nb, block, H, d).sum(2)
    n = torch.full((nb,), block, device=x.device)
    n[-1] = T - (nb - 1) * block
    return (s / n.view(1, nb, 1, 1)).permute(2, 0, 1, 3)


def _prepare_attn(case, seed):
    g = _gen(seed)
    sh = _shape(case)
    H, d, T, F, S, fc = sh.H, sh.d, sh.T, sh.n_hist, sh.n_sink, sh.n_cur_frames
    nb, nqb, kf, kb, kc = _counts(case)
    ncur = fc * T
    bf = torch.bfloat16
    # keys around one centre per (head, frame), queries drawn towards a history frame
    cent = _normal(g, F + S + fc, 1, H, d, std=0.5)
    order = torch.randperm(max(sh.n_slots, 1), generator=torch.Generator().manual_seed(seed)).tolist()
    sinks, hist = order[:S], order[S:S + F]
    k_cache = _normal(g, max(sh.n_slots, 1), T, H, d)
    for i, s in enumerate(sinks + hist):
        k_cache[s] += cent[i]
    k_cache = k_cache.to(bf)
    v_cache = _normal(g, max(sh.n_slots, 1), T, H, d).to(bf)
    pull = cent[S + torch.randint(0, F, (fc,), generator=g, device=DEV)] if F else cent[F + S:]
    q = (_normal(g, fc, T, H, d) + 0.5 * pull).view(ncur, H, d).to(bf)
    k_cur = (_normal(g, fc, T, H, d) + cent[F + S:]).view(ncur, H, d).to(bf)
    v_cur = _normal(g, ncur, H, d).to(bf)
    dout = _normal(g, ncur, H, d).to(bf)
    block_idx = cur_idx = None
    q_blk = _block_means(q, T, sh.block).reshape(H, nqb, d) if F or kc else None
    if F:
        k_blk = _block_means(k_cache[hist].view(-1, H, d), T, sh.block)
        k_frm = k_cache[hist].float().mean(1).permute(1, 0, 2)
        frames = _topk_sorted(q_blk @ k_frm.transpose(1, 2), kf)              # [H, nqb, kf]
        sc = torch.einsum("hqd,hfbd->hqfb", q_blk, k_blk)
        sc = sc.gather(2, frames[..., None].expand(-1, -1, -1, nb))
        block_idx = (frames[..., None] * nb + _topk_sorted(sc, kb)).view(H, nqb, kf * kb)
        block_idx = block_idx.to(torch.int32).contiguous()
    if kc:
        sc = q_blk @ _block_means(k_cur, T, sh.block).reshape(H, nqb, d).transpose(1, 2)
        sc.diagonal(dim1=1, dim2=2).fill_(float("inf"))                       # its own block
        cur_idx = _topk_sorted(sc, kc).to(torch.int32).contiguous()
    st = dict(shape=sh, q=q, k_cur=k_cur, v_cur=v_cur, k_cache=k_cache, v_cache=v_cache,
              hist=hist, sinks=sinks, block_idx=block_idx, cur_idx=cur_idx, dout=dout,
              dq=torch.empty_like(q), dk_cur=torch.empty_like(q), dv_cur=torch.empty_like(q),
              dk_cache=None, dv_cache=None, workspace=None,
              out=torch.empty_like(q), lse=torch.empty(H, ncur, device=DEV), case=case)
    if case["cache_grad"] and F + S:
        st["dk_cache"], st["dv_cache"] = torch.zeros_like(k_cache), torch.zeros_like(v_cache)
    # the forward pass that training ran before: output and log-normaliser
    for h, chunk, idx, msk in _plain_chunks(st):
        k, v = _head_keys(st, h)
        s = (chunk["q"][:, h].float() @ k[idx].transpose(1, 2)) * sh.scale
        s.masked_fill_(msk[:, None, :], float("-inf"))
        m = torch.logsumexp(s, -1)
        o = torch.exp(s - m[..., None]) @ v[idx]
        st["out"][chunk["rows"], h] = o[chunk["valid"]].to(bf)
        st["lse"][h, chunk["rows"]] = m[chunk["valid"]]
    if own:
        import block_sparse_attention_46_b200 as lf
        st["workspace"] = torch.empty(max(lf.lf_attn_backward_workspace_size(sh), 256),
                                      dtype=torch.uint8, device=DEV)
    return st


# --------------------------------------------------------------------------- plain forms
def _angles(case, pos, f64=torch.float64):
    """[frames, T, pairs]: position along the pair's axis x its frequency, in 64 bits."""
    out = []
    hh = torch.arange(case["height"], device=DEV, dtype=f64)
    ww = torch.arange(case["width"], device=DEV, dtype=f64)
    tt = torch.tensor(pos, device=DEV, dtype=f64)
    F, h, w = len(pos), case["height"], case["width"]
    for axis, n in zip((tt.view(F, 1, 1), hh.view(1, h, 1), ww.view(1, 1, w)), _axes(case["d"])):
        freq = BASE ** (-torch.arange(n, device=DEV, dtype=f64) / n)
        out.append((axis[..., None] * freq).expand(F, h, w, n))
    return torch.cat(out, -1).view(F, h * w, -1)


def _rotate(x, cos, sin, halves):
    """Channel pairs of x [..., d] turned by their angles; cos, sin [F, T, 1, d/2]."""
    half = x.shape[-1] // 2
    a, b = (x[..., :half], x[..., half:]) if halves else (x[..., 0::2], x[..., 1::2])
    ra, rb = a * cos - b * sin, a * sin + b * cos
    return torch.cat([ra, rb], -1) if halves else torch.stack([ra, rb], -1).flatten(-2)


def _run_rope(st):
    case = st["case"]
    ang = _angles(case, st["pos"])[:, :, None, :]
    cos, sin = ang.cos().float(), ang.sin().float()
    x = (st["x"] if st["slots"] is None else st["x"][st["slots"]]).float()
    H, d = case["H"], case["d"]
    over = (-1,) if case["norm"] == "head" else (-2, -1)
    r = w = None
    if case["norm"] != "none":
        r = torch.rsqrt((x * x).mean(over, keepdim=True) + EPS)
        w = st["weight"] if case["norm"] == "head" else st["weight"].view(H, d)
    if not case["bwd"]:
        st["out"].copy_(_rotate(x if r is None else x * r * w, cos, sin, case["halves"]))
        return st["out"]
    g = _rotate(st["dout"].float(), cos, -sin, case["halves"])
    if r is not None:
        xn = x * r
        dw = g * xn
        st["dweight"].copy_(dw.sum((0, 1, 2) if case["norm"] == "head" else (0, 1)).flatten())
        g = g * w
        g = r * (g - xn * (g * xn).mean(over, keepdim=True))
    if st["slots"] is None:
        st["dx"].copy_(g)
    else:
        st["dx"][st["slots"]] = g.to(torch.bfloat16)
    return [st["dx"]] if r is None else [st["dx"], st["dweight"]]


def _head_keys(st, h):
    """Keys and values of one head in 32 bits: current chunk, sinks, history, and a zero row."""
    fr = st["sinks"] + st["hist"]
    out = []
    for cur, cache in ((st["k_cur"], st["k_cache"]), (st["v_cur"], st["v_cache"])):
        out.append(torch.cat([cur[:, h], cache[fr][:, :, h].reshape(-1, cur.shape[2]),
                              cur.new_zeros(1, cur.shape[2])]).float())
    return out


def _plain_chunks(st):
    """Per head and group of query blocks: the queries' rows, and for each query block the
    rows of _head_keys that it attends to with the mask of its padding."""
    sh = st["shape"]
    T, B = sh.T, sh.block
    nb, nqb, kf, kb, kc = _counts(st["case"])
    ncur, dev = sh.n_cur_frames * T, st["q"].device
    lane = torch.arange(B, device=dev)
    def tokens(frame, blk):                    # token in frame (-1 past its end), frame
        t = blk[..., None] * B + lane
        return torch.where(t < T, frame[..., None] * T + t, -1)
    qb = torch.arange(nqb, device=dev)
    q_rows = tokens(qb // nb, qb % nb)                                        # [nqb, B]
    end = ncur + (sh.n_sink + sh.n_hist) * T                                  # the zero row
    n_keys = (kc * B if kc else ncur) + sh.n_sink * T + kf * kb * B
    group = max(1, min(nqb, (1 << 28) // max(1, n_keys * max(B, sh.d))))
    for h in range(sh.H):
        for a in range(0, nqb, group):
            rows = q_rows[a:a + group]
            n = rows.shape[0]
            parts = []
            if kc:
                c = st["cur_idx"][h, a:a + group].long()
                parts.append(tokens(c // nb, c % nb).view(n, -1))
            else:
                parts.append(torch.arange(ncur, device=dev).expand(n, -1))
            parts.append(torch.arange(ncur, ncur + sh.n_sink * T, device=dev).expand(n, -1))
            if kf:
                c = st["block_idx"][h, a:a + group].long()
                t = tokens(c // nb, c % nb).view(n, -1)
                parts.append(torch.where(t < 0, t, t + ncur + sh.n_sink * T))
            idx = torch.cat(parts, 1)
            msk = idx < 0
            idx = torch.where(msk, end, idx)
            valid = rows >= 0
            safe = rows.clamp(min=0)
            yield h, dict(rows=rows[valid], valid=valid, safe=safe, q=_Rows(st["q"], safe)), idx, msk


class _Rows:
    """Rows of a [tokens, H, d] tensor, picked for one head at a time."""

    def __init__(self, x, rows):
        self.x, self.rows = x, rows

    def __getitem__(self, key):
        return self.x[:, key[1]][self.rows]


def _run_attn(st):
    sh, bf = st["shape"], torch.bfloat16
    ncur, T = sh.n_cur_frames * sh.T, sh.T
    last, acc = -1, None

    def flush(h, dk, dv):
        for grad, cur, cache in ((dk, st["dk_cur"], st["dk_cache"]), (dv, st["dv_cur"], st["dv_cache"])):
            cur[:, h] = grad[:ncur].to(bf)
            if cache is not None:
                cache[st["sinks"] + st["hist"], :, h] = grad[ncur:-1].view(-1, T, sh.d).to(bf)

    for h, chunk, idx, msk in _plain_chunks(st):
        if h != last:
            if acc is not None:
                flush(last, *acc)
            k, v = _head_keys(st, h)
            last, acc = h, (torch.zeros_like(k), torch.zeros_like(v))
        valid = chunk["valid"][..., None]
        q = chunk["q"][:, h].float()
        do = torch.where(valid, _Rows(st["dout"], chunk["safe"])[:, h].float(), 0.0)
        delta = (do * _Rows(st["out"], chunk["safe"])[:, h].float()).sum(-1, keepdim=True)
        kk, vv = k[idx], v[idx]
        s = (q @ kk.transpose(1, 2)) * sh.scale
        p = torch.exp(s - st["lse"][h][chunk["safe"]][..., None])
        p.masked_fill_(msk[:, None, :], 0.0)
        p = torch.where(valid, p, 0.0)
        ds = p * (do @ vv.transpose(1, 2) - delta) * sh.scale
        st["dq"][chunk["rows"], h] = (ds @ kk)[chunk["valid"]].to(bf)
        flat = idx.reshape(-1)
        acc[0].index_add_(0, flat, (ds.transpose(1, 2) @ q).reshape(-1, sh.d))
        acc[1].index_add_(0, flat, (p.transpose(1, 2) @ do).reshape(-1, sh.d))
    flush(last, *acc)
    return _grads(st)


def _grads(st):
    out = dict(dq=st["dq"], dk_cur=st["dk_cur"], dv_cur=st["dv_cur"])
    if st["dk_cache"] is not None:
        out.update(dk_cache=st["dk_cache"], dv_cache=st["dv_cache"])
    return out


def run(st):
    rope = st["case"]["op"] == "rope"
    if not own:
        return _run_rope(st) if rope else _run_attn(st)
    import block_sparse_attention_46_b200 as lf
    if rope and not st["case"]["bwd"]:
        lf.lf_rope_frames(st["rope"], st["x"], st["out"], frame_pos=st["pos"],
                          weight=st["weight"], in_slots=st["slots"])
        return st["out"]
    if rope:
        lf.lf_rope_frames_backward(st["rope"], st["x"], st["dout"], st["dx"], frame_pos=st["pos"],
                                   weight=st["weight"], dweight=st["dweight"],
                                   in_slots=st["slots"], workspace=st["workspace"])
        return [st["dx"]] if st["weight"] is None else [st["dx"], st["dweight"]]
    lf.lf_block_sparse_attn_backward(
        st["shape"], st["q"], st["k_cur"], st["v_cur"], st["k_cache"], st["v_cache"], st["hist"],
        st["sinks"], st["block_idx"], st["out"], st["dout"], st["lse"], st["dq"], st["dk_cur"],
        st["dv_cur"], st["dk_cache"], st["dv_cache"], workspace=st["workspace"],
        cur_idx=st["cur_idx"])
    return _grads(st)


# --------------------------------------------------------------------------- 64 bits
def exact(case, seed):
    global own
    was, own = own, False
    try:
        st = prepare(case, seed)
    finally:
        own = was
    return _exact_rope(st) if case["op"] == "rope" else _exact_attn(st)


def _turn(x, turns, halves):
    """Channel pairs as complex numbers times the unit numbers `turns`."""
    if halves:
        z = torch.complex(*x.chunk(2, -1)) * turns
        return torch.cat([z.real, z.imag], -1)
    return torch.view_as_real(torch.view_as_complex(x.unflatten(-1, (-1, 2)).contiguous()) * turns).flatten(-2)


def _exact_rope(st):
    case = st["case"]
    H, d, f64 = case["H"], case["d"], torch.float64
    names, w = (case["height"], case["width"]), None
    rows = st["slots"] if st["slots"] is not None else list(range(case["frames"]))
    res = torch.empty(st["dout" if case["bwd"] else "out"].shape, dtype=f64, device=DEV)
    if st["weight"] is not None:
        w = st["weight"].to(f64).requires_grad_(case["bwd"])
    dw = torch.zeros_like(w) if w is not None else None
    for f, pos in enumerate(st["pos"]):
        x = st["x"][rows[f]].to(f64).requires_grad_(case["bwd"])
        ii = torch.arange(names[0], dtype=f64, device=DEV).repeat_interleave(names[1])
        jj = torch.arange(names[1], dtype=f64, device=DEV).repeat(names[0])
        cols = []
        for p, n in zip((torch.full_like(ii, pos), ii, jj), _axes(d)):
            e = torch.linspace(0, n - 1, n, dtype=f64, device=DEV) / n
            cols.append(torch.outer(p, torch.exp(-math.log(BASE) * e)))
        turns = torch.polar(torch.ones((), dtype=f64, device=DEV), torch.cat(cols, 1))[:, None]
        y = x
        if w is not None:
            dims = 2 if case["norm"] == "head" else (1, 2)
            y = x / torch.sqrt(x.pow(2).mean(dims, keepdim=True) + EPS) * w.view(-1, d)
        y = _turn(y, turns, case["halves"])
        if case["bwd"]:
            (y * st["dout"][f].to(f64)).sum().backward()
            res[f] = x.grad
        else:
            res[f] = y
    if not case["bwd"]:
        return res
    dx = st["dx"].to(f64)
    dx[rows] = res
    return [dx] if w is None else [dx, w.grad]


def _exact_attn(st):
    sh, f64 = st["shape"], torch.float64
    T, B, ncur, d = sh.T, sh.block, sh.n_cur_frames * sh.T, sh.d
    nb = -(-T // B)
    frames = list(st["sinks"]) + list(st["hist"])
    tok = torch.arange(ncur, device=DEV)
    q_block = tok // T * nb + tok % T // B
    res = {n: torch.zeros_like(t, dtype=f64) for n, t in _grads(st).items()}
    kt = torch.arange(sh.n_hist * T, device=DEV)
    k_block = kt // T * nb + kt % T // B
    for h in range(sh.H):
        pick = lambda cur, cache: torch.cat([cur[:, h], cache[frames][:, :, h].reshape(-1, d)]).to(f64)
        k, v = pick(st["k_cur"], st["k_cache"]), pick(st["v_cur"], st["v_cache"])
        dk, dv = torch.zeros_like(k), torch.zeros_like(v)
        for a in range(0, ncur, 2048):
            r = slice(a, min(a + 2048, ncur))
            n = r.stop - a
            see = torch.ones(n, k.shape[0], dtype=torch.bool, device=DEV)
            if st["cur_idx"] is not None:
                tab = torch.zeros(sh.n_cur_frames * nb, sh.n_cur_frames * nb, dtype=torch.bool, device=DEV)
                tab.scatter_(1, st["cur_idx"][h].long(), True)
                see[:, :ncur] = tab[q_block[r]][:, q_block]
            if sh.n_hist:
                tab = torch.zeros(sh.n_cur_frames * nb, sh.n_hist * nb, dtype=torch.bool, device=DEV)
                tab.scatter_(1, st["block_idx"][h].long(), True)
                see[:, ncur + sh.n_sink * T:] = tab[q_block[r]][:, k_block]
            q, do, o = (st[x][r, h].to(f64) for x in ("q", "dout", "out"))
            p = torch.exp(q @ k.T * sh.scale - st["lse"][h, r, None].to(f64)) * see
            dv += p.T @ do
            ds = p * (do @ v.T - (do * o).sum(1, keepdim=True))
            dk += ds.T @ q * sh.scale
            res["dq"][r, h] = ds @ k * sh.scale
        for name, g in (("k", dk), ("v", dv)):
            res[f"d{name}_cur"][:, h] = g[:ncur]
            if st[f"d{name}_cache"] is not None:
                res[f"d{name}_cache"][frames, :, h] = g[ncur:].view(-1, T, d)
    return res
