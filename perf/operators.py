"""The cached-attention operators on measured sizes: per-head norm and position rotation of queries and
keys, the append to a paged KV cache, and attention of a batch that shares a prefix.

Each case is run in one of two forms on the same inputs: a plain one of elementary torch operations in
fp32, and (own = True) the calls that a program makes of rank_decomposed_gb300.

  rotate   q', k' = rotation(rms_norm(q) * q_gain), rotation(rms_norm(k) * k_gain), head by head
  append   the same for the new tokens' keys, written with the values to their rows of the paged cache
           (and the queries' rotation, where the case has queries)
  attend   softmax(q K^T / sqrt(head_dim)) V over a prefix that all sequences share followed by the
           sequence's own tokens; its query rows are its last tokens (each sees itself and what is before)
"""

import math

import torch

own = False

# n_heads, n_kv_heads, head_dim: the shapes of the repository's 7B, 70B and OPT-30B-shaped configurations
# and of its small test stack, and two uneven groups.
H7B, H70B, HOPT, HSMALL = (32, 32, 128), (64, 8, 128), (56, 56, 128), (8, 2, 64)
HEADS = (H7B, H70B, HOPT, HSMALL, (40, 8, 128), (12, 4, 64))
EPS = 1e-6


def _rotate_case(name, m, heads, norm, rot, style, f32, max_pos):
    c = dict(op="rotate", m=m, heads=heads[0], kv_heads=heads[1], head_dim=heads[2], norm=norm, rot=rot,
             style=style, f32=f32, max_pos=max_pos)
    return dict(c, name=name) if name else c


def _append_case(name, m, heads, norm, rot, style, f32, max_pos, with_q, per_seq, block_rows):
    c = _rotate_case(name, m, heads, norm, rot, style, f32, max_pos)
    return dict(c, op="append", with_q=with_q, per_seq=per_seq, block_rows=block_rows)


def _attend_case(name, n_seq, heads, prefix, own_lo, own_hi, q_lo, q_hi, block_rows):
    c = dict(op="attend", n_seq=n_seq, heads=heads[0], kv_heads=heads[1], head_dim=heads[2], prefix=prefix,
             own_lo=own_lo, own_hi=own_hi, q_lo=q_lo, q_hi=q_hi, block_rows=block_rows)
    return dict(c, name=name) if name else c


def listed():
    return [
        # one token of a single request: the smallest call of a decode step, all latency
        _rotate_case("rotate 1 token", 1, H70B, True, 128, "half", False, 8192),
        # a full decode batch with the fp32 outputs of the projections, rotation of a quarter of each head
        _rotate_case("rotate 256 rows fp32", 256, H7B, True, 32, "pair", True, 4096),
        # the prompts of a prefill batch, bound by memory
        _rotate_case("rotate 8191 rows", 8191, H70B, True, 128, "half", False, 131072),
        # a decode step of 64 sequences: queries, keys and values in one go, one new row a sequence
        _append_case("append 64 rows with q", 64, H70B, True, 128, "half", False, 131072, True, 1, 16),
        # a prompt chunk of MHA keys and values into scattered pages, without norms
        _append_case("append 4099 rows", 4099, H7B, False, 128, "half", False, 32768, False, 683, 16),
        # small heads, paired rotation of half a head, fp32 projections, large pages
        _append_case("append 777 rows fp32", 777, HSMALL, True, 32, "pair", True, 4096, False, 111, 64),
        # three chats just begun behind a short system prompt: all latency
        _attend_case("attend 3 seqs, prefix 200", 3, HSMALL, 200, 1, 40, 1, 1, 16),
        # a serving batch behind a long system prompt, one token each
        _attend_case("attend 64 seqs, prefix 8K", 64, H70B, 8192, 1, 512, 1, 1, 16),
        # the same for MHA: one query row for each key head and sequence
        _attend_case("attend 32 seqs MHA", 32, H7B, 4099, 1, 1000, 1, 1, 16),
        # few answers about one book: nearly all of the work lies along the keys
        _attend_case("attend 5 seqs, prefix 128K", 5, H70B, 131000, 16, 64, 1, 1, 64),
        # new turns of some hundred tokens behind a shared prompt, in one ragged call
        _attend_case("attend ragged turns", 12, H70B, 4096, 150, 700, 33, 300, 16),
        # many samples of one prompt, small heads
        _attend_case("attend 256 seqs, hd 64", 256, HSMALL, 1500, 1, 128, 1, 1, 16),
    ]


def _spread(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(("rotate", "append", "attend", "attend"))
    heads = rng.choice(HEADS)
    hd = heads[2]
    if op != "attend":
        norm, style, f32 = rng.random() < 0.7, rng.choice(("half", "half", "pair")), rng.random() < 0.3
        rot = rng.choice((hd, hd, hd // 2, hd // 4, 16))
        max_pos = rng.choice((4096, 32768, 131072))
        if op == "rotate":
            return _rotate_case(None, _spread(rng, 1, 8191), heads, norm, rot, style, f32, max_pos)
        return _append_case(None, _spread(rng, 1, 4099), heads, norm, rot, style, f32, max_pos, rng.random() < 0.5,
                            rng.choice((1, 1, _spread(rng, 2, 700))), rng.choice((16, 16, 32, 64)))
    block_rows = rng.choice((16, 16, 32, 64))
    if rng.random() < 0.7:  # one token each
        n_seq = _spread(rng, 1, 256)
        wide = max(8, heads[1])  # both bounds hold the cache that is read under that of the longest listed prefix
        prefix = _spread(rng, 1, min(800000 // wide, 6000000 // n_seq))
        hi = _spread(rng, 2, max(2, min(1500, 240000 // wide // n_seq)))
        return _attend_case(None, n_seq, heads, prefix, rng.randint(1, hi), hi, 1, 1, block_rows)
    n_seq = _spread(rng, 1, 12)
    q_hi = _spread(rng, 2, 300)
    hi = q_hi + rng.randint(0, 400)
    return _attend_case(None, n_seq, heads, _spread(rng, 1, 4096), q_hi, hi, rng.randint(1, q_hi), q_hi, block_rows)


# ------------------------------------------------------------------ inputs
def _table(max_pos, rot, dev):
    """fp32 [max_pos][rot]: the cosines of a position's rot/2 angles, then the sines, from 64-bit angles."""
    f = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device=dev) / rot)
    a = torch.arange(max_pos, dtype=torch.float64, device=dev)[:, None] * f[None]
    return torch.cat((a.cos(), a.sin()), 1).float()


def _lengths(case):
    """The batch's lengths: a fixed spread of the case's range, so that its work does not depend on the seed."""
    n, lo, hi = case["n_seq"], case["own_lo"], case["own_hi"]
    lens = [lo + ((i * 7919 + 13) % n) * (hi - lo) // max(1, n - 1) for i in range(n)]
    qs = [case["q_lo"] + ((i * 104729 + 5) % n) * (case["q_hi"] - case["q_lo"]) // max(1, n - 1) for i in range(n)]
    return lens, [min(a, b) for a, b in zip(qs, lens)]


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)
    H, K, D = case["heads"], case["kv_heads"], case["head_dim"]
    normal = lambda *s: torch.randn(*s, generator=g, device=dev)  # noqa: E731
    s = dict(case, status=torch.zeros(1, dtype=torch.int32, device=dev))
    i32 = lambda v: torch.tensor(v, dtype=torch.int32).to(dev)  # noqa: E731
    if case["op"] != "attend":
        m, t = case["m"], torch.float32 if case["f32"] else torch.bfloat16
        # one row of the projections' joint output a token: queries, keys, values
        s["qkv"] = (normal(m, (H + 2 * K) * D) * 1.5).to(t)
        s["q_gain"] = (1 + 0.2 * normal(D)).bfloat16() if case["norm"] else None
        s["k_gain"] = (1 + 0.2 * normal(D)).bfloat16() if case["norm"] else None
        s["table"] = _table(case["max_pos"], case["rot"], dev)
        s["pos"] = torch.randint(0, case["max_pos"], (m,), generator=g, device=dev, dtype=torch.int32)
        s["q_out"] = torch.zeros(m, H * D, dtype=torch.bfloat16, device=dev)
        s["k_out"] = torch.zeros(m, K * D, dtype=torch.bfloat16, device=dev)
        if case["op"] == "append":
            # runs of per_seq consecutive positions, each run's rows in pages of its own
            br, per = case["block_rows"], case["per_seq"]
            j = torch.arange(m, device=dev)
            pages = -(-per // br) + 1
            n_seq = -(-m // per)
            start = torch.randint(0, max(1, case["max_pos"] - per), (n_seq,), generator=g, device=dev)
            s["pos"] = (start[j // per] + j % per).clamp_(max=case["max_pos"] - 1).int()
            perm = torch.randperm(n_seq * pages, generator=g, device=dev)
            at = torch.randint(0, br, (n_seq,), generator=g, device=dev)[j // per] + j % per
            s["rows"] = (perm[(j // per) * pages + at // br] * br + at % br).int()
            s["k_pool"] = normal(n_seq * pages * br, K * D).bfloat16()
            s["v_pool"] = normal(n_seq * pages * br, K * D).bfloat16()
        return s
    lens, qs = _lengths(case)
    n, br, P = case["n_seq"], case["block_rows"], case["prefix"]
    pblocks, bps = -(-P // br), -(-max(lens) // br)
    perm = torch.randperm(pblocks + n * bps, generator=g, device=dev).int()
    s["prefix_blocks"], s["block_table"] = perm[:pblocks].contiguous(), perm[pblocks:].view(n, bps).contiguous()
    s["prefix_len"], s["lengths"] = i32([P]), i32(lens)
    starts = [0]
    for x in qs:
        starts.append(starts[-1] + x)
    s["q_start"] = i32(starts) if max(qs) > 1 else None
    s["max_q"], s["m"], s["max_own"] = max(qs), starts[-1], max(lens)
    # a few channels carry most of a score, as after a trained norm
    loud = torch.ones(D, device=dev)
    loud[torch.randperm(D, generator=g, device=dev)[:4]] = 3.0
    rows = perm.numel() * br
    s["k_pool"] = (normal(rows, K, D) * loud).bfloat16().view(rows, K * D)
    s["v_pool"] = normal(rows, K * D).bfloat16()
    s["q"] = (normal(s["m"], H, D) * loud).bfloat16().view(s["m"], H * D)
    s["out"] = torch.zeros(s["m"], H * D, dtype=torch.bfloat16, device=dev)
    s["workspace"] = torch.empty(512 << 20, dtype=torch.uint8, device=dev)
    # the plain form's padding of the batch: each row's sequence, and its place among that one's rows
    s["seq"] = torch.repeat_interleave(torch.arange(n, device=dev), i32(qs).long())
    s["place"] = torch.arange(s["m"], device=dev) - i32(starts).long()[s["seq"]]
    s["n_q"] = i32(qs)
    return s


# -------------------------------------------------------------- plain forms
def _plain_heads(x, heads, gain, s):
    """RMS norm of each head and its rotation, in fp32; [rows][heads][head_dim]."""
    m, D, r = x.shape[0], s["head_dim"], s["rot"]
    x = x.float().view(m, heads, D)
    if s["norm"]:
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * gain.float()
    cs = s["table"][s["pos"].long()][:, None]
    c, sn = cs[..., : r // 2], cs[..., r // 2:]
    if s["style"] == "half":
        a, b = x[..., : r // 2], x[..., r // 2: r]
        turned = torch.cat((a * c - b * sn, b * c + a * sn), -1)
    else:
        a, b = x[..., 0:r:2], x[..., 1:r:2]
        turned = torch.stack((a * c - b * sn, b * c + a * sn), -1).flatten(-2)
    return torch.cat((turned, x[..., r:]), -1).view(m, heads * D).bfloat16()


def _split(s):
    H, K, D = s["heads"], s["kv_heads"], s["head_dim"]
    x = s["qkv"]
    return x[:, : H * D], x[:, H * D: (H + K) * D], x[:, (H + K) * D:]


def _plain_attend(s):
    H, K, D, n, br = s["heads"], s["kv_heads"], s["head_dim"], s["n_seq"], s["block_rows"]
    G, m, Q, L, P = H // K, s["m"], s["max_q"], s["max_own"], s["prefix"]
    dev = s["q"].device
    step = torch.arange(br, device=dev)
    prow = (s["prefix_blocks"].long()[:, None] * br + step).flatten()[:P]
    orow = (s["block_table"].long()[:, :, None] * br + step).view(n, -1)[:, :L]
    q = s["q"].float().view(m, K, G, D) / math.sqrt(D)
    # the prefix: all rows of the batch against the same keys
    kp = s["k_pool"][prow].float().view(P, K, D).permute(1, 2, 0)
    vp = s["v_pool"][prow].float().view(P, K, D).transpose(0, 1)
    sp = torch.matmul(q.transpose(0, 1).reshape(K, m * G, D), kp).view(K, m, G, P)
    # the own tokens, padded to [sequences][most rows]
    qo = q.new_zeros(n, Q, K, G, D)
    qo[s["seq"], s["place"]] = q
    ko = s["k_pool"][orow].float().view(n, L, K, D).permute(0, 2, 3, 1)
    vo = s["v_pool"][orow].float().view(n, L, K, D).transpose(1, 2)
    so = torch.matmul(qo.transpose(1, 2).reshape(n, K, Q * G, D), ko).view(n, K, Q, G, L)
    last = (s["lengths"] - s["n_q"]).long()[:, None] + torch.arange(Q, device=dev)  # a row's own position
    so = so.masked_fill((torch.arange(L, device=dev) > last[..., None])[:, None, :, None], -math.inf)
    so = so.permute(0, 2, 1, 3, 4)[s["seq"], s["place"]]  # [m][K][G][L]
    top = torch.maximum(sp.amax(-1).permute(1, 0, 2), so.amax(-1))
    ep = torch.exp(sp - top.permute(1, 0, 2)[..., None])
    eo = torch.exp(so - top[..., None])
    total = ep.sum(-1).permute(1, 0, 2) + eo.sum(-1)
    op = torch.matmul(ep.view(K, m * G, P), vp).view(K, m, G, D).permute(1, 0, 2, 3)
    pad = eo.new_zeros(n, Q, K, G, L)
    pad[s["seq"], s["place"]] = eo
    oo = torch.matmul(pad.transpose(1, 2).reshape(n, K, Q * G, L), vo).view(n, K, Q, G, D)
    oo = oo.permute(0, 2, 1, 3, 4)[s["seq"], s["place"]]
    s["out"].copy_(((op + oo) / total[..., None]).reshape(m, H * D))
    return s["out"]


def _plain(s):
    if s["op"] == "attend":
        return _plain_attend(s)
    q, k, v = _split(s)
    if s["op"] == "rotate":
        s["q_out"].copy_(_plain_heads(q, s["heads"], s["q_gain"], s))
        s["k_out"].copy_(_plain_heads(k, s["kv_heads"], s["k_gain"], s))
        return s["q_out"], s["k_out"]
    at = s["rows"].long()
    s["k_pool"][at] = _plain_heads(k, s["kv_heads"], s["k_gain"], s)
    s["v_pool"][at] = v.bfloat16()
    if not s["with_q"]:
        return s["k_pool"], s["v_pool"]
    s["q_out"].copy_(_plain_heads(q, s["heads"], s["q_gain"], s))
    return s["k_pool"], s["v_pool"], s["q_out"]


# -------------------------------------------------- the framework's operators
def _own(s):
    import rank_decomposed_gb300 as lr

    if s["op"] == "attend":
        cache = lr.PagedKV(s["k_pool"], s["v_pool"], s["kv_heads"], s["head_dim"], s["block_rows"])
        lr.prefix_attention(s["q"], s["heads"], cache, s["prefix_blocks"], s["prefix_len"], s["block_table"],
                            s["lengths"], s["out"], s["workspace"], s["status"], q_start=s["q_start"],
                            max_q=s["max_q"])
        return s["out"]
    q, k, v = _split(s)
    hm = lr.HeadMap(s["head_dim"], norm=s["norm"], eps=EPS, q_gain=s["q_gain"], k_gain=s["k_gain"],
                    rot_dim=s["rot"], rot_style=lr.ROT_HALF if s["style"] == "half" else lr.ROT_PAIR,
                    cos_sin=s["table"])
    if s["op"] == "rotate":
        lr.qk_norm_rope(q, k, s["pos"], hm, s["q_out"], s["k_out"], s["status"])
        return s["q_out"], s["k_out"]
    with_q = s["with_q"]
    cache = lr.PagedKV(s["k_pool"], s["v_pool"], s["kv_heads"], s["head_dim"], s["block_rows"])
    lr.kv_append(k, v, s["pos"], s["rows"], hm, cache, s["status"], q=q if with_q else None,
                 q_out=s["q_out"] if with_q else None)
    return (s["k_pool"], s["v_pool"], s["q_out"]) if with_q else (s["k_pool"], s["v_pool"])


def run(state):
    return _own(state) if own else _plain(state)


# ------------------------------------------------------------------ 64 bits
def _exact_heads(x, heads, gain, s):
    out = x.double().reshape(x.shape[0], heads, s["head_dim"]).clone()
    if s["norm"]:
        out /= (out.square().sum(-1, keepdim=True) / s["head_dim"] + EPS).sqrt()
        out *= gain.double()
    half = s["rot"] // 2
    first = torch.arange(half, device=x.device)
    first, second = (first, first + half) if s["style"] == "half" else (2 * first, 2 * first + 1)
    # the pair (a, b) as the complex number a + ib, turned by cos + i sin of its angle
    turn = torch.complex(s["table"][:, :half].double(), s["table"][:, half:].double())[s["pos"].long()]
    z = torch.complex(out[..., first], out[..., second]) * turn[:, None]
    out[..., first], out[..., second] = z.real, z.imag
    return out.flatten(1)


def exact(case, seed):
    s = prepare(case, seed)
    H, K, D = case["heads"], case["kv_heads"], case["head_dim"]
    if case["op"] != "attend":
        q, k, v = _split(s)
        if case["op"] == "rotate":
            return _exact_heads(q, H, s["q_gain"], s), _exact_heads(k, K, s["k_gain"], s)
        kp, vp = s["k_pool"].double(), s["v_pool"].double()
        kp[s["rows"].long()] = _exact_heads(k, K, s["k_gain"], s)
        vp[s["rows"].long()] = v.double()
        return (kp, vp, _exact_heads(q, H, s["q_gain"], s)) if case["with_q"] else (kp, vp)
    lens, qs = _lengths(case)
    br, P, G = case["block_rows"], case["prefix"], H // K
    kb, vb = (s[x].view(-1, br, K, D) for x in ("k_pool", "v_pool"))
    out, at = [], 0
    kpre, vpre = (x[s["prefix_blocks"].long()].flatten(0, 1)[:P].double() for x in (kb, vb))
    for b, (L, nq) in enumerate(zip(lens, qs)):
        blocks = s["block_table"][b].long()
        keys = torch.cat((kpre, kb[blocks].flatten(0, 1)[:L].double()))
        vals = torch.cat((vpre, vb[blocks].flatten(0, 1)[:L].double()))
        q = s["q"][at: at + nq].double().view(nq, K, G, D)
        at += nq
        sees = torch.arange(P + L, device=q.device)[None] <= P + L - nq + torch.arange(nq, device=q.device)[:, None]
        o = q.new_empty(nq, K, G, D)
        for h in range(K):
            w = torch.einsum("qgd,kd->qgk", q[:, h], keys[:, h]) / math.sqrt(D)
            w = torch.softmax(w.masked_fill(~sees[:, None], -math.inf), -1)
            o[:, h] = torch.einsum("qgk,kd->qgd", w, vals[:, h])
        out.append(o.flatten(1))
    return torch.cat(out)


# --------------------------------------------------------------------- work
def work(case):
    """Inputs read once, outputs written once; the products and the per-element arithmetic."""
    H, K, D = case["heads"], case["kv_heads"], case["head_dim"]
    if case["op"] != "attend":
        m, e = case["m"], 4 if case["f32"] else 2
        qs = H if case["op"] == "rotate" or case["with_q"] else 0
        vs = K if case["op"] == "append" else 0
        # a row's position and angles (and its place in the cache) beside its heads
        side = m * (4 + 4 * min(case["rot"], case["rot"] * case["max_pos"] // m) + (4 if vs else 0))
        return {"bytes": m * (qs + K + vs) * D * (e + 2) + side, "flops": m * (qs + K) * D * (9 if case["norm"] else 3)}
    lens, qs = _lengths(case)
    m = sum(qs)
    seen = m * case["prefix"] + sum(nq * (L - nq) + nq * (nq + 1) // 2 for L, nq in zip(lens, qs))
    return {"bytes": (case["prefix"] + sum(lens)) * K * D * 4 + m * H * D * 4, "flops": 4 * seen * H * D}
