"""Cases, plain forms and 64-bit values of the operators over a KV cache held in 4 bits.

Three passes, each as a program makes it:
  append  a chunk's K and V (slices of one fused projection) into the cache, in place of the
          chunk's rows of the step before, and the stored values read back;
  attend  one attention over the rows held, with the attention weight each row drew added to
          its sum where the case asks for it;
  evict   a rolling step at a full cache: append, evict down to `keep` rows by accumulated
          weight, and one query token's attention over what stays.

Where `own` is false the passes are elementary torch operations in 32 bits.
"""

import math

import torch

own = False

E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)  # magnitudes of the codes 0..7; bit 3 is the sign
MAX_SCALE = 10240.0
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


# ------------------------------------------------------------------ cases

def _case(name, op, batch, kv_heads, group, head_dim, dtype, tokens, rows, ragged=False,
          causal=False, weights=False):
    """rows: rows held before the pass (append: with the rows to be replaced; evict: the rows
    that stay, `keep`); group: query heads per KV head; tokens: rows appended or query tokens."""
    case = dict(op=op, batch=batch, kv_heads=kv_heads, group=group, head_dim=head_dim, dtype=dtype,
                tokens=tokens, rows=rows, ragged=ragged, causal=causal, weights=weights)
    return dict(case, name=name) if name else case


def listed():
    return [
        # one decoded token of eight sequences: launch latency
        _case("append, a token each", "append", 8, 8, 1, 128, "bf16", 1, 4096),
        # the generating chunk of a 720p stream, re-appended at every denoising step
        _case("append, a 720p chunk", "append", 1, 12, 1, 128, "bf16", 10800, 43200),
        # a single conversation's next token, short history: launch latency
        _case("decode, one short sequence", "attend", 1, 8, 4, 128, "bf16", 1, 700),
        # a serving batch of uneven histories, one slot idle, collecting weights for eviction
        _case("decode, a ragged batch, weights", "attend", 16, 8, 4, 128, "bf16", 1, 16300,
              ragged=True, weights=True),
        # long histories, few heads: the cache is all the traffic
        _case("decode, long histories", "attend", 4, 8, 8, 128, "bf16", 1, 131071),
        # five draft tokens checked at once, small heads
        _case("verify, five drafts", "attend", 8, 8, 4, 64, "fp16", 5, 8000, ragged=True,
              causal=True),
        # a 540p chunk attends to its history and itself, both ways
        _case("chunk, 540p", "attend", 1, 12, 1, 128, "bf16", 6120, 24480),
        # the same at 720p, with the weights that decide what is evicted
        _case("chunk, 720p, weights", "attend", 1, 12, 1, 128, "bf16", 10800, 43200, weights=True),
        # prompts of different lengths, causal, grouped heads
        _case("prompt, ragged, causal", "attend", 4, 8, 4, 128, "fp16", 4093, 4093, ragged=True,
              causal=True, weights=True),
        # decoding at a full cache: a row in, a row out, every step
        _case("evict, a token each", "evict", 8, 8, 4, 128, "bf16", 1, 4096),
        # a 720p chunk in, as many rows out, per head
        _case("evict, a 720p chunk", "evict", 1, 12, 1, 128, "bf16", 10800, 43200),
    ]


def draw(rng):
    def spread(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    while True:
        op = rng.choice(("append", "attend", "attend", "attend", "evict"))
        head_dim = rng.choice((64, 128, 128))
        kv_heads = rng.choice((1, 2, 3, 4, 8, 12))
        group = rng.choice((1, 1, 2, 3, 4, 6, 8))
        batch = spread(1, 24)
        tokens = rng.choice((1, 1, spread(2, 16), spread(17, 600), spread(601, 9000)))
        rows = max(tokens, spread(1, 150000))
        case = _case(None, op, batch, kv_heads, 1 if op == "append" else group, head_dim,
                     rng.choice(("bf16", "fp16")), tokens, rows,
                     ragged=op != "evict" and rng.random() < 0.5,
                     causal=op == "attend" and rng.random() < 0.5,
                     weights=op == "attend" and rng.random() < 0.5)
        queries = tokens if op == "attend" else 1
        if 4.0 * batch * kv_heads * group * queries * rows <= 8e9 and \
                8.0 * batch * kv_heads * rows * head_dim <= 6e9 and \
                batch * kv_heads * (rows + tokens) <= 6e6:
            return case


def _counts(case):
    """Valid tokens of each sequence of the call."""
    t, n = case["tokens"], case["batch"]
    if not case["ragged"]:
        return [t] * n
    return [0 if b == 2 else t - (b * 389) % (t // 2 + 1) for b in range(n)]


def _lens(case):
    """Rows held by each sequence when the pass begins."""
    r, n = case["rows"], case["batch"]
    if not case["ragged"]:
        return [r] * n
    c = _counts(case)
    return [0 if b == 2 else max(c[b], r - (b * 2477) % (3 * r // 4 + 1)) for b in range(n)]


def _capacity(case):
    need = case["rows"] + (case["tokens"] if case["op"] == "evict" else 0)
    return -(-need // 128) * 128


def _protect(case):
    """(first, recent) rows that an eviction leaves alone."""
    return min(16, case["rows"] // 8), min(case["tokens"] + 64, case["rows"] // 2)


# ------------------------------------------------------------------ the format, plain

def _quantise(x):
    """x [..., D] -> (codes uint8 [..., D / 2], scales uint8 [..., D / 16])."""
    blocks = x.float().unflatten(-1, (-1, 16))
    u = blocks.abs().amax(-1)
    u = u / torch.full_like(u, 6.0)  # by a tensor: a true division, so that 6 s / 6 is s
    e = torch.frexp(u).exponent - 1  # u = 1.m * 2^e
    step = ((e.clamp(min=-14) - 3 + 127) << 23).view(torch.float32)  # 2^(e - 3)
    s = torch.where(u > 0, torch.ceil(u / step) * step, u).clamp(max=MAX_SCALE)
    a = torch.where(s[..., None] > 0, blocks / s[..., None], torch.zeros_like(blocks))
    m = a.abs()
    code = ((m > 0.25).to(torch.uint8) + (m >= 0.75) + (m > 1.25) + (m >= 1.75) + (m > 2.5)
            + (m >= 3.5) + (m > 5.0))
    code = (code + (a < 0).to(torch.uint8) * 8).flatten(-2)
    scales = (s.half().view(torch.int16) >> 7).to(torch.uint8)
    return code[..., 0::2] | (code[..., 1::2] << 4), scales


def _dequantise(codes, scales):
    """The values in fp32, [..., D]."""
    lut = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=codes.device)
    v = torch.stack((lut[(codes & 15).long()], lut[(codes >> 4).long()]), -1).flatten(-2)
    s = (scales.to(torch.int16) << 7).view(torch.float16).float()
    return (v.unflatten(-1, (-1, 16)) * s[..., None]).flatten(-2)


# ------------------------------------------------------------------ states

def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed * 7919 + 17)
    B, H, G, D, T = (case[k] for k in ("batch", "kv_heads", "group", "head_dim", "tokens"))
    dt, cap = DTYPES[case["dtype"]], _capacity(case)

    def normal(*shape):
        return torch.randn(shape, generator=gen, device=dev)

    # keys have a few wide channels, as trained projections have; queries are narrower there
    wide = 1.0 + 3.0 * (torch.rand((H, D), generator=gen, device=dev) < 0.06).float()
    lens = torch.tensor(_lens(case), dtype=torch.int32, device=dev)
    counts = torch.tensor(_counts(case), dtype=torch.int32, device=dev)
    last = counts if case["op"] != "evict" else torch.zeros_like(counts)
    # rows held, rows ever appended, rows of the last append, rows appended since an eviction
    seq = torch.stack((lens, lens, last, last)).contiguous()
    state = {"case": case, "seq": seq}
    for name in ("k", "v"):
        x = normal(B, H, cap, D)
        x *= wide[None, :, None] if name == "k" else 0.5
        state[name + "_codes"], state[name + "_scales"] = _quantise(x)
        del x
    state["pos"] = torch.arange(cap, dtype=torch.int32, device=dev).expand(B, H, cap).contiguous()
    # what earlier steps gave: a few rows draw most of the weight
    state["weight"] = torch.exp(2.0 * normal(B, H, cap))
    state["status"] = torch.zeros(4, dtype=torch.int32, device=dev)
    if case["op"] != "attend":
        kv = normal(B, T, 2 * H, D)
        kv[:, :, :H] *= wide
        kv[:, :, H:] *= 0.5
        kv = kv.to(dt)
        state["k"], state["v"] = kv[:, :, :H], kv[:, :, H:]
    if case["op"] == "append":
        state["k_out"] = torch.zeros((B, T, H, D), dtype=dt, device=dev)
        state["v_out"] = torch.zeros_like(state["k_out"])
    else:
        n_q = T if case["op"] == "attend" else 1
        q = normal(B, n_q, H, G, D) / wide[:, None, :].sqrt()
        state["q"] = q.reshape(B, n_q, H * G, D).to(dt)
        state["out"] = torch.zeros((B, n_q, H * G, D), dtype=dt, device=dev)
        state["lse"] = torch.zeros((B, H * G, n_q), dtype=torch.float32, device=dev)
    state["counts"] = counts if case["ragged"] else None
    return state


# ------------------------------------------------------------------ the plain forms

def _put(dst, rows, valid, x):
    """dst [B, H, cap, ...] at rows [B, T] <- x [B, H, T, ...] where valid [B, T]."""
    b, t = valid.nonzero(as_tuple=True)
    dst[b, :, rows[b, t]] = x.transpose(1, 2)[b, t]


def _plain_append(s, replace):
    c, seq = s["case"], s["seq"]
    T, dev = c["tokens"], seq.device
    n_new = s["counts"] if s["counts"] is not None else torch.full_like(seq[0], T)
    back = seq[2] if replace else torch.zeros_like(seq[2])
    base = seq[0] - back
    t = torch.arange(T, device=dev)
    rows, valid = base[:, None] + t, t < n_new[:, None]
    for name in ("k", "v"):
        codes, scales = _quantise(s[name].transpose(1, 2))
        _put(s[name + "_codes"], rows, valid, codes)
        _put(s[name + "_scales"], rows, valid, scales)
    first = (seq[1] - back)[:, None] + t
    H = c["kv_heads"]
    _put(s["pos"], rows, valid, first[:, None].expand(-1, H, -1).to(torch.int32))
    _put(s["weight"], rows, valid, torch.zeros(rows.shape, device=dev)[:, None].expand(-1, H, -1))
    seq.copy_(torch.stack((base + n_new, seq[1] - back + n_new, n_new, seq[3] - back + n_new)))
    return rows, valid


def _plain_read(s, rows, valid):
    """The stored values of rows [B, T] into k_out, v_out where valid."""
    at = rows.clamp(max=_capacity(s["case"]) - 1).long()[:, None, :, None]
    for name in ("k", "v"):
        codes, scales = s[name + "_codes"], s[name + "_scales"]
        codes = codes.gather(2, at.expand(-1, codes.shape[1], -1, codes.shape[3]))
        scales = scales.gather(2, at.expand(-1, scales.shape[1], -1, scales.shape[3]))
        x = _dequantise(codes, scales).transpose(1, 2)
        out = s[name + "_out"]
        out.copy_(torch.where(valid[:, :, None, None], x.to(out.dtype), out))


def _plain_attend(s, causal, weights):
    c, seq = s["case"], s["seq"]
    B, H, G, D = (c[k] for k in ("batch", "kv_heads", "group", "head_dim"))
    n, T, dev = c["rows"], s["q"].shape[1], seq.device
    keys = _dequantise(s["k_codes"][:, :, :n], s["k_scales"][:, :, :n])
    q = s["q"].float().unflatten(2, (H, G)).permute(0, 2, 3, 1, 4).reshape(B, H, G * T, D)
    sc = torch.matmul(q, keys.transpose(2, 3)).mul_(1.0 / math.sqrt(D)).view(B, H, G, T, n)
    del keys
    n_q = s["counts"] if s["counts"] is not None else torch.full_like(seq[0], T)
    t, j = torch.arange(T, device=dev), torch.arange(n, device=dev)
    valid = t < n_q[:, None]
    end = seq[0][:, None].expand(-1, T)
    if causal:
        end = end - n_q[:, None] + t + 1
    if c["ragged"] or causal:
        seen = (j < end[:, :, None]) & valid[:, :, None]
        sc.masked_fill_(~seen[:, None, None], -math.inf)
    m = sc.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    p = sc.sub_(m).exp_()
    total = p.sum(-1, keepdim=True)
    p.div_(torch.where(total > 0, total, torch.ones_like(total)))
    lse = (m + total.log()).squeeze(-1)
    vals = _dequantise(s["v_codes"][:, :, :n], s["v_scales"][:, :, :n])
    o = torch.matmul(p.view(B, H, G * T, n), vals).view(B, H, G, T, D)
    o = o.permute(0, 3, 1, 2, 4).reshape(B, T, H * G, D)
    s["out"].copy_(torch.where(valid[:, :, None, None], o.to(s["out"].dtype), s["out"]))
    s["lse"].copy_(torch.where(valid[:, None], lse.view(B, H * G, T), s["lse"]))
    if weights:
        s["weight"][:, :, :n] += p.sum((2, 3))


def _plain_evict(s, keep, first, recent):
    seq, cap = s["seq"], s["weight"].shape[2]
    j = torch.arange(cap, device=seq.device)
    held = (j < seq[0][:, None])[:, None]
    w, pos = s["weight"], s["pos"]
    w = torch.where(w.isnan(), -math.inf, w.double())
    kept_anyway = (pos < first) | (pos >= (seq[1] - recent)[:, None, None])
    # three classes kept apart in one 64-bit key: protected, held, not held
    key = torch.where(kept_anyway, math.inf, w.clamp(-1e300, 1e300))
    key = torch.where(held, key, -math.inf)
    order = key.argsort(dim=-1, descending=True, stable=True)
    kept = torch.zeros_like(order, dtype=torch.bool).scatter_(2, order[:, :, :keep], True) & held
    holes = (j < keep) & held & ~kept
    movers = (j >= keep) & kept
    movers_in_order = (~movers).to(torch.uint8).argsort(dim=-1, stable=True)
    nth = (holes.cumsum(-1) - 1).clamp(min=0)
    src = torch.where(holes, movers_in_order.gather(2, nth), j.expand_as(nth))
    for name in ("pos", "weight"):
        s[name].copy_(s[name].gather(2, src))
    for name in ("k_codes", "k_scales", "v_codes", "v_scales"):
        x = s[name]
        x.copy_(x.gather(2, src[..., None].expand(-1, -1, -1, x.shape[3])))
    more = seq[0] > keep
    seq[0].clamp_(max=keep)
    seq[2:] *= ~more


# ------------------------------------------------------------------ one pass

def _cache(s):
    """The program's cache object over the state's tensors, made once."""
    if "cache" not in s:
        from block_causal_streaming_sa_b200 import QuantKVCache

        names = ("k_codes", "v_codes", "k_scales", "v_scales", "pos", "weight", "seq", "status")
        s["cache"] = QuantKVCache.from_tensors(**{n: s[n] for n in names})
    return s["cache"]


def run(state):
    s, c = state, state["case"]
    if c["op"] == "append":
        if own:
            cache = _cache(s)
            cache.append(s["k"], s["v"], counts=s["counts"], replace=True)
            cache.read_last(s["k_out"], s["v_out"])
        else:
            rows, valid = _plain_append(s, replace=True)
            _plain_read(s, rows, valid)
        return {"k": s["k_out"], "v": s["v_out"], "seq": s["seq"]}
    if c["op"] == "attend":
        if own:
            _cache(s).attend(s["q"], counts=s["counts"], causal=c["causal"], out=s["out"],
                             lse=s["lse"], add_weight=c["weights"])
        else:
            _plain_attend(s, c["causal"], c["weights"])
        got = {"out": s["out"], "lse": s["lse"]}
        return dict(got, weight=s["weight"]) if c["weights"] else got
    first, recent = _protect(c)
    if own:
        cache = _cache(s)
        cache.append(s["k"], s["v"])
        cache.evict(c["rows"], first=first, recent=recent)
        cache.attend(s["q"], out=s["out"], lse=s["lse"])
    else:
        _plain_append(s, replace=False)
        _plain_evict(s, c["rows"], first, recent)
        _plain_attend(s, False, False)
    return {"out": s["out"], "lse": s["lse"], "pos": s["pos"], "weight": s["weight"],
            "seq": s["seq"]}


# ------------------------------------------------------------------ what a pass cannot do without

def work(case):
    B, H, G, D, T = (case[k] for k in ("batch", "kv_heads", "group", "head_dim", "tokens"))
    row = D + D // 8  # K and V codes and scales of one row of one head
    counts, lens = _counts(case), _lens(case)
    if case["op"] == "append":
        # K and V in, codes, scales, position and weight out; the codes back in, the values out
        return {"bytes": H * sum(counts) * (4 * D + row + 8 + row + 4 * D), "flops": 0}
    if case["op"] == "attend":
        byts = H * sum(lens) * (row + (8 if case["weights"] else 0))
        byts += H * G * sum(counts) * (4 * D + 4)
        pairs = 0
        for n, t in zip(lens, counts):
            pairs += t * n - (t * (t - 1) // 2 if case["causal"] else 0)
        return {"bytes": byts, "flops": 4 * D * H * G * pairs}
    keep = case["rows"]
    byts = B * H * (T * (4 * D + row + 8)            # append
                    + 8 * (keep + T) + 2 * T * (row + 8)  # weights and positions, rows moved
                    + keep * row + G * (4 * D + 4))  # the attention
    return {"bytes": byts, "flops": 4 * D * B * H * G * keep}


# ------------------------------------------------------------------ 64-bit values

def _scale_table64(device):
    return torch.tensor([i * 2.0 ** -17 if i < 8 else (1 + i % 8 / 8) * 2.0 ** (i // 8 - 15)
                         for i in range(256)], dtype=torch.float64, device=device)


def _values64(codes, scales):
    """Stored values from the definition of the format: sign, two exponent bits, one fraction
    bit; the scale's byte has five exponent bits and three fraction bits."""
    nib = torch.empty(codes.shape[:-1] + (2 * codes.shape[-1],), dtype=torch.int64,
                      device=codes.device)
    nib[..., 0::2], nib[..., 1::2] = codes.long() % 16, codes.long() // 16
    e, f = (nib // 2) % 4, (nib % 2).double()
    mag = torch.where(e == 0, 0.5 * f, (1 + 0.5 * f) * (1 << e).double() / 2)
    s = _scale_table64(codes.device)[scales.long()]
    return mag * (1 - 2 * (nib >= 8).double()) * s.repeat_interleave(16, dim=-1)


def _nearest64(x):
    """What the format makes of x [..., D]: the smallest scale that covers the block, the
    nearest code, an even fraction bit at a tie."""
    x = x.double()
    blocks = x.reshape(x.shape[:-1] + (x.shape[-1] // 16, 16))
    table = _scale_table64(x.device)[:227]
    want = blocks.abs().amax(-1)
    s = table[torch.searchsorted(6 * table, want).clamp(max=226)]
    grid = torch.tensor(E2M1, dtype=torch.float64, device=x.device)
    a = torch.where(s[..., None] > 0, blocks.abs() / s[..., None], 0.0 * blocks)
    i = torch.searchsorted(grid, a.contiguous()).clamp(1, 7)  # grid[i-1] < a <= grid[i]
    lo, hi = grid[i - 1], grid[i]
    up = (hi - a < a - lo) | ((hi - a == a - lo) & (i % 2 == 0))
    q = torch.where(up, hi, lo) * torch.sign(blocks) * s[..., None]
    return q.reshape(x.shape)


def _attend64(q, keys, vals, end, scale):
    """(O, lse, weight) of queries [R, D] over keys, vals [n, D], query r seeing end[r] rows."""
    sc = (q @ keys.T) * scale
    sc[torch.arange(keys.shape[0], device=q.device)[None] >= end[:, None]] = -math.inf
    lse = torch.logsumexp(sc, dim=1)
    p = torch.exp(sc - torch.where(lse == -math.inf, 0.0, lse)[:, None])
    return p @ vals, lse, p.sum(0)


def exact(case, seed):
    s = prepare(case, seed)
    B, H, G, D, T = (case[k] for k in ("batch", "kv_heads", "group", "head_dim", "tokens"))
    counts, lens = _counts(case), _lens(case)
    if case["op"] == "append":
        got = {}
        for name in ("k", "v"):
            got[name] = torch.zeros((B, T, H, D), dtype=torch.float64, device="cuda")
            for b in range(B):
                got[name][b, :counts[b]] = _nearest64(s[name][b, :counts[b]])
        return dict(got, seq=None)
    if 4.0 * D * B * H * G * T * case["rows"] > 6e12:
        return None
    n_q = s["q"].shape[1]
    out = torch.zeros((B, n_q, H * G, D), dtype=torch.float64, device="cuda")
    lse = torch.zeros((B, H * G, n_q), dtype=torch.float64, device="cuda")
    weight = s["weight"].double()
    first, recent = _protect(case)
    for b in range(B):
        for h in range(H):
            n = lens[b]
            at = slice(0, n)
            keys = _values64(s["k_codes"][b, h, at], s["k_scales"][b, h, at])
            vals = _values64(s["v_codes"][b, h, at], s["v_scales"][b, h, at])
            c = counts[b]
            end = torch.full((c,), n, device="cuda")
            if case["causal"]:
                end = torch.arange(n - c + 1, n + 1, device="cuda")
            if case["op"] == "evict":
                # the rows that stay: protected ones, then by weight, then by place
                w = weight[b, h, :n + T].clone()
                w[n:] = 0.0
                at = torch.arange(n + T, device="cuda")
                safe = (at < first) | (at >= n + T - recent)
                w[safe] = math.inf
                kept = torch.sort(torch.sort(w, descending=True, stable=True).indices[:n]).values
                stay = torch.zeros(n + T, dtype=torch.bool, device="cuda")
                stay[kept] = True
                to = torch.nonzero(~stay[:n]).flatten()
                weight[b, h, n:n + T] = 0.0
                weight[b, h, to] = weight[b, h, kept[kept >= n]]
                keys = torch.cat((keys, _nearest64(s["k"][b, :, h])))[kept]
                vals = torch.cat((vals, _nearest64(s["v"][b, :, h])))[kept]
                c, end = 1, torch.full((1,), n, device="cuda")
            for g in range(G):
                hq = h * G + g
                o, l, w = _attend64(s["q"][b, :c, hq].double(), keys, vals, end, D ** -0.5)
                out[b, :c, hq], lse[b, hq, :c] = o, l
                if case["weights"]:
                    weight[b, h, :n] += w
    got = {"out": out, "lse": lse}
    if case["op"] == "evict":
        return dict(got, pos=None, weight=weight, seq=None)
    return dict(got, weight=weight) if case["weights"] else got
