"""Rotary positions, appending to the paged cache and shared-prefix decode, as cases to measure.

`listed()` and `draw()` give cases, `prepare()` what a program holds before the
call, `run()` one call: in plain torch operations, or, with `own` set, through
this package's entry points. `exact()` gives the same results in 64 bits.
"""
import math

import torch

own = False

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
RANK = 32  # components of a projected key


# ------------------------------------------------------------------ cases
def _rotate(name, **kw):
    c = dict(op="rotate", name=name, dtype="bf16", head_dim=128, heads=32, tokens=1, first=0, stride_heads=0,
             layout="half", rot_dim=128, scaling="none", transpose=False)
    c.update(kw)
    return c


def _append(name, **kw):
    c = dict(op="append", name=name, dtype="bf16", head_dim=128, q_heads=32, kv_heads=8, page=16, proxy="exact",
             batch=1, tokens=1, first=4000, last=4000, fused=False, rotate_q=True, layout="half", rot_dim=128,
             scaling="none")
    c.update(kw)
    return c


def _shared(name, **kw):
    c = dict(op="shared", name=name, dtype="bf16", head_dim=128, q_heads=32, kv_heads=8, page=16, batch=8, groups=1,
             prefix_min=1024, prefix_max=1024, own_min=1, own_max=64)
    c.update(kw)
    return c


def listed():
    return [
        # the queries of a single sequence at one decode step
        _rotate("rotate_token", first=20000),
        # a prompt's queries, a view of the fused q/k/v product, positions scaled band by band
        _rotate("rotate_prompt", tokens=8192, stride_heads=48, scaling="bands"),
        # the gradient of a partly rotated head in fp32, an odd number of tokens
        _rotate("rotate_gradient", tokens=4001, heads=12, dtype="f32", head_dim=64, rot_dim=32, layout="interleaved",
                first=100, transpose=True),
        # one sequence, one new token: latency
        _append("append_token"),
        # a served batch at one step, every sequence somewhere in a long context
        _append("append_batch", batch=256, tokens=256, first=16384, last=65536, scaling="yarn"),
        # three prompts at once out of the fused product
        _append("append_prompts", batch=3, tokens=12001, first=0, last=300, fused=True),
        # a prompt into a contiguous cache with the dim-major copy of the keys
        _append("append_sparq", tokens=8192, first=17, last=17, page=16384, proxy="sparq", scaling="linear"),
        # a long prompt continued, with projected keys
        _append("append_loki", batch=2, tokens=8190, first=1000, last=30000, proxy="loki", rotate_q=False),
        # two short fp32 sequences over one short prefix
        _shared("shared_small", dtype="f32", head_dim=64, q_heads=4, kv_heads=4, batch=2, prefix_min=500,
                prefix_max=500, own_max=40),
        # a batch that shares one long document
        _shared("shared_document", batch=32, prefix_min=32768, prefix_max=32768, own_min=100, own_max=1000),
        # several instructions of different lengths, groups of different sizes
        _shared("shared_groups", batch=48, groups=6, prefix_min=2000, prefix_max=16000, page=64, own_max=700),
        # many short answers to one instruction
        _shared("shared_many", batch=256, prefix_min=8192, prefix_max=8192, own_max=300),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rotate", "append", "append", "shared", "shared"])
    d = rng.choice([64, 128, 128])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    rope = dict(layout=rng.choice(["half", "interleaved"]), rot_dim=rng.choice([d, d, d // 2, d // 4, 2 * rng.randint(1, d // 2)]),
                scaling=rng.choice(["none", "linear", "base", "bands", "yarn"]))
    kv = rng.choice([1, 2, 4, 8])
    g = rng.choice([1, 2, 4, 8])
    page = rng.choice([16, 16, 32, 48, 64, 256])
    if op == "rotate":
        heads = rng.randint(1, 32)
        c = _rotate("", dtype=dtype, head_dim=d, heads=heads, tokens=_log(rng, 1, 8192 if dtype == "bf16" else 4096),
                    first=_log(rng, 1, 1 << 20), stride_heads=rng.choice([0, heads + 16]),
                    transpose=rng.random() < 0.3, **rope)
    elif op == "append":
        proxy = rng.choice(["exact", "exact", "sparq", "loki"])
        batch = _log(rng, 1, 256)
        tokens = batch if rng.random() < 0.5 else batch + _log(rng, 1, 4000)
        first = _log(rng, 1, 20000)
        c = _append("", dtype=dtype, head_dim=d, q_heads=kv * g, kv_heads=kv, page=page, proxy=proxy, batch=batch,
                    tokens=tokens, first=first, last=first + _log(rng, 1, 20000), fused=rng.random() < 0.5,
                    rotate_q=rng.random() < 0.7, **rope)
    else:
        groups = rng.choice([1, 1, 2, 3, 5])
        batch = groups + _log(rng, 1, 100 if dtype == "bf16" else 40)
        lo = _log(rng, 100, 5000 if dtype == "bf16" else 2000)
        own_min = _log(rng, 1, 100)
        c = _shared("", dtype=dtype, head_dim=d, q_heads=kv * g, kv_heads=kv, page=page, batch=batch, groups=groups,
                    prefix_min=lo, prefix_max=lo + _log(rng, 1, lo), own_min=own_min, own_max=own_min + _log(rng, 1, 700))
    del c["name"]
    return c


# ------------------------------------------------------------------ rotary settings
BASE, FACTOR, ORIGINAL = 500000.0, 8.0, 8192
LOW, HIGH = 1.0, 4.0            # bands: wavelengths above ORIGINAL / LOW divided, below ORIGINAL / HIGH kept
SLOW, FAST = 1.0, 32.0          # yarn: turns over ORIGINAL positions where the ramp ends and begins


def _amplitude(c):
    return 0.1 * math.log(FACTOR) + 1.0 if c["scaling"] == "yarn" else 1.0


def _frequencies(c):
    """Angle per position of each pair, float64."""
    r, kind = c["rot_dim"], c["scaling"]
    i = torch.arange(r // 2, dtype=torch.float64)
    base = BASE * FACTOR ** (r / (r - 2)) if kind == "base" and r > 2 else BASE
    f = base ** (-2.0 * i / r)
    if kind == "linear":
        f = f / FACTOR
    elif kind == "bands":
        turns = ORIGINAL * f / (2 * math.pi)
        keep = ((turns - LOW) / (HIGH - LOW)).clamp(0, 1)
        f = keep * f + (1 - keep) * f / FACTOR
    elif kind == "yarn":
        at = lambda turns: r * math.log(ORIGINAL / (turns * 2 * math.pi)) / (2 * math.log(BASE))  # noqa: E731
        lo, hi = max(math.floor(at(FAST)), 0), min(math.ceil(at(SLOW)), r - 1)
        ramp = ((i - lo) / (hi - lo if hi > lo else 0.001)).clamp(0, 1)
        f = f * (1 - ramp) + f / FACTOR * ramp
    return f


def _rotary(c):
    """The package's plan of the same rotation."""
    from verified_sparse_attention_b200.rotary import Rotary
    return Rotary(head_dim=c["head_dim"], rot_dim=c["rot_dim"], layout=c["layout"], base=BASE, scaling=c["scaling"],
                  factor=FACTOR, original_ctx=ORIGINAL, low=LOW, high=HIGH, slow=SLOW, fast=FAST)


def _turned(x, pos, freq, c, sign=1.0):
    """x [T, H, d] rotated to positions pos [T], in fp32 (angles in fp64)."""
    r = c["rot_dim"]
    ang = pos.double()[:, None] * freq
    cos = (ang.cos() * _amplitude(c)).float()[:, None]
    sin = (ang.sin() * (sign * _amplitude(c))).float()[:, None]
    x = x.float()
    y = x.clone()
    if c["layout"] == "half":
        a, b = x[..., :r // 2], x[..., r // 2:r]
        y[..., :r // 2] = a * cos - b * sin
        y[..., r // 2:r] = b * cos + a * sin
    else:
        a, b = x[..., 0:r:2], x[..., 1:r:2]
        y[..., 0:r:2] = a * cos - b * sin
        y[..., 1:r:2] = b * cos + a * sin
    return y


# ------------------------------------------------------------------ inputs
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _randn(shape, g, dt):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).to(dt)


def _spread(total, parts, seed):
    """`total` cut into `parts` lengths of at least one."""
    g = torch.Generator()
    g.manual_seed(seed)
    cuts = sorted((torch.randperm(total - 1, generator=g)[:parts - 1] + 1).tolist()) if parts > 1 else []
    return [b - a for a, b in zip([0] + cuts, cuts + [total])]


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def prepare(case, seed):
    c = dict(case)
    g = _gen(seed)
    s = {"case": c}
    if c["op"] == "rotate":
        dt = DT[c["dtype"]]
        T, H, d = c["tokens"], c["heads"], c["head_dim"]
        wide = _randn((T, max(H, c["stride_heads"]), d), g, dt)
        s["x"] = wide[:, :H]
        s["positions"] = torch.arange(c["first"], c["first"] + T, dtype=torch.int32, device="cuda")
        s["freq"] = _frequencies(c).cuda()
        s["out"] = torch.empty((T, H, d), dtype=dt, device="cuda")
        if own:
            s["rotary"] = _rotary(c)
    elif c["op"] == "append":
        _prepare_append(c, seed, g, s)
    else:
        _prepare_shared(c, seed, g, s)
    return s


def _decoder(c, batch, max_ctx):
    from verified_sparse_attention_b200.decoder import SparseDecoder
    proxy = c.get("proxy", "exact")
    return SparseDecoder(num_q_heads=c["q_heads"], num_kv_heads=c["kv_heads"], head_dim=c["head_dim"],
                         dtype=DT[c["dtype"]], page_size=c["page"], max_batch=batch, max_ctx=max_ctx, proxy=proxy,
                         proxy_rank={"exact": 0, "sparq": 32, "loki": RANK}[proxy])


def _prepare_append(c, seed, g, s):
    dt = DT[c["dtype"]]
    B, T, d, Hq, Hkv, ps = c["batch"], c["tokens"], c["head_dim"], c["q_heads"], c["kv_heads"], c["page"]
    new = [1] * B if T == B else _spread(T, B, seed)
    h = torch.Generator()
    h.manual_seed(seed + 1)
    before = torch.randint(c["first"], c["last"] + 1, (B,), generator=h).tolist()
    lens = [a + n for a, n in zip(before, new)]
    max_ctx = max(lens)
    pps = -(-max_ctx // ps)
    # every new token's page is its own; the pages of earlier positions are not touched by the call and
    # stand on page 0
    table = torch.zeros((B, pps), dtype=torch.int32)
    pages = 1
    for b in range(B):
        lo, hi = before[b] // ps, (lens[b] - 1) // ps
        table[b, lo:hi + 1] = torch.arange(pages, pages + hi + 1 - lo, dtype=torch.int32)
        pages += hi + 1 - lo
    pages = 1 + T // ps + 2 * B  # the pool: at least the pages used
    order = torch.cat([torch.zeros(1, dtype=torch.int64), torch.randperm(pages - 1, generator=h) + 1])
    s["page_table"] = order[table.long()].int().cuda()
    s["seq_lens"] = _ints(lens)
    s["cu_tokens"] = None if T == B else torch.tensor([0] + new, dtype=torch.int64).cumsum(0).int().cuda()
    s["num_pages"] = pages
    if c["fused"]:
        wide = _randn((T, Hq + 2 * Hkv, d), g, dt)
        s["q"], s["k"], s["v"] = wide[:, :Hq], wide[:, Hq:Hq + Hkv], wide[:, Hq + Hkv:]
    else:
        s["q"], s["k"], s["v"] = _randn((T, Hq, d), g, dt), _randn((T, Hkv, d), g, dt), _randn((T, Hkv, d), g, dt)
    if not c["rotate_q"]:
        s["q"] = None
    s["q_out"] = torch.empty((T, Hq, d), dtype=dt, device="cuda") if c["rotate_q"] else None
    s["k_cache"] = torch.zeros((pages, Hkv, ps, d), dtype=dt, device="cuda")
    s["v_cache"] = torch.zeros((pages, Hkv, ps, d), dtype=dt, device="cuda")
    s["k_t_cache"] = torch.zeros((pages, Hkv, d, ps), dtype=dt, device="cuda") if c["proxy"] == "sparq" else None
    s["k_proj_cache"] = s["basis"] = None
    if c["proxy"] == "loki":
        s["k_proj_cache"] = torch.zeros((pages, Hkv, ps, RANK), dtype=dt, device="cuda")
        s["basis"] = torch.linalg.qr(_randn((Hkv, d, RANK), g, torch.float32))[0].contiguous()
    s["freq"] = _frequencies(c).cuda()
    if own:
        s["rotary"] = _rotary(c)
        s["decoder"] = _decoder(c, B, max_ctx)


def _prepare_shared(c, seed, g, s):
    dt = DT[c["dtype"]]
    B, n, d, Hq, Hkv, ps = c["batch"], c["groups"], c["head_dim"], c["q_heads"], c["kv_heads"], c["page"]
    h = torch.Generator()
    h.manual_seed(seed + 1)
    sizes = _spread(B, n, seed)
    prefix = torch.randint(c["prefix_min"], c["prefix_max"] + 1, (n,), generator=h).tolist()
    rest = torch.randint(c["own_min"], c["own_max"] + 1, (B,), generator=h).tolist()
    start = [0]
    for z in sizes:
        start.append(start[-1] + z)
    lens = [prefix[k] + rest[b] for k in range(n) for b in range(start[k], start[k + 1])]
    max_ctx = max(lens)
    # whole pages of a prefix are shared by its group; the page in which it ends is each sequence's own
    table = torch.zeros((B, -(-max_ctx // ps)), dtype=torch.int64)
    pages, copies = 0, []
    for k in range(n):
        whole = prefix[k] // ps
        table[start[k]:start[k + 1], :whole] = torch.arange(pages, pages + whole)
        pages += whole
        for b in range(start[k], start[k + 1]):
            more = -(-lens[b] // ps) - whole
            table[b, whole:whole + more] = torch.arange(pages, pages + more)
            if prefix[k] % ps and b > start[k]:
                copies.append((int(table[start[k], whole]), int(table[b, whole]), prefix[k] % ps))
            pages += more
    order = torch.randperm(pages, generator=h)
    s["k_cache"], s["v_cache"] = _randn((pages, Hkv, ps, d), g, dt), _randn((pages, Hkv, ps, d), g, dt)
    if copies:
        src, dst, rows = (torch.tensor(v) for v in zip(*copies))
        src, dst = order[src].cuda(), order[dst].cuda()
        keep = (torch.arange(ps)[None] < rows[:, None]).cuda()[:, None, :, None]
        for cache in (s["k_cache"], s["v_cache"]):
            cache[dst] = torch.where(keep, cache[src], cache[dst])
    s["page_table"] = order[table].int().cuda()
    s["seq_lens"], s["group_start"], s["prefix_lens"] = _ints(lens), _ints(start), _ints(prefix)
    s["num_pages"] = pages
    s["q"] = _randn((B, Hq, d), g, dt)
    s["out"] = torch.empty((B, Hq, d), dtype=torch.float32, device="cuda")
    # what a program that batches requests knows of its groups on the host
    s["sizes"] = (max(sizes), max(prefix), max(rest))
    if own:
        s["decoder"] = _decoder(c, B, max_ctx)


# ------------------------------------------------------------------ one pass
def run(s):
    op = s["case"]["op"]
    return (_run_rotate if op == "rotate" else _run_append if op == "append" else _run_shared)(s)


def _run_rotate(s):
    c = s["case"]
    if own:
        return s["rotary"].rotate(s["x"], s["positions"], out=s["out"], transpose=c["transpose"])
    return _turned(s["x"], s["positions"], s["freq"], c, -1.0 if c["transpose"] else 1.0).to(DT[c["dtype"]])


def _run_append(s):
    c = s["case"]
    if own:
        s["decoder"].append(s["k"], s["v"], s["k_cache"], s["v_cache"], s["page_table"], s["seq_lens"], s["num_pages"],
                            cu_tokens=s["cu_tokens"], rotary=s["rotary"], q=s["q"], q_out=s["q_out"],
                            k_t_cache=s["k_t_cache"], k_proj_cache=s["k_proj_cache"], proj_basis=s["basis"])
        q = s["q_out"]
    else:
        dt, ps = DT[c["dtype"]], c["page"]
        t = torch.arange(c["tokens"], device="cuda")
        if s["cu_tokens"] is None:
            seq, pos = t, s["seq_lens"].long() - 1
        else:
            cu = s["cu_tokens"].long()
            seq = torch.searchsorted(cu[1:], t, right=True)
            pos = s["seq_lens"].long()[seq] - cu[seq + 1] + t
        page, slot = s["page_table"][seq, pos // ps].long(), pos % ps
        key = _turned(s["k"], pos, s["freq"], c).to(dt)
        s["k_cache"][page, :, slot] = key
        s["v_cache"][page, :, slot] = s["v"]
        if s["k_t_cache"] is not None:
            s["k_t_cache"][page, :, :, slot] = key
        if s["k_proj_cache"] is not None:
            s["k_proj_cache"][page, :, slot] = torch.einsum("thd,hdr->thr", key.float(), s["basis"]).to(dt)
        q = None if s["q"] is None else _turned(s["q"], pos, s["freq"], c).to(dt)
    return {"k": s["k_cache"], "v": s["v_cache"], "q": [] if q is None else q,
            "t": [] if s["k_t_cache"] is None else s["k_t_cache"],
            "proj": [] if s["k_proj_cache"] is None else s["k_proj_cache"]}


def _rows(s, key, table, pos):
    """Cache rows of positions pos [N, P] under page-table rows [N, pages] as [N, Hkv, P, d] fp32."""
    ps = s["case"]["page"]
    pos = pos.clamp(0, table.shape[1] * ps - 1)
    page = table.gather(1, pos // ps).long()
    return s[key][page, :, pos % ps].float().transpose(1, 2)


def _part(q, k, v, valid):
    """Row maxima, weight sums and weighted values of q [N, H, R, d] over k, v [N, H, P, d]; valid [N, 1, 1, P]."""
    x = torch.matmul(q, k.transpose(-1, -2)) * (1.0 / math.sqrt(q.shape[-1]))
    x = x.masked_fill(~valid, -math.inf)
    m = x.amax(-1, keepdim=True).clamp_min(-3e38)
    w = (x - m).exp()
    return m, w.sum(-1, keepdim=True), torch.matmul(w, v)


def _run_shared(s):
    c = s["case"]
    if own:
        return s["decoder"].shared_dense(s["q"], s["k_cache"], s["v_cache"], s["page_table"], s["seq_lens"],
                                         s["num_pages"], s["group_start"], s["prefix_lens"], out=s["out"])
    B, Hq, Hkv, d = c["batch"], c["q_heads"], c["kv_heads"], c["head_dim"]
    most, longest, rest = s["sizes"]
    dev = s["q"].device
    start, lens, prefix = s["group_start"].long(), s["seq_lens"].long(), s["prefix_lens"].long()
    # the prefix: one product per group over the rows of all its sequences
    member = start[:-1, None] + torch.arange(most, device=dev)
    real = member < start[1:, None]
    qg = s["q"].float().view(B, Hkv, Hq // Hkv, d)[member.clamp(max=B - 1)]
    qg = qg.transpose(1, 2).reshape(c["groups"], Hkv, most * (Hq // Hkv), d)
    pos = torch.arange(longest, device=dev).expand(c["groups"], longest)
    first = s["page_table"][start[:-1]]
    m, l, a = _part(qg, _rows(s, "k_cache", first, pos), _rows(s, "v_cache", first, pos),
                    (pos < prefix[:, None])[:, None, None])
    back = [x.view(c["groups"], Hkv, most, Hq // Hkv, -1).transpose(1, 2)[real] for x in (m, l, a)]
    # each sequence's own positions
    group = torch.searchsorted(start[1:], torch.arange(B, device=dev), right=True)
    pos = prefix[group][:, None] + torch.arange(rest, device=dev)
    mo, lo, ao = _part(s["q"].float().view(B, Hkv, Hq // Hkv, d), _rows(s, "k_cache", s["page_table"], pos),
                       _rows(s, "v_cache", s["page_table"], pos), (pos < lens[:, None])[:, None, None])
    top = torch.maximum(back[0], mo)
    wp, wo = (back[0] - top).exp(), (mo - top).exp()
    return ((back[2] * wp + ao * wo) / (back[1] * wp + lo * wo)).reshape(B, Hq, d)


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    c = case
    e = 2 if c["dtype"] == "bf16" else 4
    d = c["head_dim"]
    if c["op"] == "rotate":
        n = c["tokens"] * c["heads"]
        return {"bytes": 2 * n * d * e + 4 * c["tokens"], "flops": 3 * n * c["rot_dim"]}
    Hq, Hkv = c["q_heads"], c["kv_heads"]
    if c["op"] == "append":
        T = c["tokens"]
        rows = 4 * Hkv + (2 * Hq if c["rotate_q"] else 0) + (Hkv if c["proxy"] == "sparq" else 0)
        b = T * (rows * d * e + 8) + (T * Hkv * RANK * e + Hkv * d * RANK * 4 if c["proxy"] == "loki" else 0)
        f = 3 * T * c["rot_dim"] * (Hkv + (Hq if c["rotate_q"] else 0))
        return {"bytes": b, "flops": f + (2 * T * Hkv * d * RANK if c["proxy"] == "loki" else 0)}
    prefix, rest = (c["prefix_min"] + c["prefix_max"]) / 2, (c["own_min"] + c["own_max"]) / 2
    keys = c["groups"] * prefix + c["batch"] * rest
    return {"bytes": 2 * keys * Hkv * d * e + c["batch"] * Hq * d * (e + 4),
            "flops": 4 * d * Hq * c["batch"] * (prefix + rest)}


# ------------------------------------------------------------------ 64-bit results
def _exact_turn(x, pos, c, sign=1):
    """Complex multiplication by amplitude * exp(i angle)."""
    r, kind = c["rot_dim"], c["scaling"]
    rate = []
    for i in range(r // 2):
        base = BASE * math.pow(FACTOR, r / (r - 2.0)) if kind == "base" and r != 2 else BASE
        w = math.exp(-math.log(base) * 2 * i / r)
        if kind == "linear":
            w /= FACTOR
        if kind == "bands":
            length = 2 * math.pi / w
            if length > ORIGINAL / LOW:
                w /= FACTOR
            elif length >= ORIGINAL / HIGH:
                t = (ORIGINAL / length - LOW) / (HIGH - LOW)
                w = (1 - t) * w / FACTOR + t * w
        if kind == "yarn":
            lo, hi = (r * math.log(ORIGINAL / (n * 2 * math.pi)) / (2 * math.log(BASE)) for n in (FAST, SLOW))
            lo, hi = max(math.floor(lo), 0), min(math.ceil(hi), r - 1)
            t = min(max((i - lo) / (hi - lo if hi > lo else 0.001), 0.0), 1.0)
            w = w / FACTOR * t + w * (1 - t)
        rate.append(w)
    turn = torch.polar(torch.full((len(pos), r // 2), _amplitude(c), dtype=torch.float64, device="cuda"),
                       sign * torch.outer(pos.double(), torch.tensor(rate, dtype=torch.float64, device="cuda")))
    x = x.double()
    head = x[..., :r]
    if c["layout"] == "half":
        z = torch.complex(head[..., :r // 2].contiguous(), head[..., r // 2:].contiguous()) * turn[:, None]
        head = torch.cat([z.real, z.imag], -1)
    else:
        z = torch.view_as_complex(head.reshape(*head.shape[:-1], r // 2, 2).contiguous()) * turn[:, None]
        head = torch.view_as_real(z).flatten(-2)
    return torch.cat([head, x[..., r:]], -1)


def exact(case, seed):
    s = prepare(case, seed)
    c = s["case"]
    if c["op"] == "rotate":
        return _exact_turn(s["x"], s["positions"], c, -1 if c["transpose"] else 1)
    ps, d = c["page"], c["head_dim"]
    lens = s["seq_lens"].tolist()
    if c["op"] == "append":
        cu = list(range(c["batch"] + 1)) if s["cu_tokens"] is None else s["cu_tokens"].tolist()
        pos, page = [], []
        table = s["page_table"].tolist()
        for b in range(c["batch"]):
            for p in range(lens[b] - (cu[b + 1] - cu[b]), lens[b]):
                pos.append(p)
                page.append(table[b][p // ps])
        pos, page = torch.tensor(pos, device="cuda"), torch.tensor(page, device="cuda")
        key = _exact_turn(s["k"], pos, c)
        res = {"k": s["k_cache"].double(), "v": s["v_cache"].double(), "q": None, "t": None, "proj": None}
        flat = lambda x: x.permute(0, 2, 1, 3).reshape(-1, x.shape[1], x.shape[3])  # noqa: E731
        for name, rows in (("k", key), ("v", s["v"].double())):
            x = flat(res[name])
            x[page * ps + pos % ps] = rows
            res[name] = x.view(-1, ps, c["kv_heads"], d).permute(0, 2, 1, 3)
        if s["q"] is not None:
            res["q"] = _exact_turn(s["q"], pos, c)
        if s["k_t_cache"] is not None:
            res["t"] = res["k"].transpose(2, 3)
        if s["k_proj_cache"] is not None:
            # the product is of the key as it is stored
            res["proj"] = torch.matmul(res["k"].to(DT[c["dtype"]]).double(), s["basis"].double())
        return res
    out = torch.empty((c["batch"], c["q_heads"], d), dtype=torch.float64, device="cuda")
    for b in range(c["batch"]):
        pages = s["page_table"][b, :-(-lens[b] // ps)].long()
        k, v = (s[n][pages].double().permute(1, 0, 2, 3).reshape(c["kv_heads"], -1, d)[:, :lens[b]]
                for n in ("k_cache", "v_cache"))
        q = s["q"][b].double().view(c["kv_heads"], -1, d)
        w = torch.softmax(torch.bmm(q, k.transpose(1, 2)) / math.sqrt(d), -1)
        out[b] = torch.bmm(w, v).view(c["q_heads"], d)
    return out
