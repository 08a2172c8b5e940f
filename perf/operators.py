"""Measured cases of the serving operators around the quantized KV cache.

Three operators:

plan    one serving step's page bookkeeping: page tables, slot map, positions and offsets
        from request lengths, with a stack of free pages (pages of ended requests return).
prompt  causal attention of each request's new tokens (a prompt, a chunk of one, a handful
        of proposed tokens) over its paged, block-quantized cache.
prefix  decode attention, one token per request, for requests that share long prefixes:
        each attends to its group's prefix and then to its own positions.

The plain form is elementary torch in 32 bits; ``exact`` is written apart from it in 64.
"""
import math

import torch

own = False

FORMATS = ("q8_0", "q4_0", "lut4", "nvfp4")
# positive half of the 16-level minimum-error quantizer of N(0, 1) (Max 1960)
LEVELS16 = (0.1284, 0.3881, 0.6568, 0.9424, 1.2562, 1.6181, 2.0690, 2.7326)
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ------------------------------------------------------------------ cases

def listed():
    return [
        # every decode step of a mid-size server: one new token per request
        dict(name="plan_decode_b256", op="plan", batch=256, page_size=64, max_pages=1024, max_old=65536 - 64,
             max_new=1, ended=0.0),
        # a busy odd-sized batch: decodes, small chunks, and a tenth of the requests ending
        dict(name="plan_mixed_b1000", op="plan", batch=1000, page_size=128, max_pages=40, max_old=4000,
             max_new=37, ended=0.1),
        # a wave of prompts: most of the work is the slot map
        dict(name="plan_prompts_b61", op="plan", batch=61, page_size=64, max_pages=128, max_old=3,
             max_new=8100, ended=0.0),
        # verification of four proposed tokens per request at long contexts
        dict(name="prompt_verify_b8", op="prompt", fmt="q8_0", head_dim=128, kv_heads=8, group=4, batch=8, page_size=64,
             min_new=4, max_new=4, min_old=7000, max_old=16384),
        # two chunks of a chunked prefill in the middle of their prompts
        dict(name="prompt_chunk_b2", op="prompt", fmt="q4_0", head_dim=128, kv_heads=4, group=8, batch=2, page_size=64,
             min_new=500, max_new=512, min_old=6000, max_old=8192),
        # a ragged batch of short prompts, small heads, odd group
        dict(name="prompt_ragged_b37_d64", op="prompt", fmt="nvfp4", head_dim=64, kv_heads=4, group=7, batch=37,
             page_size=192, min_new=1, max_new=700, min_old=0, max_old=1000),
        # one long prompt from the start
        dict(name="prompt_8k", op="prompt", fmt="q8_0", head_dim=128, kv_heads=8, group=4, batch=1, page_size=64,
             min_new=8192, max_new=8192, min_old=0, max_old=0),
        # a few users on one system prompt: latency
        dict(name="prefix_4k_b4", op="prefix", fmt="q4_0", head_dim=128, kv_heads=8, group=4, batch=4, groups=1,
             page_size=64, prefix=4096, max_own=200),
        # a server's batch on one long document
        dict(name="prefix_32k_b64", op="prefix", fmt="q4_0", head_dim=128, kv_heads=4, group=8, batch=64, groups=1,
             page_size=64, prefix=32768, max_own=1024),
        # three documents with ragged groups, rotated codebook, odd lengths
        dict(name="prefix_groups_b93_lut4", op="prefix", fmt="lut4", head_dim=128, kv_heads=8, group=5, batch=93,
             groups=3, page_size=64, prefix=9973, max_own=333),
        # many samples from one short prompt, small heads
        dict(name="prefix_2k_b200_nvfp4", op="prefix", fmt="nvfp4", head_dim=64, kv_heads=2, group=8, batch=200,
             groups=1, page_size=128, prefix=2047, max_own=500),
        # the largest: a big batch on a 64K prefix
        dict(name="prefix_64k_b256", op="prefix", fmt="q8_0", head_dim=128, kv_heads=4, group=8, batch=256, groups=1,
             page_size=64, prefix=65536, max_own=512),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def _plain_size(c):
    """Scores that the plain form holds at once."""
    heads = c["kv_heads"] * c["group"]
    if c["op"] == "prompt":
        return c["batch"] * heads * c["max_new"] * (c["max_old"] + c["max_new"])
    return heads * c["batch"] * (c["prefix"] * min(c["groups"], 2) + c["max_own"])


def draw(rng):
    op = rng.choice(("plan", "prompt", "prompt", "prefix", "prefix"))
    if op == "plan":
        ps = rng.choice((64, 128, 192))
        batch = _log(rng, 1, 1024)
        max_new = rng.choice((1, _log(rng, 2, 40), _log(rng, 2, max(2, 240000 // batch))))
        max_old = _log(rng, 1, 30000)
        return dict(op=op, batch=batch, page_size=ps, max_pages=(max_old + max_new) // ps + rng.randint(1, 9),
                    max_old=max_old, max_new=max_new, ended=rng.choice((0.0, 0.0, 0.2)))
    while True:
        c = dict(op=op, fmt=rng.choice(FORMATS), head_dim=rng.choice((64, 128, 128)), kv_heads=rng.randint(1, 8),
                 group=rng.randint(1, 8), page_size=rng.choice((64, 64, 128, 192)))
        if op == "prompt":
            max_new, max_old = _log(rng, 1, 6000), rng.choice((0, _log(rng, 1, 20000)))
            c.update(batch=_log(rng, 1, 40), min_new=rng.choice((0, max_new // 2, max_new)), max_new=max_new,
                     min_old=rng.choice((0, max_old // 2)), max_old=max_old)
        else:
            c.update(batch=_log(rng, 1, 300), groups=rng.choice((1, 1, 2, 5)), prefix=_log(rng, 64, 50000),
                     max_own=rng.choice((1, _log(rng, 1, 1000))))
            c["groups"] = min(c["groups"], c["batch"])
        if _plain_size(c) <= 1000000000 and work(c)["flops"] <= 2.5e11:
            return c


# ------------------------------------------------------------------ inputs

def _lengths(case):
    """Request lengths of a case, from the case alone (host): work() and prepare() agree on them."""
    g = torch.Generator().manual_seed(1234 + 7 * case["batch"])
    b = case["batch"]
    if case["op"] == "prompt":
        new = torch.randint(case["min_new"], case["max_new"] + 1, (b,), generator=g)
        old = torch.randint(case["min_old"], case["max_old"] + 1, (b,), generator=g)
        new[0] = case["max_new"]
        return old, new
    n = case["groups"]
    prefix = torch.randint(case["prefix"] // 2, case["prefix"] + 1, (n,), generator=g)
    prefix[0] = case["prefix"]
    own_lens = torch.randint(1, case["max_own"] + 1, (b,), generator=g)
    cuts = torch.sort(torch.randperm(b - 1, generator=g)[:n - 1] + 1)[0] if n > 1 else torch.zeros(0, dtype=torch.int64)
    offsets = torch.cat((torch.zeros(1, dtype=torch.int64), cuts, torch.tensor([b])))
    return prefix, own_lens, offsets


def _row_bytes(fmt, d):
    codes = d if fmt == "q8_0" else d // 2
    scales = {"q8_0": d // 16, "q4_0": d // 16, "lut4": 2, "nvfp4": (d // 16 + 11) // 8 * 8}[fmt]
    return codes, scales


def _hadamard(d, device, dtype):
    h = torch.ones(1, 1, device=device, dtype=dtype)
    while h.shape[0] < d:
        h = torch.cat((torch.cat((h, h), 1), torch.cat((h, -h), 1)), 0)
    return h / math.sqrt(d)


def _quantize(fmt, x, codebook, signs):
    """Codes (uint8) and scale rows (fp16 slots) of fp32 vectors x[..., D], as the cache stores them."""
    d = x.shape[-1]
    if fmt in ("q8_0", "q4_0"):
        xb = x.unflatten(-1, (d // 32, 32))
        if fmt == "q8_0":
            s = xb.abs().amax(-1) / 127
            q = torch.round(xb / s.clamp_min(1e-30).unsqueeze(-1)).clamp(-127, 127).to(torch.int8).flatten(-2)
            return q.view(torch.uint8), s.half()
        m = torch.take_along_dim(xb, xb.abs().argmax(-1, keepdim=True), -1).squeeze(-1)
        s = m / -8
        q = torch.floor(xb / torch.where(s == 0, 1.0, s).unsqueeze(-1) + 8.5).clamp(0, 15).to(torch.uint8).flatten(-2)
        s = s.half()
    elif fmt == "lut4":
        y = (x * signs.float()) @ _hadamard(d, x.device, torch.float32)
        s = y.norm(dim=-1, keepdim=True)
        cb = codebook.float()
        q = torch.bucketize(y / s.clamp_min(1e-30), (cb[1:] + cb[:-1]) / 2).to(torch.uint8)
        s = s.half()
    else:
        g = x.abs().amax(-1, keepdim=True) / 2688
        xb = x.unflatten(-1, (d // 16, 16))
        e = (xb.abs().amax(-1) / (6 * g).clamp_min(1e-30)).to(torch.float8_e4m3fn)
        t = xb / (e.float() * g).clamp_min(1e-30).unsqueeze(-1)
        v = torch.tensor(E2M1, device=x.device)
        q = (torch.bucketize(t.abs(), (v[1:] + v[:-1]) / 2) + 8 * (t < 0)).to(torch.uint8).flatten(-2)
        row = torch.zeros(x.shape[:-1] + (_row_bytes(fmt, d)[1],), dtype=torch.uint8, device=x.device)
        row[..., :d // 16] = e.view(torch.uint8)
        row[..., d // 16:d // 16 + 4] = g.contiguous().view(torch.uint8)
        s = row.view(torch.float16)
    return q[..., 0::2] | (q[..., 1::2] << 4), s


def _plan_inputs(case, gen, dev):
    b, ps, mp = case["batch"], case["page_size"], case["max_pages"]
    old = torch.randint(0, case["max_old"] + 1, (b,), generator=gen, device=dev)
    new = torch.randint(1, case["max_new"] + 1, (b,), generator=gen, device=dev)
    new[torch.rand(b, generator=gen, device=dev) < case["ended"]] = -1
    pages = (old + ps - 1) // ps
    used = int(pages.sum())
    num_pages = b * ((case["max_old"] + case["max_new"] + ps - 1) // ps) + 100  # every request at its longest, and some more
    order = torch.randperm(num_pages, generator=gen, device=dev).int()
    table = torch.full((b, mp), -1, dtype=torch.int32, device=dev)
    table[torch.arange(mp, device=dev) < pages.unsqueeze(1)] = order[:used]
    free = torch.zeros(num_pages, dtype=torch.int32, device=dev)
    free[:num_pages - used] = order[used:]
    return dict(op="plan", page_size=ps, num_pages=num_pages, seq_lens=old.int(), new_lens=new.int(), page_table=table,
                free_pages=free, free_count=torch.tensor([num_pages - used], dtype=torch.int32, device=dev),
                max_tokens=b * case["max_new"])


def _inputs(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(int(seed) * 1000003 + 17)
    if case["op"] == "plan":
        return _plan_inputs(case, gen, dev)
    fmt, d, hkv, ps, b = case["fmt"], case["head_dim"], case["kv_heads"], case["page_size"], case["batch"]
    hq = hkv * case["group"]
    # rows of pages: the requests' own, then the shared prefixes'
    if case["op"] == "prompt":
        old, new = _lengths(case)
        lens, prefix, offsets = old + new, torch.zeros(0, dtype=torch.int64), None
        tokens = int(new.sum())
    else:
        prefix, lens, offsets = _lengths(case)
        tokens = b
    rows = (torch.cat((lens, prefix)) + ps - 1) // ps
    num_pages, max_pages = int(rows.sum()) + 3, max(1, int(rows.max()))
    table = torch.full((rows.numel(), max_pages), -1, dtype=torch.int32, device=dev)
    table[torch.arange(max_pages, device=dev) < rows.to(dev).unsqueeze(1)] = \
        torch.randperm(num_pages, generator=gen, device=dev)[:int(rows.sum())].int()
    # keys and queries share a direction: some keys (about 1 in 500) score high for every query
    u = torch.where(torch.rand(d, generator=gen, device=dev) < 0.5, -1.0, 1.0)
    k = torch.randn(num_pages, hkv, ps, d, generator=gen, device=dev)
    strong = torch.rand(num_pages, hkv, ps, 1, generator=gen, device=dev)
    k += torch.where(strong < 0.002, 0.7 + 500 * strong, 0.0) * u
    v = torch.randn(num_pages, hkv, ps, d, generator=gen, device=dev)
    q = (torch.randn(tokens, hq, d, generator=gen, device=dev) + 0.7 * u).half()
    signs = torch.where(torch.rand(d, generator=gen, device=dev) < 0.5, -1, 1).to(torch.int8)
    half = torch.tensor(LEVELS16, device=dev) / math.sqrt(d)
    codebook = torch.cat((-half.flip(0), half)).half()
    kc, ks = _quantize(fmt, k.half().float(), codebook, signs)
    vc, vs = _quantize(fmt, v.half().float(), codebook, signs)
    del k, v, strong
    state = dict(op=case["op"], fmt=fmt, head_dim=d, kv_heads=hkv, page_size=ps, q=q, k_codes=kc, k_scales=ks,
                 v_codes=vc, v_scales=vs, codebook=codebook, signs=signs, seq_lens=lens.int().to(dev),
                 page_table=table[:b].contiguous(), max_pages=max_pages, max_seq_len=int(lens.max()))
    if case["op"] == "prompt":
        state["token_offsets"] = torch.cat((torch.zeros(1, dtype=torch.int64), new.cumsum(0))).int().to(dev)
        state["max_new"] = int(new.max())
    else:
        state.update(prefix_table=table[b:].contiguous(), prefix_lens=prefix.int().to(dev),
                     max_prefix_len=int(prefix.max()), group_offsets=offsets.int().to(dev),
                     max_group=int((offsets[1:] - offsets[:-1]).max()))
    return state


def prepare(case, seed):
    s = _inputs(case, seed)
    if own:  # the handles that a user's program keeps: a planner, a cache filled earlier
        import quantized_kv_cache_split_b200 as kvq
        if case["op"] == "plan":
            b, max_pages = s["page_table"].shape
            s["planner"] = kvq.PagePlanner(b, s["page_size"], s["num_pages"], max_pages, s["max_tokens"], s["seq_lens"].device)
        else:
            s["cache"] = kvq.QuantizedKVCache(s["fmt"], s["head_dim"], s["kv_heads"], s["page_size"], s["k_codes"].shape[0],
                                              s["q"].device, s["codebook"], s["signs"])
            for plane in ("k_codes", "k_scales", "v_codes", "v_scales"):
                getattr(s["cache"], plane).copy_(s.pop(plane))
    return s


# ------------------------------------------------------------------ the plain form

def _values(s, which, table):
    """fp32 values [rows, positions, heads, D] of the pages of a table (negative entries: page 0, masked later)."""
    t = table.long().clamp_min(0)
    codes = s[which + "_codes"][t].transpose(2, 3).flatten(1, 2)      # [rows, positions, heads, bytes]
    scales = s[which + "_scales"][t].transpose(2, 3).flatten(1, 2)
    d = s["head_dim"]
    if s["fmt"] == "q8_0":
        return codes.view(torch.int8).float() * scales.float().repeat_interleave(32, -1)
    q = torch.stack((codes & 15, codes >> 4), -1).flatten(-2)
    if s["fmt"] == "q4_0":
        return (q.float() - 8) * scales.float().repeat_interleave(32, -1)
    if s["fmt"] == "lut4":
        return s["codebook"].float()[q.long()] * scales.float()
    raw = scales.contiguous().view(torch.uint8)
    e = raw[..., :d // 16].contiguous().view(torch.float8_e4m3fn).float().repeat_interleave(16, -1)
    g = raw[..., d // 16:d // 16 + 4].contiguous().view(torch.float32)
    levels = torch.tensor(E2M1 + tuple(-x for x in E2M1), device=q.device)
    return levels[q.long()] * e * g


def _rotate(s, x, back=False):
    if s["fmt"] != "lut4":
        return x
    h, signs = _hadamard(s["head_dim"], x.device, x.dtype), s["signs"].to(x.dtype)
    return (x @ h) * signs if back else (x * signs) @ h


def _softmax_parts(parts):
    """exp weights of score parts along their last axes under a common maximum, and the sums (1 where a row is empty)."""
    m = torch.stack([p.amax(-1) for p in parts]).amax(0)
    m = torch.where(m == -math.inf, 0.0, m).unsqueeze(-1)
    e = [torch.exp(p - m) for p in parts]
    z = torch.stack([x.sum(-1) for x in e]).sum(0).unsqueeze(-1)
    return e, torch.where(z == 0, 1.0, z)


def _plain_prompt(s):
    d, hkv = s["head_dim"], s["kv_heads"]
    off, lens = s["token_offsets"].long(), s["seq_lens"].long()
    new, dev = off[1:] - off[:-1], off.device
    b, n, total = new.numel(), s["max_new"], s["q"].shape[0]
    req = torch.repeat_interleave(torch.arange(b, device=dev), new, output_size=total)
    i = torch.arange(total, device=dev) - off[req]
    q = torch.zeros(b, n, hkv, s["q"].shape[1] // hkv, d, device=dev)
    q[req, i] = _rotate(s, s["q"].float()).unflatten(1, (hkv, -1))
    pages = (s["max_seq_len"] + s["page_size"] - 1) // s["page_size"]
    k = _values(s, "k", s["page_table"][:, :pages])
    p = torch.matmul(q.permute(0, 2, 3, 1, 4), k.permute(0, 2, 3, 1).unsqueeze(2)) / math.sqrt(d)  # [b, hkv, g, n, pos]
    last = (lens - new).unsqueeze(1) + torch.arange(n, device=dev)
    p.masked_fill_((torch.arange(p.shape[-1], device=dev) > last.unsqueeze(-1))[:, None, None], -math.inf)
    (p,), z = _softmax_parts([p])
    o = torch.matmul(p, _values(s, "v", s["page_table"][:, :pages]).permute(0, 2, 1, 3).unsqueeze(2)) / z
    return _rotate(s, o.permute(0, 3, 1, 2, 4).flatten(2, 3)[req, i], back=True).half()


def _plain_prefix(s):
    d, hkv, dev = s["head_dim"], s["kv_heads"], s["q"].device
    b, hq, off = s["q"].shape[0], s["q"].shape[1], s["group_offsets"].long()
    ng, ps = off.numel() - 1, s["page_size"]
    grp = torch.repeat_interleave(torch.arange(ng, device=dev), off[1:] - off[:-1], output_size=b)
    i = torch.arange(b, device=dev) - off[grp]
    q = _rotate(s, s["q"].float()).unflatten(1, (hkv, hq // hkv))                                   # [b, hkv, g, d]
    qg = torch.zeros(ng, s["max_group"], hkv, hq // hkv, d, device=dev)
    qg[grp, i] = q
    tab = s["prefix_table"][:, :(s["max_prefix_len"] + ps - 1) // ps]
    sp = torch.matmul(qg.permute(0, 2, 1, 3, 4).flatten(2, 3), _values(s, "k", tab).permute(0, 2, 3, 1))
    sp = sp.unflatten(2, (s["max_group"], -1)).permute(0, 2, 1, 3, 4)[grp, i] / math.sqrt(d)        # [b, hkv, g, pos]
    sp.masked_fill_((torch.arange(sp.shape[-1], device=dev) >= s["prefix_lens"].long()[grp].unsqueeze(1))[:, None, None],
                    -math.inf)
    own_tab = s["page_table"][:, :(s["max_seq_len"] + ps - 1) // ps]
    so = torch.matmul(q, _values(s, "k", own_tab).permute(0, 2, 3, 1)) / math.sqrt(d)
    so.masked_fill_((torch.arange(so.shape[-1], device=dev) >= s["seq_lens"].long().unsqueeze(1))[:, None, None], -math.inf)
    (sp, so), z = _softmax_parts([sp, so])
    pg = torch.zeros((ng, s["max_group"]) + sp.shape[1:], device=dev)
    pg[grp, i] = sp
    op = torch.matmul(pg.permute(0, 2, 1, 3, 4).flatten(2, 3), _values(s, "v", tab).permute(0, 2, 1, 3))
    op = op.unflatten(2, (s["max_group"], -1)).permute(0, 2, 1, 3, 4)[grp, i]
    oo = torch.matmul(so, _values(s, "v", own_tab).permute(0, 2, 1, 3))
    return _rotate(s, ((op + oo) / z).flatten(1, 2), back=True).half()


def _plain_plan(s):
    dev, ps = s["seq_lens"].device, s["page_size"]
    old, new = s["seq_lens"].long(), s["new_lens"].long()
    b, mp = s["page_table"].shape
    had = (old + ps - 1) // ps
    col = torch.arange(mp, device=dev)
    # pages of ended requests return to the top of the stack
    ended = new < 0
    back = s["page_table"][ended.unsqueeze(1) & (col < had.unsqueeze(1))]
    count = s["free_count"].long()
    free = s["free_pages"].clone()
    free[count + torch.arange(back.numel(), device=dev)] = back
    top = count + back.numel()
    # the j-th page needed comes from the top of the stack
    add = new.clamp_min(0)
    need = (old + add + ps - 1) // ps - had
    need = torch.where(ended, 0, need)
    first = need.cumsum(0) - need
    table = s["page_table"].clone()
    fresh = (col >= had.unsqueeze(1)) & (col < (had + need).unsqueeze(1))
    j = (first.unsqueeze(1) + col - had.unsqueeze(1))[fresh]
    table[fresh] = free[top - 1 - j]
    offsets = torch.cat((torch.zeros(1, dtype=torch.int64, device=dev), add.cumsum(0)))
    t = torch.arange(s["max_tokens"], device=dev)
    req = torch.searchsorted(offsets[1:], t, right=True).clamp_max(b - 1)
    live = t < offsets[-1]
    pos = torch.where(live, old[req] + t - offsets[req], 0)
    slots = torch.where(live, table[req, (pos // ps).clamp_max(mp - 1)].long() * ps + pos % ps, -1)
    return dict(page_table=table, seq_lens=torch.where(ended, 0, old + add).int(), token_offsets=offsets.int(),
                slots=slots.int(), positions=pos.int(), free_pages=free, free_count=(top - need.sum()).int())


# ------------------------------------------------------------------ one pass

def run(state):
    s = state
    if not own:
        return {"plan": _plain_plan, "prompt": _plain_prompt, "prefix": _plain_prefix}[s["op"]](s)
    if s["op"] == "plan":
        p = s["planner"]
        p.step(s["new_lens"], s["page_table"], s["seq_lens"], s["free_pages"], s["free_count"])
        return dict(page_table=s["page_table"], seq_lens=p.seq_lens, token_offsets=p.token_offsets, slots=p.slots,
                    positions=p.positions, free_pages=s["free_pages"], free_count=p.free_count)
    if s["op"] == "prompt":
        return s["cache"].prompt_attention(s["q"], s["token_offsets"], s["seq_lens"], s["max_seq_len"], s["page_table"],
                                           s["max_pages"], out_dtype=torch.float16)
    return s["cache"].prefix_attention(s["q"], s["prefix_table"], s["prefix_lens"], s["max_prefix_len"], s["seq_lens"],
                                       s["max_seq_len"], s["page_table"], s["max_pages"],
                                       group_offsets=s["group_offsets"], out_dtype=torch.float16)


# ------------------------------------------------------------------ what a pass cannot do without

def work(case):
    if case["op"] == "plan":
        # lengths in and out, offsets, slots and positions, about half of the new pages' entries twice
        b, tokens = case["batch"], case["batch"] * case["max_new"]
        pages = tokens // 2 // case["page_size"] + 1
        return {"bytes": 4 * (4 * b + 2 * tokens + 2 * pages), "flops": 0}
    d, hkv, hq = case["head_dim"], case["kv_heads"], case["kv_heads"] * case["group"]
    row = 2 * hkv * sum(_row_bytes(case["fmt"], d))
    if case["op"] == "prompt":
        old, new = (x.double() for x in _lengths(case))
        pairs, tokens, positions = float((new * old + new * (new + 1) / 2).sum()), float(new.sum()), float((old + new).sum())
    else:
        prefix, lens, off = _lengths(case)
        size = (off[1:] - off[:-1])
        pairs, tokens = float((prefix * size).sum() + lens.sum()), float(case["batch"])
        positions = float(prefix.sum() + lens.sum())
    return {"bytes": positions * row + tokens * hq * d * 4, "flops": 4.0 * pairs * hq * d}


# ------------------------------------------------------------------ the definition, in 64 bits

def _exact_rows(s, which, pages, n):
    """[n, heads, D] values of one sequence: its positions in order, read page by page."""
    pages = [int(p) for p in pages[:(n + s["page_size"] - 1) // s["page_size"]]]
    codes = torch.cat([s[which + "_codes"][p] for p in pages], 1)[:, :n].transpose(0, 1)
    scales = torch.cat([s[which + "_scales"][p] for p in pages], 1)[:, :n].transpose(0, 1).contiguous()
    d, fmt = s["head_dim"], s["fmt"]
    x = torch.empty(n, s["kv_heads"], d, dtype=torch.float64, device=codes.device)
    if fmt == "q8_0":
        x.copy_(codes.contiguous().view(torch.int8))
    else:
        lo, hi = codes % 16, codes // 16
        if fmt == "q4_0":
            x[..., 0::2], x[..., 1::2] = lo.double() - 8, hi.double() - 8
        else:
            of = s["codebook"].double() if fmt == "lut4" else torch.tensor(
                [(1 - 2 * (c // 8)) * E2M1[c % 8] for c in range(16)], dtype=torch.float64, device=codes.device)
            x[..., 0::2], x[..., 1::2] = of[lo.long()], of[hi.long()]
    if fmt == "lut4":
        return x * scales.double()
    if fmt == "nvfp4":
        by = scales.view(torch.uint8)
        per = by[..., :d // 16].contiguous().view(torch.float8_e4m3fn).double()
        vec = by[..., d // 16:d // 16 + 4].contiguous().view(torch.float32).double()
        return (x.view(n, -1, d // 16, 16) * per.unsqueeze(-1)).flatten(-2) * vec
    return (x.view(n, -1, d // 32, 32) * scales.double().unsqueeze(-1)).flatten(-2)


def _exact_plan(s):
    ps = s["page_size"]
    old, new = s["seq_lens"].tolist(), s["new_lens"].tolist()
    table, stack = s["page_table"].cpu().clone(), s["free_pages"].cpu().clone()
    n = int(s["free_count"])
    for b, a in enumerate(new):
        if a < 0:
            for j in range(-(-old[b] // ps)):
                stack[n] = table[b, j]
                n += 1
    slots, positions, offsets = [], [], [0]
    for b, a in enumerate(new):
        for j in range(-(-old[b] // ps), -(-(old[b] + max(a, 0)) // ps) if a > 0 else 0):
            n -= 1
            table[b, j] = stack[n]
        row = table[b].tolist()
        for p in range(old[b], old[b] + max(a, 0)):
            slots.append(row[p // ps] * ps + p % ps)
            positions.append(p)
        offsets.append(len(slots))
    rest = s["max_tokens"] - len(slots)
    ints = lambda v: torch.tensor(v, dtype=torch.int32)  # noqa: E731
    return dict(page_table=table, seq_lens=ints([o + a if a >= 0 else 0 for o, a in zip(old, new)]),
                token_offsets=ints(offsets), slots=ints(slots + [-1] * rest), positions=ints(positions + [0] * rest),
                free_pages=stack, free_count=ints([n]))


def exact(case, seed):
    s = _inputs(case, seed)
    if case["op"] == "plan":
        return _exact_plan(s)
    d, hkv, g = case["head_dim"], case["kv_heads"], case["group"]
    q = s["q"].double()
    had = torch.ones(1, 1, dtype=torch.float64, device=q.device)
    while had.shape[0] < d:
        had = torch.kron(torch.tensor([[1.0, 1.0], [1.0, -1.0]], dtype=torch.float64, device=q.device), had)
    turn = s["signs"].double().unsqueeze(1) * had / d ** 0.5 if case["fmt"] == "lut4" else None  # x' = x turn
    out = torch.zeros_like(q)

    def attend(rows, keys, values, last):
        """Rows of q over [n, heads, D] keys and values; row r sees the positions up to last[r] (None: all)."""
        qr = q[rows] if turn is None else q[rows] @ turn
        for h in range(hkv):
            w = torch.einsum("rgd,nd->rgn", qr[:, h * g:(h + 1) * g], keys[:, h]) / d ** 0.5
            if last is not None:
                hidden = torch.arange(keys.shape[0], device=q.device)[None] > last[:, None]
                w.masked_fill_(hidden.unsqueeze(1), -math.inf)
            w = torch.softmax(w, -1)
            o = torch.einsum("rgn,nd->rgd", w, values[:, h])
            out[rows, h * g:(h + 1) * g] = o if turn is None else o @ turn.T

    if case["op"] == "prompt":
        old, new = (x.tolist() for x in _lengths(case))
        at = 0
        for b in range(case["batch"]):
            n = old[b] + new[b]
            if new[b]:
                pages = s["page_table"][b].tolist()
                keys, values = _exact_rows(s, "k", pages, n), _exact_rows(s, "v", pages, n)
                for i in range(0, new[b], 1024):
                    rows = torch.arange(at + i, at + min(i + 1024, new[b]), device=q.device)
                    attend(rows, keys, values, old[b] + rows - at)
            at += new[b]
        return out
    prefix, lens, off = (x.tolist() for x in _lengths(case))
    for gi in range(case["groups"]):
        pages = s["prefix_table"][gi].tolist()
        pk, pv = _exact_rows(s, "k", pages, prefix[gi]), _exact_rows(s, "v", pages, prefix[gi])
        for b in range(off[gi], off[gi + 1]):
            own_pages = s["page_table"][b].tolist()
            keys = torch.cat((pk, _exact_rows(s, "k", own_pages, lens[b])))
            values = torch.cat((pv, _exact_rows(s, "v", own_pages, lens[b])))
            attend(torch.tensor([b], device=q.device), keys, values, None)
    return out
