"""Cases that measure the cache and attention operators around the retrieval path:

  append        new key and value rows quantised to 8 bits as they are written into the pages
  read          a range of an 8-bit cache read back as bf16 rows
  attn          one new token per sequence attending to every key of its paged cache
  block_select  the blocks that a mean-key score selects for each query
  block_attn    attention over the selected blocks, one list per query and KV group

Shapes follow the Llama-3.1-8B layout used throughout the repository (32 query heads over 8 KV
heads of 128 channels, pages of 32 keys, up to 128K keys) and its block indexer (blocks of 128
keys, 64 queries at a time); drawn cases vary every size around them.

An 8-bit cache holds, per key row and KV head, 128 e4m3 values and one exponent byte x: the row is
value * 2^(x - 127). The exponent is the smallest e in [-117, 119] with max|row| <= 448 * 2^e
(-117 for a row of zeros), so every row is divided by a power of two, exactly, and rounded once.
"""
import math

import torch

own = False

D = 128  # channels of a head
GOLD = 0.6180339887498949


# ------------------------------------------------------------------------------------- cases

def listed():
    base = {"heads": 32, "kv_heads": 8, "page": 32}
    return [
        # One generated token for each of 8 sequences of 32K keys: written, quantised, and the
        # mean of its page kept up to date for the block selection. Latency counts.
        dict(base, name="append_decode", op="append", batch=8, lo=32768, hi=32768, new=1,
             mean=True, fused_qkv=True),
        # A prefill of 4 prompts of 2K to 8K tokens, rows strided as a fused QKV product leaves them.
        dict(base, name="append_prefill", op="append", batch=4, lo=2048, hi=8192, new=8192,
             mean=False, fused_qkv=True),
        # A short shared prefix read back.
        dict(base, name="read_prefix", op="read", batch=1, page=16, lo=700, hi=700),
        # Four whole 32K caches read back (a cache that moves to another layout or another host).
        dict(base, name="read_32k", op="read", batch=4, lo=32768, hi=32768),
        # The first tokens of one conversation: 517 keys. Latency counts.
        dict(base, name="attn_short", op="attn", batch=1, lo=517, hi=517, kv8=False,
             append=False, out_bf16=False),
        # One 32K sequence whose new key and value are written by the same call.
        dict(base, name="attn_32k", op="attn", batch=1, lo=32768, hi=32768, kv8=False,
             append=True, out_bf16=False),
        # Eight sequences of 128K keys: the largest dense step.
        dict(base, name="attn_128k_b8", op="attn", batch=8, lo=131072, hi=131072, kv8=False,
             append=False, out_bf16=False),
        # A ragged serving batch over an 8-bit cache.
        dict(base, name="attn_ragged_kv8", op="attn", batch=16, lo=8192, hi=131072, kv8=True,
             append=False, out_bf16=True),
        # Block selection of one decode step at 128K: 256 of 4096 pages, one sink page and two
        # local pages forced.
        dict(base, name="select_128k_b8", op="block_select", batch=8, lo=131072, hi=131072,
             queries=1, keep=256, sink=1, local=2),
        # Block selection of a chunk of 64 queries over blocks of 128 keys.
        dict(base, name="select_chunk", op="block_select", batch=1, page=128, lo=131072,
             hi=131072, queries=64, keep=64, sink=0, local=1),
        # Attention over 64 selected pages of 128K keys, 8-bit cache, one token a sequence.
        dict(base, name="block_decode_kv8", op="block_attn", batch=8, lo=131072, hi=131072,
             queries=1, keep=64, kv8=True, out_bf16=True),
        # A chunk of 64 queries, each with its own 16 blocks of 128 keys for each KV head.
        dict(base, name="block_chunk", op="block_attn", batch=1, page=128, lo=131072, hi=131072,
             queries=64, keep=16, kv8=False, out_bf16=False),
    ]


def _spread(rng, lo, hi):
    """A whole number of [lo, hi], even over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["append", "read", "attn", "attn", "block_select", "block_attn"])
    kv_heads = rng.choice([1, 2, 4, 8])
    group = rng.choice([1, 2, 3, 4, 4, 5, 7, 8])
    page = rng.choice([5, 8, 16, 17, 32, 32, 64, 100, 128, 256])
    batch = _spread(rng, 1, 32)
    # Rows of all sequences and heads, bounded by half of the largest listed case.
    most = 131072 if op in ("attn", "block_select", "block_attn") else 32768
    hi = _spread(rng, 1, max(1, min(most, 4 * 131072 * 8 // (batch * kv_heads))))
    if op == "block_select":
        hi = max(hi, 64 * page)  # a choice among enough blocks
    c = {"op": op, "heads": kv_heads * group, "kv_heads": kv_heads, "page": page, "batch": batch,
         "lo": rng.randint(1, hi), "hi": hi}
    pages = -(-hi // page)
    if op == "append":
        c.update(new=_spread(rng, 1, max(1, min(hi, 32768 * 8 // (batch * kv_heads)))),
                 mean=rng.random() < 0.5, fused_qkv=rng.random() < 0.5)
    elif op == "attn":
        c.update(kv8=rng.random() < 0.5, append=rng.random() < 0.3 and batch * hi <= 1 << 18,
                 out_bf16=rng.random() < 0.5)
    elif op in ("block_select", "block_attn"):
        queries = _spread(rng, 1, max(1, 64 // batch))
        if op == "block_attn":
            keep = _spread(rng, 1, max(1, min(256, pages)))
            # Selected rows of all queries, bounded by the listed chunk.
            keep = max(1, min(keep, 64 * 8 * 2048 // (batch * queries * kv_heads * page)))
            c.update(queries=queries, keep=keep, kv8=rng.random() < 0.5,
                     out_bf16=rng.random() < 0.5)
        else:
            c.update(queries=queries, keep=_spread(rng, 4, min(256, pages // 2)),
                     sink=rng.choice([0, 1]), local=rng.choice([0, 1, 2]))
    return c


def _lens(case):
    """Keys of each sequence after the call: between lo and hi, the first one hi."""
    lo, hi = case["lo"], case["hi"]
    return [hi - int((hi - lo) * ((b * GOLD) % 1.0)) for b in range(case["batch"])]


def _news(case):
    """Appended rows of each sequence: at most "new", and at most its length."""
    return [min(case["new"], n) for n in _lens(case)]


def work(case):
    G, H, P, B = case["kv_heads"], case["heads"], case["page"], case["batch"]
    lens, op = _lens(case), case["op"]
    row = 2 * (D + 1 if case.get("kv8") else 2 * D)  # K and V of one key and head
    if op == "append":
        news = _news(case)
        n = sum(news)
        b = n * G * (4 * D + 2 * (D + 1))
        if case["mean"]:  # the rows that the first touched page held, and the means
            b += sum(((l - k) % P) * G * (D + 1) + (-(-l // P) - (l - k) // P) * G * 4 * D
                     for l, k in zip(lens, news))
        return {"bytes": b, "flops": 4 * n * G * D}
    if op == "read":
        return {"bytes": sum(lens) * G * (2 * (D + 1) + 4 * D), "flops": 2 * sum(lens) * G * D}
    if op == "attn":
        b = sum(lens) * G * row + B * H * D * (2 + (2 if case["out_bf16"] else 4))
        return {"bytes": b, "flops": 4 * sum(lens) * H * D}
    T, keep = case["queries"], case["keep"]
    if op == "block_select":
        pages = sum(-(-n // P) for n in lens)
        b = pages * G * D * 4 + B * T * H * D * 2 + B * T * G * keep * 4
        return {"bytes": b, "flops": 2 * pages * T * G * D}
    keys = [min(n, T * keep * P) for n in lens]
    each = [min(n, keep * P) for n in lens]
    b = sum(keys) * G * row + B * T * H * D * (2 + (2 if case["out_bf16"] else 4))
    return {"bytes": b, "flops": 4 * sum(each) * T * H * D}


# ------------------------------------------------------------------------------------ inputs

def _pow2(e):
    """2^e as float32 for a whole-number tensor e of [-126, 127], exactly."""
    return ((e.to(torch.int32) + 127) << 23).view(torch.float32)


def _quantise(x):
    """e4m3 values and exponent bytes of float32 rows."""
    m, ex = torch.frexp(x.abs().amax(-1, keepdim=True))  # max = m 2^ex; 448 = 0.875 * 2^9
    e = torch.where(m > 0, ex - 9 + (m > 0.875), torch.full_like(ex, -117)).clamp(-117, 119)
    return (x * _pow2(-e)).to(torch.float8_e4m3fn), (e.squeeze(-1) + 127).to(torch.uint8)


def _positions(case, lens, dev):
    """A chunk's queries are the last ones of the sequence."""
    T = case["queries"]
    back = torch.arange(T - 1, -1, -1, device=dev)
    return (lens[:, None] - 1 - back[None]).clamp(min=0).to(torch.int32).contiguous()


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed)
    G, H, P, B = case["kv_heads"], case["heads"], case["page"], case["batch"]
    lens_h = _lens(case)
    lens = torch.tensor(lens_h, dtype=torch.int32, device=dev)
    pages = [-(-n // P) for n in lens_h]
    maxp, n_phys = max(pages), sum(pages) + 3
    # Every sequence's pages lie anywhere in the pool; columns past its pages hold -1.
    order = torch.randperm(n_phys, generator=gen, device=dev).to(torch.int32)
    page_table = torch.full((B, maxp), -1, dtype=torch.int32, device=dev)
    at = 0
    for b, n in enumerate(pages):
        page_table[b, :n] = order[at:at + n]
        at += n
    s = {"case": case, "seq_len": lens, "page_table": page_table, "n_phys": n_phys}

    def rows(*shape):
        return torch.randn(*shape, D, generator=gen, device=dev, dtype=torch.bfloat16)

    def keys(*shape):  # a few channels of larger size, as keys have them
        k = rows(*shape)
        k[..., 3::41] *= 6
        return k

    op = case["op"]
    if op == "block_select":
        mean = keys(n_phys, G).float() / math.sqrt(P)
        # Means of real keys are not bf16 numbers.
        mean += 0.01 * torch.randn(mean.shape, generator=gen, device=dev)
        s["block_mean"] = mean
        s["q"] = rows(B, case["queries"], H)
        s["q_pos"] = _positions(case, lens, dev)
        s["blocks"] = torch.empty(B, case["queries"], G, min(case["keep"], maxp),
                                  dtype=torch.int32, device=dev)
        s["count"] = torch.empty(B, case["queries"], G, dtype=torch.int32, device=dev)
        return s
    k, v = keys(n_phys, G, P), rows(n_phys, G, P)
    if case.get("kv8", True):
        (s["k"], s["k_exp"]), (s["v"], s["v_exp"]) = _quantise(k.float()), _quantise(v.float())
    else:
        s["k"], s["v"], s["k_exp"], s["v_exp"] = k, v, None, None
    if op == "append":
        news = torch.tensor(_news(case), dtype=torch.int32, device=dev)
        s["start"], s["n_new"] = lens - news, news
        n = int(case["new"])
        if case["fused_qkv"]:
            qkv = rows(B, n, H + 2 * G)
            s["k_new"], s["v_new"] = qkv[:, :, H:H + G], qkv[:, :, H + G:]
        else:
            s["k_new"], s["v_new"] = keys(B, n, G), rows(B, n, G)
        s["block_mean"] = (torch.zeros(n_phys, G, D, device=dev) if case["mean"] else None)
        return s
    if op == "read":
        s["start"] = torch.zeros_like(lens)
        # Rows past a sequence's end stay as the caller left them.
        s["k_out"] = torch.zeros(B, max(lens_h), G, D, dtype=torch.bfloat16, device=dev)
        s["v_out"] = torch.zeros_like(s["k_out"])
        return s
    T = case.get("queries")
    s["scale"] = 1.0 / math.sqrt(D)
    shape = (B, H) if T is None else (B, T, H)
    s["q"] = rows(*shape)
    s["out"] = torch.empty(*shape, D, device=dev,
                           dtype=torch.bfloat16 if case["out_bf16"] else torch.float32)
    s["lse"] = torch.empty(*shape, device=dev)
    if op == "attn":
        s["k_new"] = keys(B, G) if case["append"] else None
        s["v_new"] = rows(B, G) if case["append"] else None
        return s
    # The blocks of each query and KV head: a random choice of its eligible ones, ascending.
    s["q_pos"] = _positions(case, lens, dev)
    m = min(case["keep"], maxp)
    n = s["q_pos"].clamp(min=0) // P + 1                                       # [B, T]
    r = torch.rand(B, T, G, maxp, generator=gen, device=dev)
    r.masked_fill_(torch.arange(maxp, device=dev) >= n[:, :, None, None], 2.0)
    pick = r.argsort(-1)[..., :m]
    count = n.clamp(max=m)[:, :, None].expand(B, T, G)
    far = torch.arange(m, device=dev) >= count[..., None]
    pick = pick.masked_fill(far, maxp).sort(-1).values
    s["blocks"] = pick.masked_fill(pick >= maxp, -1).to(torch.int32).contiguous()
    s["count"] = count.to(torch.int32).contiguous()
    return s


# ------------------------------------------------------------------------------ plain forms

def _values(s, name, at):
    """The float32 rows that cache `name` stands for at the index `at`."""
    if s[name + "_exp"] is None:
        return s[name][at].float()
    x = s[name].view(torch.uint8)[at].view(torch.float8_e4m3fn).float()
    return x * _pow2(s[name + "_exp"][at].to(torch.int32) - 127)[..., None]


def _gathered(s, name, pages):
    """float32 rows [..., G, P, D] of the physical pages `pages` (-1: any page, masked later)."""
    return _values(s, name, (pages.clamp(min=0).long(),))


def _softmax_rows(q, k, v, ok, scale):
    """Attention of q [..., h, D] over rows k, v [..., n, D], where ok [..., n]; and the
    logarithm of the weights' sum. A row with no key gives zeros and -inf."""
    x = (q @ k.transpose(-1, -2)) * scale
    x = x.masked_fill(~ok[..., None, :], -math.inf)
    lse = torch.logsumexp(x, -1)
    p = torch.exp(x - torch.where(torch.isinf(lse), torch.zeros_like(lse), lse)[..., None])
    return p @ v.masked_fill(~ok[..., None], 0.0), lse


def _slots(s, pos):
    """(physical page, slot) of the positions pos [B, n] of each sequence."""
    P = s["case"]["page"]
    return s["page_table"].gather(1, (pos // P).clamp(max=s["page_table"].shape[1] - 1)), pos % P


def _plain_append(s):
    B, n, G, _ = s["k_new"].shape
    i = torch.arange(n, device=s["k_new"].device)
    ok = i[None] < s["n_new"][:, None]
    phys, slot = _slots(s, (s["start"][:, None] + i[None]).long())
    phys, slot = phys[ok].long(), slot[ok].long()
    for name in ("k", "v"):
        q, e = _quantise(s[name + "_new"][ok].float())
        # Byte views: an indexed write of 8-bit floats.
        s[name].view(torch.uint8)[phys, :, slot] = q.view(torch.uint8)
        s[name + "_exp"][phys, :, slot] = e
    outs = [s["k"], s["v"], s["k_exp"], s["v_exp"]]
    if s["block_mean"] is not None:
        P, pt = s["case"]["page"], s["page_table"]
        end = s["start"] + s["n_new"]
        j = torch.arange(pt.shape[1], device=pt.device)
        hit = (j[None] >= (s["start"] // P)[:, None]) & (j[None] * P < end[:, None])
        x = _gathered(s, "k", pt[hit])                                       # [hits, G, P, D]
        valid = (end[:, None] - j[None] * P).clamp(max=P)[hit]
        ok = torch.arange(P, device=pt.device)[None] < valid[:, None]
        x = x.masked_fill(~ok[:, None, :, None], 0.0)
        s["block_mean"][pt[hit].long()] = x.sum(2) / valid[:, None, None]
        outs.append(s["block_mean"])
    return outs


def _plain_read(s):
    n = s["k_out"].shape[1]
    i = torch.arange(n, device=s["k_out"].device)
    ok = i[None] < s["seq_len"][:, None]
    phys, slot = _slots(s, i[None].expand(len(ok), n))
    phys, slot = phys[ok].long(), slot[ok]
    for name in ("k", "v"):
        x = _values(s, name, (phys, slice(None), slot))
        s[name + "_out"][ok] = x.to(torch.bfloat16)
    return [s["k_out"], s["v_out"]]


def _plain_attn(s):
    c = s["case"]
    B, G, P = c["batch"], c["kv_heads"], c["page"]
    pt, n = s["page_table"], s["seq_len"].long()
    outs = []
    if s["k_new"] is not None:
        phys, slot = _slots(s, (n - 1)[:, None])
        phys, slot = phys[:, 0].long(), slot[:, 0]
        for name in ("k", "v"):
            if c["kv8"]:
                q, e = _quantise(s[name + "_new"].float())
                s[name].view(torch.uint8)[phys, :, slot] = q.view(torch.uint8)
                s[name + "_exp"][phys, :, slot] = e
                outs += [s[name], s[name + "_exp"]]
            else:
                s[name][phys, :, slot] = s[name + "_new"]
                outs.append(s[name])
    k, v = (_gathered(s, name, pt).transpose(1, 2).reshape(B, G, -1, D) for name in ("k", "v"))
    ok = (torch.arange(pt.shape[1] * P, device=pt.device) < n[:, None])[:, None].expand(B, G, -1)
    o, lse = _softmax_rows(s["q"].float().reshape(B, G, -1, D), k, v, ok, s["scale"])
    return [o.reshape(B, -1, D).to(s["out"].dtype), lse.reshape(B, -1)] + outs


def _plain_block_select(s):
    c = s["case"]
    B, G, P, T = c["batch"], c["kv_heads"], c["page"], c["queries"]
    pt, m = s["page_table"], s["blocks"].shape[-1]
    # 64 bits: a choice hangs on which of two close scores is the larger.
    mean = s["block_mean"][pt.clamp(min=0).long()].double()                       # [B, p, G, D]
    q = s["q"].double().reshape(B, T, G, -1, D).sum(3)
    x = torch.einsum("btgd,bpgd->btgp", q, mean).float()
    limit = torch.minimum(s["seq_len"][:, None], s["q_pos"] + 1).clamp(min=0)
    n = ((limit + P - 1) // P)[:, :, None, None]                                  # [B, T, 1, 1]
    p = torch.arange(pt.shape[1], device=pt.device)
    x = torch.where(torch.isnan(x), torch.full_like(x, -math.inf), x)   # never chosen
    forced = (p < c["sink"]) | (p >= n - c["local"])
    x = torch.where(forced, torch.full_like(x, math.inf), x)
    x = torch.where(p < n, x, torch.full_like(x, -math.inf))
    pick = x.sort(dim=-1, descending=True, stable=True).indices[..., :m]
    count = (x > -math.inf).sum(-1, keepdim=True).clamp(max=m)
    far = torch.arange(m, device=pt.device) >= count
    pick = pick.masked_fill(far, 1 << 30).sort(-1).values
    return [pick.masked_fill(pick >= 1 << 30, -1).to(torch.int32),
            count.squeeze(-1).to(torch.int32)]


def _plain_block_attn(s):
    c = s["case"]
    B, G, P, T = c["batch"], c["kv_heads"], c["page"], c["queries"]
    blocks, m = s["blocks"].long(), s["blocks"].shape[-1]
    dev = blocks.device
    b = torch.arange(B, device=dev)[:, None, None, None]
    g = torch.arange(G, device=dev)[:, None]
    phys = s["page_table"][b, blocks.clamp(min=0)].clamp(min=0).long()            # [B, T, G, m]

    k, v = (_values(s, name, (phys, g)).reshape(B, T, G, m * P, D) for name in ("k", "v"))
    limit = torch.minimum(s["seq_len"][:, None], s["q_pos"] + 1)[:, :, None, None, None]
    pos = blocks[..., None] * P + torch.arange(P, device=dev)
    listed_ = torch.arange(m, device=dev) < s["count"][..., None]
    ok = (listed_[..., None] & (pos < limit)).reshape(B, T, G, m * P)
    o, lse = _softmax_rows(s["q"].float().reshape(B, T, G, -1, D), k, v, ok, s["scale"])
    return [o.reshape(B, T, -1, D).to(s["out"].dtype), lse.reshape(B, T, -1)]


# ------------------------------------------------------------------- the framework's calls

def _dims(s):
    """The dims that a user's program keeps beside its buffers, made at its first call."""
    if "dims" not in s:
        from hash_hierarchical_top_b200 import hhr
        c = s["case"]
        s["hhr"] = hhr
        s["dims"] = d = hhr.make_dims(c["batch"], c["heads"], c["kv_heads"], c["page"],
                                      s["page_table"].shape[1], s["n_phys"])
        n = {"attn": lambda: hhr.hhr_paged_attn_workspace_bytes(d),
             "block_select": lambda: hhr.hhr_block_select_workspace_bytes(d, c["queries"]),
             "block_attn": lambda: hhr.hhr_block_attn_workspace_bytes(
                 d, c["queries"], s["blocks"].shape[-1])}.get(c["op"], lambda: 0)()
        s["ws"] = torch.empty(n, dtype=torch.uint8, device=s["page_table"].device)
        if c["op"] == "block_select":
            s["opts"] = hhr.make_opts(c["sink"], c["local"])
    return s["hhr"], s["dims"]


def _own(s):
    hhr, d = _dims(s)
    op = s["case"]["op"]
    if op == "append":
        hhr.hhr_append_kv8(d, s["k_new"], s["v_new"], s["start"], s["n_new"], s["page_table"],
                           s["k"], s["v"], s["k_exp"], s["v_exp"], s["block_mean"])
        return [s["k"], s["v"], s["k_exp"], s["v_exp"]] + (
            [s["block_mean"]] if s["block_mean"] is not None else [])
    if op == "read":
        hhr.hhr_read_kv8(d, s["k"], s["v"], s["k_exp"], s["v_exp"], s["page_table"], s["start"],
                         s["seq_len"], s["k_out"], s["v_out"])
        return [s["k_out"], s["v_out"]]
    if op == "attn":
        hhr.hhr_paged_attn(d, s["q"], s["k_new"], s["v_new"], s["k"], s["v"], s["k_exp"],
                           s["v_exp"], s["page_table"], s["seq_len"], s["scale"], s["out"],
                           s["ws"], lse=s["lse"])
        outs = [s["out"], s["lse"]]
        if s["k_new"] is not None:
            outs += ([s["k"], s["k_exp"], s["v"], s["v_exp"]] if s["case"]["kv8"]
                     else [s["k"], s["v"]])
        return outs
    if op == "block_select":
        hhr.hhr_block_select(d, s["q"], s["seq_len"], s["q_pos"], s["page_table"],
                             s["block_mean"], s["case"]["keep"], s["blocks"], s["count"],
                             s["ws"], opts=s["opts"])
        return [s["blocks"], s["count"]]
    hhr.hhr_block_attn(d, s["q"], s["k"], s["v"], s["k_exp"], s["v_exp"], s["page_table"],
                       s["seq_len"], s["q_pos"], s["blocks"], s["count"], s["scale"], s["out"],
                       s["ws"], lse=s["lse"])
    return [s["out"], s["lse"]]


def run(state):
    if own:
        return _own(state)
    return {"append": _plain_append, "read": _plain_read, "attn": _plain_attn,
            "block_select": _plain_block_select,
            "block_attn": _plain_block_attn}[state["case"]["op"]](state)


# ---------------------------------------------------------------- the definitions in 64 bits

def _nearest_e4m3(x):
    """x (float64) rounded to the nearest e4m3 number, ties to the even one: a step of 2^-3 of
    the value's power of two, no finer than 2^-9."""
    step = torch.exp2(torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -6))) - 3)
    return torch.round(x / step) * step


def _exact_row(x):
    """(e4m3 values, exponent bytes) of float64 rows, by searching the exponents' range."""
    top = x.abs().amax(-1)
    e = torch.ceil(torch.log2(top / 448))                # -inf for a row of zeros
    e = torch.where(top > 448 * torch.exp2(e), e + 1, e)
    e = torch.where(top <= 448 * torch.exp2(e - 1), e - 1, e).clamp(-117, 119)
    return _nearest_e4m3(x / torch.exp2(e)[..., None]), (e + 127).to(torch.uint8)


def _exact_cache(s, name, b, g, n):
    """float64 rows [n, D] of sequence b and KV head g."""
    P = s["case"]["page"]
    phys = s["page_table"][b, :-(-n // P)].long()
    x = s[name].view(torch.uint8)[phys, g].view(torch.float8_e4m3fn) if s[name + "_exp"] is not None \
        else s[name][phys, g]
    x = x.double()
    if s[name + "_exp"] is not None:
        x = x * torch.exp2(s[name + "_exp"][phys, g].double() - 127)[..., None]
    return x.reshape(-1, D)[:n]


def _exact_attention(q, k, v, scale):
    """float64 attention of q [h, D] over k, v [n, D], and the log of the weights' sum."""
    if not len(k):
        return torch.zeros_like(q), torch.full((len(q),), -math.inf, dtype=q.dtype, device=q.device)
    x = scale * (q @ k.T)
    top = x.max(1, keepdim=True).values
    w = (x - top).exp()
    return (w @ v) / w.sum(1, keepdim=True), top[:, 0] + w.sum(1).log()


def _exact_write(s, b, pos, k_rows, v_rows):
    """Quantised rows written at the positions pos of sequence b."""
    P = s["case"]["page"]
    phys, slot = s["page_table"][b, pos // P].long(), pos % P
    for name, x in (("k", k_rows), ("v", v_rows)):
        q, e = _exact_row(x.double())
        s[name].view(torch.uint8)[phys, :, slot] = q.to(torch.float8_e4m3fn).view(torch.uint8)
        s[name + "_exp"][phys, :, slot] = e


def exact(case, seed):
    s = prepare(case, seed)
    op, G, H, P = case["op"], case["kv_heads"], case["heads"], case["page"]
    gs, lens, dev = H // G, _lens(case), s["page_table"].device
    if op == "append":
        for b, (n, new) in enumerate(zip(lens, _news(case))):
            pos = torch.arange(n - new, n, device=dev)
            _exact_write(s, b, pos, s["k_new"][b, :new], s["v_new"][b, :new])
        outs = [s["k"].double(), s["v"].double(), None, None]
        if case["mean"]:
            mean = s["block_mean"].double()
            for b, (n, new) in enumerate(zip(lens, _news(case))):
                first = (n - new) // P
                for g in range(G):
                    x = _exact_cache(s, "k", b, g, n)[first * P:]
                    whole = torch.zeros(-(-len(x) // P) * P, D, dtype=x.dtype, device=dev)
                    whole[:len(x)] = x
                    size = torch.full((len(whole) // P, 1), P, dtype=x.dtype, device=dev)
                    size[-1] = len(x) - (len(whole) - P)
                    mean[s["page_table"][b, first:-(-n // P)].long(), g] = \
                        whole.reshape(-1, P, D).sum(1) / size
            outs.append(mean)
        return outs
    if op == "read":
        outs = []
        for name in ("k", "v"):
            x = torch.zeros(s["k_out"].shape, dtype=torch.float64, device=dev)
            for b, n in enumerate(lens):
                for g in range(G):
                    x[b, :n, g] = _exact_cache(s, name, b, g, n)
            outs.append(x)
        return outs
    if op == "block_select":
        return None  # whole numbers
    if op == "attn":
        caches = []
        if case["append"]:
            for b, n in enumerate(lens):
                pos = torch.tensor([n - 1], device=dev)
                if case["kv8"]:
                    _exact_write(s, b, pos, s["k_new"][b:b + 1], s["v_new"][b:b + 1])
                else:
                    at = int(s["page_table"][b, (n - 1) // P])
                    s["k"][at, :, (n - 1) % P], s["v"][at, :, (n - 1) % P] = \
                        s["k_new"][b], s["v_new"][b]
            caches = ([s["k"].double(), None, s["v"].double(), None] if case["kv8"]
                      else [s["k"].double(), s["v"].double()])
        o = torch.zeros(len(lens), H, D, dtype=torch.float64, device=dev)
        lse = torch.zeros(len(lens), H, dtype=torch.float64, device=dev)
        for b, n in enumerate(lens):
            for g in range(G):
                h = slice(g * gs, (g + 1) * gs)
                o[b, h], lse[b, h] = _exact_attention(
                    s["q"][b, h].double(), _exact_cache(s, "k", b, g, n),
                    _exact_cache(s, "v", b, g, n), s["scale"])
        return [o, lse] + caches
    T = case["queries"]
    o = torch.zeros(len(lens), T, H, D, dtype=torch.float64, device=dev)
    lse = torch.zeros(len(lens), T, H, dtype=torch.float64, device=dev)
    pos, blocks, count = s["q_pos"].tolist(), s["blocks"], s["count"].tolist()
    for b, n in enumerate(lens):
        for g in range(G):
            k, v = _exact_cache(s, "k", b, g, n), _exact_cache(s, "v", b, g, n)
            h = slice(g * gs, (g + 1) * gs)
            for t in range(T):
                chosen = blocks[b, t, g, :count[b][t][g]].long()
                at = (chosen[:, None] * P + torch.arange(P, device=dev)).reshape(-1)
                at = at[at < min(n, pos[b][t] + 1)]
                o[b, t, h], lse[b, t, h] = _exact_attention(s["q"][b, t, h].double(), k[at],
                                                            v[at], s["scale"])
    return [o, lse]
