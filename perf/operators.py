"""Measured cases of the 4-bit cache and page operators.

Operators (``case["op"]``):

``decode``   attention of new tokens over a paged cache held in 4 bits
             (``pa_decode_v2_kv4``, ``pa_decode_v2_mq_kv4``)
``append``   new tokens quantised into the cache, and tokens read back as
             16-bit rows (``pa_kv4_append``, ``pa_kv4_gather``)
``fork``     child sequences that share their parents' full pages
             (``pa_pages_fork``)
``resize``   sequences grown, truncated and freed (``pa_pages_resize``)
``compact``  the pages in use moved to the front of the pool
             (``pa_pages_compact``)

The 4-bit cache is uint8 ``[num_blocks, KH, BS * (D + 8)]``: one record per
(block, kv head) with the key codes, the value codes (each ``[D / x][BS][x / 2]``
bytes with x = min(D, 128), two codes a byte, the even dim in the low nibble)
and ``[BS][4]`` 16-bit floats (key scale, key zero, value scale, value zero).
A code c stands for ``scale * c + zero``.

With ``own`` false ``run`` computes each operator from elementary torch
operations; with ``own`` true it calls the framework.
"""
import math
import random

import torch

own = False

_T = {"fp16": torch.float16, "bf16": torch.bfloat16}


def _dev():
    return torch.device("cuda", torch.cuda.current_device())


# ------------------------------------------------------------------ cases
def _decode(name, dtype, S, H, KH, D, BS, q_len, lens, P=512):
    return dict(name=name, op="decode", dtype=dtype, S=S, H=H, KH=KH, D=D, BS=BS, q_len=q_len, lens=lens, P=P)


def _append(name, dtype, S, KH, D, BS, new, ctx, back):
    return dict(name=name, op="append", dtype=dtype, S=S, KH=KH, D=D, BS=BS, new=new, ctx=ctx, back=back)


def _pages(name, op, S, BS, lens, NB, caches, page, **kw):
    return dict(name=name, op=op, S=S, BS=BS, lens=lens, NB=NB, caches=caches, page=page, **kw)


def listed():
    return [
        # A handful of short chats on a small model: the time of the call itself.
        _decode("decode_small_mha", "fp16", 4, 4, 4, 64, 16, 1, "1:300"),
        # A full serving batch of a grouped-query model.
        _decode("decode_batch_gqa", "bf16", 128, 32, 8, 128, 16, 1, "2048:8192"),
        # One very long document next to ordinary and tiny requests.
        _decode("decode_long_skew", "bf16", 8, 64, 8, 128, 32, 1, "131072,16384,8192,4096,2048,1024,1000,17"),
        # Four draft tokens a sequence verified at once, odd lengths.
        _decode("decode_draft4", "fp16", 48, 32, 8, 128, 16, 4, "1001:4999"),
        # One new token of each running sequence, written and read back.
        _append("append_step", "bf16", 128, 8, 128, 16, "1:1", "2048:8192", "new"),
        # A chunk of each prompt, and the whole context back for its prefill attention.
        _append("append_prompt", "fp16", 24, 8, 128, 16, "257:2049", "0:4096", "all"),
        # Beams of a few requests split in two; 4-bit pages of one layer.
        _pages("fork_beams", "fork", 8, 16, "33:500", 1024, 1, 8 * 2176, children=16, parents="each"),
        # Eight samples of each of 32 prompts over eight layers of 4-bit pages.
        _pages("fork_samples", "fork", 32, 16, "500:4000", 16384, 8, 8 * 2176, children=256, parents="each"),
        # A decode step: every sequence gets room for one more token.
        _pages("resize_step", "resize", 128, 16, "2048:8192", 65536, 1, 16384, grow="one"),
        # Turnover: sequences end, drafts are taken back, prompts come in.
        _pages("resize_turnover", "resize", 512, 16, "100:6000", 262144, 4, 2048, grow="mixed"),
        # A small pool with half of its pages in use.
        _pages("compact_small", "compact", 16, 16, "1:600", 1536, 2, 4096, fill=0.5),
        # A large pool after a burst of requests: keys and values of four layers.
        _pages("compact_pool", "compact", 96, 16, "500:3000", 16384, 8, 32768, fill=0.65),
    ]


def _logint(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["decode", "decode", "append", "fork", "resize", "compact"])
    if op == "decode":
        D, BS = rng.choice([64, 80, 96, 112, 128, 128, 256]), rng.choice([8, 16, 16, 32, 64])
        KH = rng.choice([1, 2, 3, 4, 8, 8])
        G = rng.choice([1, 2, 4, 4, 5, 8, 12])
        S, q_len = _logint(rng, 1, 128), rng.choice([1, 1, 1, 2, 3, 4, 7])
        top = _logint(rng, 8, 65536)
        # No more cached tokens x heads x head size than the largest listed case has.
        top = max(q_len, min(top, 128 * 8192 * 8 * 128 // (2 * S * KH * D * max(1, G // 4) * max(1, q_len // 2))))
        return dict(op=op, dtype=rng.choice(["fp16", "bf16"]), S=S, H=KH * G, KH=KH, D=D, BS=BS, q_len=q_len,
                    lens=f"{q_len}:{top}", P=rng.choice([256, 512, 512, 1024]))
    if op == "append":
        D, BS = rng.choice([64, 80, 96, 112, 128, 128, 256]), rng.choice([8, 16, 16, 32, 64])
        S, KH = _logint(rng, 1, 128), rng.choice([1, 2, 3, 4, 8, 8])
        top, ctx = _logint(rng, 1, 2048), _logint(rng, 1, 4096)
        room = max(1, 24 * 4096 * 8 * 128 // (S * KH * D))
        return dict(op=op, dtype=rng.choice(["fp16", "bf16"]), S=S, KH=KH, D=D, BS=BS,
                    new=f"{rng.choice([0, 1, top])}:{min(top, room)}" if min(top, room) == top else f"0:{room}",
                    ctx=f"0:{min(ctx, room)}", back=rng.choice(["new", "all"]))
    BS = rng.choice([8, 16, 16, 32, 64])
    page = 16 * _logint(rng, 16, 2048)
    caches = rng.choice([1, 2, 3, 4, 6, 8])
    S = _logint(rng, 1, 256)
    top = _logint(rng, 4, 4000)
    MB = -(-top // BS) + 2
    if op == "fork":
        children = _logint(rng, 1, 256)
        NB = S * MB + children + _logint(rng, 1, 4096)
        extra = dict(children=children, parents=rng.choice(["each", "any"]))
    elif op == "resize":
        NB = 2 * S * MB + _logint(rng, 1, 65536)
        extra = dict(grow=rng.choice(["one", "mixed"]))
    else:
        NB = 0
        extra = dict(fill=rng.choice([0.25, 0.5, 0.65, 0.9]))
    # The pool of a drawn case holds no more than that of the largest listed one.
    total = max(NB, S * MB * 4) * page * caches
    page = max(256, min(page, int(page * 3e9 / total) // 16 * 16))
    return dict(op=op, S=S, BS=BS, lens=f"1:{top}", NB=NB, caches=caches, page=page, **extra)


def _lens(text, n, rng):
    if ":" in text:
        lo, hi = (int(v) for v in text.split(":"))
        return [rng.randint(lo, hi) for _ in range(n)]
    return [int(v) for v in text.split(",")]


def _fixed(case):
    """The lengths of a case are its own; a seed gives their order (and all the data)."""
    return random.Random(repr(sorted((k, v) for k, v in case.items() if k != "name")))


def _shuffled(seed, *lists):
    order = list(range(len(lists[0])))
    random.Random(seed).shuffle(order)
    return [[v[i] for i in order] for v in lists]


def _nominal(text, n):
    """The mean of a length rule, times n."""
    if ":" in text:
        lo, hi = (int(v) for v in text.split(":"))
        return n * (lo + hi) / 2
    return sum(int(v) for v in text.split(","))


# ------------------------------------------------------------------ the cache format
def _pack(kc, vc, params):
    """Codes uint8 [..., BS, D] and params T [..., BS, 4] as records uint8 [..., BS * (D + 8)]."""
    BS, D = kc.shape[-2:]
    x = min(D, 128)

    def rows(c):
        c = c.unflatten(-1, (D // x, x)).transpose(-3, -2)
        return (c[..., 0::2] | (c[..., 1::2] << 4)).flatten(-3)

    return torch.cat([rows(kc), rows(vc), params.contiguous().view(torch.uint8).flatten(-2)], dim=-1)


def _unpack(rec, D, BS, dtype):
    """Records as fp32 keys and values [..., BS, D]."""
    x, n = min(D, 128), BS * D // 2

    def codes(b):
        b = b.unflatten(-1, (D // x, BS, x // 2))
        c = torch.stack([b & 15, b >> 4], dim=-1).flatten(-2)
        return c.transpose(-3, -2).flatten(-2).float()

    p = rec[..., 2 * n:].contiguous().view(dtype).unflatten(-1, (BS, 4)).float()
    return (codes(rec[..., :n]) * p[..., 0:1] + p[..., 1:2],
            codes(rec[..., n:2 * n]) * p[..., 2:3] + p[..., 3:4])


def _quantise(x):
    """[..., D] of T: codes uint8, scale and zero of T ([...])."""
    f = x.float()
    lo, hi = f.amin(dim=-1), f.amax(dim=-1)
    # (A divisor on the device: torch turns a scalar one into a product with its reciprocal.)
    s = ((hi - lo) / torch.full_like(lo, 15.0)).to(x.dtype)
    s32 = s.float().unsqueeze(-1)
    c = torch.where(s32 > 0, torch.round((f - lo.unsqueeze(-1)) / s32), torch.zeros_like(f)).clamp(0, 15)
    return c.to(torch.uint8), s, lo.to(x.dtype)


def _randn(shape, gen):
    return torch.randn(shape, generator=gen, device=gen.device)


def _fill_cache(NB, KH, D, BS, dtype, gen, offset):
    """A pool whose records hold N(0, 1) keys (about the channel offsets) and values."""
    cache = torch.empty((NB, KH, BS * (D + 8)), dtype=torch.uint8, device=gen.device)
    step = max(1, (1 << 25) // (KH * BS * D))
    for b in range(0, NB, step):
        n = min(step, NB - b)
        kc, ks, kz = _quantise((_randn((n, KH, BS, D), gen) + offset).to(dtype))
        vc, vs, vz = _quantise(_randn((n, KH, BS, D), gen).to(dtype))
        cache[b:b + n] = _pack(kc, vc, torch.stack([ks, kz, vs, vz], dim=-1))
    return cache


def _tables(lens, MB, NB, BS, gen):
    """Shuffled distinct pages per sequence, int32 [S, MB] (unused entries 0)."""
    S = len(lens)
    perm = torch.randperm(NB, generator=gen, device=gen.device)[: S * MB].to(torch.int32).view(S, MB)
    used = torch.tensor([-(-v // BS) for v in lens], device=gen.device)
    cols = torch.arange(MB, device=gen.device)
    return torch.where(cols[None] < used[:, None], perm, torch.zeros_like(perm)).contiguous()


def _channel_offset(KH, D, gen):
    """Keys of trained models have a few channels far from zero."""
    off = torch.zeros((KH, 1, D), device=gen.device)
    off[:, :, 3 % D] = 3.0
    off[:, :, (D // 2 + 1) % D] = -2.0
    return off


# ------------------------------------------------------------------ prepare
def prepare(case, seed):
    gen = torch.Generator(device=_dev()).manual_seed(seed)
    st = dict(case=case)
    {"decode": _prepare_decode, "append": _prepare_append}.get(case["op"], _prepare_pages)(case, st, seed, gen)
    return st


def _prepare_decode(case, st, seed, gen):
    S, H, KH, D, BS, q_len = (case[k] for k in ("S", "H", "KH", "D", "BS", "q_len"))
    dtype = _T[case["dtype"]]
    lens, = _shuffled(seed, _lens(case["lens"], S, _fixed(case)))
    MB = max(1, max(-(-v // BS) for v in lens))
    NB = S * MB if S * MB * KH * BS * (D + 8) < 3e9 else max(MB, int(3e9 / (KH * BS * (D + 8))))
    st["lens_host"] = lens
    st["lens"] = torch.tensor(lens, dtype=torch.int32, device=gen.device)
    st["cache"] = _fill_cache(NB, KH, D, BS, dtype, gen, _channel_offset(KH, D, gen))
    if NB >= S * MB:
        st["tables"] = _tables(lens, MB, NB, BS, gen)
    else:  # sequences drawn from one pool that is smaller than all their tables
        st["tables"] = torch.randint(0, NB, (S, MB), generator=gen, device=gen.device, dtype=torch.int32)
    shape = (S, H, D) if q_len == 1 else (S, q_len, H, D)
    st["query"] = _randn(shape, gen).to(dtype)
    st["out"] = torch.empty_like(st["query"])
    st["scale"] = 1.0 / math.sqrt(D)
    if own:
        import decode_attention_paged_pa_gb300 as pa
        n = pa.workspace_bytes(S * q_len, H, KH, D, MB, BS, case["P"])
        st["ws"] = torch.empty(max(n, 256), dtype=torch.uint8, device=gen.device)


def _prepare_append(case, st, seed, gen):
    S, KH, D, BS = (case[k] for k in ("S", "KH", "D", "BS"))
    dtype = _T[case["dtype"]]
    rng = _fixed(case)
    new, ctx = _lens(case["new"], S, rng), _lens(case["ctx"], S, rng)
    new[0] = max(new[0], 0 if sum(new) else 1)
    new, ctx = _shuffled(seed, new, ctx)
    lens = [a + b for a, b in zip(new, ctx)]
    back = new if case["back"] == "new" else lens
    MB = max(1, max(-(-v // BS) for v in lens))
    NB = S * MB
    dev = gen.device
    st["lens_host"], st["new_host"], st["back_host"] = lens, new, back
    st["lens"] = torch.tensor(lens, dtype=torch.int32, device=dev)
    st["cu_new"] = torch.tensor([0] + new, dtype=torch.int32).cumsum(0, dtype=torch.int32).to(dev)
    st["cu_back"] = torch.tensor([0] + back, dtype=torch.int32).cumsum(0, dtype=torch.int32).to(dev)
    st["tables"] = _tables(lens, MB, NB, BS, gen)
    off = _channel_offset(KH, D, gen)
    st["cache"] = _fill_cache(NB, KH, D, BS, dtype, gen, off)
    # Keys and values as they leave a fused projection: slices of wider rows.
    n = sum(new)
    qkv = _randn((max(n, 1), 3 * KH, D), gen)
    qkv[:, KH:2 * KH] += off.transpose(0, 1)
    st["qkv"] = qkv.to(dtype)
    st["key"], st["value"] = st["qkv"][:n, KH:2 * KH], st["qkv"][:n, 2 * KH:]
    st["key_out"] = torch.empty((sum(back), KH, D), dtype=dtype, device=dev)
    st["value_out"] = torch.empty_like(st["key_out"])
    if own:
        st["ws"] = torch.empty(256, dtype=torch.uint8, device=dev)


def _prepare_pages(case, st, seed, gen):
    S, BS, op = case["S"], case["BS"], case["op"]
    dev, rng = gen.device, _fixed(case)
    lens = _lens(case["lens"], S, rng)
    hi = int(case["lens"].split(":")[1])
    new = list(lens)
    if op == "resize":
        if case["grow"] == "one":
            new = [v + 1 for v in lens]
        else:
            for i in range(S):
                kind = rng.randrange(4)
                if kind == 0:      # ends
                    new[i] = 0
                elif kind == 1:    # takes drafts back
                    new[i] = max(0, lens[i] - rng.randint(1, 40))
                elif kind == 2:    # a prompt comes in
                    lens[i], new[i] = 0, rng.randint(1, hi)
                else:              # goes on
                    new[i] = lens[i] + rng.randint(0, 7)
    lens, new = _shuffled(seed, lens, new)
    MB = max(1, max(-(-v // BS) for v in lens + new)) + 1
    NB = case["NB"]
    used = sum(-(-v // BS) for v in lens)
    if op == "compact":
        NB = max(NB, int(used / case["fill"]))
    ids = torch.randperm(NB, generator=gen, device=dev).to(torch.int32)
    tables = torch.zeros((S, MB), dtype=torch.int32, device=dev)
    held = torch.tensor([-(-v // BS) for v in lens], device=dev)
    mask = torch.arange(MB, device=dev)[None] < held[:, None]
    tables[mask] = ids[:used]
    # Requests with the same system prompt share its pages (four rows a group).
    share = max(0, min(lens) // BS) if op != "resize" else 0
    for g in range(0, S, 4):
        if share:
            tables[g:g + 4, :share] = tables[g, :share].clone()
    if op == "resize" and S >= 2 and lens[0] > BS and lens[1] > BS:
        # Two samples of one prompt: one of them is cut back into the shared part.
        k = min(lens[0], lens[1]) // BS
        tables[1, :k] = tables[0, :k]
        if case["grow"] == "mixed":
            new[1] = k * BS - 1
    refs = torch.zeros((NB,), dtype=torch.int32, device=dev)
    flat = tables[mask].long()
    refs.index_add_(0, flat, torch.ones_like(flat, dtype=torch.int32))
    st["start"] = [tables, torch.tensor(lens, dtype=torch.int32, device=dev), refs]
    st["now"] = [t.clone() for t in st["start"]]
    st["new"] = torch.tensor(new, dtype=torch.int32, device=dev)
    st["caches"] = [torch.randint(0, 256, (NB, case["page"]), generator=gen, device=dev, dtype=torch.uint8)
                    for _ in range(case["caches"])]
    rows = S
    if op == "fork":
        n = case["children"]
        rows = n
        if case["parents"] == "each":
            par = [i % S for i in range(n)]
        else:
            par = random.Random(seed).choices(range(S), k=n)
        st["parents"] = torch.tensor(par, dtype=torch.int32, device=dev)
        st["tables_out"] = torch.zeros((n, MB), dtype=torch.int32, device=dev)
        st["lens_out"] = torch.zeros((n,), dtype=torch.int32, device=dev)
    if own:
        import decode_attention_paged_pa_gb300 as pa
        st["ws"] = torch.empty(pa.pages_workspace_bytes(rows, MB, NB), dtype=torch.uint8, device=dev)


# ------------------------------------------------------------------ run
def run(st):
    return {"decode": _run_decode, "append": _run_append, "fork": _run_fork, "resize": _run_resize,
            "compact": _run_compact}[st["case"]["op"]](st)


def _run_decode(st):
    c = st["case"]
    if own:
        import decode_attention_paged_pa_gb300 as pa
        call = pa.pa_decode_v2_kv4 if c["q_len"] == 1 else pa.pa_decode_v2_mq_kv4
        call(st["out"], st["query"], st["cache"], st["tables"], st["lens"], st["scale"], partition_size=c["P"],
             workspace=st["ws"])
        return st["out"]
    S, H, KH, D, BS, q_len = (c[k] for k in ("S", "H", "KH", "D", "BS", "q_len"))
    G = H // KH
    q = st["query"].view(S, q_len, KH, G, D).float()
    out = torch.zeros_like(q)
    for s, L in enumerate(st["lens_host"]):
        if L == 0:
            continue
        nb = -(-L // BS)
        k, v = _unpack(st["cache"][st["tables"][s, :nb].long()], D, BS, _T[c["dtype"]])  # [nb, KH, BS, D]
        k = k.transpose(0, 1).reshape(KH, nb * BS, D)[:, :L]
        v = v.transpose(0, 1).reshape(KH, nb * BS, D)[:, :L]
        qs = q[s].permute(1, 0, 2, 3).reshape(KH, q_len * G, D)
        z = torch.matmul(qs, k.transpose(1, 2)) * st["scale"]
        if q_len > 1:
            last = torch.arange(q_len, device=z.device).repeat_interleave(G) + (L - q_len)
            z = z.masked_fill(torch.arange(L, device=z.device)[None, None] > last[None, :, None], -math.inf)
        p = torch.exp(z - z.amax(dim=-1, keepdim=True))
        o = torch.matmul(p, v) / p.sum(dim=-1, keepdim=True)
        out[s] = o.view(KH, q_len, G, D).transpose(0, 1)
    return out.view(st["query"].shape).to(st["query"].dtype)


def _run_append(st):
    c = st["case"]
    if own:
        import decode_attention_paged_pa_gb300 as pa
        pa.pa_kv4_append(st["cache"], st["key"], st["value"], st["tables"], st["lens"], cu_tokens=st["cu_new"],
                         workspace=st["ws"])
        pa.pa_kv4_gather(st["key_out"], st["value_out"], st["cache"], st["tables"], st["lens"],
                         cu_tokens=st["cu_back"], workspace=st["ws"])
        return [st["key_out"], st["value_out"]]
    D, BS, dtype = c["D"], c["BS"], _T[c["dtype"]]
    cache, tables, lens = st["cache"], st["tables"], st["lens"].long()

    def places(cu, total):
        """Block and slot of the rows of cu: each sequence's last tokens."""
        n = torch.diff(cu).long()
        seq = torch.repeat_interleave(torch.arange(n.numel(), device=cu.device), n, output_size=total)
        pos = lens[seq] - n[seq] + torch.arange(total, device=cu.device) - cu.long()[seq]
        return tables[seq, pos // BS].long(), pos % BS

    n, x, half = sum(st["new_host"]), min(D, 128), BS * D // 2
    blk, slot = places(st["cu_new"], n)
    kq, ks, kz = _quantise(st["key"])
    vq, vs, vz = _quantise(st["value"])
    codes = cache[..., :2 * half].unflatten(-1, (2, D // x, BS, x // 2))
    params = cache.view(dtype)[..., half:].unflatten(-1, (BS, 4))
    for i, q in enumerate((kq, vq)):
        codes[blk, :, i, :, slot] = (q[..., 0::2] | (q[..., 1::2] << 4)).unflatten(-1, (D // x, x // 2))
    params[blk, :, slot] = torch.stack([ks, kz, vs, vz], dim=-1)
    blk, slot = places(st["cu_back"], sum(st["back_host"]))
    out = []
    p = params[blk, :, slot].float()  # [N, KH, 4]
    for i in range(2):
        b = codes[blk, :, i, :, slot].flatten(-2)
        q = torch.stack([b & 15, b >> 4], dim=-1).flatten(-2).float()
        out.append((q * p[..., 2 * i:2 * i + 1] + p[..., 2 * i + 1:2 * i + 2]).to(dtype))
    return out


def _restart(st):
    # The pass starts from the pool as the step before left it.
    now = st["now"] + ([st["tables_out"], st["lens_out"]] if "tables_out" in st else [])
    if "tables_out" in st and "zeros" not in st:
        st["zeros"] = [torch.zeros_like(st["tables_out"]), torch.zeros_like(st["lens_out"])]
    torch._foreach_copy_(now, st["start"] + st.get("zeros", []))
    return st["now"]


def _lowest_free(refs):
    return torch.argsort((refs > 0).to(torch.uint8), stable=True)


def _move(caches, src, dst):
    for c in caches:
        c[dst] = c[src]


def _run_fork(st):
    c = st["case"]
    tables, lens, refs = _restart(st)
    if own:
        import decode_attention_paged_pa_gb300 as pa
        pa.pa_pages_fork(st["tables_out"], st["lens_out"], tables, lens, st["parents"], refs, st["caches"], c["BS"],
                         workspace=st["ws"])
        return dict(tables=st["tables_out"], lens=st["lens_out"], refs=refs, caches=st["caches"])
    par, BS, MB = st["parents"].long(), c["BS"], tables.shape[1]
    t, L = tables[par], lens[par].long()
    cols = torch.arange(MB, device=t.device)[None]
    full, part = L // BS, L % BS != 0
    shared = cols < full[:, None]
    free = _lowest_free(refs)
    fresh = free[(torch.cumsum(part, 0) - 1).clamp(min=0)]
    row = torch.arange(t.shape[0], device=t.device)[part]
    src, dst = t[row, full[part]].long(), fresh[part]
    flat = t[shared].long()
    refs.index_add_(0, flat, torch.ones_like(flat, dtype=torch.int32))
    refs[dst] = 1
    out = torch.where(shared, t, st["tables_out"])
    out[row, full[part]] = dst.to(torch.int32)
    st["tables_out"].copy_(out)
    st["lens_out"].copy_(L)
    _move(st["caches"], src, dst)
    return dict(tables=st["tables_out"], lens=st["lens_out"], refs=refs, caches=st["caches"])


def _run_resize(st):
    c = st["case"]
    tables, lens, refs = _restart(st)
    if own:
        import decode_attention_paged_pa_gb300 as pa
        pa.pa_pages_resize(tables, lens, st["new"], refs, st["caches"], c["BS"], workspace=st["ws"])
        return dict(tables=tables, lens=lens, refs=refs, caches=st["caches"])
    BS, MB = c["BS"], tables.shape[1]
    L, N = lens.long(), st["new"].long()
    old, new, keep = (L + BS - 1) // BS, (N + BS - 1) // BS, torch.minimum(L, N)
    cols = torch.arange(MB, device=L.device)[None]
    edge = (cols == (keep // BS)[:, None]) & (keep % BS != 0)[:, None]
    own_copy = edge & (refs[tables.long()] > 1)
    fresh = own_copy | ((cols >= old[:, None]) & (cols < new[:, None]))
    gone = own_copy | ((cols >= new[:, None]) & (cols < old[:, None]))
    rank = (torch.cumsum(fresh.flatten(), 0) - 1).view_as(fresh)
    ids = _lowest_free(refs)[rank.clamp(min=0)].to(torch.int32)
    src, dst, taken = tables[own_copy].long(), ids[own_copy].long(), ids[fresh].long()
    flat = tables[gone].long()
    refs.index_add_(0, flat, -torch.ones_like(flat, dtype=torch.int32))
    refs[taken] = 1
    tables.copy_(torch.where(fresh, ids, tables))
    lens.copy_(st["new"])
    _move(st["caches"], src, dst)
    return dict(tables=tables, lens=lens, refs=refs, caches=st["caches"])


def _run_compact(st):
    c = st["case"]
    tables, lens, refs = _restart(st)
    if own:
        import decode_attention_paged_pa_gb300 as pa
        pa.pa_pages_compact(tables, lens, refs, st["caches"], c["BS"], workspace=st["ws"])
        return dict(tables=tables, lens=lens, refs=refs, caches=st["caches"])
    ids = torch.arange(refs.numel(), device=refs.device)
    used = refs > 0
    front = ids < used.sum()
    src, dst = ids[used & ~front], ids[~used & front]
    to = ids.to(torch.int32)
    to[src] = dst.to(torch.int32)
    held = torch.arange(tables.shape[1], device=refs.device)[None] < ((lens + c["BS"] - 1) // c["BS"])[:, None]
    tables.copy_(torch.where(held, to[tables.long()], tables))
    refs[dst] = refs[src]
    refs[src] = 0
    _move(st["caches"], src, dst)
    return dict(tables=tables, lens=lens, refs=refs, caches=st["caches"])


# ------------------------------------------------------------------ work
def work(case):
    op = case["op"]
    if op == "decode":
        S, H, KH, D, q_len = (case[k] for k in ("S", "H", "KH", "D", "q_len"))
        tok = _nominal(case["lens"], S)
        return {"bytes": tok * KH * (D + 8) + 4 * S * q_len * H * D + 4 * tok / case["BS"] + 4 * S,
                "flops": 4 * tok * H * D * q_len}
    if op == "append":
        S, KH, D = (case[k] for k in ("S", "KH", "D"))
        new = _nominal(case["new"], S)
        back = new if case["back"] == "new" else new + _nominal(case["ctx"], S)
        return {"bytes": (new + back) * KH * (D + 8 + 4 * D), "flops": (new + back) * KH * D * 8}
    S, BS = case["S"], case["BS"]
    tok = _nominal(case["lens"], S)
    page, moved, NB, entries = case["page"] * case["caches"], 0, case["NB"], tok / BS + S / 2
    if op == "fork":
        moved = case["children"] * (1 - 1 / BS)
        entries = 2 * entries * case["children"] / S
    elif op == "resize":
        moved = 1
    else:
        NB = max(NB, int(entries / case["fill"]))
        fill = min(1.0, entries / NB)
        moved = fill * (1 - fill) * NB
        entries *= 2
    return {"bytes": 2 * moved * page + 8 * NB + 4 * entries + 8 * S, "flops": 0}


# ------------------------------------------------------------------ exact
def exact(case, seed):
    """What ``run`` returns, in 64 bits; None where pages are moved rather than computed."""
    if case["op"] == "decode":
        return _exact_decode(case, prepare(case, seed))
    if case["op"] == "append":
        return _exact_append(case, prepare(case, seed))
    return None


def _offsets(D, BS, dev):
    """Byte of each (slot, dim) code within a code array."""
    t, d = torch.arange(BS, device=dev)[:, None], torch.arange(D, device=dev)[None]
    w = D if D < 128 else 128
    return (d // w) * (BS * w // 2) + t * (w // 2) + (d % w) // 2


def _read64(rec, D, BS, dtype):
    """Records [nb, KH, R] as fp64 keys and values [nb, KH, BS, D]."""
    at, high = _offsets(D, BS, rec.device), (torch.arange(D, device=rec.device) % 2 * 4).to(torch.uint8)
    f = rec.view(dtype)[..., BS * D // 2:].double()
    res = []
    for i in range(2):
        code = (rec[..., at + i * BS * D // 2] >> high) & 15
        s, z = f[..., 2 * i::4], f[..., 2 * i + 1::4]
        res.append(code.double() * s[..., None] + z[..., None])
    return res


def _exact_decode(case, st):
    S, H, KH, D, BS, n = (case[k] for k in ("S", "H", "KH", "D", "BS", "q_len"))
    q = st["query"].double().view(S, n, H, D)
    res = torch.zeros_like(q)
    for s, L in enumerate(st["lens_host"]):
        for kv in range(KH if L else 0):
            ids = st["tables"][s, : (L + BS - 1) // BS].long()
            K, V = _read64(st["cache"][ids, kv:kv + 1], D, BS, _T[case["dtype"]])
            K, V = K.reshape(-1, D)[:L], V.reshape(-1, D)[:L]
            for i in range(n):
                see = L - n + 1 + i
                h = slice(kv * (H // KH), (kv + 1) * (H // KH))
                w = torch.softmax(q[s, i, h] @ K[:see].T * st["scale"], dim=1)
                res[s, i, h] = w @ V[:see]
    return res.view(st["query"].shape)


def _exact_append(case, st):
    D, BS, dtype = case["D"], case["BS"], _T[case["dtype"]]
    out = [[], []]
    row = 0
    for s, L in enumerate(st["lens_host"]):
        n, back = st["new_host"][s], st["back_host"][s]
        ids = st["tables"][s, : (L + BS - 1) // BS].long()
        for i, x in enumerate((st["key"], st["value"])):
            old = _read64(st["cache"][ids], D, BS, dtype)[i].transpose(1, 2).reshape(-1, case["KH"], D)[: L - n]
            v = x[row:row + n].double()
            lo = v.amin(-1, keepdim=True)
            # The definition's roundings: the spread and its fifteenth to fp32, the scale to T.
            scale = ((v.amax(-1, keepdim=True) - lo).float().double() / 15.0).float().to(dtype).double()
            code = ((v - lo).float().double() / scale).float().double().round().clamp(0, 15)
            fresh = torch.where(scale > 0, code * scale, torch.zeros_like(code)) + lo
            out[i].append(torch.cat([old, fresh])[L - back:])
        row += n
    return [torch.cat(o) for o in out]
