"""Measured cases of windowed and tree attention over a paged cache, and of the
steps around them.

Operators (``case["op"]``):

``window``  attention of new tokens to a sliding window of the cache and to its
            first tokens (``pa_decode_v2_window``, ``pa_decode_v2_window_fp8``)
``tree``    attention of a tree of drafted tokens to the cache and to each
            node's ancestors (``pa_decode_v2_tree``, ``pa_decode_v2_tree_fp8``)
``slots``   the rows of a step numbered from its requests' lengths: sequence,
            position and cache slot of each, and the trees' masks
            (``pa_pages_slots``, ``pa_tree_masks``)
``write``   new keys and values written into the cache by their slots
            (``pa_cache_write``)
``accept``  the accepted nodes of each tree moved together in the caches of
            every layer (``pa_tree_accept``)

Caches are the paged ones of the framework: keys ``[NB, KH, D / x, BS, x]`` with
x = 16 bytes of elements, values ``[NB, KH, D, BS]``; E4M3 caches hold a code a
byte, and a code c stands for ``scale * c``.

With ``own`` false ``run`` computes each operator from elementary torch
operations; with ``own`` true it calls the framework.
"""
import math
import random

import torch

own = False

_T = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}
_K_SCALE, _V_SCALE = 0.5, 1.5


def _dev():
    return torch.device("cuda", torch.cuda.current_device())


# ------------------------------------------------------------------ cases
def _attention(name, op, dtype, S, H, KH, D, BS, n, lens, window, sinks, P=512, e4m3=False, pad=False):
    return dict(name=name, op=op, dtype=dtype, S=S, H=H, KH=KH, D=D, BS=BS, n=n, lens=lens, window=window,
                sinks=sinks, P=P, e4m3=e4m3, pad=pad)


def _slots(name, S, BS, new, ctx, nodes, room):
    return dict(name=name, op="slots", S=S, BS=BS, new=new, ctx=ctx, nodes=nodes, room=room)


def _write(name, dtype, S, KH, D, BS, new, ctx, e4m3, room):
    return dict(name=name, op="write", dtype=dtype, S=S, KH=KH, D=D, BS=BS, new=new, ctx=ctx, e4m3=e4m3, room=room)


def _accept(name, dtype, S, KH, D, BS, n, ctx, layers, e4m3=False):
    return dict(name=name, op="accept", dtype=dtype, S=S, KH=KH, D=D, BS=BS, n=n, ctx=ctx, layers=layers, e4m3=e4m3)


def listed():
    return [
        # A handful of short chats on a small model: the time of the call itself.
        _attention("window_small", "window", "fp16", 4, 4, 4, 64, 16, 1, "1:300", 128, 4),
        # A full serving batch of a grouped-query model, the layers with a window.
        _attention("window_batch", "window", "bf16", 128, 32, 8, 128, 16, 1, "2048:8192", 1024, 4),
        # A chunk of each prompt over a window of 8-bit cache, odd lengths.
        _attention("window_chunk", "window", "fp16", 24, 32, 8, 128, 16, 128, "1001:4999", 1024, 4, e4m3=True),
        # Seven drafted nodes of two requests: latency again.
        _attention("tree_small", "tree", "fp16", 2, 8, 2, 64, 16, 7, "40:300", 0, 0),
        # A serving batch with sixteen nodes a request, some of them padding.
        _attention("tree_batch", "tree", "bf16", 48, 32, 8, 128, 16, 16, "1001:4999", 0, 0, pad=True),
        # Few requests with wide trees over long caches.
        _attention("tree_wide", "tree", "bf16", 16, 32, 8, 128, 32, 64, "2048:8192", 0, 0, P=1024),
        # One new token of each running sequence.
        _slots("slots_step", 128, 16, "1:1", "2048:8192", 0, 0),
        # A mixed step: chunks of prompts next to single tokens, room for more rows.
        _slots("slots_mixed", 512, 16, "1:257", "0:4096", 0, 4096),
        # One new token of each running sequence, written into one layer's cache.
        _write("write_step", "bf16", 128, 8, 128, 16, "1:1", "500:2000", False, 0),
        # Chunks of prompts rounded into an 8-bit cache, rows of padding behind them.
        _write("write_prompt", "fp16", 24, 8, 128, 16, "257:2049", "0:1024", True, 63),
        # A few requests, one layer: latency.
        _accept("accept_small", "fp16", 2, 2, 64, 16, 7, "40:300", 1),
        # A serving batch over the caches of eight layers.
        _accept("accept_batch", "bf16", 48, 8, 128, 16, 16, "301:999", 8),
    ]


def _logint(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def _shape(rng):
    return rng.choice([64, 80, 96, 112, 128, 128, 256]), rng.choice([8, 16, 16, 32, 64]), rng.choice([1, 2, 3, 4, 8, 8])


def draw(rng):
    op = rng.choice(["window", "window", "tree", "tree", "slots", "write", "accept"])
    if op in ("window", "tree"):
        D, BS, KH = _shape(rng)
        G = rng.choice([1, 1, 2, 4, 4, 5, 8, 12])
        e4m3 = rng.random() < 0.25
        dtype = rng.choice(["fp16", "bf16"] if e4m3 else ["fp16", "fp16", "bf16", "bf16", "fp32"])
        n = rng.choice([1, 1, 1, 2, 4, 7, 16, 61, 128]) if op == "window" else _logint(rng, 1, 100)
        if dtype == "fp32":  # (whose blocks hold at most 32 tokens of 256 dims)
            n, BS = min(n, 16), min(BS, 32) if D == 256 else BS
        S = _logint(rng, 1, 128)
        if op == "window" or rng.random() < 0.3:
            window, sinks = max(_logint(rng, 1, 4096), n if op == "tree" else 1), rng.choice([0, 0, 1, 4, 4, 33, 128])
        else:
            window, sinks = 0, 0
        top = _logint(rng, 8, 65536)
        # No more rows x cached tokens, and no more cached tokens, than the largest listed cases have.
        seen = min(top, window + sinks + n) if window else top
        seen = max(1, min(seen, 16 * 5120 * 64 * 32 * 128 // (S * n * KH * G * D), 128 * 2048 * 8 * 128 // (S * KH * D)))
        if dtype == "fp32":
            seen = max(1, seen // 8)
        if window:
            window, top = max(min(window, seen), n if op == "tree" else 1), min(top, 16 * seen)
        else:
            top = min(top, seen)
        return dict(op=op, dtype=dtype, S=S, H=KH * G, KH=KH, D=D, BS=BS, n=n, lens=f"{n}:{max(n, top)}", window=window,
                    sinks=sinks, P=rng.choice([256, 512, 512, 1024]), e4m3=e4m3,
                    pad=op == "tree" and rng.random() < 0.5)
    if op == "slots":
        nodes = rng.choice([0, 0, _logint(rng, 1, 100)])
        new = f"{nodes}:{nodes}" if nodes else f"{rng.choice([0, 1])}:{_logint(rng, 1, 512)}"
        return dict(op=op, S=_logint(rng, 1, 512), BS=rng.choice([8, 16, 16, 32, 64]), new=new,
                    ctx=f"0:{_logint(rng, 1, 8192)}", nodes=nodes, room=rng.choice([0, 1, 511, 4096]))
    D, BS, KH = _shape(rng)
    e4m3 = rng.random() < 0.35
    dtype = rng.choice(["fp16", "bf16", "bf16", "fp32"])
    S, ctx = _logint(rng, 1, 128), _logint(rng, 1, 2000)
    room = max(1, 24 * 2048 * 8 * 128 // (S * KH * D))
    if op == "write":
        top = min(_logint(rng, 1, 2048), room)
        return dict(op=op, dtype=dtype, S=S, KH=KH, D=D, BS=BS, new=f"{rng.choice([0, 1])}:{top}",
                    ctx=f"0:{min(ctx, room)}", e4m3=e4m3, room=rng.choice([0, 1, 63]))
    return dict(op=op, dtype=dtype, S=S, KH=KH, D=D, BS=BS, n=_logint(rng, 1, 100), ctx=f"0:{min(ctx, room)}",
                layers=rng.choice([1, 2, 3, 8]), e4m3=e4m3)


def _lens(text, n, rng):
    lo, hi = (int(v) for v in text.split(":"))
    return [rng.randint(lo, max(lo, hi)) for _ in range(n)]


def _fixed(case):
    """The lengths of a case are its own; a seed gives their order (and all the data)."""
    return random.Random(repr(sorted((k, v) for k, v in case.items() if k != "name")))


def _shuffled(seed, *lists):
    order = list(range(len(lists[0])))
    random.Random(seed).shuffle(order)
    return [[v[i] for i in order] for v in lists]


# ------------------------------------------------------------------ data
def _randn(shape, gen):
    return torch.randn(shape, generator=gen, device=gen.device)


def _fill(shape, dtype, e4m3, scale, gen):
    """A cache of N(0, 1) values, or of the E4M3 codes of N(0, 1) / scale."""
    out = torch.empty(shape, dtype=torch.uint8 if e4m3 else dtype, device=gen.device)
    flat = out.view(-1)
    for i in range(0, flat.numel(), 1 << 28):
        part = flat[i:i + (1 << 28)]
        x = _randn((part.numel(),), gen)
        part.copy_((x / scale).to(torch.float8_e4m3fn).view(torch.uint8) if e4m3 else x)
    return out


def _caches(case, NB, gen):
    KH, D, BS, e4m3 = (case[k] for k in ("KH", "D", "BS", "e4m3"))
    dtype = _T[case["dtype"]]
    x = 16 if e4m3 else 16 // torch.empty((), dtype=dtype).element_size()
    return (_fill((NB, KH, D // x, BS, x), dtype, e4m3, _K_SCALE, gen),
            _fill((NB, KH, D, BS), dtype, e4m3, _V_SCALE, gen))


def _tables(lens, MB, NB, BS, gen):
    """Shuffled distinct pages per sequence, int32 [S, MB] (unused entries 0)."""
    S = len(lens)
    if NB < S * MB:  # sequences drawn from one pool that is smaller than all their tables
        return torch.randint(0, NB, (S, MB), generator=gen, device=gen.device, dtype=torch.int32)
    perm = torch.randperm(NB, generator=gen, device=gen.device)[: S * MB].to(torch.int32).view(S, MB)
    used = torch.tensor([-(-v // BS) for v in lens], device=gen.device)
    cols = torch.arange(MB, device=gen.device)
    return torch.where(cols[None] < used[:, None], perm, torch.zeros_like(perm)).contiguous()


def _parents(S, n, pad, seed, dev):
    """Trees as a drafter makes them: a few children of the last token, most nodes below recent ones."""
    rng = random.Random(seed)
    rows = []
    for _ in range(S):
        live = rng.randint(max(1, n // 2), n) if pad else n
        row = []
        for i in range(n):
            if i >= live:
                row.append(-2)
            elif i == 0 or rng.random() < 0.15:
                row.append(-1)
            else:
                row.append(rng.randint(max(0, i - 5), i - 1))
        rows.append(row)
    return torch.tensor(rows, dtype=torch.int32, device=dev)


def _ancestors(parents):
    """bool [S, n, n]: node i sees node j."""
    S, n = parents.shape
    see = torch.zeros((S, n, n), dtype=torch.bool, device=parents.device)
    rows = torch.arange(S, device=parents.device)
    for i in range(n):
        p = parents[:, i].long()
        see[:, i] = see[rows, p.clamp(min=0)] & (p >= 0)[:, None]
        see[:, i, i] = p >= -1
    return see


def _packed(see):
    """bool [S, n, n] as int32 [S, n, ceil(n / 32)], bit j % 32 of word j // 32."""
    S, n, _ = see.shape
    words = -(-n // 32)
    bits = torch.zeros((S, n, words * 32), dtype=torch.int64, device=see.device)
    bits[..., :n] = see
    w = (bits.view(S, n, words, 32) << torch.arange(32, device=see.device)).sum(-1)
    return torch.where(w >= 1 << 31, w - (1 << 32), w).to(torch.int32)


# ------------------------------------------------------------------ prepare
def prepare(case, seed):
    gen = torch.Generator(device=_dev()).manual_seed(seed)
    st = dict(case=case)
    {"window": _prepare_attention, "tree": _prepare_attention, "slots": _prepare_slots, "write": _prepare_write,
     "accept": _prepare_accept}[case["op"]](case, st, seed, gen)
    return st


def _prepare_attention(case, st, seed, gen):
    S, H, KH, D, BS, n = (case[k] for k in ("S", "H", "KH", "D", "BS", "n"))
    dtype, dev = _T[case["dtype"]], gen.device
    lens, = _shuffled(seed, _lens(case["lens"], S, _fixed(case)))
    MB = max(1, max(-(-v // BS) for v in lens))
    page = KH * BS * D * (1 if case["e4m3"] else torch.empty((), dtype=dtype).element_size())
    NB = S * MB if S * MB * page < 2.5e9 else max(MB, int(2.5e9 / page))
    st["lens_host"] = lens
    # Positions that some row of a sequence may see, at most (what a plain form gathers).
    st["most"] = max(min(v, case["window"] + n + case["sinks"]) if case["window"] else v for v in lens)
    st["lens"] = torch.tensor(lens, dtype=torch.int32, device=dev)
    st["key_cache"], st["value_cache"] = _caches(case, NB, gen)
    st["tables"] = _tables(lens, MB, NB, BS, gen)
    st["query"] = _randn((S, n, H, D) if case["op"] == "tree" or n > 1 else (S, H, D), gen).to(dtype)
    st["out"] = torch.empty_like(st["query"])
    st["scale"] = 1.0 / math.sqrt(D)
    if case["op"] == "tree":
        st["masks"] = _packed(_ancestors(_parents(S, n, case["pad"], seed, dev)))


def _rows(case, st, seed, gen):
    """Lengths, tables and new tokens of a step."""
    S, BS = case["S"], case["BS"]
    rng = _fixed(case)
    new, ctx = _lens(case["new"], S, rng), _lens(case["ctx"], S, rng)
    new[0] = max(new[0], 0 if sum(new) else 1)
    new, ctx = _shuffled(seed, new, ctx)
    lens = [a + b for a, b in zip(new, ctx)]
    MB = max(1, max(-(-v // BS) for v in lens))
    st["lens_host"], st["new_host"] = lens, new
    st["lens"] = torch.tensor(lens, dtype=torch.int32, device=gen.device)
    st["new"] = torch.tensor(new, dtype=torch.int32, device=gen.device)
    st["tables"] = _tables(lens, MB, S * MB, BS, gen)
    return sum(new), S * MB


def _prepare_slots(case, st, seed, gen):
    total, _ = _rows(case, st, seed, gen)
    S, dev, n = case["S"], gen.device, case["nodes"]
    N = total + case["room"]
    st["slots"] = torch.empty((N,), dtype=torch.int64, device=dev)
    st["positions"] = torch.empty((N,), dtype=torch.int32, device=dev)
    st["seq_ids"] = torch.empty((N,), dtype=torch.int32, device=dev)
    st["cu"] = torch.empty((S + 1,), dtype=torch.int32, device=dev)
    if n:
        st["parents"] = _parents(S, n, True, seed, dev)
        st["masks"] = torch.empty((S, n, -(-n // 32)), dtype=torch.int32, device=dev)
        st["node_positions"] = torch.empty((S, n), dtype=torch.int32, device=dev)


def _slots_of(st, BS, room):
    """The slots of a step's rows, -1 for the room behind them (made where the data is)."""
    out = []
    tables = st["tables"].tolist()
    for s, (L, n) in enumerate(zip(st["lens_host"], st["new_host"])):
        out += [tables[s][t // BS] * BS + t % BS for t in range(L - n, L)]
    return torch.tensor(out + [-1] * room, dtype=torch.int64, device=st["tables"].device)


def _prepare_write(case, st, seed, gen):
    _, NB = _rows(case, st, seed, gen)
    KH, D = case["KH"], case["D"]
    st["key_cache"], st["value_cache"] = _caches(case, NB, gen)
    st["slots"] = _slots_of(st, case["BS"], case["room"])
    # Keys and values as they leave a fused projection: slices of wider rows.
    st["qkv"] = _randn((st["slots"].numel(), 3 * KH, D), gen).to(_T[case["dtype"]])
    st["key"], st["value"] = st["qkv"][:, KH:2 * KH], st["qkv"][:, 2 * KH:]
    st["scales"] = (_K_SCALE, _V_SCALE) if case["e4m3"] else (1.0, 1.0)


def _prepare_accept(case, st, seed, gen):
    S, n, BS, dev = case["S"], case["n"], case["BS"], gen.device
    ctx, = _shuffled(seed, _lens(case["ctx"], S, _fixed(case)))
    lens = [v + n for v in ctx]
    MB = max(-(-v // BS) for v in lens)
    st["lens"] = torch.tensor(lens, dtype=torch.int32, device=dev)
    st["tables"] = _tables(lens, MB, S * MB, BS, gen)
    pairs = [_caches(case, S * MB, gen) for _ in range(case["layers"])]
    st["key_caches"], st["value_caches"] = [p[0] for p in pairs], [p[1] for p in pairs]
    # The accepted path of each tree: ascending nodes, none to most of them.
    rng = random.Random(seed)
    most = max(1, min(n, 8))
    paths = [sorted(rng.sample(range(n), rng.randint(0, most))) for _ in range(S)]
    st["accepted"] = torch.tensor([p + [0] * (most - len(p)) for p in paths], dtype=torch.int32, device=dev)
    st["num_accepted"] = torch.tensor([len(p) for p in paths], dtype=torch.int32, device=dev)
    st["new_lens"] = torch.empty((S,), dtype=torch.int32, device=dev)


# ------------------------------------------------------------------ run
def run(st):
    return {"window": _run_attention, "tree": _run_attention, "slots": _run_slots, "write": _run_write,
            "accept": _run_accept}[st["case"]["op"]](st)


def _own_attention(st):
    import decode_attention_paged_pa_gb300 as pa
    c = st["case"]
    args = [st["out"], st["query"], st["key_cache"], st["value_cache"], st["tables"], st["lens"]]
    more = dict(partition_size=c["P"], workspace=st.get("ws"))  # the workspace of the first pass is kept
    if c["e4m3"]:
        more |= dict(k_scale=_K_SCALE, v_scale=_V_SCALE)
    if c["op"] == "window":
        call = pa.pa_decode_v2_window_fp8 if c["e4m3"] else pa.pa_decode_v2_window
        st["ws"] = call(*args, st["scale"], c["window"], c["sinks"], **more)
    else:
        call = pa.pa_decode_v2_tree_fp8 if c["e4m3"] else pa.pa_decode_v2_tree
        st["ws"] = call(*args, st["masks"], st["scale"], window=c["window"], sinks=c["sinks"], **more)
    return st["out"]


def _values(cache, e4m3, scale):
    return cache.view(torch.float8_e4m3fn).float() * scale if e4m3 else cache.float()


def _run_attention(st):
    if own:
        return _own_attention(st)
    c = st["case"]
    S, H, KH, D, BS, n, window, sinks = (c[k] for k in ("S", "H", "KH", "D", "BS", "n", "window", "sinks"))
    dev = st["query"].device
    L = st["lens"].long()
    base = L - n  # the position of a sequence's first new token
    # The positions that some row may see: the first ones, and those from `low` on.
    low = (base + 1 - window).clamp(min=0) if window else torch.zeros_like(L)
    first = low.clamp(max=sinks)
    j = torch.arange(st["most"], device=dev)[None]
    pos = torch.where(j < first[:, None], j, j - first[:, None] + low[:, None])
    there = pos < L[:, None]
    pos = torch.where(there, pos, torch.zeros_like(pos))
    block, slot = st["tables"].gather(1, pos // BS).long(), pos % BS
    k = _values(st["key_cache"][block, :, :, slot], c["e4m3"], _K_SCALE).flatten(-2)  # [S, T, KH, D]
    v = _values(st["value_cache"][block, :, :, slot], c["e4m3"], _V_SCALE)
    i = torch.arange(n, device=dev)
    if c["op"] == "tree":
        bits = (st["masks"].unsqueeze(-1) >> torch.arange(32, device=dev, dtype=torch.int32)) & 1
        bits = bits.flatten(-2)[..., :n].bool()  # [S, n, n]
        depth = bits.sum(-1)
        at = base[:, None] + depth - 1  # a node's position in its sequence
        node = (pos - base[:, None]).clamp(min=0, max=n - 1)
        see = torch.where((pos < base[:, None])[:, None], (depth > 0)[..., None],
                          bits.gather(2, node[:, None].expand(S, n, pos.shape[1])))
    else:
        at = base[:, None] + i
        see = pos[:, None] <= at[..., None]
    if window:
        drafted = (pos >= base[:, None])[:, None] & (c["op"] == "tree")
        see = see & ((pos[:, None] > at[..., None] - window) | (pos < sinks)[:, None] | drafted)
    see = see & there[:, None]  # [S, n, T]
    q = st["query"].view(S, n, KH, H // KH, D).permute(0, 2, 1, 3, 4).reshape(S, KH, -1, D).float()
    z = torch.matmul(q, k.permute(0, 2, 3, 1)) * st["scale"]  # [S, KH, n * G, T]
    z = z.view(S, KH, n, H // KH, -1).masked_fill_(~see[:, None, :, None], -math.inf)
    m = z.amax(dim=-1, keepdim=True)
    p = torch.exp(z.sub_(torch.where(m == -math.inf, torch.zeros_like(m), m)))
    s = p.sum(dim=-1, keepdim=True)
    o = torch.matmul(p.flatten(2, 3), v.permute(0, 2, 1, 3)).view(S, KH, n, -1, D)
    o = torch.where(s > 0, o / s, torch.zeros_like(o))
    return o.permute(0, 2, 1, 3, 4).reshape(st["query"].shape).to(st["query"].dtype)


def _run_slots(st):
    c = st["case"]
    n, BS = c["nodes"], c["BS"]
    if own:
        import decode_attention_paged_pa_gb300 as pa
        st["ws"] = pa.pa_pages_slots(st["slots"], st["positions"], st["seq_ids"], st["cu"], st["tables"], st["lens"],
                                     st["new"], BS, workspace=st.get("ws"))
        if n:
            st["ws"] = pa.pa_tree_masks(st["masks"], st["node_positions"], st["parents"], st["lens"],
                                        workspace=st["ws"])
    else:
        new, L = st["new"].long(), st["lens"].long()
        cu = torch.nn.functional.pad(torch.cumsum(new, 0), (1, 0))
        row = torch.arange(st["slots"].numel(), device=L.device)
        seq = torch.bucketize(row, cu[1:], right=True)
        there = row < cu[-1]
        seq = torch.where(there, seq, torch.zeros_like(seq))
        pos = torch.where(there, L[seq] - new[seq] + row - cu[seq], torch.zeros_like(row))
        slot = st["tables"][seq, pos // BS].long() * BS + pos % BS
        none = torch.full_like(row, -1)
        st["slots"].copy_(torch.where(there, slot, none))
        st["positions"].copy_(torch.where(there, pos, none))
        st["seq_ids"].copy_(torch.where(there, seq, none))
        st["cu"].copy_(cu)
        if n:
            # Each node's ancestors, by doubling: those of its ancestor 1, 2, 4, ... levels up.
            par = st["parents"].long()
            eye = torch.eye(n, dtype=torch.float32, device=par.device)
            live = (par >= -1)[..., None]
            up = torch.nn.functional.one_hot(par.clamp(min=0), n).float() * (par >= 0)[..., None]
            see = eye + up
            for _ in range((n - 1).bit_length()):
                see = (torch.matmul(see, see) > 0).float()
            see = (see > 0) & live
            st["masks"].copy_(_packed(see))
            depth = see.sum(-1)
            st["node_positions"].copy_(torch.where(depth > 0, L[:, None] - n + depth - 1, torch.full_like(depth, -1)))
    trees = [st["masks"], st["node_positions"]] if n else []
    return [st["slots"], st["positions"], st["seq_ids"], st["cu"], *trees]


def _run_write(st):
    c = st["case"]
    kc, vc = st["key_cache"], st["value_cache"]
    ks, vs = st["scales"]
    if own:
        import decode_attention_paged_pa_gb300 as pa
        st["ws"] = pa.pa_cache_write(kc, vc, st["key"], st["value"], st["slots"], k_scale=ks, v_scale=vs,
                                     workspace=st.get("ws"))
    else:
        keep = st["slots"] >= 0
        slots = st["slots"][keep]
        block, off = slots // c["BS"], slots % c["BS"]
        key, value = st["key"][keep], st["value"][keep]
        if c["e4m3"]:
            # (Divisors on the device: torch turns a scalar one into a product with its reciprocal.)
            key, value = ((t.float() / torch.full((), s, device=t.device)).clamp(-448, 448).to(torch.float8_e4m3fn)
                          .view(torch.uint8) for t, s in ((key, ks), (value, vs)))
        kc[block, :, :, off] = key.unflatten(-1, kc.shape[2::2])
        vc[block, :, :, off] = value
    # (Codes are looked at as the values that they stand for.)
    return [t.view(torch.float8_e4m3fn) if c["e4m3"] else t for t in (kc, vc)]


def _run_accept(st):
    c = st["case"]
    n, BS = c["n"], c["BS"]
    if own:
        import decode_attention_paged_pa_gb300 as pa
        st["ws"] = pa.pa_tree_accept(st["new_lens"], st["key_caches"], st["value_caches"], st["tables"], st["lens"],
                                     st["accepted"], st["num_accepted"], n, workspace=st.get("ws"))
    else:
        L, count = st["lens"].long(), st["num_accepted"].long()
        i = torch.arange(st["accepted"].shape[1], device=L.device)[None]
        live = i < count[:, None]
        base = (L - n)[:, None]
        src, dst = base + st["accepted"].long(), base + i
        rows = torch.arange(L.numel(), device=L.device)[:, None].expand_as(src)[live]
        src, dst = src[live], dst[live]
        from_block, to_block = st["tables"][rows, src // BS].long(), st["tables"][rows, dst // BS].long()
        st["new_lens"].copy_(L - n + count)
        _move(st["key_caches"] + st["value_caches"], from_block, src % BS, to_block, dst % BS)
    out = [t.view(torch.float8_e4m3fn) if c["e4m3"] else t for t in st["key_caches"] + st["value_caches"]]
    return [st["new_lens"], *out]


def _move(caches, from_block, from_off, to_block, to_off):
    for t in caches:
        t[to_block, :, :, to_off] = t[from_block, :, :, from_off]


# ------------------------------------------------------------------ work
def _seen(case):
    """Per sequence: positions that some row sees, and the rows' positions summed."""
    n, window, sinks = case["n"], case["window"], case["sinks"]
    for L in _lens(case["lens"], case["S"], _fixed(case)):
        if not window:
            yield L, n * (L - n) + (n * (n + 1) // 2 if case["op"] == "window" else n * 4)
            continue
        low = max(0, L - n + 1 - window)
        rows = sum(min(p + 1, window + max(0, min(sinks, p + 1 - window))) for p in range(L - n, L))
        yield L - low + min(sinks, low), rows


def work(case):
    op = case["op"]
    size = 1 if case.get("e4m3") else 4 if case.get("dtype") == "fp32" else 2
    if op in ("window", "tree"):
        S, H, KH, D, n = (case[k] for k in ("S", "H", "KH", "D", "n"))
        seen = list(_seen(case))
        tok, pairs = sum(a for a, _ in seen), sum(b for _, b in seen)
        io = 2 * S * n * H * D * (4 if case["dtype"] == "fp32" else 2)
        return {"bytes": 2 * tok * KH * D * size + io + 4 * tok / case["BS"] + 4 * S, "flops": 4 * pairs * H * D}
    if op == "accept":
        S, KH, D = (case[k] for k in ("S", "KH", "D"))
        moved = S * min(case["n"], 8) / 2
        return {"bytes": 4 * moved * case["layers"] * KH * D * size + 8 * S, "flops": 0}
    S = case["S"]
    rng = _fixed(case)
    rows = sum(_lens(case["new"], S, rng))
    if op == "slots":
        n = case["nodes"]
        trees = S * n * (8 + 4 * -(-n // 32))
        return {"bytes": 16 * (rows + case["room"]) + 12 * S + 4 * max(S, rows / case["BS"]) + trees, "flops": 0}
    wide = 4 if case["dtype"] == "fp32" else 2
    return {"bytes": rows * (2 * case["KH"] * case["D"] * (wide + size) + 8), "flops": 0}


# ------------------------------------------------------------------ exact
def exact(case, seed):
    """What ``run`` returns, in 64 bits; None where values are placed rather than computed."""
    if case["op"] in ("window", "tree"):
        return _exact_attention(case, prepare(case, seed))
    if case["op"] == "write" and case["e4m3"]:
        return _exact_write(case, prepare(case, seed))
    return None


def _tokens64(cache, ids, e4m3, scale, keys):
    """The tokens of the blocks `ids` as fp64 [KH, tokens, D]."""
    t = cache[ids]
    t = (t.view(torch.float8_e4m3fn) if e4m3 else t).double() * (scale if e4m3 else 1.0)
    t = t.permute(1, 0, 3, 2, 4).flatten(3) if keys else t.permute(1, 0, 3, 2)  # [KH, blocks, BS, D]
    return t.flatten(1, 2)


def _exact_attention(case, st):
    S, H, KH, D, BS, n, window, sinks = (case[k] for k in ("S", "H", "KH", "D", "BS", "n", "window", "sinks"))
    if sum(b for _, b in _seen(case)) * H * D > 5e11:
        return None
    q = st["query"].double().view(S, n, KH, H // KH, D)
    res = torch.zeros_like(q)
    tree = case["op"] == "tree"
    words = st["masks"].tolist() if tree else None
    for s, L in enumerate(st["lens_host"]):
        if L == 0:
            continue
        ids = st["tables"][s, : (L + BS - 1) // BS].long()
        K = _tokens64(st["key_cache"], ids, case["e4m3"], _K_SCALE, True)[:, :L]
        V = _tokens64(st["value_cache"], ids, case["e4m3"], _V_SCALE, False)[:, :L]
        t = torch.arange(L, device=K.device)
        hide = torch.ones((n, L), dtype=torch.bool, device=K.device)
        for i in range(n):
            here = L - n + i
            hide[i] = t > here
            if tree:
                mine = [j for j in range(n) if (words[s][i][j // 32] >> (j % 32)) & 1]
                here = L - n + len(mine) - 1
                hide[i] = (t >= L - n) if mine else True
            if window:
                hide[i] |= (t <= here - window) & (t >= sinks)
            if tree and mine:
                hide[i, [L - n + j for j in mine]] = False
        for i in range(n):
            keep = ~hide[i]
            if not bool(keep.any()):
                continue
            z = torch.einsum("kgd,ktd->kgt", q[s, i], K[:, keep]) * st["scale"]
            res[s, i] = torch.einsum("kgt,ktd->kgd", torch.softmax(z, dim=-1), V[:, keep])
    return res.view(st["query"].shape)


def _exact_write(case, st):
    res = []
    for cache, rows, scale in ((st["key_cache"], st["key"], st["scales"][0]), (st["value_cache"], st["value"], st["scales"][1])):
        out = cache.view(torch.float8_e4m3fn).double()
        x = (rows.double() / scale).clamp(-448.0, 448.0)
        at = st["slots"].tolist()
        keep = [r for r, a in enumerate(at) if a >= 0]
        block = torch.tensor([at[r] // case["BS"] for r in keep], device=out.device)
        off = torch.tensor([at[r] % case["BS"] for r in keep], device=out.device)
        if out.dim() == 5:
            for d in range(0, case["D"], out.shape[4]):
                out[block, :, d // out.shape[4], off] = x[keep, :, d:d + out.shape[4]]
        else:
            out[block, :, :, off] = x[keep]
        res.append(out)
    return res
