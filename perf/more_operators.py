"""The attention operators as they are measured: cases, inputs, and each operator in its plain form (elementary
torch operations in 32 bits) beside the library's call.

A step has S sequences, whose new tokens are packed rows of one matrix, [q | k | v] as a packed qkv projection
leaves them. "prompt" attends over the rows of a sequence themselves; "paged" over a cache of pages that holds the
sequence's keys and values, its new ones among them; "write" puts the new rows into that cache. A paged case with
"step" is the whole of a layer: the step's plan, the write, the attention."""
import math
import random

import torch

own = False

NEG = float("-inf")


# ----------------------------------------------------------------------------- cases

def _case(name, op, heads, q, ctx=(0, 0), page=16, dtype="bf16", causal=True, lse=False, mix=0, step=False):
    """heads: (query heads, key-value heads, head size); q and ctx: (sequences, fewest, most) new tokens and
    (fewest, most) tokens in the cache before them; mix: which lengths of those ranges; step: with plan and write."""
    case = dict(op=op, Hq=heads[0], Hkv=heads[1], D=heads[2], S=q[0], q_min=q[1], q_max=q[2], c_min=ctx[0], c_max=ctx[1],
                page=page, dtype=dtype, causal=causal, lse=lse, mix=mix, step=step)
    return dict(case, name=name) if name else case


def listed():
    big = (32, 8, 128)      # the packed qkv projection of 4096 + 1024 + 1024 columns
    return [
        # The new token of each of 256 decoding requests into the cache.
        _case("write_decode", "write", big, (256, 1, 1), (0, 400)),
        # Sixteen prompts' rows into the cache.
        _case("write_prefill", "write", big, (16, 128, 2048)),
        # Six short requests in fp32, an accuracy run: latency.
        _case("prompt_toy_f32", "prompt", (4, 2, 64), (6, 1, 37), dtype="f32", lse=True),
        # One short prompt: latency.
        _case("prompt_short", "prompt", big, (1, 117, 117)),
        # A prefill step of sixteen prompts of different lengths.
        _case("prompt_packed", "prompt", big, (16, 128, 2048)),
        # Eight documents, every token seeing all of its own, heads of 64 without groups: an encoder's layer.
        _case("prompt_full_d64", "prompt", (20, 20, 64), (8, 301, 1999), causal=False, lse=True),
        # One long prompt.
        _case("prompt_long", "prompt", big, (1, 16381, 16381)),
        # One decoding request: latency.
        _case("decode_single", "paged", big, (1, 1, 1), (999, 999)),
        # A decode step of 256 requests, from short to long contexts.
        _case("decode_batch", "paged", big, (256, 1, 1), (1, 4000)),
        # A few requests over very long contexts, a layer of groups of eight.
        _case("decode_long", "paged", (64, 8, 128), (3, 1, 1), (90001, 131000), page=64, lse=True),
        # Prompts cut into chunks of up to 512 tokens, attending over what came before them.
        _case("chunk_prefill", "paged", big, (12, 65, 512), (0, 7600), page=32),
        # A layer of a decode step with a few draft tokens a request: plan, write and attention.
        _case("step_draft", "paged", (28, 4, 128), (48, 1, 5), (17, 2000), step=True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


_HEADS = [(32, 8, 128), (64, 8, 128), (28, 4, 128), (40, 8, 128), (16, 2, 128), (20, 20, 64), (12, 12, 64), (16, 1, 64), (6, 2, 64), (9, 3, 64)]


def draw(rng):
    op = rng.choice(["write", "prompt", "prompt", "paged", "paged", "paged", "paged"])
    step = op == "paged" and rng.random() < 0.25
    mix = rng.randrange(1 << 20)
    f32 = op != "write" and rng.random() < 0.1
    page = rng.choice([16, 16, 32, 64, 128])
    if f32:         # accuracy runs are small
        heads = rng.choice([(4, 2, 64), (6, 2, 64), (4, 1, 80), (3, 3, 128)])
        q, ctx = (_log(rng, 1, 12), 1, _log(rng, 1, 200)), (0, _log(rng, 1, 300))
        return _case(None, op, heads, q, ctx, page, "f32", rng.random() < 0.7, rng.random() < 0.5, mix, step)
    heads = rng.choice(_HEADS)
    if op == "write":
        n = _log(rng, 1, 2048)
        return _case(None, op, heads, (max(1, min(300, _log(rng, 1, 16000) // n)), rng.randint(1, n), n), (0, _log(rng, 1, 400)), page, mix=mix)
    if op == "prompt":
        n = _log(rng, 1, 9000)
        S = max(1, min(40, _log(rng, 1, 20000) // n))
        while S > 1 and S * heads[0] * n * n > 3 << 30:
            S -= 1
        return _case(None, op, heads, (S, max(1, int(n * rng.random())), n), (0, 0), page, "bf16", rng.random() < 0.7, rng.random() < 0.3, mix)
    decode = rng.random() < 0.5
    n = 1 if decode else _log(rng, 1, 6 if step else 1000)
    c = _log(rng, 1, 131000 if decode else 8000)
    S = _log(rng, 1, 256)
    while S > 1 and (S * (c + n) * heads[1] * heads[2] > 1 << 30 or S * heads[0] * n * (c + n) > 3 << 30):
        S = S * 3 // 4
    return _case(None, op, heads, (S, max(1, int(n * rng.random())), n), (int(c * rng.random()), c), page, "bf16", rng.random() < 0.8,
                 rng.random() < 0.3, mix, step)


def _lengths(case):
    """New tokens and tokens before them of every sequence: the same for every seed."""
    r = random.Random(case["mix"])
    n = [r.randint(case["q_min"], case["q_max"]) for _ in range(case["S"])]
    c = [r.randint(case["c_min"], case["c_max"]) for _ in range(case["S"])]
    return n, [0] * len(n) if case["op"] == "prompt" else c


# ----------------------------------------------------------------------------- inputs

def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    s = dict(case)
    n, c = _lengths(case)
    T, S, Hq, Hkv, D, ps = sum(n), case["S"], case["Hq"], case["Hkv"], case["D"], case["page"]
    dtype = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
    qkv = torch.empty(T, (Hq + 2 * Hkv) * D, dtype=dtype, device="cuda")
    qkv.normal_(generator=g)
    qkv[:, :Hq * D] *= 2                                        # some keys matter more than others
    s["q"], s["k"], s["v"] = qkv.split([Hq * D, Hkv * D, Hkv * D], 1)
    s["out"] = torch.zeros(T, Hq * D, dtype=dtype, device="cuda")
    s["lse_out"] = torch.zeros(T, Hq, dtype=torch.float32, device="cuda") if case["lse"] else None
    start = [0]
    for x in n:
        start.append(start[-1] + x)
    s["q_start"] = torch.tensor(start, dtype=torch.int32, device="cuda")
    s["n"], s["T"], s["n_most"] = n, T, max(n)
    kv = [a + b for a, b in zip(n, c)]
    s["kv_len"] = torch.tensor(kv, dtype=torch.int32, device="cuda")
    s["kv_most"] = max(kv)
    paged = case["op"] != "prompt"
    pages = -(-max(kv) // ps)
    if paged:
        # Pages in the order in which a pool hands them out after a while of use: any.
        need = [-(-x // ps) for x in kv]
        pool = sum(need) + 7
        perm = torch.randperm(pool, device="cuda", generator=g, dtype=torch.int32)
        table = torch.zeros(S, pages, dtype=torch.int32, device="cuda")
        here = torch.arange(pages, device="cuda")[None] < torch.tensor(need, device="cuda")[:, None]
        table[here] = perm[:sum(need)]
        s["table"] = table
        cache = torch.empty(2, pool, ps, Hkv, D, dtype=dtype, device="cuda").normal_(generator=g)
        s["k_cache"], s["v_cache"] = cache[0], cache[1]
        row_seq = torch.repeat_interleave(torch.arange(S, device="cuda"), torch.tensor(n, device="cuda"))
        pos = torch.arange(T, device="cuda") - s["q_start"].long()[row_seq] + torch.tensor(c, device="cuda")[row_seq]
        s["page_of"], s["slot_of"] = table[row_seq, pos // ps].long(), pos % ps
        if case["op"] == "paged" and not case["step"]:          # the new rows are in the cache already
            s["k_cache"][s["page_of"], s["slot_of"]] = s["k"].reshape(T, Hkv, D)
            s["v_cache"][s["page_of"], s["slot_of"]] = s["v"].reshape(T, Hkv, D)
    if own:
        # The step's plan (one serves all layers of a step) and what a serving loop keeps.
        import rank_adapter_gb300 as ra
        att = ra.Attention(Hq, Hkv, D, causal=case["causal"], dtype=ra.LORA_BF16 if case["dtype"] == "bf16" else ra.LORA_F32)
        s["seqs"] = ra.SeqMeta(att, T, S, page_size=ps if paged else 0, max_pages=pages if paged else 0)
        s["seqs"].prepare(T, s["q_start"], s["kv_len"] if paged else None, s["table"] if paged else None)
        s["ws"] = ra.attn_workspace(s["seqs"])
        if paged:
            s["cache"] = ra.KVCache(s["k_cache"], s["v_cache"])
    return s


# ----------------------------------------------------------------------------- one pass

def _plain_write(s):
    s["k_cache"][s["page_of"], s["slot_of"]] = s["k"].reshape(s["T"], s["Hkv"], s["D"])
    s["v_cache"][s["page_of"], s["slot_of"]] = s["v"].reshape(s["T"], s["Hkv"], s["D"])


def _plain_attention(s):
    """Every sequence padded to the longest: [S, Hkv, group, rows, keys] scores in one product."""
    S, Hq, Hkv, D, T = s["S"], s["Hq"], s["Hkv"], s["D"], s["T"]
    G, Lq, Lk, ps = Hq // Hkv, s["n_most"], s["kv_most"], s["page"]
    dev = s["q"].device
    start, kv = s["q_start"].long(), s["kv_len"].long()
    n = start[1:] - start[:-1]
    i, j = torch.arange(Lq, device=dev), torch.arange(Lk, device=dev)
    live_q, live_k = i[None] < n[:, None], j[None] < kv[:, None]
    rows = (start[:-1, None] + i[None]).clamp(max=T - 1)
    q = s["q"].reshape(T, Hkv, G, D)[rows].float().permute(0, 2, 3, 1, 4).reshape(S, Hkv, G * Lq, D)
    if s["op"] == "prompt":
        at = (start[:-1, None] + j[None]).clamp(max=T - 1)
        k, v = s["k"].reshape(T, Hkv, D)[at], s["v"].reshape(T, Hkv, D)[at]
    else:
        page, slot = s["table"].long()[:, j // ps], (j % ps)[None].expand(S, Lk)
        k, v = s["k_cache"][page, slot], s["v_cache"][page, slot]
    k = k.float().permute(0, 2, 3, 1)                                           # [S, Hkv, D, Lk]
    v = v.float().masked_fill_(~live_k[:, :, None, None], 0).permute(0, 2, 1, 3)
    x = torch.matmul(q, k).mul_(D ** -0.5).view(S, Hkv, G, Lq, Lk)
    hidden = ~live_k[:, None, :].expand(S, Lq, Lk)
    if s["causal"]:
        hidden = hidden | (j[None, None] > (kv - n)[:, None, None] + i[None, :, None])
    x.masked_fill_(hidden[:, None, None], NEG)
    m = x.amax(-1, keepdim=True)
    m = torch.where(torch.isinf(m), torch.zeros_like(m), m)
    x.sub_(m).exp_()
    total = x.sum(-1, keepdim=True)
    o = torch.matmul(x.view(S, Hkv, G * Lq, Lk), v).view(S, Hkv, G, Lq, D)
    o = o / torch.where(total > 0, total, torch.ones_like(total))
    s["out"][rows[live_q]] = o.permute(0, 3, 1, 2, 4).reshape(S, Lq, Hq * D)[live_q].to(s["out"].dtype)
    if not s["lse"]:
        return s["out"]
    lse = (m + torch.log(total)).squeeze(-1).permute(0, 3, 1, 2).reshape(S, Lq, Hq)
    s["lse_out"][rows[live_q]] = lse[live_q]
    return s["out"], s["lse_out"]


def run(state):
    s = state
    op, step = s["op"], s["step"]
    if own:
        import rank_adapter_gb300 as ra
        if step:
            s["seqs"].prepare(s["T"], s["q_start"], s["kv_len"], s["table"])
        if op == "write" or step:
            ra.kv_write(s["seqs"], s["cache"], s["k"], s["v"])
        if op == "prompt":
            ra.attn_prompt(s["seqs"], s["q"], s["k"], s["v"], s["out"], lse=s["lse_out"], ws=s["ws"])
        elif op != "write":
            ra.attn_paged(s["seqs"], s["cache"], s["q"], s["out"], lse=s["lse_out"], ws=s["ws"])
    else:
        if op == "write" or step:
            _plain_write(s)
        if op != "write":
            _plain_attention(s)
    outputs = []
    if op != "write":
        outputs += [s["out"]] + ([s["lse_out"]] if s["lse"] else [])
    if op == "write" or step:
        outputs += [s["k_cache"], s["v_cache"]]
    return outputs


# ----------------------------------------------------------------------------- what a pass cannot do without

def work(case):
    n, c = _lengths(case)
    e = 2 if case["dtype"] == "bf16" else 4
    T, Hq, Hkv, D = sum(n), case["Hq"], case["Hkv"], case["D"]
    written = 4 * T * Hkv * D * e
    if case["op"] == "write":
        return {"bytes": written, "flops": 0}
    seen = sum(a * b + a * (a + 1) // 2 if case["causal"] else a * (a + b) for a, b in zip(n, c))   # (row, key) pairs
    keys = sum(n) + sum(c)
    total = 2 * T * Hq * D * e + 2 * keys * Hkv * D * e + (4 * T * Hq if case["lse"] else 0)
    return {"bytes": total + (written // 2 if case["step"] else 0), "flops": 4 * D * Hq * seen}


# ----------------------------------------------------------------------------- 64 bits

def exact(case, seed):
    n, c = _lengths(case)
    w = work(case)
    if w["flops"] > 3e11 or w["bytes"] > 4e9:     # most of the time is in 64-bit products: a few seconds for these
        return None
    s = prepare(case, seed)
    Hq, Hkv, D, ps = case["Hq"], case["Hkv"], case["D"], case["page"]
    if case["op"] == "write" or case["step"]:
        for b, (a, before) in enumerate(zip(n, c)):
            r0 = int(s["q_start"][b])
            p = torch.arange(before, before + a, device="cuda")
            page = s["table"][b].long()[torch.div(p, ps, rounding_mode="floor")]
            s["k_cache"][page, p % ps] = s["k"][r0:r0 + a].reshape(a, Hkv, D)
            s["v_cache"][page, p % ps] = s["v"][r0:r0 + a].reshape(a, Hkv, D)
        if case["op"] == "write":
            return [s["k_cache"].double(), s["v_cache"].double()]
    out = torch.zeros(s["T"], Hq, D, dtype=torch.float64, device="cuda")
    lse = torch.zeros(s["T"], Hq, dtype=torch.float64, device="cuda")
    for b, (a, before) in enumerate(zip(n, c)):
        r0, L = int(s["q_start"][b]), a + before
        if case["op"] == "prompt":
            k, v = s["k"][r0:r0 + L].reshape(L, Hkv, D), s["v"][r0:r0 + L].reshape(L, Hkv, D)
        else:
            ids = s["table"][b, :-(-L // ps)].long()
            k, v = s["k_cache"][ids].reshape(-1, Hkv, D)[:L], s["v_cache"][ids].reshape(-1, Hkv, D)[:L]
        q = s["q"][r0:r0 + a].reshape(a, Hq, D).double()
        sees = torch.ones(a, L, dtype=torch.bool, device="cuda")
        if case["causal"]:
            sees = sees.tril(before)
        for h in range(Hkv):
            heads = slice(h * (Hq // Hkv), (h + 1) * (Hq // Hkv))
            z = torch.einsum("ahd,kd->hak", q[:, heads], k[:, h].double()) / math.sqrt(D)
            z = z.masked_fill(~sees, NEG)
            lse[r0:r0 + a, heads] = torch.logsumexp(z, -1).T
            out[r0:r0 + a, heads] = torch.einsum("hak,kd->ahd", torch.softmax(z, -1), v[:, h].double())
    outputs = [out.reshape(s["T"], Hq * D)] + ([lse] if case["lse"] else [])
    return outputs + ([s["k_cache"].double(), s["v_cache"].double()] if case["step"] else [])
