"""Cases of the batch builder, the latent cache writer and dense MLA attention.

`run` computes an operator in elementary torch operations (`own` false) or
through the library (`own` true) on what `prepare` puts on the GPU; `exact`
computes the same results in 64 bits.
"""
from __future__ import annotations

import math
import random

import numpy as np
import torch

own = False

DK, DV = 576, 512  # a latent row: 512 latent dims (the values), then 64 rope dims
FP8_ROW = 656      # 512 e4m3 codes, 4 fp32 group scales, 64 bf16 rope dims
SCALE = 1.0 / math.sqrt(DK)
MAX_FLOPS = 4.5e12      # of a drawn attention case
MAX_KEYS = 8 * 131072   # cached keys of a drawn attention case


def _attention(name, B, L, q, H, fp8=False, block=64, shape_seed=7):
    """L (cached keys, the new tokens among them) and q (new tokens): the
    lowest and the highest of the requests, drawn from shape_seed."""
    return {"name": name, "op": "attention", "B": B, "L_lo": L[0], "L_hi": L[1], "q_lo": q[0], "q_hi": q[1], "H": H,
            "fp8": fp8, "block": block, "shape_seed": shape_seed}


def _batch(name, B, ctx, new, pad, block, shape_seed):
    return {"name": name, "op": "batch", "B": B, "ctx_lo": ctx[0], "ctx_hi": ctx[1], "new_lo": new[0],
            "new_hi": new[1], "pad": pad, "block": block, "shape_seed": shape_seed}


def _cache(name, T, rows, stride, pad, block):
    return {"name": name, "op": "cache", "T": T, "rows": rows, "stride": stride, "pad": pad, "block": block}


def listed():
    return [
        # the metadata of one decode step: 32 requests with one new token each
        _batch("batch_decode_b32", 32, (1, 8192), (1, 1), 0, 64, 1),
        # a large ragged batch of prompts and decoding requests, in buffers padded for a captured graph
        _batch("batch_prompts_b512", 512, (0, 4096), (0, 511), 517, 128, 2),
        # the new latent rows of a decode batch
        _cache("cache_decode_t32", 32, 16384, DK, 0, 64),
        # the latent rows of a prompt, cut out of a wider projection's rows, some slots padding
        _cache("cache_prompt_t16384", 16384, 32768, 2112, 100, 64),
        # one short request: what a call costs at least
        _attention("dense_b1_l256", 1, (256, 256), (1, 1), 128),
        # a decode batch over moderate contexts
        _attention("dense_decode_b32_l8192", 32, (8192, 8192), (1, 1), 128),
        # the same over the fp8 cache
        _attention("dense_decode_fp8_b32_l8192", 32, (8192, 8192), (1, 1), 128, fp8=True),
        # few requests with long contexts
        _attention("dense_decode_b8_l131072", 8, (131072, 131072), (1, 1), 128),
        # ragged steps of two tokens (a drafted one beside the last)
        _attention("dense_mixed_b64_q2", 64, (1024, 32768), (2, 2), 128),
        # one rank's share of the heads, ragged lengths from one key on
        _attention("dense_decode_h16_b64", 64, (1, 8192), (1, 1), 16),
        # a chunk of a long prompt
        _attention("dense_chunk_1024_of_16384", 1, (16384, 16384), (1024, 1024), 128),
        # ragged chunks over the fp8 cache
        _attention("dense_chunks_fp8_b5", 5, (700, 9000), (1, 700), 128, fp8=True, block=192),
    ]


def _log_int(rng, lo, hi):
    """A whole number from lo to hi, uniform in its logarithm."""
    return min(hi, max(lo, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    op = rng.choice(["batch", "cache", "attention", "attention", "attention"])
    block = rng.choice([64, 64, 128, 192, 256])
    seed = rng.randrange(1 << 30)
    if op == "batch":
        B = _log_int(rng, 1, 512)
        ctx_hi = _log_int(rng, 1, 32768)
        new_hi = _log_int(rng, 1, max(1, 131072 // B))
        return _without_name(_batch("", B, (0, ctx_hi), (rng.choice([0, 1]), new_hi), rng.choice([0, 1, 300]), block,
                                    seed))
    if op == "cache":
        T = _log_int(rng, 1, 16384)
        return _without_name(_cache("", T, 16384 + T, rng.choice([576, 584, 2112]), rng.choice([0, 3]), block))
    H = rng.choice([1, 8, 16, 32, 40, 64, 100, 128])
    B = _log_int(rng, 1, 64)
    L_hi = _log_int(rng, 1, MAX_KEYS // max(B, 8))
    q_hi = 1 if rng.random() < 0.5 else _log_int(rng, 1, 1024)
    q_hi = max(1, min(q_hi, L_hi, int(MAX_FLOPS / (2 * (DK + DV) * H * B * L_hi))))
    return _without_name(_attention("", B, (rng.randint(1, L_hi), L_hi), (rng.randint(1, q_hi), q_hi), H,
                                    fp8=rng.random() < 0.4, block=block, shape_seed=seed))


def _without_name(case):
    del case["name"]
    return case


def _shape(case):
    """The requests' lengths: (L, q) of an attention case, (ctx, new) of a batch."""
    rng = random.Random(case["shape_seed"])
    if case["op"] == "attention":
        L = [rng.randint(case["L_lo"], case["L_hi"]) for _ in range(case["B"])]
        q = [min(n, rng.randint(case["q_lo"], case["q_hi"])) for n in L]
        return L, q
    ctx = [rng.randint(case["ctx_lo"], case["ctx_hi"]) for _ in range(case["B"])]
    new = [rng.randint(case["new_lo"], case["new_hi"]) for _ in range(case["B"])]
    return ctx, new


def _blocks(n, block):
    return (n + block - 1) // block


def work(case):
    if case["op"] == "cache":
        n = case["T"] - min(case["pad"], case["T"] // 2)
        return {"bytes": n * 2 * DK * 2 + case["T"] * 8, "flops": 0}
    B, block = case["B"], case["block"]
    if case["op"] == "batch":
        ctx, new = _shape(case)
        taken = sum(_blocks(c + n, block) - _blocks(c, block) for c, n in zip(ctx, new))
        tokens = sum(new) + case["pad"]
        # lengths in and out, the blocks taken and stored, per token a request, a position and a slot
        held = sum(1 for c, n in zip(ctx, new) if n and c % block)
        return {"bytes": 4 * (4 * B + 3) + 8 * taken + 4 * held + 16 * tokens, "flops": 0}
    L, q = _shape(case)
    H, T = case["H"], sum(q)
    row = FP8_ROW if case["fp8"] else 2 * DK
    pairs = sum(n * (l - n) + n * (n + 1) // 2 for l, n in zip(L, q))  # (token, visible key) pairs
    return {"bytes": sum(L) * row + T * H * (2 * (DK + DV) + (0 if case["fp8"] else 4))
            + 4 * (2 * B + 1 + sum(_blocks(l, block) for l in L)),
            "flops": 2 * (DK + DV) * H * pairs}


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return {"attention": _prepare_attention, "batch": _prepare_batch, "cache": _prepare_cache}[case["op"]](case, gen)


def _tables(lens, block, num_blocks, gen):
    """Block tables over a random permutation of the pool, -1 behind a request's blocks."""
    need = [_blocks(n, block) for n in lens]
    perm = torch.randperm(num_blocks, generator=gen, device="cuda").to(torch.int32)
    table = torch.full((len(lens), max(1, max(need))), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = perm[at:at + n]
        at += n
    return table


def _int32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _prepare_attention(case, gen):
    L, q = _shape(case)
    block, H, T = case["block"], case["H"], sum(q)
    num_blocks = sum(_blocks(n, block) for n in L) + 2
    row = FP8_ROW if case["fp8"] else DK
    cache = torch.empty((num_blocks, block, row), dtype=torch.uint8 if case["fp8"] else torch.bfloat16, device="cuda")
    step = max(1, (1 << 18) // block)
    for i in range(0, num_blocks, step):
        n = min(step, num_blocks - i)
        kv = torch.randn((n, block, DK), generator=gen, device="cuda") * 0.5
        if case["fp8"]:
            groups = kv[..., :DV].reshape(n, block, 4, 128)
            scale = groups.abs().amax(-1) / 448.0
            codes = (groups / scale[..., None]).to(torch.float8_e4m3fn).reshape(n, block, DV)
            cache[i:i + n, :, :DV] = codes.view(torch.uint8)
            cache[i:i + n, :, DV:DV + 16] = scale.view(torch.uint8)
            cache[i:i + n, :, DV + 16:] = kv[..., DV:].to(torch.bfloat16).view(torch.uint8)
        else:
            cache[i:i + n] = kv
    # queries whose scaled scores have a deviation of about 1.5: some keys stand out, none rules
    queries = (torch.randn((T, H, DK), generator=gen, device="cuda") * 3.0).to(torch.bfloat16)
    state = {"case": case, "L": L, "q_lens": q, "q": queries, "cache": cache,
             "block_table": _tables(L, block, num_blocks, gen), "seq_lens": _int32(L), "qsl": _int32(np.concatenate([[0], np.cumsum(q)]).tolist()),
             "out": torch.empty((T, H, DV), dtype=torch.bfloat16, device="cuda"),
             "lse": None if case["fp8"] else torch.empty((T, H), dtype=torch.float32, device="cuda")}
    if own:
        from deepseek_sparse_attention_fp8_gb300 import api
        state["workspace"] = torch.empty(max(16, api.dense_mla_workspace_size(T, H, DV, 0)), dtype=torch.uint8,
                                         device="cuda")
    return state


def _prepare_batch(case, gen):
    ctx, new = _shape(case)
    block = case["block"]
    held = [_blocks(c, block) for c in ctx]
    need = [_blocks(c + n, block) for c, n in zip(ctx, new)]
    num_blocks = sum(need) + 64
    ids = torch.randperm(num_blocks, generator=gen, device="cuda").to(torch.int32)
    table = torch.full((case["B"], max(1, max(need))), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(held):
        table[b, :n] = ids[at:at + n]
        at += n
    # the free ids as a queue whose first entries went to earlier steps
    free = torch.cat([ids[:at][:7], ids[at:]]).contiguous()
    T = sum(new) + case["pad"]
    dev = {"device": "cuda"}
    return {"case": case, "ctx": _int32(ctx), "new": _int32(new), "table": table, "free": free,
            "head": _int32([min(at, 7)]), "max_tokens": T,
            "seq_lens": torch.empty(case["B"], dtype=torch.int32, **dev),
            "qsl": torch.empty(case["B"] + 1, dtype=torch.int32, **dev),
            "token_req": torch.empty(T, dtype=torch.int32, **dev),
            "positions": torch.empty(T, dtype=torch.int32, **dev),
            "slot_map": torch.empty(T, dtype=torch.int64, **dev),
            "head_out": torch.empty(1, dtype=torch.int32, **dev)}


def _prepare_cache(case, gen):
    T, block = case["T"], case["block"]
    num_blocks = _blocks(case["rows"], block) + 1
    wide = torch.randn((T, case["stride"]), generator=gen, device="cuda").to(torch.bfloat16)
    kv = wide[:, case["stride"] - DK:]
    # the last block is nobody's
    slots = torch.randperm((num_blocks - 1) * block, generator=gen, device="cuda")[:T]
    pad = min(case["pad"], T // 2)
    if pad:
        slots[torch.randperm(T, generator=gen, device="cuda")[:pad]] = -1
    cache = torch.randn((num_blocks, block, DK), generator=gen, device="cuda").to(torch.bfloat16)
    return {"case": case, "kv": kv, "slots": slots, "cache": cache}


def run(state):
    op = state["case"]["op"]
    if own:
        return {"attention": _own_attention, "batch": _own_batch, "cache": _own_cache}[op](state)
    return {"attention": _plain_attention, "batch": _plain_batch, "cache": _plain_cache}[op](state)


def _own_attention(s):
    from deepseek_sparse_attention_fp8_gb300 import api
    call = api.dense_mla_attention_fp8 if s["case"]["fp8"] else api.dense_mla_attention
    call(s["q"], s["cache"], s["block_table"], s["seq_lens"], s["qsl"], SCALE, DV, s["out"], lse=s["lse"],
         workspace=s["workspace"])
    return {"out": s["out"]} if s["lse"] is None else {"out": s["out"], "lse": s["lse"]}


def _own_batch(s):
    from deepseek_sparse_attention_fp8_gb300 import api
    api.dsa_build_batch(s["ctx"], s["new"], s["table"], s["case"]["block"], s["max_tokens"], free_blocks=s["free"],
                        free_head=s["head"], free_head_out=s["head_out"], seq_lens=s["seq_lens"],
                        query_start_loc=s["qsl"], token_req=s["token_req"], positions=s["positions"],
                        slot_map=s["slot_map"])
    return {k: s[k] for k in ("table", "seq_lens", "qsl", "token_req", "positions", "slot_map", "head_out")}


def _own_cache(s):
    from deepseek_sparse_attention_fp8_gb300 import api
    api.dsa_mla_kv_cache(s["kv"], s["slots"], s["cache"])
    return {"cache": s["cache"]}


def _rows(s, b, dtype):
    """The latent rows of request b, decoded."""
    L, block = s["L"][b], s["case"]["block"]
    pages = s["cache"][s["block_table"][b, :_blocks(L, block)].long()]
    rows = pages.reshape(-1, pages.shape[-1])[:L]
    if not s["case"]["fp8"]:
        return rows.to(dtype)
    codes = rows[:, :DV].contiguous().view(torch.float8_e4m3fn).to(dtype)
    scale = rows[:, DV:DV + 16].contiguous().view(torch.float32).to(dtype)
    rope = rows[:, DV + 16:].contiguous().view(torch.bfloat16).to(dtype)
    return torch.cat([(codes.view(L, 4, 128) * scale[..., None]).view(L, DV), rope], dim=1)


def _plain_attention(s):
    H = s["case"]["H"]
    t0 = 0
    for b, (L, n) in enumerate(zip(s["L"], s["q_lens"])):
        k = _rows(s, b, torch.float32)
        step = max(1, (1 << 28) // (H * L))
        for i in range(0, n, step):
            m = min(step, n - i)
            q = s["q"][t0 + i:t0 + i + m].float().reshape(m * H, DK)
            scores = (q @ k.T).mul_(SCALE).view(m, H, L)
            pos = torch.arange(L - n + i, L - n + i + m, device="cuda")
            hidden = torch.arange(L, device="cuda")[None, :] > pos[:, None]
            scores.masked_fill_(hidden[:, None, :], -math.inf)
            top = scores.amax(-1, keepdim=True)
            p = scores.sub_(top).exp_()
            total = p.sum(-1, keepdim=True)
            out = (p.view(m * H, L) @ k[:, :DV]).view(m, H, DV) / total
            s["out"][t0 + i:t0 + i + m] = out.to(torch.bfloat16)
            if s["lse"] is not None:
                s["lse"][t0 + i:t0 + i + m] = (top + total.log())[..., 0]
        t0 += n
    return {"out": s["out"]} if s["lse"] is None else {"out": s["out"], "lse": s["lse"]}


def _plain_batch(s):
    ctx, new, table, block = s["ctx"], s["new"], s["table"], s["case"]["block"]
    seq = ctx + new
    qsl = torch.cat([torch.zeros_like(new[:1]), new.cumsum(0, dtype=torch.int32)])
    held, need = (ctx + block - 1) // block, (seq + block - 1) // block
    taken = (need - held).cumsum(0, dtype=torch.int32)
    first = s["head"] + taken - (need - held)
    j = torch.arange(table.shape[1], dtype=torch.int32, device="cuda")[None, :]
    grown = (j >= held[:, None]) & (j < need[:, None])
    source = (first[:, None] + j - held[:, None]).clamp(0, s["free"].shape[0] - 1)
    table.copy_(torch.where(grown, s["free"][source.long()], table))
    t = torch.arange(s["max_tokens"], dtype=torch.int32, device="cuda")
    req = torch.searchsorted(qsl[1:], t, right=True)
    live = t < qsl[-1]
    b = req.clamp(max=ctx.shape[0] - 1)
    pos = ctx[b] + t - qsl[b]
    slot = table[b, torch.where(live, pos // block, 0).long()].long() * block + pos % block
    s["seq_lens"].copy_(seq)
    s["qsl"].copy_(qsl)
    s["token_req"].copy_(torch.where(live, b, -1))
    s["positions"].copy_(torch.where(live, pos, 0))
    s["slot_map"].copy_(torch.where(live, slot, -1))
    s["head_out"].copy_(s["head"] + taken[-1])
    return {k: s[k] for k in ("table", "seq_lens", "qsl", "token_req", "positions", "slot_map", "head_out")}


def _plain_cache(s):
    rows = s["cache"].view(-1, DK)
    # padding is stored in the last row, and that row put back
    kept = rows[-1].clone()
    rows[torch.where(s["slots"] >= 0, s["slots"], rows.shape[0] - 1)] = s["kv"]
    rows[-1] = kept
    return {"cache": s["cache"]}


def exact(case, seed):
    if case["op"] == "attention":
        # about 1e12 double operations a second
        return None if work(case)["flops"] > 8e12 else _exact_attention(prepare(case, seed))
    return _exact_batch(prepare(case, seed)) if case["op"] == "batch" else _exact_cache(prepare(case, seed))


def _exact_attention(s):
    case, table, cache = s["case"], s["block_table"].tolist(), s["cache"]
    outs, lses, t = [], [], 0
    for b in range(case["B"]):
        n_keys, n_new = s["L"][b], s["q_lens"][b]
        keys = torch.cat([cache[p] for p in table[b][:_blocks(n_keys, case["block"])]])[:n_keys]
        if case["fp8"]:
            lat = keys[:, :DV].contiguous().view(torch.float8_e4m3fn).double()
            grp = keys[:, DV:DV + 16].contiguous().view(torch.float32).double()
            keys = torch.hstack([lat * grp.repeat_interleave(128, dim=1),
                                 keys[:, DV + 16:].contiguous().view(torch.bfloat16).double()])
        else:
            keys = keys.double()
        values = keys[:, :DV].contiguous()
        for i in range(n_new):
            seen = n_keys - n_new + i + 1
            x = torch.einsum("hd,kd->hk", s["q"][t].double(), keys[:seen]) * SCALE
            lse = torch.logsumexp(x, dim=1)
            outs.append(torch.einsum("hk,kd->hd", torch.exp(x - lse[:, None]), values[:seen]))
            lses.append(lse)
            t += 1
    out = torch.stack(outs)
    return {"out": out} if s["lse"] is None else {"out": out, "lse": torch.stack(lses)}


def _exact_batch(s):
    block = s["case"]["block"]
    ctx, new, table, free = s["ctx"].tolist(), s["new"].tolist(), s["table"].tolist(), s["free"].tolist()
    head = s["head"].item()
    qsl, req, pos, slot = [0], [], [], []
    for b, (c, n) in enumerate(zip(ctx, new)):
        for p in range(c, c + n):
            if p % block == 0:
                table[b][p // block] = free[head]
                head += 1
            req.append(b)
            pos.append(p)
            slot.append(table[b][p // block] * block + p % block)
        qsl.append(qsl[-1] + n)
    pad = s["max_tokens"] - qsl[-1]
    res = {"table": table, "seq_lens": [c + n for c, n in zip(ctx, new)], "qsl": qsl, "token_req": req + [-1] * pad,
           "positions": pos + [0] * pad, "slot_map": slot + [-1] * pad, "head_out": [head]}
    return {k: torch.tensor(v, dtype=s[k].dtype, device="cuda") for k, v in res.items()}


def _exact_cache(s):
    want = s["cache"].double().reshape(-1, DK)
    for t, slot in enumerate(s["slots"].tolist()):
        if slot >= 0:
            want[slot] = s["kv"][t]
    return {"cache": want.reshape(s["cache"].shape)}
