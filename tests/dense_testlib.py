"""Cases and 64-bit references for dense MLA attention and the batch builder."""
from __future__ import annotations

import math

import numpy as np
import torch

DK, DV = 576, 512
SCALE = 1.0 / math.sqrt(DK)


def make_dense_case(lens, q_lens, H, *, fp8=False, block=64, seed=0, q_std=3.0, kv_std=0.5, pad_tokens=0,
                    extra_rows=0, extra_cols=0, poison=True, device="cuda"):
    """A ragged batch over a permuted pool of blocks. What no request owns
    (spare blocks, rows behind a request's last key) is NaN with poison;
    extra_rows adds unused rows between the blocks (a wider block stride)."""
    rng = np.random.default_rng(seed)
    gen = torch.Generator().manual_seed(seed)
    B, T = len(lens), sum(q_lens)
    need = [max(0, -(-n // block)) for n in lens]
    nb = sum(need) + 3
    perm = rng.permutation(nb)
    table = np.full((B, max(need + [1]) + extra_cols), -1, dtype=np.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = perm[at:at + n]
        at += n
    row = 656 if fp8 else DK
    cache = torch.zeros((nb, block + extra_rows, row), dtype=torch.uint8 if fp8 else torch.bfloat16)
    cache.fill_(0x7F if fp8 else float("nan")) if poison else None
    for b, n in enumerate(lens):
        for j in range(need[b]):
            m = min(block, n - j * block)
            kv = torch.randn((m, DK), generator=gen) * kv_std
            cache[table[b, j], :m] = encode_fp8(kv) if fp8 else kv.to(torch.bfloat16)
    q = (torch.randn((T + pad_tokens, H, DK), generator=gen) * q_std).to(torch.bfloat16)
    qsl = np.concatenate([[0], np.cumsum(q_lens)]).astype(np.int32)
    to = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(device)
    return dict(q=q.to(device), cache=cache.to(device), table=to(table), seq=to(np.array(lens, dtype=np.int32)),
                qsl=to(qsl), fp8=fp8, block=block, H=H, T=T, stride=block + extra_rows, lens=list(lens),
                q_lens=list(q_lens))


def encode_fp8(kv):
    """Latent rows as fp8 cache rows (uint8 [n, 656])."""
    n = kv.shape[0]
    rope = kv[:, DV:].to(torch.bfloat16)
    lat = kv[:, :DV].reshape(n, 4, 128)
    amax = lat.abs().amax(-1)
    scale = torch.where(amax > 0, amax / 448.0, torch.ones_like(amax))
    codes = (lat / scale[..., None]).to(torch.float8_e4m3fn).reshape(n, DV)
    return torch.cat([codes.view(torch.uint8), scale.contiguous().view(torch.uint8), rope.view(torch.uint8)], dim=1)


def decode_rows(rows, fp8):
    if not fp8:
        return rows.double()
    n = rows.shape[0]
    codes = rows[:, :DV].contiguous().view(torch.float8_e4m3fn).to(torch.float32).double()
    scale = rows[:, DV:DV + 16].contiguous().view(torch.float32).double()
    rope = rows[:, DV + 16:].contiguous().view(torch.bfloat16).double()
    return torch.cat([(codes.view(n, 4, 128) * scale[..., None]).view(n, DV), rope], dim=1)


def dense_reference(c, scale=SCALE, tokens=None, blocked=()):
    """out, lse in 64 bits, and the bounds of what the kernels' roundings may
    move them, per element. `blocked`: table blocks (b, j) whose keys count as
    masked.

    The roundings counted, each at most half a step: the weights to bf16
    (2^-8 of a weight: 2^-8 A, A = sum p |v|), the result to bf16 (2^-8
    |out|), and with the fp8 cache the decoded values to bf16 (2^-8 of a
    value: 2^-8 A in the sum over values, and 2^-8 scale sum |q k| =: d in a
    score, which moves every weight by at most a factor e^(2d)). Scores,
    exponentials and sums in 32 bits: 576 products and a few more roundings
    of 2^-24 of sum |q k| scale, and 2^-20 for the exponentials, the running
    maximum's factors and the sums."""
    outs, tols, lses, ltols = [], [], [], []
    t = 0
    eps = 2.0 ** -8
    for b, (n, m) in enumerate(zip(c["lens"], c["q_lens"])):
        nblk = -(-n // c["block"]) if n > 0 else 0
        bad = torch.zeros(max(n, 0), dtype=torch.bool, device=c["q"].device)
        rows = []
        for j in range(nblk):
            p = int(c["table"][b, j])
            if (b, j) in blocked:
                bad[j * c["block"]:(j + 1) * c["block"]] = True
                p = 0
            rows.append(c["cache"][p, :c["block"]])
        if rows:
            raw = torch.cat(rows)[:n]
            k = torch.where(bad[:, None], torch.zeros((), dtype=torch.float64, device=raw.device),
                            decode_rows(raw, c["fp8"]))
        for i in range(m):
            if tokens is not None and t not in tokens:
                t += 1
                continue
            seen = n - m + i + 1
            ok = (~bad[:seen]).nonzero()[:, 0] if seen > 0 else bad[:0].nonzero()[:, 0]
            if ok.numel() == 0:
                outs.append(torch.zeros((c["H"], DV), dtype=torch.float64, device=c["q"].device))
                tols.append(torch.zeros_like(outs[-1]))
                lses.append(torch.full((c["H"],), -math.inf, dtype=torch.float64, device=c["q"].device))
                ltols.append(torch.zeros_like(lses[-1]))
                t += 1
                continue
            kk, q = k[ok], c["q"][t].double()
            s = (q @ kk.T) * scale
            mag = (q.abs() @ kk.abs().T).amax(1) * scale  # of a score's terms
            lse = torch.logsumexp(s, 1)
            p = torch.exp(s - lse[:, None])
            out = p @ kk[:, :DV]
            A = p @ kk[:, :DV].abs()
            d32 = mag * 600 * 2.0 ** -24 + 2.0 ** -20
            d = d32 + (eps * mag if c["fp8"] else 0.0)
            grow = torch.expm1(2 * d)[:, None]
            values = eps if c["fp8"] else 0.0
            tol = eps * out.abs() + (1 + eps) * ((1 + grow) * (1 + eps) * (1 + values) - 1) * A
            outs.append(out)
            tols.append(tol)
            lses.append(lse)
            ltols.append(d + lse.abs() * 2.0 ** -23)
            t += 1
    if not outs:
        return None
    return torch.stack(outs), torch.stack(tols), torch.stack(lses), torch.stack(ltols)


def check_dense(got, lse, ref, rows=None):
    out, tol, rl, rt = ref
    g = got.double() if rows is None else got[rows].double()
    assert torch.isfinite(g).all(), "non-finite output"
    over = (g - out).abs() - tol
    assert (over <= 0).all(), f"output off by {over.max().item():.3g} more than its bound"
    if lse is not None:
        l = lse.double() if rows is None else lse[rows].double()
        fin = torch.isfinite(rl)
        assert torch.equal(torch.isneginf(l), ~fin), "lse of empty rows"
        over = (l[fin] - rl[fin]).abs() - rt[fin]
        assert over.numel() == 0 or (over <= 0).all(), f"lse off by {over.max().item():.3g} more than its bound"


def batch_reference(ctx, new, table, block, max_tokens, free=None, head=0):
    """What dsa_build_batch leaves, in plain loops over tokens."""
    table = np.array(table, dtype=np.int64)
    B, cols = table.shape
    qsl, req, pos, slot, seq = [0], [], [], [], []
    head0, ok = head, free is not None and 0 <= head <= len(free)
    err = 0
    for b in range(B):
        c, n = int(ctx[b]), int(new[b])
        if c < 0 or n < 0 or c + n > 2 ** 31 - 1:
            err |= 8
            c, n = max(c, 0), 0
        room = max_tokens - qsl[-1]
        if n > room:
            err |= 8
            n = room
        held = -(-c // block)
        for p in range(c, c + n):
            j = p // block
            s = -1
            if j >= cols:
                err |= 8
            else:
                if free is not None and j >= held and p % block == 0:
                    if ok and head < len(free):
                        table[b, j] = free[head]
                        if free[head] < 0:
                            err |= 1
                    else:
                        table[b, j] = -1
                        err |= 16
                    head += 1
                elif table[b, j] < 0 and not (free is not None and j >= held):
                    err |= 1
                if table[b, j] >= 0:
                    s = int(table[b, j]) * block + p % block
            req.append(b)
            pos.append(p)
            slot.append(s)
        seq.append(c + n)
        qsl.append(qsl[-1] + n)
    pad = max_tokens - qsl[-1]
    new_head = (min(head, len(free)) if ok else head0) if free is not None else head0
    return dict(table=table, seq=np.array(seq), qsl=np.array(qsl), req=np.array(req + [-1] * pad),
                pos=np.array(pos + [0] * pad), slot=np.array(slot + [-1] * pad), head=new_head, err=err)
