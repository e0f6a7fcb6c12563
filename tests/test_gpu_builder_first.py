"""Top-k and sparse attention as the first kernel behind the batch builder: they
see the lengths that it has just written."""
import numpy as np
import pytest
import torch

from dense_testlib import DK, DV, SCALE

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from deepseek_sparse_attention_fp8_gb300 import api

B, COLS, BLOCK, STEPS = 8, 32, 64, 40


def dev(a, dtype=np.int32):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=dtype)).cuda()


def steps_of(call, make_out):
    """call(seq, qsl, out) behind a builder of other lengths each step, all
    enqueued without a pause; the same with a pause in between."""
    rng = np.random.default_rng(3)
    lens = rng.integers(1, COLS * BLOCK, (STEPS, B))
    table = dev(np.arange(B * COLS).reshape(B, COLS))
    ctx, one = [dev(n - 1) for n in lens], dev(np.ones(B))
    results = []
    for pause in (False, True):
        seq, qsl = dev(np.ones(B)), dev(np.arange(B + 1))
        bufs = dict(seq_lens=seq, query_start_loc=qsl, token_req=dev(np.zeros(B)), positions=dev(np.zeros(B)),
                    slot_map=dev(np.zeros(B), np.int64))
        outs = [make_out() for _ in range(STEPS)]
        torch.cuda.synchronize()
        for i in range(STEPS):
            api.dsa_build_batch(ctx[i], one, table, BLOCK, B, **bufs)
            if pause:
                torch.cuda.synchronize()
            call(table, seq, qsl, outs[i])
        torch.cuda.synchronize()
        results.append(outs)
    for i in range(STEPS):
        assert torch.equal(results[0][i], results[1][i])
    return lens, results[0]


@pytest.mark.parametrize("ld,k", [(COLS * BLOCK, 64), (COLS * BLOCK * 32, 128)])
def test_topk(ld, k):
    logits = torch.randn((B, ld), device="cuda")
    ws = torch.empty(max(16, api.dsa_topk_workspace_size(B, ld, k)), dtype=torch.uint8, device="cuda")
    lens, outs = steps_of(lambda table, seq, qsl, out: api.dsa_topk(logits, seq, qsl, k, out, ws),
                          lambda: torch.full((B, k), -7, dtype=torch.int32, device="cuda"))
    for n, out in zip(lens, outs):
        for b in range(B):
            want = torch.topk(logits[b, :n[b]], min(k, int(n[b]))).indices.sort().values.int()
            got = out[b][out[b] >= 0].sort().values
            assert torch.equal(got, want)


@pytest.mark.parametrize("splits", [1, 2])
def test_sparse_attention(splits):
    gen = torch.Generator(device="cuda").manual_seed(5)
    q = torch.randn((B, 16, DK), generator=gen, device="cuda").to(torch.bfloat16)
    cache = torch.randn((B * COLS, BLOCK, DK), generator=gen, device="cuda").to(torch.bfloat16)
    idx = torch.arange(512, dtype=torch.int32, device="cuda").repeat(B, 1)  # what lies behind the length is masked
    ws = torch.empty(max(16, api.sparse_mla_workspace_size(B, 16, DV, splits)), dtype=torch.uint8, device="cuda")
    lse = torch.empty((B, 16), device="cuda")
    steps_of(lambda table, seq, qsl, out: api.sparse_mla_decode(q, cache, table, seq, qsl, idx, SCALE, DV, out, lse,
                                                                splits, ws),
             lambda: torch.full((B, 16, DV), float("nan"), dtype=torch.bfloat16, device="cuda"))
