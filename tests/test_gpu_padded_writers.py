"""The writers that find a token's place from the batch's lengths, on a padded
batch: rows from query_start_loc[B] on are nobody's."""
import numpy as np
import pytest
import torch

from dense_testlib import DK, DV, SCALE, check_dense, dense_reference

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from deepseek_sparse_attention_fp8_gb300 import api

BLOCK = 64


def dev(a, dtype=np.int32):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=dtype)).cuda()


def batches():
    # the last request ends inside a block, at a block's end, without a token; the entry behind its
    # last block is block 0, which belongs to the first request
    return [([70, 60], [2, 3]), ([70, 64], [1, 64]), ([70, 64], [2, 0]), ([40], [40])]


@pytest.mark.parametrize("pad", [1, 5, 200])
@pytest.mark.parametrize("lens,news", batches())
def test_fp8_latent_rows(lens, news, pad):
    n, B = sum(news), len(lens)
    table = dev([[0, 1, 0, 0, 0], [2, 0, 0, 0, 0]][:B])
    kv = torch.randn((n + pad, 576), device="cuda").to(torch.bfloat16)
    seq, qsl = dev(lens), dev(np.concatenate([[0], np.cumsum(news)]))
    caches, st = [], dev([0])
    for T in (n, n + pad):
        cache = torch.full((3, BLOCK, 656), 0x55, dtype=torch.uint8, device="cuda")
        api.dsa_mla_kv_fp8_quant_and_cache(kv[:T], cache, table, seq, qsl, BLOCK, dev_status=st)
        caches.append(cache)
    assert int(st.item()) == 0 and torch.equal(caches[0], caches[1])


@pytest.mark.parametrize("di", [32, 64, 128])
@pytest.mark.parametrize("lens,news", batches())
def test_indexer_keys(lens, news, di):
    n, B, pad = sum(news), len(lens), 70
    table = dev([[0, 1, 0, 0, 0], [2, 0, 0, 0, 0]][:B])
    k = torch.randn((n + pad, di), device="cuda").to(torch.bfloat16)
    seq, qsl = dev(lens), dev(np.concatenate([[0], np.cumsum(news)]))
    caches, st = [], dev([0])
    for T in (n, n + pad):
        cache = torch.full((3, BLOCK * (di + 4)), 0x55, dtype=torch.uint8, device="cuda")
        api.dsa_indexer_k_quant_and_cache(k[:T], cache, table, seq, qsl, BLOCK, dev_status=st)
        caches.append(cache)
    assert int(st.item()) == 0 and torch.equal(caches[0], caches[1])


def test_captured_loop_over_the_fp8_caches():
    """One graph builds the batch, stores latent rows and indexer keys and
    attends, in buffers padded to a fixed size; rows once stored stay."""
    B, H, T, cols, di = 4, 16, 150, 6, 64
    rng = np.random.default_rng(7)
    gen = torch.Generator().manual_seed(8)
    nb = B * cols + 2
    # entries behind a request's blocks are not -1, as in a table whose rows are used again
    table, free = dev(rng.integers(0, nb, (B, cols))), dev(rng.permutation(nb))
    head, st, ctx, new = dev([0]), dev([0]), dev(np.zeros(B)), dev(np.zeros(B))
    bufs = dict(seq_lens=dev(np.zeros(B)), query_start_loc=dev(np.zeros(B + 1)), token_req=dev(np.zeros(T)),
                positions=dev(np.zeros(T)), slot_map=dev(np.zeros(T), np.int64))
    seq, qsl = bufs["seq_lens"], bufs["query_start_loc"]
    cache = torch.full((nb, BLOCK, 656), 0x7F, dtype=torch.uint8, device="cuda")
    keys = torch.zeros((nb, BLOCK * (di + 4)), dtype=torch.uint8, device="cuda")
    q = torch.zeros((T, H, DK), dtype=torch.bfloat16, device="cuda")
    kv, k = (torch.zeros((T, d), dtype=torch.bfloat16, device="cuda") for d in (DK, di))
    out, lse = torch.zeros((T, H, DV), dtype=torch.bfloat16, device="cuda"), torch.zeros((T, H), device="cuda")
    ws = torch.empty(max(16, api.dense_mla_workspace_size(T, H, DV, 0)), dtype=torch.uint8, device="cuda")

    def step():
        api.dsa_build_batch(ctx, new, table, BLOCK, T, free_blocks=free, free_head=head, dev_status=st, **bufs)
        api.dsa_mla_kv_fp8_quant_and_cache(kv, cache, table, seq, qsl, BLOCK, dev_status=st)
        api.dsa_indexer_k_quant_and_cache(k, keys, table, seq, qsl, BLOCK, dev_status=st)
        api.dense_mla_attention_fp8(q, cache, table, seq, qsl, SCALE, DV, out, lse=lse, workspace=ws, dev_status=st)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    lens = np.zeros(B, dtype=np.int64)
    kept = [torch.zeros((0, 656), dtype=torch.uint8, device="cuda") for _ in range(B)]
    for i in range(6):
        add = np.array([30, 64, 1, 50]) if i == 0 else rng.integers(0, 20, B)
        kv.copy_((torch.randn((T, DK), generator=gen) * 0.5).to(torch.bfloat16))
        k.copy_(torch.randn((T, di), generator=gen).to(torch.bfloat16))
        q.copy_((torch.randn((T, H, DK), generator=gen) * 3).to(torch.bfloat16))
        ctx.copy_(dev(lens))
        new.copy_(dev(add))
        out.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        n = int(add.sum())
        lens += add
        assert int(st.item()) == 0 and torch.isnan(out[n:]).all()
        for b in range(B):
            rows = cache[table[b, :-(-int(lens[b]) // BLOCK)].long()].reshape(-1, 656)[:lens[b]]
            assert torch.equal(rows[:len(kept[b])], kept[b])
            kept[b] = rows.clone()
        case = dict(q=q, cache=cache, table=table, fp8=True, block=BLOCK, H=H, T=n, lens=lens.tolist(),
                    q_lens=add.tolist())
        check_dense(out[:n], lse[:n], dense_reference(case))
