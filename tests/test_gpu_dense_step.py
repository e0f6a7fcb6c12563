"""The batch builder, the cache writers and dense attention together: a dense
DsaStep beside the sparse one, and a serving loop that keeps its metadata on
the GPU."""

import numpy as np
import pytest
import torch

from deepseek_sparse_attention_fp8_gb300.inputs import make_workload

from dense_testlib import DK, DV, SCALE, check_dense, dense_reference

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from deepseek_sparse_attention_fp8_gb300 import api
    from deepseek_sparse_attention_fp8_gb300.step import DsaStep


def _as_case(step, wl, fp8):
    return dict(q=step.q, cache=step.kv_cache, table=step.block_table, seq=step.seq_lens, qsl=step.qsl, fp8=fp8,
                block=wl.block_size, H=wl.H, T=wl.T, stride=wl.block_size, lens=wl.seq_lens.tolist(),
                q_lens=np.diff(wl.query_start_loc).tolist())


@pytest.mark.parametrize("splits", [0, -1])
@pytest.mark.parametrize("fp8", [False, True])
def test_dense_step(fp8, splits):
    wl = make_workload("mixed_b64_mtp2", lens=[1500, 2049, 130, 65], q_lens=[2, 1, 3, 1], H=16, kv_fp8=True)
    step = DsaStep(wl, kv_fp8=fp8, dense=True, num_kv_splits=splits)
    step.run()
    torch.cuda.synchronize()
    assert int(step.dev_status.item()) == 0 and step.kernel_launches() == (2 if splits == 0 else 1)
    check_dense(step.out, step.lse, dense_reference(_as_case(step, wl, fp8), wl.softmax_scale))


def test_dense_step_from_host_memory():
    wl = make_workload("decode_b32_l8192", lens=[300, 64, 1000], H=16)
    step = DsaStep(wl, dense=True)
    ref = dense_reference(_as_case(step, wl, False), wl.softmax_scale)
    h_in, h_q = step.inputs.cpu().pin_memory(), step.inputs_q.cpu().pin_memory()
    h_out = torch.empty_like(step.outputs, device="cpu").pin_memory()
    step.inputs_q.zero_()
    step.run_host(h_in, h_q, h_out)
    torch.cuda.synchronize()
    check_dense(step.out, step.lse, ref)
    assert torch.equal(h_out, step.outputs.cpu())


def test_dense_step_refuses_split_counts():
    wl = make_workload("decode_b32_l8192", lens=[64], H=16)
    with pytest.raises(ValueError):
        DsaStep(wl, dense=True, num_kv_splits=4)


def test_serving_loop_in_one_graph():
    """Prompts, then decode steps of one to three tokens, in buffers padded to
    a fixed size: one captured graph builds the batch, stores the new latent
    rows and indexer keys and attends, densely and through the sparse path
    with index_topk above every length. Lengths, block tables and the free
    queue live on the GPU only; requests idle and stop along the way."""
    B, H, block, T, cols, steps = 5, 16, 64, 200, 8, 7
    Hi, Di, K = 16, 64, 512
    rng = np.random.default_rng(0)
    gen = torch.Generator().manual_seed(1)
    dev = torch.device("cuda")
    nb = B * cols + 3
    i32 = dict(dtype=torch.int32, device=dev)
    table, free = torch.full((B, cols), -1, **i32), torch.from_numpy(rng.permutation(nb).astype(np.int32)).to(dev)
    head, st = torch.zeros(1, **i32), torch.zeros(1, **i32)
    ctx, new = torch.zeros(B, **i32), torch.zeros(B, **i32)
    seq, qsl = torch.zeros(B, **i32), torch.zeros(B + 1, **i32)
    req, pos = torch.zeros(T, **i32), torch.zeros(T, **i32)
    slots = torch.zeros(T, dtype=torch.int64, device=dev)
    cache = torch.full((nb, block, DK), float("nan"), dtype=torch.bfloat16, device=dev)
    k_cache = torch.zeros((nb, block * (Di + 4)), dtype=torch.uint8, device=dev)
    q = torch.zeros((T, H, DK), dtype=torch.bfloat16, device=dev)
    kv = torch.zeros((T, DK), dtype=torch.bfloat16, device=dev)
    q_idx = torch.zeros((T, Hi, Di), dtype=torch.bfloat16, device=dev)
    w = torch.ones((T, Hi), dtype=torch.float32, device=dev)
    ki = torch.zeros((T, Di), dtype=torch.bfloat16, device=dev)
    logits = torch.zeros((T, cols * block), dtype=torch.float32, device=dev)
    idx = torch.zeros((T, K), **i32)
    out, out2 = (torch.zeros((T, H, DV), dtype=torch.bfloat16, device=dev) for _ in range(2))
    lse = torch.zeros((T, H), dtype=torch.float32, device=dev)
    ws = torch.empty(max(16, api.dense_mla_workspace_size(T, H, DV, 0)), dtype=torch.uint8, device=dev)

    def step():
        api.dsa_build_batch(ctx, new, table, block, T, free_blocks=free, free_head=head, seq_lens=seq,
                            query_start_loc=qsl, token_req=req, positions=pos, slot_map=slots, dev_status=st)
        api.dsa_mla_kv_cache(kv, slots, cache, dev_status=st)
        api.dense_mla_attention(q, cache, table, seq, qsl, SCALE, DV, out, lse=lse, workspace=ws, dev_status=st)

    def sparse(n):  # the sparse calls take the batch's tokens without padding
        api.dsa_indexer_k_quant_and_cache(ki[:n], k_cache, table, seq, qsl, block, dev_status=st)
        api.dsa_indexer_logits(q_idx[:n], w[:n], k_cache, table, seq, qsl, block, T, logits[:n], st)
        api.dsa_topk(logits[:n], seq, qsl, K, idx[:n])
        api.sparse_mla_prefill(q[:n], cache, table, seq, qsl, idx[:n], SCALE, DV, out2[:n], dev_status=st)

    step()  # first use outside the capture; no request has a token
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    lens = np.zeros(B, dtype=np.int64)
    history = [torch.zeros((0, DK), dtype=torch.bfloat16) for _ in range(B)]
    for i in range(steps):
        add = np.array([30, 64, 1, 0, 90]) if i == 0 else rng.integers(0, 4, B) * (rng.random(B) < 0.8)
        if i == 1:
            add[3] = 100  # a request that joins later
        n = int(add.sum())
        rows = (torch.randn((T, DK), generator=gen) * 0.5).to(torch.bfloat16)
        kv.copy_(rows)
        q.copy_((torch.randn((T, H, DK), generator=gen) * 3).to(torch.bfloat16))
        q_idx.copy_(torch.randn((T, Hi, Di), generator=gen).to(torch.bfloat16))
        ki.copy_(torch.randn((T, Di), generator=gen).to(torch.bfloat16))
        ctx.copy_(torch.from_numpy(lens.astype(np.int32)))
        new.copy_(torch.from_numpy(add.astype(np.int32)))
        out.fill_(float("nan"))
        graph.replay()
        sparse(n)
        torch.cuda.synchronize()
        assert int(st.item()) == 0
        at = 0
        for b in range(B):
            history[b] = torch.cat([history[b], rows[at:at + add[b]]])
            at += int(add[b])
        lens += add
        assert seq.tolist() == lens.tolist() and torch.isnan(out[n:]).all()
        assert int(head.item()) == sum(-(-int(x) // block) for x in lens)
        # the reference reads the rows that were fed, not the cache
        pages = torch.zeros((B * cols, block, DK), dtype=torch.bfloat16)
        for b in range(B):
            pages.view(B, cols * block, DK)[b, :lens[b]] = history[b]
        case = dict(q=q, cache=pages.to(dev), table=torch.arange(B * cols, **i32).view(B, cols), fp8=False, block=block,
                    H=H, T=n, lens=lens.tolist(), q_lens=add.tolist())
        ref = dense_reference(case)
        check_dense(out[:n], lse[:n], ref)
        # the sparse path over every key: its normaliser sums bf16 weights, 2^-8 more
        assert ((out2[:n].double() - ref[0]).abs() <= ref[1] + 2.0 ** -8 * ref[0].abs()).all()
