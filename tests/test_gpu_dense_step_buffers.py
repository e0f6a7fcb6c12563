"""What a dense DsaStep holds and moves: nothing of the indexer and the top-k."""
import numpy as np
import pytest
import torch

from deepseek_sparse_attention_fp8_gb300.inputs import make_workload

from dense_testlib import check_dense, dense_reference

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from deepseek_sparse_attention_fp8_gb300.step import DsaStep


def test_inputs_hold_the_batch_alone():
    wl = make_workload("decode_b32_l8192", lens=[300, 64, 1000], H=16)
    step = DsaStep(wl, dense=True)
    need = sum(-(-4 * int(np.size(a)) // 256) * 256 for a in (wl.block_table, wl.seq_lens, wl.query_start_loc))
    assert step.inputs.numel() == need
    assert all(x is None for x in (step.q_idx, step.w, step.k_cache, step.logits, step.topk_idx, step.ws_topk))
    for call in (step.indexer, step.topk):
        with pytest.raises(ValueError):
            call()
    # the batch and q come from host memory
    case = dict(q=step.q.clone(), cache=step.kv_cache, table=step.block_table.clone(), fp8=False, block=wl.block_size,
                H=wl.H, T=wl.T, lens=wl.seq_lens.tolist(), q_lens=np.diff(wl.query_start_loc).tolist())
    h_in, h_q = step.inputs.cpu().pin_memory(), step.inputs_q.cpu().pin_memory()
    h_out = torch.empty_like(step.outputs, device="cpu").pin_memory()
    step.inputs.zero_()
    step.inputs_q.zero_()
    step.run_host(h_in, h_q, h_out)
    torch.cuda.synchronize()
    check_dense(step.out, step.lse, dense_reference(case, wl.softmax_scale))
