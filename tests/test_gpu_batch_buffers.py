"""The batch builder's results in buffers made for more requests and tokens."""
import pytest
import torch

from dense_testlib import DK, DV, SCALE, check_dense, dense_reference

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from deepseek_sparse_attention_fp8_gb300 import api


def test_longer_buffers():
    """What comes back serves the attention as it is, whatever lies behind it."""
    i32 = dict(dtype=torch.int32, device="cuda")
    ctx, new, T, H = [100, 3, 200], [1, 5, 2], 12, 16
    table = torch.arange(12, **i32).view(3, 4)
    cache = (torch.randn((12, 64, DK), device="cuda") * 0.5).to(torch.bfloat16)
    bufs = [torch.full((n,), 50, **i32) for n in (9, 10, 40, 40)] + [torch.full((40,), 50, dtype=torch.int64,
                                                                                 device="cuda")]
    res = api.dsa_build_batch(torch.tensor(ctx, **i32), torch.tensor(new, **i32), table, 64, T, seq_lens=bufs[0],
                              query_start_loc=bufs[1], token_req=bufs[2], positions=bufs[3], slot_map=bufs[4])
    assert [tuple(t.shape) for t in res] == [(3,), (4,), (T,), (T,), (T,)]
    assert all(t.data_ptr() == b.data_ptr() and (b[t.shape[0]:] == 50).all() for t, b in zip(res, bufs))
    assert res[0].tolist() == [101, 8, 202] and res[1].tolist() == [0, 1, 6, 8]
    q = torch.randn((T, H, DK), device="cuda").to(torch.bfloat16)
    out = torch.full((T, H, DV), float("nan"), dtype=torch.bfloat16, device="cuda")
    lse = torch.full((T, H), float("nan"), device="cuda")
    api.dense_mla_attention(q, cache, table, res[0], res[1], SCALE, DV, out, lse=lse)
    torch.cuda.synchronize()
    n = sum(new)
    case = dict(q=q, cache=cache, table=table, fp8=False, block=64, H=H, T=n, lens=res[0].tolist(), q_lens=new)
    check_dense(out[:n], lse[:n], dense_reference(case))
    assert torch.isnan(out[n:]).all()
    pos = [100, *range(3, 8), 200, 201]  # request b's blocks are 4 b and the following
    want = [256 * b + p for b, p in zip([0, 1, 1, 1, 1, 1, 2, 2], pos)]
    assert res[4].tolist() == want + [-1] * (T - n)
