"""Dense MLA attention on clusters of four CTAs: batches that the device gives
to them, against 64-bit references. Every case first shows that it is one."""
import pytest
import torch

from dense_kinds import QUAD, kinds, takes_quads
from dense_testlib import DV, SCALE, check_dense, dense_reference, make_dense_case

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from deepseek_sparse_attention_fp8_gb300 import api
    from test_gpu_dense_mla import call


def check_quads(c, scale=SCALE, status=0, every=1, **kw):
    """The call's results, checked at every `every`-th token and at the last."""
    T, H = c["q"].shape[:2]
    ws = torch.full((api.dense_mla_workspace_size(T, H, DV, 0),), 0xFF, dtype=torch.uint8, device="cuda")
    out, lse, st = call(c, scale=scale, workspace=ws)
    torch.cuda.synchronize()
    assert int(st.item()) == status
    assert kinds(ws) == {QUAD}
    tokens = sorted(set(range(0, c["T"], every)) | {c["T"] - 1})
    assert torch.isfinite(out[:c["T"]].float()).all(), "rows left out"
    check_dense(out[tokens], lse[tokens], dense_reference(c, scale, tokens=set(tokens), **kw))
    return out, lse


FEW_HEADS = {
    "one_head": ([16384], [1024], 1),
    "one_head_odd": ([16390], [701], 1),
    "one_head_ragged": ([16000, 12000, 300], [1024, 700, 257], 1),
    "two_heads": ([20000, 9000], [600, 500], 2),
}


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("name", sorted(FEW_HEADS))
def test_row_tiles_of_many_tokens(name, fp8):
    lens, q_lens, H = FEW_HEADS[name]
    assert takes_quads(lens, q_lens, H)
    check_quads(make_dense_case(lens, q_lens, H, fp8=fp8, seed=len(name)), every=13)
