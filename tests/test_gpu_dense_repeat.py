"""Dense MLA attention, the same call many times: its results are the same to
the last bit, so that an access that two CTAs do not order would be seen."""
import pytest
import torch

from dense_kinds import PAIR, QUAD, kinds, takes_quads
from dense_testlib import DV, SCALE, check_dense, dense_reference, make_dense_case

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from deepseek_sparse_attention_fp8_gb300 import api
    from test_gpu_dense_mla import call


def repeat(c, kind, calls):
    T, H = c["q"].shape[:2]
    ws = torch.full((api.dense_mla_workspace_size(T, H, DV, 0),), 0xFF, dtype=torch.uint8, device="cuda")
    out, lse, st = call(c, workspace=ws)
    torch.cuda.synchronize()
    assert int(st.item()) == 0 and kinds(ws) == {kind}
    check_dense(out, lse, dense_reference(c))
    differs = torch.zeros((), dtype=torch.int64, device="cuda")
    again, lse2 = torch.empty_like(out), torch.empty_like(lse)
    fn = api.dense_mla_attention_fp8 if c["fp8"] else api.dense_mla_attention
    for _ in range(calls):
        again.fill_(float("nan"))
        lse2.fill_(float("nan"))
        fn(c["q"], c["cache"], c["table"], c["seq"], c["qsl"], SCALE, DV, again, lse=lse2, workspace=ws, dev_status=st)
        differs += (again != out).sum() + (lse2 != lse).sum()
    assert int(differs.item()) == 0 and int(st.item()) == 0


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("lens,q_lens,H", [([8192] * 16, [1] * 16, 128), ([900, 300, 2000, 64] * 8, [1] * 32, 100)])
def test_pairs(lens, q_lens, H, fp8):
    repeat(make_dense_case(lens, q_lens, H, fp8=fp8, seed=61), PAIR, 600)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("lens,q_lens,H", [([9000, 5000, 12000], [16, 40, 8], 128), ([6100, 3000], [150, 90], 40)])
def test_quads(lens, q_lens, H, fp8):
    assert takes_quads(lens, q_lens, H)
    repeat(make_dense_case(lens, q_lens, H, fp8=fp8, seed=62), QUAD, 600)


@pytest.mark.parametrize("fp8", [False, True])
def test_quads_of_several_row_tiles(fp8):
    """A run of many row tiles: maxima and sums go to the output CTAs tile after tile."""
    lens, q_lens = [900, 700, 800], [200, 151, 177]
    assert takes_quads(lens, q_lens, 128)
    repeat(make_dense_case(lens, q_lens, 128, fp8=fp8, seed=63), QUAD, 300)
