"""Dense MLA attention on clusters of four CTAs: batches that the device gives
to them, against 64-bit references. Every case shows that it is one, by what it
leaves in the workspace."""
import pytest
import torch

from dense_kinds import PAIR, QUAD, kinds, takes_quads
from dense_testlib import DV, SCALE, check_dense, dense_reference, encode_fp8, make_dense_case

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from deepseek_sparse_attention_fp8_gb300 import api


def call(c, scale=SCALE, kind=QUAD, out=None):
    """out, lse and the status word, through the C entry point (blocks may be
    further apart than their rows)."""
    T, H = c["q"].shape[:2]
    row = c["cache"].shape[2]
    ws = torch.full((api.dense_mla_workspace_size(T, H, DV, 0),), 0xFF, dtype=torch.uint8, device="cuda")
    out = torch.full((T, H, DV), float("nan"), dtype=torch.bfloat16, device="cuda") if out is None else out
    lse = torch.full((T, H), float("nan"), dtype=torch.float32, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    fn = api.lib.dense_mla_attention_fp8 if c["fp8"] else api.lib.dense_mla_attention
    rc = fn(api._ptr(c["q"]), api._ptr(c["cache"]), c["stride"] * row, c["cache"].shape[0], api._ptr(c["table"]),
            c["table"].shape[1], api._ptr(c["seq"]), api._ptr(c["qsl"]), c["seq"].shape[0], T, H, 576, DV, c["block"],
            scale, 0, api._ptr(out), api._ptr(lse), api._ptr(ws), ws.numel(), api._ptr(st), api._stream(None))
    assert rc == 0, api.lib.dsa_last_error()
    torch.cuda.synchronize()
    assert kinds(ws) == {kind}
    return out, lse, int(st.item())


def check(c, scale=SCALE, status=0, every=1, **kw):
    """The call's results, at every `every`-th token and at the last."""
    assert takes_quads(c["lens"], c["q_lens"], c["H"])
    out, lse, st = call(c, scale)
    assert st == status
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
    check(make_dense_case(lens, q_lens, H, fp8=fp8, seed=len(name)), every=13)


CASES = {
    "several_tokens": ([8000, 9000], [8, 16], 128, 64),
    "odd_tokens": ([12000, 8003], [17, 9], 128, 192),
    "heads100": ([9000, 4000], [16, 21], 100, 64),
    "heads40": ([8000, 9100], [50, 41], 40, 128),
    "heads64": ([9000, 5000], [41, 30], 64, 64),
    "heads3": ([9000], [601], 3, 64),
    "long_and_short": ([20000, 1, 64, 130, 9000], [20, 1, 2, 1, 9], 64, 64),
    "idle_requests": ([0, 9000, 5, 7000], [0, 12, 0, 9], 128, 64),
    "row_tiles_in_a_run": ([2500, 900], [200, 151], 128, 256),
}


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("name", sorted(CASES))
def test_ragged_batches(name, fp8):
    lens, q_lens, H, block = CASES[name]
    check(make_dense_case(lens, q_lens, H, fp8=fp8, block=block, seed=len(name)), every=3)


@pytest.mark.parametrize("fp8", [False, True])
def test_bad_blocks_and_lengths(fp8):
    """Masked blocks, a request with fewer keys than tokens, padded rows, and
    blocks further apart than their rows."""
    c = make_dense_case([6000, 3, 7000], [24, 5, 16], 128, fp8=fp8, seed=71, pad_tokens=3, extra_rows=8, extra_cols=2)
    bad = ((0, 1, 10 ** 6), (0, 93, -5), (2, 40, int(c["cache"].shape[0])), (2, 109, -1))
    for b, j, v in bad:
        c["table"][b, j] = v
    out, lse = check(c, status=api.DSA_DEVERR_BLOCK_OOB | api.DSA_DEVERR_SEQ_LEN, blocked={(b, j) for b, j, _ in bad})
    assert torch.isnan(out[45:]).all() and torch.isnan(lse[45:]).all()
    assert (out[24:26] == 0).all() and torch.isneginf(lse[24:26]).all()


@pytest.mark.parametrize("fp8", [False, True])
def test_keys_past_the_table(fp8):
    c = make_dense_case([8192, 6000], [16, 12], 128, fp8=fp8, seed=72)
    c["seq"][0] = 8200  # the table holds 8192 keys: the first 8 tokens see less, the others all of them
    out, lse, st = call(c)
    assert st == api.DSA_DEVERR_SEQ_LEN
    want = dense_reference(dict(c, lens=[8192, 6000], q_lens=[1, 12], q=c["q"][15:]))
    check_dense(out[15:], lse[15:], want)
    check_dense(out[:8], lse[:8], dense_reference(dict(c, lens=[8192], q_lens=[8])))


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("q_std", [0.0, 30.0, 300.0])
def test_score_ranges(fp8, q_std):
    check(make_dense_case([7000, 5000], [16, 24], 128, fp8=fp8, q_std=q_std, seed=73), every=3)


@pytest.mark.parametrize("fp8", [False, True])
def test_rising_scores(fp8):
    """Scores that grow along the keys rescale the outputs step after step."""
    c = make_dense_case([6000], [32], 128, fp8=False, seed=74)
    q = c["q"][0, 0].float()
    n = (torch.arange(6000, device="cuda", dtype=torch.float32) / (50.0 if fp8 else 10.0))[:, None]
    rows = (q / q.pow(2).sum() / SCALE)[None, :] * n + 0.05 * torch.randn((6000, 576), device="cuda")
    pages = torch.zeros((94, 64, 576), device="cuda")
    pages.view(-1, 576)[:6000] = rows
    if fp8:
        cache = torch.zeros((c["cache"].shape[0], 64, 656), dtype=torch.uint8, device="cuda")
        new = encode_fp8(pages.view(-1, 576).cpu()).cuda().view(94, 64, 656)
    else:
        cache, new = torch.zeros_like(c["cache"]), pages.to(torch.bfloat16)
    cache[c["table"][0].long()] = new
    c["q"][:, 1:] = c["q"][0, 0]  # head 0 keeps its tokens' own queries
    c.update(cache=cache, fp8=fp8)
    check(c, every=5)


@pytest.mark.parametrize("fp8", [False, True])
def test_nan_stays_in_its_row(fp8):
    c = make_dense_case([6000, 9000], [16, 8], 128, fp8=fp8, seed=75)
    want, want_lse = check(c, every=5)
    c["q"][0, 3] = float("nan")
    c["q"][17, 7, 5] = float("inf")
    out, lse, _ = call(c)
    keep = torch.ones(out.shape[:2], dtype=torch.bool, device="cuda")
    keep[0, 3] = keep[17, 7] = False
    assert torch.equal(out[keep], want[keep]) and torch.equal(lse[keep], want_lse[keep])
    assert torch.isnan(out[0, 3]).all() and torch.isnan(lse[0, 3])


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("lens,q_lens,kind", [([2500, 900], [60, 51], QUAD), ([500, 300, 700] * 30, [1] * 90, PAIR)])
def test_results_at_16_bytes(lens, q_lens, kind, fp8):
    """`out` aligned to 16 bytes and not to 32."""
    c = make_dense_case(lens, q_lens, 128, fp8=fp8, seed=76)
    want, want_lse, _ = call(c, kind=kind)
    buf = torch.full((want.numel() + 8,), float("nan"), dtype=torch.bfloat16, device="cuda")
    out, lse, _ = call(c, kind=kind, out=buf[8:].view(want.shape))
    assert out.data_ptr() % 32 == 16 and torch.equal(out, want) and torch.equal(lse, want_lse)
    assert torch.isnan(buf[:8]).all()
