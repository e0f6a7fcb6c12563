"""Dense MLA attention over the paged latent caches against 64-bit references,
with bounds counted from the kernels' roundings (dense_testlib)."""
import numpy as np
import pytest
import torch

from dense_testlib import DV, SCALE, check_dense, dense_reference, make_dense_case

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from deepseek_sparse_attention_fp8_gb300 import api


def call(c, splits=0, scale=SCALE, lse=True, out=None, stream=None, workspace=None, status=None):
    T, H = c["q"].shape[:2]
    out = torch.full((T, H, DV), float("nan"), dtype=torch.bfloat16, device="cuda") if out is None else out
    l = torch.full((T, H), float("nan"), dtype=torch.float32, device="cuda") if lse else None
    st = torch.zeros(1, dtype=torch.int32, device="cuda") if status is None else status
    fn = api.dense_mla_attention_fp8 if c["fp8"] else api.dense_mla_attention
    if c["stride"] == c["block"]:
        fn(c["q"], c["cache"], c["table"], c["seq"], c["qsl"], scale, DV, out, lse=l, num_kv_splits=splits,
           workspace=workspace, dev_status=st, stream=stream)
    else:  # blocks further apart than their rows: through the C entry point
        row = c["cache"].shape[2]
        ws = torch.empty(max(16, api.dense_mla_workspace_size(T, H, DV, splits)), dtype=torch.uint8, device="cuda")
        rc = getattr(api.lib, fn.__name__)(
            api._ptr(c["q"]), api._ptr(c["cache"]), c["stride"] * row, c["cache"].shape[0], api._ptr(c["table"]),
            c["table"].shape[1], api._ptr(c["seq"]), api._ptr(c["qsl"]), c["seq"].shape[0], T, H, 576, DV, c["block"],
            scale, splits, api._ptr(out), api._ptr(l), api._ptr(ws), ws.numel(), api._ptr(st), api._stream(stream))
        assert rc == 0, api.lib.dsa_last_error()
    return out, l, st


def check(c, splits=0, scale=SCALE, status=0, **kw):
    out, lse, st = call(c, splits, scale)
    torch.cuda.synchronize()
    assert int(st.item()) == status
    check_dense(out[:c["T"]], lse[:c["T"]], dense_reference(c, scale, **kw))
    return out, lse


CASES = {
    "one_key": ([1], [1], 128, 64),
    "two_keys": ([2], [1], 1, 64),
    "edges": ([63, 64, 65, 127, 128, 129, 191, 192, 193, 255, 256, 257], [1] * 12, 16, 64),
    "edges_h128": ([1, 64, 65, 128, 129, 300], [1] * 6, 128, 64),
    "heads3": ([200, 5], [3, 5], 3, 64),
    "heads40": ([333, 130, 1], [7, 2, 1], 40, 128),
    "heads100": ([150, 700], [2, 9], 100, 64),
    "heads64_mtp": ([1000, 129, 64], [2, 2, 2], 64, 64),
    "idle_requests": ([100, 0, 40, 0, 0, 300], [1, 0, 0, 0, 0, 4], 32, 64),
    "prompt": ([130, 64, 1], [130, 64, 1], 16, 64),
    "prompt_h128": ([150], [150], 128, 64),
    "chunk": ([1000], [257], 16, 192),
    "chunk_h8": ([500, 260], [200, 37], 8, 64),
    "long": ([9000, 3], [1, 1], 128, 256),
    "many": ([(37 * i) % 300 + 1 for i in range(200)], [1] * 200, 16, 64),
    "more_than_threads": ([(11 * i) % 90 + 1 for i in range(700)], [1] * 700, 4, 64),
}


@pytest.mark.parametrize("splits", [0, -1])
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("name", sorted(CASES))
def test_dense_attention(name, fp8, splits):
    lens, q_lens, H, block = CASES[name]
    check(make_dense_case(lens, q_lens, H, fp8=fp8, block=block, seed=len(name)), splits)


# several row tiles a request over long contexts: the four-CTA kernel's
LONG_CASES = {
    "two_tokens": ([9000, 12000, 3000, 7000], [2, 2, 2, 2], 128, 64),
    "odd_tokens": ([5000, 4097], [3, 5], 128, 64),
    "chunks": ([2500, 900], [40, 33], 128, 192),
    "heads100": ([6000, 2049], [7, 3], 100, 64),
    "heads40": ([4000, 8191, 5000], [13, 6, 20], 40, 128),
    "heads16": ([6100, 3000], [150, 17], 16, 64),
    "heads3": ([9000], [300], 3, 64),
    "one_cut_tile": ([30000], [2], 128, 256),
    "long_and_short": ([20000, 1, 64, 130, 9000], [20, 1, 2, 1, 9], 64, 64),
    "idle_requests": ([0, 8000, 5, 7000], [0, 6, 0, 4], 128, 64),
}


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("name", sorted(LONG_CASES))
def test_long_chunks(name, fp8):
    lens, q_lens, H, block = LONG_CASES[name]
    check(make_dense_case(lens, q_lens, H, fp8=fp8, block=block, seed=len(name)))


@pytest.mark.parametrize("fp8", [False, True])
def test_long_chunks_with_bad_blocks_and_lengths(fp8):
    """Masked blocks, a request with fewer keys than tokens, padded rows, and
    blocks further apart than their rows."""
    c = make_dense_case([6000, 3, 7000], [6, 5, 4], 128, fp8=fp8, seed=31, pad_tokens=3, extra_rows=8, extra_cols=2)
    for b, j, v in ((0, 1, 10 ** 6), (0, 93, -5), (2, 40, int(c["cache"].shape[0])), (2, 109, -1)):
        c["table"][b, j] = v
    out, lse = check(c, status=api.DSA_DEVERR_BLOCK_OOB | api.DSA_DEVERR_SEQ_LEN,
                     blocked={(0, 1), (0, 93), (2, 40), (2, 109)})
    assert torch.isnan(out[15:]).all() and torch.isnan(lse[15:]).all()
    assert (out[6:8] == 0).all() and torch.isneginf(lse[6:8]).all()


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("q_std", [0.0, 300.0])
def test_long_chunks_score_ranges(fp8, q_std):
    check(make_dense_case([7000, 5000], [4, 6], 128, fp8=fp8, q_std=q_std, seed=32))


def test_long_chunks_rising_scores():
    """Scores that grow along the keys rescale the outputs step after step."""
    c = make_dense_case([6000], [4], 128, seed=33)
    q = c["q"][0, 0].float()
    n = (torch.arange(6000, device="cuda", dtype=torch.float32) / 50.0)[:, None]
    rows = (q / q.pow(2).sum() / SCALE)[None, :] * n + 0.05 * torch.randn((6000, 576), device="cuda")
    pages = torch.zeros((94, 64, 576), device="cuda")
    pages.view(-1, 576)[:6000] = rows
    c["cache"][c["table"][0].long()] = pages.to(torch.bfloat16)
    c["q"][:] = c["q"][0, 0]
    check(c)


# few rows a request: one rank's share of the heads
FEW_CASES = {
    "h16": ([3000, 1, 64, 130, 8193, 127], [1] * 6, 16, 64),
    "h32": ([5000, 129, 2, 128, 7777], [1] * 5, 32, 128),
    "h17": ([999, 4000, 33], [1] * 3, 17, 64),
    "h1": ([1, 700, 20000], [1] * 3, 1, 64),
    "h5_three_tokens": ([2500, 3, 640], [3, 3, 3], 5, 64),
    "h8_two_tokens": ([130, 2, 4500, 65], [2, 2, 2, 2], 8, 192),
    "h16_two_tokens": ([4000, 70, 129], [2, 2, 2], 16, 64),
    "a_prompt_among_tokens": ([1000, 30, 90, 2000, 5, 0, 300, 77], [1, 9, 1, 1, 1, 0, 1, 1], 16, 64),
    "a_chunk_and_idle": ([6000] + [0] * 99, [90] + [0] * 99, 16, 64),
    "one_cut_tile": ([60000], [1], 16, 256),
    "many_short": ([(13 * i) % 500 + 1 for i in range(300)], [1] * 300, 32, 64),
}


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("name", sorted(FEW_CASES))
def test_few_rows(name, fp8):
    lens, q_lens, H, block = FEW_CASES[name]
    check(make_dense_case(lens, q_lens, H, fp8=fp8, block=block, seed=len(name)))


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("H", [16, 32])
@pytest.mark.parametrize("q_std", [0.0, 300.0])
def test_few_rows_score_ranges(H, q_std, fp8):
    check(make_dense_case([7000, 5000, 90], [1, 1, 1], H, fp8=fp8, q_std=q_std, seed=41))


@pytest.mark.parametrize("H", [16, 32])
def test_few_rows_rising_scores(H):
    c = make_dense_case([6000], [1], H, seed=42)
    q = c["q"][0, 0].float()
    n = (torch.arange(6000, device="cuda", dtype=torch.float32) / 50.0)[:, None]
    rows = (q / q.pow(2).sum() / SCALE)[None, :] * n + 0.05 * torch.randn((6000, 576), device="cuda")
    pages = torch.zeros((94, 64, 576), device="cuda")
    pages.view(-1, 576)[:6000] = rows
    c["cache"][c["table"][0].long()] = pages.to(torch.bfloat16)
    c["q"][:, 1:] = c["q"][0, 0]
    check(c)


@pytest.mark.parametrize("fp8", [False, True])
def test_few_rows_with_bad_blocks_and_lengths(fp8):
    c = make_dense_case([6000, 1, 7000], [1, 2, 1], 16, fp8=fp8, seed=43, pad_tokens=3, extra_rows=8, extra_cols=2)
    for b, j, v in ((0, 1, 10 ** 6), (0, 93, -5), (2, 40, int(c["cache"].shape[0])), (2, 109, -1)):
        c["table"][b, j] = v
    out, lse = check(c, status=api.DSA_DEVERR_BLOCK_OOB | api.DSA_DEVERR_SEQ_LEN,
                     blocked={(0, 1), (0, 93), (2, 40), (2, 109)})
    assert torch.isnan(out[4:]).all() and torch.isnan(lse[4:]).all()
    assert (out[1] == 0).all() and torch.isneginf(lse[1]).all()


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("lens,q_lens,H", [([500, 3000], [1, 1], 16), ([500, 3000], [1, 1], 128),
                                           ([6000, 9000], [2, 4], 128)])
def test_nan_stays_in_its_row(lens, q_lens, H, fp8):
    """A head whose q is NaN, and one whose scores are infinite, leave the
    other heads of the row tile as they are."""
    c = make_dense_case(lens, q_lens, H, fp8=fp8, seed=44)
    want, want_lse = check(c)
    c["q"][0, 3] = float("nan")
    c["q"][1, 7, 5] = float("inf")
    out, lse, _ = call(c)
    keep = torch.ones(out.shape[:2], dtype=torch.bool, device="cuda")
    keep[0, 3] = keep[1, 7] = False
    assert torch.equal(out[keep], want[keep]) and torch.equal(lse[keep], want_lse[keep])
    assert torch.isnan(out[0, 3]).all() and torch.isnan(lse[0, 3])


def test_captured_graph_follows_lengths_between_the_kernels():
    """Long and short contexts, chunks and none, in replays of one graph."""
    c = make_dense_case([9000, 7000], [8, 8], 128, seed=34)
    ws = torch.full((api.dense_mla_workspace_size(16, 128, DV, 0),), 0xFF, dtype=torch.uint8, device="cuda")
    out, lse = torch.empty((16, 128, DV), dtype=torch.bfloat16, device="cuda"), torch.empty((16, 128), device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    args = (c["q"], c["cache"], c["table"], c["seq"], c["qsl"], SCALE, DV, out)
    api.dense_mla_attention(*args, lse=lse, workspace=ws, dev_status=st)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        api.dense_mla_attention(*args, lse=lse, workspace=ws, dev_status=st)
    for lens, q_lens in (([9000, 7000], [8, 8]), ([60, 100], [8, 8]), ([8, 0], [0, 0]), ([8999, 6000], [16, 0]),
                         ([9000, 300], [1, 15])):
        c["seq"].copy_(torch.tensor(lens, dtype=torch.int32))
        c["qsl"].copy_(torch.tensor(np.concatenate([[0], np.cumsum(q_lens)]), dtype=torch.int32))
        out.fill_(float("nan"))
        ws.fill_(0xFF)
        g.replay()
        torch.cuda.synchronize()
        n = sum(q_lens)
        assert int(st.item()) == 0 and torch.isnan(out[n:]).all()
        if n:
            check_dense(out[:n], lse[:n], dense_reference(dict(c, lens=lens, q_lens=q_lens, T=n)))


@pytest.mark.parametrize("fp8", [False, True])
def test_block_stride_and_wide_table(fp8):
    check(make_dense_case([300, 70, 129], [3, 1, 2], 16, fp8=fp8, extra_rows=8, extra_cols=5, seed=3))


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("q_std", [0.0, 30.0, 300.0])
def test_score_ranges(fp8, q_std):
    """Uniform weights, and scores of several hundred, where one key rules."""
    check(make_dense_case([700, 200], [2, 1], 16, fp8=fp8, q_std=q_std, seed=5))


@pytest.mark.parametrize("fp8", [False, True])
def test_rising_scores(fp8):
    """Scores that grow along the keys move the running maximum in every tile."""
    c = make_dense_case([1500], [1], 128, fp8=False, seed=6)
    q = c["q"][0, 0].float()
    n = (torch.arange(1500, device="cuda", dtype=torch.float32) / 50.0)[:, None]
    rows = (q / q.pow(2).sum() / SCALE)[None, :] * n + 0.05 * torch.randn((1500, 576), device="cuda")
    pages = torch.zeros((24, 64, 576), device="cuda")
    pages.view(-1, 576)[:1500] = rows
    if fp8:
        from dense_testlib import encode_fp8
        cache = torch.zeros((c["cache"].shape[0], 64, 656), dtype=torch.uint8, device="cuda")
        enc = encode_fp8(pages.view(-1, 576).cpu()).cuda().view(24, 64, 656)
    else:
        cache, enc = torch.zeros_like(c["cache"]), pages.to(torch.bfloat16)
    cache[c["table"][0].long()] = enc
    c["q"][:] = c["q"][0, 0]
    c.update(cache=cache, fp8=fp8)
    check(c)


@pytest.mark.parametrize("fp8", [False, True])
def test_token_without_a_key(fp8):
    """seq_lens below the query count: the first tokens have no key."""
    c = make_dense_case([100, 2, 0, 70], [1, 5, 2, 3], 16, fp8=fp8, seed=8)
    out, lse = check(c, status=api.DSA_DEVERR_SEQ_LEN)
    assert (out[1:4] == 0).all() and torch.isneginf(lse[1:4]).all()
    assert (out[6:8] == 0).all()


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("splits", [0, -1])
def test_bad_blocks_count_as_masked(fp8, splits):
    c = make_dense_case([300, 64, 500], [2, 1, 1], 16, fp8=fp8, seed=9)
    for b, j, v in ((0, 1, 10 ** 6), (1, 0, -3), (2, 7, -1), (2, 0, int(c["cache"].shape[0]))):
        c["table"][b, j] = v
    check(c, splits, status=api.DSA_DEVERR_BLOCK_OOB, blocked={(0, 1), (1, 0), (2, 7), (2, 0)})


def test_keys_past_the_table_are_masked():
    c = make_dense_case([256, 64], [1, 1], 16, seed=10)
    c["seq"][0] = 300  # the table holds 256 keys
    out, lse, st = call(c)
    torch.cuda.synchronize()
    assert int(st.item()) == api.DSA_DEVERR_SEQ_LEN
    c["seq"][0] = 256
    check_dense(out, lse, dense_reference(c))


@pytest.mark.parametrize("splits", [0, -1])
def test_rows_behind_the_batch_stay(splits):
    c = make_dense_case([100, 200], [1, 3], 128, pad_tokens=5, seed=11)
    out, lse = check(c, splits)
    assert torch.isnan(out[4:]).all() and torch.isnan(lse[4:]).all()


def test_lse_is_optional():
    c = make_dense_case([300], [2], 128, seed=12)
    out, lse, _ = call(c)
    out2, none, _ = call(c, lse=False)
    assert none is None and torch.equal(out, out2)


@pytest.mark.parametrize("fp8", [False, True])
def test_batch_invariant_mode_is_bit_identical(fp8):
    lens, q_lens = [700, 129, 2000, 64, 1], [3, 1, 2, 5, 1]
    c = make_dense_case(lens, q_lens, 16, fp8=fp8, seed=13)
    out, lse, _ = call(c, -1)
    t = 0
    for b in range(5):
        one = dict(c, q=c["q"][t:t + q_lens[b]].contiguous(), table=c["table"][b:b + 1].contiguous(),
                   seq=c["seq"][b:b + 1].contiguous(),
                   qsl=torch.tensor([0, q_lens[b]], dtype=torch.int32, device="cuda"))
        o, l, _ = call(one, -1)
        assert torch.equal(o, out[t:t + q_lens[b]]) and torch.equal(l, lse[t:t + q_lens[b]])
        t += q_lens[b]


def test_repeated_calls_agree_bit_for_bit():
    c = make_dense_case([5000, 900, 3000], [1, 2, 1], 128, seed=14)
    first = call(c)
    for _ in range(3):
        again = call(c)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


def test_other_stream_and_garbage_workspace():
    c = make_dense_case([5000, 900, 3000], [1, 2, 1], 128, seed=15)
    n = api.dense_mla_workspace_size(4, 128, DV, 0)
    ws = torch.full((max(n, 16),), 0xFF, dtype=torch.uint8, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    out, lse, st = call(c, workspace=ws, stream=s)
    s.synchronize()
    assert int(st.item()) == 0
    check_dense(out, lse, dense_reference(c))


def test_captured_graph_follows_new_lengths():
    """One captured call serves later steps whose lengths changed on the device."""
    c = make_dense_case([900, 300, 2000], [2, 2, 2], 16, seed=16)
    ws = torch.empty(max(16, api.dense_mla_workspace_size(6, 16, DV, 0)), dtype=torch.uint8, device="cuda")
    out = torch.empty((6, 16, DV), dtype=torch.bfloat16, device="cuda")
    call(c, workspace=ws, out=out)
    torch.cuda.synchronize()
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    lse = torch.empty((6, 16), dtype=torch.float32, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        api.dense_mla_attention(c["q"], c["cache"], c["table"], c["seq"], c["qsl"], SCALE, DV, out, lse=lse,
                                workspace=ws, dev_status=st)
    for lens, q_lens in (([900, 300, 2000], [2, 2, 2]), ([5, 250, 1999], [1, 4, 1]), ([64, 1, 130], [0, 1, 5])):
        c["seq"].copy_(torch.tensor(lens, dtype=torch.int32))
        c["qsl"].copy_(torch.tensor(np.concatenate([[0], np.cumsum(q_lens)]), dtype=torch.int32))
        out.fill_(float("nan"))
        g.replay()
        torch.cuda.synchronize()
        now = dict(c, lens=lens, q_lens=q_lens, T=sum(q_lens))
        check_dense(out[:sum(q_lens)], lse[:sum(q_lens)], dense_reference(now))


def test_own_workspace_on_another_stream():
    """The workspace a call takes itself is not given to the current stream
    while the call still waits on its own."""
    c = make_dense_case([9000, 3000], [1, 1], 128, seed=51)
    n = api.dense_mla_workspace_size(2, 128, DV, 0)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        torch.cuda._sleep(20_000_000)
    out = torch.full((2, 128, DV), float("nan"), dtype=torch.bfloat16, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    lse = torch.empty((2, 128), device="cuda")
    torch.cuda.current_stream().synchronize()
    api.dense_mla_attention(c["q"], c["cache"], c["table"], c["seq"], c["qsl"], SCALE, DV, out, lse=lse,
                            dev_status=st, stream=s)
    other = [torch.zeros(n, dtype=torch.uint8, device="cuda") for _ in range(3)]
    torch.cuda.synchronize()
    assert int(st.item()) == 0 and all(int(o.max().item()) == 0 for o in other)
    check_dense(out, lse, dense_reference(c))


def test_two_calls_at_once_with_a_workspace_each():
    cs = [make_dense_case([4000 + 100 * i, 700], [1, 3], 128, seed=20 + i, fp8=bool(i)) for i in range(2)]
    ws = [torch.empty(max(16, api.dense_mla_workspace_size(4, 128, DV, 0)), dtype=torch.uint8, device="cuda")
          for _ in cs]
    streams = [torch.cuda.Stream() for _ in cs]
    torch.cuda.synchronize()
    res = [[], []]
    for _ in range(4):
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                res[i].append(call(cs[i], workspace=ws[i]))
    torch.cuda.synchronize()
    for i in range(2):
        ref = dense_reference(cs[i])
        for out, lse, st in res[i]:
            assert int(st.item()) == 0
            check_dense(out, lse, ref)


@pytest.mark.parametrize("fp8", [False, True])
def test_cache_past_32_bit_offsets(fp8):
    c = make_dense_case([300, 64], [2, 1], 16, fp8=fp8, seed=17)
    row = c["cache"].shape[2]
    nb = (1 << 32) // (64 * row * (1 if fp8 else 2)) * (2 if not fp8 else 1) + 60
    big = torch.zeros((nb, 64, row), dtype=c["cache"].dtype, device="cuda")
    n = c["cache"].shape[0]
    big[nb - n:] = c["cache"]
    c["table"][c["table"] >= 0] += nb - n
    c["cache"] = big
    check(c)


def test_full_selection_of_the_sparse_path_agrees():
    """The sparse path over every key is the same sum; both are within their
    roundings of it, the sparse normaliser of bf16 weights (2^-9 each) included."""
    c = make_dense_case([500, 129, 64], [2, 1, 1], 128, seed=18)
    out, lse, _ = call(c)
    idx = torch.full((4, 512), -1, dtype=torch.int32, device="cuda")
    for t, n in enumerate([499, 500, 129, 64]):
        idx[t, :n] = torch.arange(n, dtype=torch.int32)
    o2 = torch.empty_like(out)
    api.sparse_mla_prefill(c["q"], c["cache"], c["table"], c["seq"], c["qsl"], idx, SCALE, DV, o2)
    ref, tol, _, _ = dense_reference(c)
    assert ((out.double() - o2.double()).abs() <= 2 * tol + 2.0 ** -8 * ref.abs()).all()


def test_refusals_of_the_binding():
    c = make_dense_case([300], [2], 16, seed=19)
    T, H = 2, 16
    out = torch.empty((T, H, DV), dtype=torch.bfloat16, device="cuda")
    args = [c["q"], c["cache"], c["table"], c["seq"], c["qsl"], SCALE, DV, out]

    def bad(err, i=None, v=None, **kw):
        a = list(args)
        if i is not None:
            a[i] = v
        with pytest.raises(err):
            api.dense_mla_attention(*a, **kw)

    bad(TypeError, 0, c["q"].float())
    bad(ValueError, 0, c["q"].transpose(0, 1))
    bad(TypeError, 1, c["cache"].view(torch.uint8))
    bad(ValueError, 1, c["cache"][:, :, :512].contiguous())
    bad(TypeError, 2, c["table"].long())
    bad(ValueError, 4, c["qsl"][:1])
    bad(ValueError, 7, out[:1])
    bad(TypeError, 7, out.float())
    bad(ValueError, lse=torch.empty((T, H + 1), dtype=torch.float32, device="cuda"))
    bad(api.DsaError, 5, -1.0)
    bad(api.DsaError, num_kv_splits=3)
    bad(ValueError, 3, c["seq"].cpu())


def test_small_workspace_is_refused():
    c = make_dense_case([300], [2], 16, seed=19)
    need = api.dense_mla_workspace_size(2, 16, DV, 0)
    if need == 0:
        pytest.skip("no workspace needed")
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    out = torch.empty((2, 16, DV), dtype=torch.bfloat16, device="cuda")

    def rc(ptr, n):
        return api.lib.dense_mla_attention(
            api._ptr(c["q"]), api._ptr(c["cache"]), 64 * 576, c["cache"].shape[0], api._ptr(c["table"]),
            c["table"].shape[1], api._ptr(c["seq"]), api._ptr(c["qsl"]), 1, 2, 16, 576, DV, 64, SCALE, 0,
            api._ptr(out), None, ptr, n, None, api._stream(None))

    assert rc(api._ptr(ws), need - 1) == api.DSA_ERR_WORKSPACE
    assert rc(None, need) == api.DSA_ERR_WORKSPACE
    assert rc(api._ptr(ws), need) == api.DSA_OK
    torch.cuda.synchronize()
