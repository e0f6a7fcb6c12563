"""The batch builder and the latent cache writer on the GPU, against plain loops."""
import numpy as np
import pytest
import torch

from dense_testlib import batch_reference

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from deepseek_sparse_attention_fp8_gb300 import api


def dev(a, dtype=np.int32):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=dtype)).cuda()


def run(ctx, new, table, block, T, free=None, head=0, inplace=False, extra=0):
    """The call's results as numpy, in buffers with `extra` sentinel entries behind what it may write."""
    B = len(ctx)
    bufs = dict(seq_lens=torch.full((B + extra,), 77, dtype=torch.int32, device="cuda"),
                query_start_loc=torch.full((B + 1 + extra,), 77, dtype=torch.int32, device="cuda"),
                token_req=torch.full((T + extra,), 77, dtype=torch.int32, device="cuda"),
                positions=torch.full((T + extra,), 77, dtype=torch.int32, device="cuda"),
                slot_map=torch.full((T + extra,), 77, dtype=torch.int64, device="cuda"))
    t, st = dev(table), torch.zeros(1, dtype=torch.int32, device="cuda")
    kw = {}
    if free is not None:
        kw = dict(free_blocks=dev(free), free_head=dev([head]))
        if not inplace:
            kw["free_head_out"] = dev([-5])
    api.dsa_build_batch(dev(ctx), dev(new), t, block, T, dev_status=st, **bufs, **kw)
    torch.cuda.synchronize()
    for name, n in (("seq_lens", B), ("query_start_loc", B + 1), ("token_req", T), ("positions", T), ("slot_map", T)):
        assert (bufs[name][n:] == 77).all(), f"{name} written behind its end"
    res = dict(table=t, seq=bufs["seq_lens"][:B], qsl=bufs["query_start_loc"][:B + 1], req=bufs["token_req"][:T],
               pos=bufs["positions"][:T], slot=bufs["slot_map"][:T])
    res = {k: v.cpu().numpy() for k, v in res.items()}
    if free is not None:
        res["head"] = int(kw["free_head" if inplace else "free_head_out"].item())
    return res, int(st.item())


def check(ctx, new, table, block, T, free=None, head=0, **kw):
    got, err = run(ctx, new, table, block, T, free, head, **kw)
    want = batch_reference(ctx, new, table, block, T, free, head)
    for k in got:
        assert np.array_equal(got[k], want[k]), k
    assert err == want["err"]
    return got


def case(seed, B, ctx_hi, new_hi, block, spare=5, cols_extra=0):
    rng = np.random.default_rng(seed)
    ctx, new = rng.integers(0, ctx_hi + 1, B), rng.integers(0, new_hi + 1, B)
    held = -(-ctx // block)
    need = -(-(ctx + new) // block)
    ids = rng.permutation(int(need.sum()) + spare)
    table = np.full((B, max(1, int(need.max())) + cols_extra), -1)
    at = 0
    for b in range(B):
        table[b, :held[b]] = ids[at:at + held[b]]
        at += held[b]
    return ctx, new, table, ids[at:]


@pytest.mark.parametrize("B,ctx_hi,new_hi,block,pad", [
    (1, 0, 1, 64, 0), (1, 1, 1, 64, 3), (1, 128, 64, 64, 0), (3, 200, 130, 64, 1), (32, 8192, 1, 64, 0),
    (33, 500, 2, 128, 31), (257, 3000, 70, 192, 100), (1024, 300, 5, 64, 0), (1025, 300, 5, 256, 7),
    (3000, 70, 3, 64, 999), (5, 0, 20000, 64, 1), (2, 100000, 60000, 64, 0),
])
def test_build_batch(B, ctx_hi, new_hi, block, pad):
    ctx, new, table, free = case(B + block, B, ctx_hi, new_hi, block, cols_extra=B % 3)
    T = int(new.sum()) + pad
    check(ctx, new, table, block, T, free, 0, extra=9)
    # from the middle of a queue, advancing the head in place
    q = np.concatenate([np.full(11, 10 ** 6), free])
    check(ctx, new, table, block, T, q, 11, inplace=True, extra=3)


def test_build_batch_takes_no_blocks_without_a_queue():
    ctx, new, table, _ = case(4, 9, 900, 200, 64)
    full = np.arange(table.size).reshape(table.shape)
    check(ctx, new, full, 64, int(new.sum()))
    # an entry that is missing: its tokens get slot -1 and the status bit
    full[2, ctx[2] // 64] = -1
    new[2] = max(new[2], 1)
    check(ctx, new, full, 64, int(new.sum()))


def test_build_batch_queue_runs_out():
    ctx, new, table, free = case(5, 20, 300, 150, 64)
    T = int(new.sum())
    taken = int((-(-(ctx + new) // 64) - -(-ctx // 64)).sum())
    assert taken > 6
    for n in (0, 1, taken - 1, taken):
        check(ctx, new, table, 64, T, free[:n], 0)
    check(ctx, new, table, 64, T, free, len(free))      # head at the end
    check(ctx, new, table, 64, T, free, len(free) + 1)  # head outside the queue
    check(ctx, new, table, 64, T, free, -1)
    bad = free.copy()
    bad[3] = -7
    check(ctx, new, table, 64, T, bad, 0)


def test_build_batch_narrow_table_and_small_buffers():
    ctx, new, table, free = case(6, 12, 400, 300, 64)
    T = int(new.sum())
    check(ctx, new, table[:, :3], 64, T, free, 0)
    for n in (T - 1, T // 2, 1, 0):
        check(ctx, new, table, 64, n, free, 0, extra=4)


def test_build_batch_bad_lengths():
    ctx, new, table, free = case(7, 6, 100, 50, 64)
    ctx[1], new[2] = -4, -1
    ctx[4], new[4] = 2 ** 31 - 5, 20
    check(ctx, new, table, 64, int(new[new > 0].sum()) + 4, free, 0)


def test_build_batch_without_requests():
    out = api.dsa_build_batch(dev([]), dev([]), dev(np.zeros((0, 4))), 64, 3)
    torch.cuda.synchronize()
    assert out[1].tolist() == [0] and out[2].tolist() == [-1] * 3 and out[4].tolist() == [-1] * 3


def test_build_batch_replayed_graph_walks_the_queue():
    """A captured call with the head in place: each replay serves the next
    step's lengths, as a decode loop does."""
    ctx, new, table, free = case(8, 7, 200, 1, 64, spare=400)
    T = 64
    d_ctx, d_new, d_table = dev(ctx), dev(new), dev(table)
    d_free, d_head = dev(free), dev([0])
    outs = api.dsa_build_batch(d_ctx, d_new, d_table, 64, T, free_blocks=d_free, free_head=d_head)
    d_table.copy_(dev(table))
    d_head.zero_()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        api.dsa_build_batch(d_ctx, d_new, d_table, 64, T, free_blocks=d_free, free_head=d_head, seq_lens=outs[0],
                            query_start_loc=outs[1], token_req=outs[2], positions=outs[3], slot_map=outs[4])
    rng = np.random.default_rng(0)
    want, head = dict(table=table), 0
    for _ in range(6):
        new = rng.integers(0, 9, 7)
        new = np.minimum(new, table.shape[1] * 64 - ctx)
        d_ctx.copy_(dev(ctx))
        d_new.copy_(dev(new))
        g.replay()
        torch.cuda.synchronize()
        want = batch_reference(ctx, new, want["table"], 64, T, free, head)
        head = want["head"]
        assert np.array_equal(d_table.cpu().numpy(), want["table"]) and int(d_head.item()) == head
        assert np.array_equal(outs[4].cpu().numpy(), want["slot"]) and np.array_equal(outs[0].cpu().numpy(),
                                                                                      want["seq"])
        ctx = ctx + new


@pytest.mark.parametrize("T,Dk,block,stride", [(1, 576, 64, 576), (31, 576, 64, 576), (257, 576, 192, 2112),
                                               (1000, 576, 128, 584), (65, 80, 64, 96), (3, 8, 64, 8)])
def test_kv_cache_writer(T, Dk, block, stride):
    gen = torch.Generator().manual_seed(T)
    nb = -(-T // block) + 4
    # any bit pattern has to arrive as it is, NaNs too
    wide = torch.randint(-2 ** 15, 2 ** 15, (T, stride), generator=gen, dtype=torch.int16)
    base = torch.randint(-2 ** 15, 2 ** 15, (nb, block, Dk), generator=gen, dtype=torch.int16)
    slots = torch.randperm(nb * block, generator=gen)[:T]
    slots[T // 2] = -1
    kv = wide.cuda().view(torch.bfloat16)[:, stride - Dk:]
    cache, st = base.cuda().view(torch.bfloat16), torch.zeros(1, dtype=torch.int32, device="cuda")
    api.dsa_mla_kv_cache(kv, slots.cuda(), cache, dev_status=st)
    want = base.clone().view(-1, Dk)
    for t, s in enumerate(slots.tolist()):
        if s >= 0:
            want[s] = wide[t, stride - Dk:]
    assert torch.equal(cache.view(torch.int16).cpu().view(-1, Dk), want) and int(st.item()) == 0


def test_kv_cache_writer_skips_and_reports_bad_slots():
    kv = torch.randn((5, 576), device="cuda").to(torch.bfloat16)
    cache, st = torch.zeros((2, 64, 576), dtype=torch.bfloat16, device="cuda"), dev([0])
    api.dsa_mla_kv_cache(kv, dev([3, 128, -2, 1 << 40, -1], np.int64), cache, dev_status=st)
    want = torch.zeros_like(cache)
    want[0, 3] = kv[0]
    assert torch.equal(cache, want) and int(st.item()) == api.DSA_DEVERR_BLOCK_OOB
    st.zero_()
    api.dsa_mla_kv_cache(kv[:1], dev([-1], np.int64), cache, dev_status=st)
    assert torch.equal(cache, want) and int(st.item()) == 0


def test_kv_cache_writer_wide_block_stride():
    """Blocks further apart than their rows, through the C entry point."""
    kv = torch.randn((70, 576), device="cuda").to(torch.bfloat16)
    cache = torch.zeros((3, 66, 576), dtype=torch.bfloat16, device="cuda")
    slots = dev(np.r_[100:130, 20:60], np.int64)
    st = api.lib.dsa_mla_kv_cache(api._ptr(kv), 576, 70, 576, api._ptr(slots), api._ptr(cache), 66 * 576, 3, 64, None,
                                  api._stream(None))
    assert st == 0
    want = torch.zeros_like(cache)
    for t, s in enumerate(slots.tolist()):
        want[s // 64, s % 64] = kv[t]
    assert torch.equal(cache, want)


def test_kv_cache_writer_past_32_bit_offsets():
    nb = (1 << 32) // (64 * 576) + 2  # elements pass 2^32
    cache = torch.zeros((nb, 64, 576), dtype=torch.bfloat16, device="cuda")
    kv = torch.randn((2, 576), device="cuda").to(torch.bfloat16)
    api.dsa_mla_kv_cache(kv, dev([nb * 64 - 1, 5], np.int64), cache)
    assert torch.equal(cache[-1, -1], kv[0]) and torch.equal(cache[0, 5], kv[1])
    assert int(cache[:, :, 0].ne(0).sum()) <= 2


def test_refusals_of_the_binding():
    t = torch.zeros((4, 576), dtype=torch.bfloat16, device="cuda")
    cache = torch.zeros((2, 64, 576), dtype=torch.bfloat16, device="cuda")
    with pytest.raises(TypeError):
        api.dsa_mla_kv_cache(t.float(), dev([0] * 4, np.int64), cache)
    with pytest.raises(TypeError):
        api.dsa_mla_kv_cache(t, dev([0] * 4), cache)
    with pytest.raises(ValueError):
        api.dsa_mla_kv_cache(t, dev([0] * 3, np.int64), cache)
    with pytest.raises(ValueError):
        api.dsa_mla_kv_cache(t.t().contiguous().t(), dev([0] * 4, np.int64), cache)
    with pytest.raises(ValueError):
        api.dsa_build_batch(dev([1]), dev([1]), dev([[0]]), 64, 4, slot_map=dev([0], np.int64))
    with pytest.raises(ValueError):
        api.dsa_build_batch(dev([1, 2]), dev([1]), dev([[0], [0]]), 64, 4)
    with pytest.raises(api.DsaError) as e:
        api.dsa_build_batch(dev([1]), dev([1]), dev([[0]]), 32, 4)
    assert e.value.status == api.DSA_ERR_UNSUPPORTED
