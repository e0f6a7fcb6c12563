"""Host-side refusals of the batch builder, the latent cache writer and dense
MLA attention: bad arguments are rejected before anything is launched."""
import ctypes

import pytest

import __graft_entry__

NULL = ctypes.c_void_p(0)
FAKE = ctypes.c_void_p(1 << 20)  # never dereferenced: validation fails first


@pytest.fixture(scope="module")
def api():
    __graft_entry__.build()
    from deepseek_sparse_attention_fp8_gb300 import api as a

    return a


@pytest.mark.parametrize("fp8", [False, True])
def test_dense_attention_rejects_bad_arguments(api, fp8):
    row = 656 if fp8 else 576
    fn = api.lib.dense_mla_attention_fp8 if fp8 else api.lib.dense_mla_attention

    def call(q=FAKE, cache=FAKE, stride=64 * row, nb=10, table=FAKE, bt=4, sl=FAKE, qsl=FAKE, B=1, T=1, H=128, Dk=576,
             Dv=512, bs=64, scale=0.04, splits=0, out=FAKE, lse=NULL, ws=NULL, ws_bytes=0):
        return fn(q, cache, stride, nb, table, bt, sl, qsl, B, T, H, Dk, Dv, bs, scale, splits, out, lse, ws, ws_bytes,
                  NULL, NULL)

    for kw in (dict(T=-1), dict(B=-1), dict(H=0), dict(nb=-1), dict(bt=-1), dict(bs=0), dict(B=0),
               dict(q=NULL), dict(cache=NULL), dict(table=NULL), dict(sl=NULL), dict(qsl=NULL), dict(out=NULL),
               dict(q=ctypes.c_void_p((1 << 20) + 8)), dict(out=ctypes.c_void_p((1 << 20) + 2)),
               dict(scale=0.0), dict(scale=-1.0), dict(scale=float("nan")), dict(scale=float("inf")),
               dict(splits=2), dict(splits=-2), dict(stride=64 * row - row)):
        assert call(**kw) == api.DSA_ERR_INVALID_ARG, kw
    for kw in (dict(Dk=80, Dv=64), dict(Dv=256), dict(H=129), dict(bs=32), dict(bs=96), dict(stride=64 * row + 8),
               dict(nb=(1 << 31) - 1)):
        assert call(**kw) == api.DSA_ERR_UNSUPPORTED, kw
    assert call(T=0) == api.DSA_OK  # nothing to do: no device touched


def test_build_batch_rejects_bad_arguments(api):
    def call(ctx=FAKE, new=FAKE, B=2, bs=64, free=FAKE, num_free=4, head=FAKE, head_out=FAKE, table=FAKE, bt=4, T=8,
             seq=FAKE, qsl=FAKE, req=FAKE, pos=FAKE, slot=FAKE):
        return api.lib.dsa_build_batch(ctx, new, B, bs, free, num_free, head, head_out, table, bt, T, seq, qsl, req,
                                       pos, slot, NULL, NULL)

    for kw in (dict(B=-1), dict(bs=0), dict(num_free=-1), dict(bt=-1), dict(T=-1), dict(ctx=NULL), dict(new=NULL),
               dict(table=NULL), dict(seq=NULL), dict(qsl=NULL), dict(req=NULL), dict(pos=NULL), dict(slot=NULL),
               dict(head=NULL), dict(head_out=NULL), dict(free=NULL)):
        assert call(**kw) == api.DSA_ERR_INVALID_ARG, kw
    assert call(bs=32) == api.DSA_ERR_UNSUPPORTED
    other = ctypes.c_void_p(1 << 21)
    assert call(seq=other, qsl=FAKE) == api.DSA_ERR_INVALID_ARG  # outputs in the inputs' memory
    assert call(seq=FAKE, qsl=other) == api.DSA_ERR_INVALID_ARG


def test_kv_cache_rejects_bad_arguments(api):
    def call(kv=FAKE, stride=576, T=4, Dk=576, slots=FAKE, cache=FAKE, bstride=64 * 576, nb=10, bs=64):
        return api.lib.dsa_mla_kv_cache(kv, stride, T, Dk, slots, cache, bstride, nb, bs, NULL, NULL)

    for kw in (dict(T=-1), dict(Dk=0), dict(bs=0), dict(nb=-1), dict(kv=NULL), dict(slots=NULL), dict(cache=NULL),
               dict(stride=568), dict(stride=580), dict(bstride=64 * 576 - 8), dict(bstride=64 * 576 + 4),
               dict(kv=ctypes.c_void_p((1 << 20) + 4))):
        assert call(**kw) == api.DSA_ERR_INVALID_ARG, kw
    assert call(Dk=580, stride=584, bstride=64 * 584) == api.DSA_ERR_UNSUPPORTED
    assert call(bs=32, bstride=64 * 576) == api.DSA_ERR_UNSUPPORTED
    assert call(T=0) == api.DSA_OK


def test_dense_workspace_does_not_grow_with_the_batch(api):
    size = api.dense_mla_workspace_size(32, 128, 512, 0)
    assert api.dense_mla_workspace_size(4096, 128, 512, 0) == size
    for splits in (1, api.DSA_KV_SPLITS_BATCH_INVARIANT):
        assert api.dense_mla_workspace_size(32, 128, 512, splits) == 0
    assert api.dense_mla_workspace_size(0, 128, 512, 0) == 0
