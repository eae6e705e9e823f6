"""Refusals of the operators behind the selection, without a GPU: every call here is rejected by the
library's or the binding's argument checks, or has nothing to do, before the HIP runtime is touched."""

import os
import struct

import pytest
import torch

from dsa_indexer_top_amd import binding as B
from test_abi_inputs import F, Stream, err, i32, on_cpu, refused  # noqa: F401 (on_cpu: a fixture)

# made-up addresses, as there
pytestmark = [pytest.mark.skipif(not os.path.exists(B.LIB_PATH), reason="library not built"),
              pytest.mark.skipif(torch.cuda.is_available(), reason="made-up addresses: only without a GPU")]

LATENT = struct.Struct("=3ifQ2qQq3i4xQqQQ3i4xQ")          # echo_latent_args
PREFIX = struct.Struct("=3ifQ2qQq7i4x5Q")                 # echo_prefix_args
INF, NAN = float("inf"), float("nan")


def latent(**kw):
    a = dict(n_rows=2, n_heads=16, type=B.BF16, scale=0.1, q=F, q_row=16 * 576, q_head=576, kv=F, kv_stride=576, n_kv=100, k=40,
             block=1, idx=F, idx_stride=40, len=0, page_table=0, page_size=0, max_pages=0, n_tables=0, req=0)
    assert set(kw) <= set(a)
    a.update(kw)
    return LATENT.pack(*a.values())


def prefix(**kw):
    a = dict(n_rows=2, n_heads=16, type=B.BF16, scale=0.1, q=F, q_row=16 * 576, q_head=576, kv=F, kv_stride=576, n_kv=100,
             page_size=16, n_groups=1, max_prefix=64, prefix_pages=4, max_own=32, own_pages=2, begin=F, prefix_len=F,
             prefix_table=F, own_len=F, own_table=F)
    assert set(kw) <= set(a)
    a.update(kw)
    return PREFIX.pack(*a.values())


def sparse_call(out=F, row=16 * 512, head=512, lse=F, ws=F, nb=1 << 30, **kw):
    return B.lib().echo_sparse_attention(latent(**kw), out, row, head, lse, ws, nb, None)


def weights_call(lse=F, w=F, stride=1 << 20, **kw):
    return B.lib().echo_attention_weights(latent(**kw), lse, w, stride, None)


def prefix_call(out=F, row=16 * 512, head=512, lse=F, ws=F, nb=1 << 30, **kw):
    return B.lib().echo_prefix_attention(prefix(**kw), out, row, head, lse, ws, nb, None)


@pytest.mark.parametrize("call", [sparse_call, weights_call, prefix_call])
def test_queries_and_cache(call):
    for name in ("n_rows", "n_heads", "n_kv"):
        assert call(**{name: -1}) == B.ECHO_EINVAL and "negative" in err(), name
    for t in (B.FP32, 3, -1):
        assert call(type=t) == B.ECHO_EINVAL and "type" in err()
    for s in (NAN, INF, -INF, 2e38):
        assert call(scale=s) == B.ECHO_EINVAL and "scale" in err()
    assert call(n_heads=1025) == call(n_rows=(1 << 22) + 1) == B.ECHO_EUNSUPPORTED
    assert call(q=0) == call(kv=0) == B.ECHO_EINVAL and "NULL" in err()
    assert call(q_row=-8) == call(q_head=-8) == call(kv_stride=-576) == call(kv_stride=568) == B.ECHO_EINVAL and "stride" in err()
    assert call(kv_stride=(1 << 30) + 8) == B.ECHO_EUNSUPPORTED
    for kw in (dict(q=F + 8), dict(kv=F + 2), dict(q_row=9220), dict(q_head=580), dict(kv_stride=580)):
        assert call(**kw) == B.ECHO_EUNSUPPORTED and "16 bytes" in err(), kw
    assert call(n_rows=0) == B.ECHO_OK


@pytest.mark.parametrize("call", [sparse_call, weights_call])
def test_lists_and_pages(call):
    paged = dict(page_table=F, page_size=16, max_pages=4, n_tables=2)
    assert call(k=-1) == B.ECHO_EINVAL
    for b in (0, -1, 3, 24, 1 << 17):
        assert call(block=b) == B.ECHO_EUNSUPPORTED and "power of two" in err(), b
    assert call(k=1 << 20, block=512) == B.ECHO_EUNSUPPORTED and "tokens" in err()
    for p in (8, 17, 1 << 17, -16):
        assert call(**dict(paged, page_size=p)) == B.ECHO_EUNSUPPORTED and "page size" in err(), p
    assert call(**dict(paged, page_table=0)) == B.ECHO_EINVAL and "NULL" in err()
    assert call(**dict(paged, max_pages=-1)) == call(**dict(paged, n_tables=-1)) == B.ECHO_EINVAL
    assert call(idx=0) == call(idx_stride=-1) == B.ECHO_EINVAL
    for name in ("idx", "len"):
        assert call(**{name: F + 2}) == B.ECHO_EINVAL and "aligned" in err(), name
    for name in ("page_table", "req"):
        assert call(**dict(paged, **{name: F + 1})) == B.ECHO_EINVAL and "aligned" in err(), name


@pytest.mark.parametrize("call", [sparse_call, prefix_call])
def test_outputs_and_workspaces(call):
    assert call(out=None) == B.ECHO_EINVAL
    assert call(row=-8192) == call(head=-512) == call(head=504) == call(row=512, head=512) == B.ECHO_EINVAL and "overlap" in err()
    assert call(out=F + 8) == call(head=516, row=16 * 516) == B.ECHO_EUNSUPPORTED
    assert call(lse=F + 2) == B.ECHO_EINVAL and "lse" in err()
    long = dict(k=4096) if call is sparse_call else dict(max_prefix=4096)
    need = B.sparse_attention_workspace_bytes(2, 16, 4096) if call is sparse_call else \
        B.prefix_attention_workspace_bytes(2, 16, 1, 4096, 32)
    assert need > 0
    assert call(ws=None, nb=0, **long) == call(ws=F, nb=need - 1, **long) == B.ECHO_EWORKSPACE and str(need) in err()
    assert call(ws=F + 8, **long) == B.ECHO_EINVAL and "workspace" in err()
    assert call(n_heads=0) == B.ECHO_OK


def test_prefix_arguments():
    assert B.lib().echo_prefix_attention(None, F, 512, 512, F, F, 1 << 30, None) == B.ECHO_EINVAL
    for name in ("n_groups", "max_prefix", "max_own", "prefix_pages", "own_pages"):
        assert prefix_call(**{name: -1}) == B.ECHO_EINVAL and "negative" in err(), name
    assert prefix_call(n_groups=65537) == prefix_call(max_prefix=(1 << 28) + 1) == prefix_call(max_own=1 << 29) == B.ECHO_EUNSUPPORTED
    for p in (0, 8, 48):
        assert prefix_call(page_size=p) == B.ECHO_EUNSUPPORTED
    for name in ("begin", "prefix_len", "prefix_table", "own_len", "own_table"):
        assert prefix_call(**{name: 0}) == B.ECHO_EINVAL and "NULL" in err(), name
        assert prefix_call(**{name: F + 2}) == B.ECHO_EINVAL and "aligned" in err(), name


def test_weights_arguments():
    assert B.lib().echo_attention_weights(None, F, F, 40, None) == B.ECHO_EINVAL
    assert B.lib().echo_sparse_attention(None, F, 512, 512, F, F, 0, None) == B.ECHO_EINVAL
    assert weights_call(n_heads=0) == B.ECHO_EINVAL
    assert weights_call(stride=39) == weights_call(stride=-1) == B.ECHO_EINVAL and "overlap" in err()
    assert weights_call(lse=None) == weights_call(w=None) == weights_call(lse=F + 2) == weights_call(w=F + 1) == B.ECHO_EINVAL
    assert weights_call(k=0, idx=0) == B.ECHO_OK
    assert weights_call(n_rows=1 << 20, k=1 << 12) == B.ECHO_EUNSUPPORTED and "launch" in err()


def test_block_topk_arguments():
    def call(scores=F, ld=1000, n=F, rows=3, most=1000, block=64, first=1, last=2, k=4, idx=F, ws=F, nb=1 << 20):
        return B.lib().echo_block_topk(scores, ld, n, rows, most, block, first, last, k, idx, ws, nb, None)
    for name in ("rows", "most", "first", "last"):
        assert call(**{name: -1}) == B.ECHO_EINVAL and "negative" in err(), name
    for b in (0, 8, 48, 1 << 17):
        assert call(block=b) == B.ECHO_EUNSUPPORTED and "power of two" in err()
    assert call(k=0) == call(k=1 << 20) == B.ECHO_EUNSUPPORTED
    assert call(ld=999) == B.ECHO_EINVAL
    for name in ("scores", "n", "idx"):
        assert call(**{name: None}) == B.ECHO_EINVAL and "NULL" in err(), name
        assert call(**{name: F + 2}) == B.ECHO_EINVAL and "aligned" in err(), name
    need = B.block_topk_workspace_bytes(3, 1000, 64)
    assert call(ws=None) == call(nb=need - 1) == B.ECHO_EWORKSPACE and call(ws=F + 1) == B.ECHO_EINVAL
    assert call(rows=1 << 22) == call(rows=1 << 21, most=1 << 20, ld=1 << 20) == B.ECHO_EUNSUPPORTED
    assert call(rows=0) == B.ECHO_OK
    assert B.block_topk_workspace_bytes(-1, 5, 16) == B.block_topk_workspace_bytes(1, 5, 0) == 0


def test_pool_weigh_arguments():
    def call(free=F, prio=F, mass=F, n=100, slot=F, w=F, entries=50, fresh=F, n_fresh=5, decay=0.5, ws=F, nb=1 << 20):
        return B.lib().echo_pool_weigh(free, prio, mass, n, slot, w, entries, fresh, n_fresh, decay, ws, nb, None)
    for name in ("n", "entries", "n_fresh"):
        assert call(**{name: -1}) == B.ECHO_EINVAL and "negative" in err(), name
    for d in (-0.1, 1.1, NAN, INF):
        assert call(decay=d) == B.ECHO_EINVAL and "decay" in err()
    assert call(n=(1 << 22) + 1) == call(entries=(1 << 21) + 1) == call(n_fresh=(1 << 21) + 1) == B.ECHO_EUNSUPPORTED
    for name in ("free", "prio", "mass", "slot", "w", "fresh"):
        assert call(**{name: None}) == B.ECHO_EINVAL and "NULL" in err(), name
        if name != "free":
            assert call(**{name: F + 2}) == B.ECHO_EINVAL and "aligned" in err(), name
    assert call(ws=None) == call(nb=799) == B.ECHO_EWORKSPACE and call(ws=F + 4) == B.ECHO_EINVAL
    assert call(n=0) == B.ECHO_OK and B.pool_weigh_workspace_bytes(100) == 800 and B.pool_weigh_workspace_bytes(0) == 0


def test_workspaces_of_sizes():
    """No sizes, none that are refused, and few rows with many tokens, which are cut."""
    S, P = B.sparse_attention_workspace_bytes, B.prefix_attention_workspace_bytes
    assert S(0, 16, 100) == S(4, 0, 100) == S(4, 16, -1) == S(4, 2000, 100) == 0
    assert S(1, 16, 33) == 0 and S(4096, 128, 2048) == 0
    for rows, heads in ((1, 1), (1, 16), (8, 128), (3, 1024)):
        parts, rest = divmod(S(rows, heads, 1 << 20), rows * heads * 2056)
        assert rest == 0 and 2 <= parts <= 256, (rows, heads)
    assert P(0, 16, 1, 64, 64) == P(4, 16, -1, 64, 64) == P(4, 16, 1, -1, 64) == P(4, 16, 0, 0, 0) == 0
    assert P(4, 16, 1, 64, 0) >= 4 * 16 * 2056 and P(4, 16, 0, 64, 64) >= 4 * 16 * 2056


# ---------------------------------------------------------------- the binding's own checks
def b16(*s):
    return torch.zeros(s, dtype=torch.bfloat16)


SHARED = dict(q=b16(3, 16, 576), kv=b16(50, 576), scale=0.1)
OUT = dict(out=b16(3, 16, 512), lse=torch.zeros(3, 16))
CACHE = [("one type", dict(q=torch.zeros(3, 16, 576))), ("one type", dict(kv=b16(50, 576).half())), ("576", dict(q=b16(3, 16, 512))),
         ("576", dict(q=b16(3, 9216))), ("576", dict(kv=b16(50, 2, 288))), ("kv", dict(kv=b16(576, 50).t())),
         ("heads of q", dict(q=b16(3, 576, 16).transpose(1, 2)))]
RESULT = [("512", dict(out=b16(3, 16, 576))), ("512", dict(out=torch.zeros(3, 16, 512))), ("lse", dict(lse=torch.zeros(3, 15))),
          ("lse", dict(lse=b16(3, 16))), ("heads of out", dict(out=b16(3, 512, 16).transpose(1, 2)))]


@pytest.mark.parametrize("what,bad", CACHE + RESULT + [
    ("idx", dict(idx=i32(2, 8))), ("idx", dict(idx=torch.zeros(3, 8))), ("idx", dict(idx=i32(8, 3).t())), ("length", dict(length=i32(4))),
    ("page_table", dict(page_table=i32(2, 4), page_size=16)), ("page_table", dict(page_table=i32(3, 4, 1), page_size=16)),
    ("page_size", dict(page_table=i32(3, 4))), ("without a page_table", dict(page_size=16)), ("without a page_table", dict(req=i32(3))),
    ("req", dict(page_table=i32(2, 4), page_size=16, req=i32(2)))])
def test_sparse_attention_tensor_checks(on_cpu, what, bad):
    refused(what, B.sparse_attention, **{**SHARED, **OUT, "idx": i32(3, 8), "ws": None, **bad})


@pytest.mark.parametrize("what,bad", CACHE + RESULT + [
    ("group_begin", dict(group_begin=i32(2))), ("prefix_table", dict(prefix_table=i32(1, 4))), ("own_table", dict(own_table=i32(2, 4))),
    ("prefix_table", dict(prefix_table=i32(4, 2).t())), ("own_len", dict(own_len=i32(4))), ("prefix_len", dict(prefix_len=torch.zeros(2)))])
def test_prefix_attention_tensor_checks(on_cpu, what, bad):
    refused(what, B.prefix_attention, **{**SHARED, **OUT, "group_begin": i32(3), "prefix_len": i32(2), "prefix_table": i32(2, 4),
                                         "own_len": i32(3), "own_table": i32(3, 4), "page_size": 16, "max_prefix": 64, "max_own": 64,
                                         "ws": None, **bad})


@pytest.mark.parametrize("what,bad", CACHE + [("lse", dict(lse=torch.zeros(3, 17))), ("w is not", dict(w=torch.zeros(3, 7))),
                                              ("w is not", dict(w=b16(3, 8))), ("rows of w", dict(w=torch.zeros(8, 3).t()))])
def test_attention_weights_tensor_checks(on_cpu, what, bad):
    refused(what, B.attention_weights, **{**SHARED, "idx": i32(3, 8), "lse": torch.zeros(3, 16), "w": torch.zeros(3, 8), **bad})


@pytest.mark.parametrize("what,bad", [
    ("scores", dict(scores=b16(3, 100))), ("scores", dict(scores=torch.zeros(100, 3).t())), ("max_len", dict(max_len=101)),
    ("length", dict(length=i32(2))), ("idx", dict(idx=i32(3, 5))), ("idx", dict(idx=torch.zeros(3, 4)))])
def test_block_topk_tensor_checks(on_cpu, what, bad):
    refused(what, B.block_topk, **{**dict(scores=torch.zeros(3, 100), length=i32(3), max_len=100, block=16, k=4, idx=i32(3, 4),
                                         ws=torch.zeros(4096, dtype=torch.uint8)), **bad})


@pytest.mark.parametrize("what,bad", [
    ("free", dict(free=i32(9))), ("priority", dict(priority=i32(8))), ("mass", dict(mass=torch.zeros(9).double())),
    ("w ", dict(w=torch.zeros(2, 4))), ("slot", dict(slot=torch.zeros(2, 5))), ("fresh", dict(fresh=torch.zeros(3)))])
def test_pool_weigh_tensor_checks(on_cpu, what, bad):
    refused(what, B.pool_weigh, **{**dict(free=torch.zeros(9, dtype=torch.uint8), priority=i32(9), mass=torch.zeros(9), slot=i32(2, 5),
                                         w=torch.zeros(2, 5), ws=torch.zeros(72, dtype=torch.uint8)), **bad})
