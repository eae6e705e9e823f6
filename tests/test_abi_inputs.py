"""Refusals of the operators in front of the scores, without a GPU: every call here is rejected by
the library's or the binding's argument checks, or has nothing to do, before the HIP runtime is
touched."""

import os
import struct

import pytest
import torch

from dsa_indexer_top_amd import binding as B

# The addresses here are no memory: a check that failed to refuse one would launch a kernel on it, so
# these tests stay off machines with a GPU.
pytestmark = [pytest.mark.skipif(not os.path.exists(B.LIB_PATH), reason="library not built"),
              pytest.mark.skipif(torch.cuda.is_available(), reason="made-up addresses: only without a GPU")]

F = 0x1000                     # never dereferenced
PAGE = struct.Struct("=5i4x13Q")          # echo_page_args
QK = struct.Struct("=11if2Q4q6Q")         # echo_qk_args


def err():
    return B.lib().echo_last_error().decode()


def page_args(**kw):
    a = dict(n_rows=4, page_size=16, max_pages=8, n_pages=32, max_new=16, len_in=F, new_len=F, done=0, page_table=F,
             free_list=F, count_in=F, len_out=F, count_out=F, row_begin=F, slot=F, row=0, pos=F, status=F)
    assert set(kw) <= set(a)
    a.update(kw)
    return PAGE.pack(*a.values())


def test_page_step_argument_errors():
    call = lambda ws=F, nb=1 << 20, **kw: B.lib().echo_page_step(page_args(**kw), ws, nb, None)
    assert B.lib().echo_page_step(None, F, 1 << 20, None) == B.ECHO_EINVAL
    for name in ("n_rows", "max_pages", "n_pages", "max_new"):
        assert call(**{name: -1}) == B.ECHO_EINVAL and "negative" in err()
    for size in (0, 8, 24, 48, 131072):
        assert call(page_size=size) == B.ECHO_EUNSUPPORTED and "power of two" in err()
    assert call(n_rows=65536) == B.ECHO_EUNSUPPORTED
    for name in ("len_in", "new_len", "page_table", "free_list", "count_in", "len_out", "count_out", "row_begin",
                 "slot", "pos", "status"):
        assert call(**{name: 0}) == B.ECHO_EINVAL and "NULL" in err(), name
    # many tokens or many requests need a workspace
    for kw in (dict(max_new=9000), dict(n_rows=3000)):
        need = B.page_workspace_bytes(kw.get("n_rows", 4), kw.get("max_new", 16))
        assert need > 0
        assert call(ws=None, nb=0, **kw) == B.ECHO_EWORKSPACE
        assert call(nb=need - 1, **kw) == B.ECHO_EWORKSPACE
    assert call(n_rows=0, max_new=0) == B.ECHO_OK
    assert B.page_workspace_bytes(-1, 4) == 0
    assert B.page_workspace_bytes(100, 4) < B.page_workspace_bytes(1000, 4)


def test_quant_argument_errors():
    def call(x=F, t=B.BF16, rows=4, cols=256, ldx=256, y=F, ldy=256, s=F, sr=2, sb=1):
        return B.lib().echo_quant_fp8(x, t, rows, cols, ldx, y, ldy, s, sr, sb, None)
    assert call(rows=-1) == B.ECHO_EINVAL and call(cols=-1) == B.ECHO_EINVAL
    assert call(t=3) == B.ECHO_EINVAL and "type" in err()
    assert call(x=None) == call(y=None) == call(s=None) == B.ECHO_EINVAL
    assert call(ldx=255) == call(ldy=255) == B.ECHO_EINVAL and "stride" in err()
    assert call(ldx=0) == B.ECHO_EINVAL                      # rows on top of each other
    assert call(sr=0) == call(sb=0) == B.ECHO_EINVAL
    assert call(x=F + 1) == call(s=F + 2) == B.ECHO_EINVAL and "aligned" in err()
    assert call(t=B.FP32, x=F + 2) == B.ECHO_EINVAL
    assert call(cols=(1 << 30) + 1, ldx=1 << 31, ldy=1 << 31) == B.ECHO_EUNSUPPORTED
    assert call(rows=1 << 40) == call(rows=1 << 30, cols=1) == B.ECHO_EUNSUPPORTED
    assert call(rows=0) == call(cols=0) == B.ECHO_OK


def test_matmul_argument_errors():
    def call(a=F, lda=256, sa=F, ar=2, ab=1, b=F, ldb=256, sb=F, br=2, bb=1, m=4, n=8, k=256, c=F, ldc=8, t=B.BF16):
        return B.lib().echo_matmul_fp8(a, lda, sa, ar, ab, b, ldb, sb, br, bb, m, n, k, c, ldc, t, None)
    assert call(m=-1) == call(n=-1) == call(k=-1) == B.ECHO_EINVAL
    assert call(t=7) == B.ECHO_EINVAL
    for name in ("a", "b", "sa", "sb", "c"):
        assert call(**{name: None}) == B.ECHO_EINVAL and "NULL" in err(), name
    assert call(lda=240) == call(ldb=240) == call(ldc=7) == B.ECHO_EINVAL and "stride" in err()
    assert call(a=F + 8) == call(b=F + 4) == call(lda=264) == call(ldb=260) == B.ECHO_EUNSUPPORTED
    assert "16" in err()
    assert call(lda=1 << 23) == call(ldb=(1 << 22) + 16) == B.ECHO_EUNSUPPORTED
    assert call(ar=-1) == call(ar=(1 << 22) + 1) == call(ab=-1) == call(br=-1) == call(bb=-1) == B.ECHO_EUNSUPPORTED
    assert call(c=F + 1) == B.ECHO_EINVAL and call(c=F + 2, t=B.FP32) == B.ECHO_EINVAL
    assert call(sa=F + 2) == call(sb=F + 1) == B.ECHO_EINVAL
    big = (1 << 26) + 1
    assert call(m=big) == call(n=big, ldc=big) == B.ECHO_EUNSUPPORTED
    assert call(m=1 << 24, n=1 << 24, ldc=1 << 24) == B.ECHO_EUNSUPPORTED
    assert call(m=0) == call(n=0, ldc=0) == B.ECHO_OK


def qk_args(**kw):
    a = dict(n_tok=4, n_q_heads=8, n_k_heads=1, head_dim=128, type=B.BF16, q_norm=0, k_norm=1, rot_begin=0, rot_dim=64,
             interleaved=0, n_pos=100, eps=1e-6, q=F, k=F, qt=1024, qh=128, kt=128, kh=128, qw=0, qb=0, kw=F, kb=0,
             pos=F, cos_sin=F)
    assert set(kw) <= set(a)
    a.update(kw)
    return QK.pack(*a.values())


def both_calls():
    L = B.lib()
    yield lambda **kw: L.echo_qk_norm_rope(qk_args(**kw), F, 1024, 128, F, 128, 128, None)
    yield lambda **kw: L.echo_indexer_qk(qk_args(**kw), F, 8, 1.0, F, F, F, F, F, 64, None)


def test_heads_argument_errors():
    L = B.lib()
    assert L.echo_qk_norm_rope(None, F, 1024, 128, F, 128, 128, None) == B.ECHO_EINVAL
    assert L.echo_indexer_qk(None, F, 8, 1.0, F, F, F, F, F, 64, None) == B.ECHO_EINVAL
    for call in both_calls():
        for name in ("n_tok", "n_q_heads", "n_k_heads", "n_pos", "rot_begin", "rot_dim"):
            assert call(**{name: -16}) == B.ECHO_EINVAL and "negative" in err(), name
        assert call(type=5) == call(q_norm=3) == call(k_norm=-1) == B.ECHO_EINVAL
        for d in (0, 4, 12, 130, 264):
            assert call(head_dim=d) == B.ECHO_EUNSUPPORTED, d
        assert call(rot_dim=24) == call(rot_begin=4) == B.ECHO_EUNSUPPORTED
        assert call(rot_dim=144) == call(rot_begin=72) == B.ECHO_EINVAL and "behind" in err()
        assert call(eps=-1.0) == call(eps=float("nan")) == B.ECHO_EINVAL
        assert call(q=0) == call(k=0) == call(pos=0) == call(cos_sin=0) == B.ECHO_EINVAL and "NULL" in err()
        assert call(n_tok=1 << 30) == B.ECHO_EUNSUPPORTED
        for kw in (dict(q=F + 8), dict(k=F + 2), dict(qt=1020), dict(qh=132), dict(kt=4), dict(kw=F + 4),
                   dict(qw=F + 8), dict(kb=F + 4), dict(cos_sin=F + 8), dict(type=B.FP32, qh=130)):
            assert call(**kw) == B.ECHO_EUNSUPPORTED and "16 bytes" in err(), kw
        assert call(n_tok=0) == call(n_q_heads=0, n_k_heads=0) == B.ECHO_OK
    rope = lambda *out: L.echo_qk_norm_rope(qk_args(), *out, None)
    assert rope(None, 1024, 128, F, 128, 128) == rope(F, 1024, 128, None, 128, 128) == B.ECHO_EINVAL
    assert rope(F + 8, 1024, 128, F, 128, 128) == rope(F, 1024, 130, F, 128, 128) == B.ECHO_EUNSUPPORTED
    assert rope(F, 1024, 128, F, 130, 128) == B.ECHO_EUNSUPPORTED
    assert rope(F, 1024, 0, F, 128, 128) == rope(F, 64, 128, F, 128, 128) == B.ECHO_EINVAL and "overlap" in err()
    assert rope(F, 1024, 128, F, 0, 128) == rope(F, -1024, 128, F, 128, 128) == B.ECHO_EINVAL
    idx = lambda w=F, q8=F, wo=F, kc=F, ks=F, sl=F, n=64, **kw: L.echo_indexer_qk(qk_args(**kw), w, 8, 1.0, q8, wo, kc, ks, sl, n, None)
    assert idx(head_dim=64) == B.ECHO_EUNSUPPORTED and idx(n_k_heads=2) == B.ECHO_EUNSUPPORTED
    assert idx(n=-1) == B.ECHO_EINVAL
    for name in ("w", "q8", "wo", "kc", "ks", "sl"):
        assert idx(**{name: None}) == B.ECHO_EINVAL and "NULL" in err(), name
    assert idx(q8=F + 4) == idx(kc=F + 1) == B.ECHO_EUNSUPPORTED
    assert idx(w=F + 2) == idx(wo=F + 1) == idx(ks=F + 2) == idx(sl=F + 4) == idx(pos=F + 2) == B.ECHO_EINVAL


# ---------------------------------------------------------------- the binding's own checks
class Stream:
    cuda_stream = 0


@pytest.fixture
def on_cpu(monkeypatch):
    """CPU tensors as the current device's; nothing in these tests gets as far as a launch."""
    monkeypatch.setattr(B, "DEVICE_TYPE", "cpu")


def refused(what, f, *a, **kw):
    with pytest.raises(B.EchoError) as e:
        f(*a, stream=Stream(), **kw)
    assert e.value.code == B.ECHO_EINVAL and what in str(e.value), str(e.value)


def i32(*s):
    return torch.zeros(s, dtype=torch.int32)


def page_tensors(**kw):
    t = dict(len_in=i32(3), new_len=i32(3), page_table=i32(3, 4), page_size=16, free_list=i32(9), count_in=i32(1),
             len_out=i32(3), count_out=i32(1), row_begin=i32(4), slot=torch.zeros(8, dtype=torch.int64), row=i32(8),
             pos=i32(8), status=i32(1), ws=None, done=torch.zeros(3, dtype=torch.uint8))
    t.update(kw)
    return t


@pytest.mark.parametrize("bad", [
    dict(new_len=i32(2)), dict(len_out=i32(4)), dict(row_begin=i32(3)), dict(pos=i32(7)), dict(row=i32(9)),
    dict(slot=i32(8)), dict(page_table=i32(2, 4)), dict(page_table=i32(4, 3).t()), dict(count_in=i32(2)),
    dict(status=torch.zeros(1)), dict(done=i32(3)), dict(done=torch.zeros(2, dtype=torch.uint8)),
    dict(len_in=torch.zeros(3, dtype=torch.int64)), dict(free_list=i32(18)[::2]), dict(pos=i32(16)[::2])],
    ids=lambda d: next(iter(d)))
def test_page_step_tensor_checks(on_cpu, bad):
    refused(next(iter(bad)), B.page_step, **page_tensors(**bad))


def test_product_and_quant_tensor_checks(on_cpu):
    u8, f = lambda *s: torch.zeros(s, dtype=torch.uint8), lambda *s: torch.zeros(s)
    refused("matrix", B.quant_fp8, f(4), u8(4), f(1))
    refused("matrix", B.quant_fp8, u8(4, 128), u8(4, 128), f(4, 1))
    refused("shapes", B.quant_fp8, f(4, 129), u8(4, 129), f(4, 1))
    refused("FP8", B.quant_fp8, f(4, 128), f(4, 128), f(4, 1))
    refused("rows of x", B.quant_fp8, f(128, 4).t(), u8(4, 128), f(4, 1))
    ok = dict(a=u8(4, 256), a_scale=f(4, 2), b=u8(130, 256), b_scale=f(2, 2), c=f(4, 130))
    def mm(what, **kw):
        t = dict(ok, **kw)
        refused(what, B.matmul_fp8, t["a"], t["a_scale"], t["b"], t["b_scale"], t["c"])
    mm("shapes", a_scale=f(4, 1))
    mm("shapes", b_scale=f(1, 2))
    mm("shapes", b=u8(130, 240))
    mm("shapes", c=f(4, 131))
    mm("matrices", c=f(4))
    mm("FP8", a=f(4, 256))
    mm("c is not", c=u8(4, 130))
    mm("scale", a_scale=f(4, 2).double())
    mm("rows of b", b=u8(256, 130).t())
    mm("16-byte piece", a=torch.zeros(4 * 256 - 2, dtype=torch.uint8).as_strided((4, 254), (256, 1)), b=u8(130, 256)[:, :254])
    mm("rows of c", c=f(130, 4).t())


def test_heads_tensor_checks(on_cpu):
    b = lambda *s: torch.zeros(s, dtype=torch.bfloat16)
    ok = dict(q=b(4, 8, 128), k=b(4, 1, 128), q_out=b(4, 8, 128), k_out=b(4, 1, 128), pos=i32(4), cos_sin=torch.zeros(9, 64))
    def rope(what, **kw):
        t = dict(ok, **kw)
        refused(what, B.qk_norm_rope, t.pop("q"), t.pop("k"), t.pop("q_out"), t.pop("k_out"), t.pop("pos"), t.pop("cos_sin"), **t)
    rope("[tokens, heads", k=b(4, 128))
    rope("[tokens, heads", k=b(4, 1, 128).float())
    rope("[tokens, heads", q=torch.zeros(4, 8, 128, dtype=torch.int8))
    rope("numbers of tokens", k=b(5, 1, 128))
    rope("head sizes", k=b(4, 1, 64))
    rope("heads of q", q=b(4, 128, 8).transpose(1, 2))
    rope("pos", pos=i32(3))
    rope("pos", pos=torch.zeros(4, dtype=torch.int64))
    rope("cos_sin", cos_sin=torch.zeros(9, 64).double())
    rope("q_weight", q_weight=torch.ones(64))
    rope("k_bias", k_bias=b(128))
    rope("does not match", q_out=b(4, 8, 64))
    rope("does not match", k_out=b(4, 1, 128).float())
    f = torch.zeros
    oki = dict(w=f(4, 8), q8=f(4, 8, 128, dtype=torch.uint8), w_out=f(4, 8), k_cache=f(32, 128, dtype=torch.uint8),
               k_scale=f(32), slot=f(4, dtype=torch.int64))
    def idx(what, **kw):
        t = dict(oki, **kw)
        refused(what, B.indexer_qk, ok["q"], ok["k"], t["w"], t["q8"], t["w_out"], t["k_cache"], t["k_scale"],
                t["slot"], ok["pos"], ok["cos_sin"])
    idx("w ", w=f(4, 7))
    idx("w ", w=b(4, 8))
    idx("rows of w", w=f(8, 4).t())
    idx("q8", q8=f(4, 8, 64, dtype=torch.uint8))
    idx("w_out", w_out=f(4, 16)[:, ::2])
    idx("numbers of keys", k_scale=f(31))
    idx("k_cache", k_cache=f(32, 128))
    idx("slot", slot=i32(4))
    idx("slot", slot=f(5, dtype=torch.int64))


def test_newest_queries_refusals(on_cpu):
    def call(q8=F, w=F, begin=F, n=F, rows=4, tok=9, heads=64, qo=F, wo=F, lo=F):
        return B.lib().echo_newest_queries(q8, w, begin, n, rows, tok, heads, qo, wo, lo, None)
    assert call(rows=-1) == call(tok=-1) == call(heads=-1) == B.ECHO_EINVAL and "negative" in err()
    for name in ("q8", "w", "begin", "n", "qo", "wo", "lo"):
        assert call(**{name: None}) == B.ECHO_EINVAL and "NULL" in err(), name
    assert call(q8=F + 4) == call(qo=F + 1) == B.ECHO_EUNSUPPORTED
    assert call(w=F + 2) == call(wo=F + 1) == call(begin=F + 2) == call(n=F + 1) == call(lo=F + 3) == B.ECHO_EINVAL
    assert call(rows=65536) == B.ECHO_EUNSUPPORTED and call(rows=0) == B.ECHO_OK
    u8 = lambda *s: torch.zeros(s, dtype=torch.uint8)
    ok = dict(q8=u8(9, 3, 128), w=torch.zeros(9, 3), row_begin=i32(5), key_len=i32(4), q_out=u8(4, 3, 128),
              w_out=torch.zeros(4, 3), len_out=i32(4))
    for bad in (dict(q8=u8(9, 3, 64)), dict(q8=torch.zeros(9, 3, 128)), dict(w=torch.zeros(9, 2)), dict(row_begin=i32(4)),
                dict(key_len=i32(5)), dict(q_out=u8(3, 3, 128)), dict(w_out=torch.zeros(5, 3)), dict(len_out=i32(3)),
                dict(q8=u8(18, 3, 128)[::2])):
        refused("", B.newest_queries, **dict(ok, **bad))


def shared(n, si, m, sj, size):
    """Whether two of the items at i * si + j * sj share one of their `size` places, one by one."""
    places = [i * si + j * sj + p for i in range(n) for j in range(m) for p in range(size)]
    return len(set(places)) < len(places)


def test_output_heads_that_overlap():
    """Strides that step over a head each and meet together are refused, those whose heads lie between
    one another are not (such a call gets as far as the key side, which overlaps here)."""
    def q_overlaps(n, st, h, sh, dim=16):
        a = qk_args(n_tok=n, n_q_heads=h, head_dim=dim, n_k_heads=2, rot_dim=0, cos_sin=0)
        assert B.lib().echo_qk_norm_rope(a, F, st, sh, F, 1024, 0, None) == B.ECHO_EINVAL and "overlap" in err()
        return "q_out" in err()
    for n in (1, 2, 3, 5):
        for h in (1, 2, 4):
            for st in range(0, 104, 8):
                for sh in range(0, 104, 8):
                    assert q_overlaps(n, st, h, sh) == shared(n, st, h, sh, 16), (n, st, h, sh)
    assert q_overlaps(4, 1 << 40, 8, 1 << 40) and q_overlaps(3, 3 << 39, 4, 1 << 40)
    assert not q_overlaps(1 << 20, 1 << 40, 8, 1 << 61) and not q_overlaps(100, 1 << 40, 8, 16)
    assert q_overlaps(4, -128, 8, 16) and q_overlaps(4, 128, 8, -16)


def test_scales_that_overlap():
    """Scale strides are checked together; those that keep every scale apart get as far as the check of
    the addresses, which are odd here."""
    for rows in (1, 2, 3, 7):
        for blocks in (1, 2, 4, 5):
            for sr in range(0, 9):
                for sb in range(0, 9):
                    rc = B.lib().echo_quant_fp8(F, B.BF16, rows, 128 * blocks, 1024, F, 1024, F + 1, sr, sb, None)
                    assert rc == B.ECHO_EINVAL
                    assert ("overlap" in err()) == shared(rows, sr, blocks, sb, 1), (rows, blocks, sr, sb)
                    assert "overlap" in err() or "aligned" in err()


def test_page_step_alignment(on_cpu):
    """The workspace, where one is used, and every array are aligned to their types."""
    call = lambda ws=F, **kw: B.lib().echo_page_step(page_args(**kw), ws, 1 << 20, None)
    for n in (1, 2, 3):
        assert call(ws=F + n, max_new=9000) == call(ws=F + n, n_rows=3000) == B.ECHO_EINVAL and "aligned" in err()
    for name in ("len_in", "new_len", "page_table", "free_list", "count_in", "len_out", "count_out", "row_begin",
                 "row", "pos", "status"):
        assert call(**{name: F + 2}) == B.ECHO_EINVAL and "aligned" in err(), name
    assert call(slot=F + 4) == B.ECHO_EINVAL
    ws = torch.zeros(B.page_workspace_bytes(3, 9000) + 8, dtype=torch.uint8)[1:]
    big = dict(slot=torch.zeros(9000, dtype=torch.int64), row=i32(9000), pos=i32(9000))
    refused("aligned", B.page_step, **page_tensors(ws=ws, **big))


def test_every_form_of_the_product_is_tested():
    """The sizes of tests/test_gpu_products.py take the kernels they are meant for, and these are all
    there are: a change of the rule that moves a case, or adds a kernel, shows here."""
    from test_gpu_products import CODE, FORMS
    for form, m, n, k, types in FORMS:
        for t in types:
            assert B.matmul_fp8_form(m, n, k, CODE[t]) == form, (m, n, k, t)
    sizes = [1, 17, 33, 65, 200, 400, 700, 1100, 1500, 2000, 2500, 2900, 4097, 6000, 9000, 17000]
    for t in CODE:
        taken = {B.matmul_fp8_form(m, n, k, CODE[t]) for m in sizes for n in sizes for k in (0, 128, 640, 641, 9000)}
        assert taken == {form for form, *_, types in FORMS if t in types}, t
    assert B.matmul_fp8_form(0, 5, 5, B.BF16) == B.matmul_fp8_form(5, 0, 5, B.BF16) == ""
