"""The 8-bit paged cache without a GPU: argument checks of the C ABI and the
pins of the 64-bit reference."""
import ctypes
import math

import pytest
import torch

from tests import q8_ref

nsa = pytest.importorskip("dynamic_block_sparse_nsa_b200.nsa")
L = nsa.LIB
FAKE = ctypes.c_void_p(256)
ODD = ctypes.c_void_p(264)


def cache(**kw):
    f = dict(k_pages=256, v_pages=256, k_scale=256, v_scale=256, page_table=256, num_pages=4)
    f.update(kw)
    return nsa.NsaQ8Cache(**f)


def rope(table=256, length=64, dim=64, style=0):
    return nsa.NsaRope(table, length, dim, style)


def detail():
    return L.nsa_last_error_detail().decode()


def append(p, c=None, k=FAKE, v=FAKE, N=2, pos=FAKE, cu=None, turn=None, q=None, q_out=None,
           k_out=None, v_out=None):
    c = cache() if c is None else c
    return L.nsa_append_q8(ctypes.byref(p), ctypes.byref(c), k, v, N, pos, cu,
                           None if turn is None else ctypes.byref(turn), q, q_out, k_out, v_out,
                           None)


def decode(p, c=None, q=FAKE, lens=FAKE, keys=0, sel=None, out=FAKE, lse=FAKE, ws=FAKE, nbytes=None):
    c = cache() if c is None else c
    nbytes = nsa.workspace_size(p, nsa.OP_DECODE_Q8) if nbytes is None else nbytes
    return L.nsa_decode_q8(ctypes.byref(p), ctypes.byref(c), q, lens, keys, sel, out, lse, ws,
                           nbytes, None)


def prefill(p, c=None, q=FAKE, N=8, cu=FAKE, lens=FAKE, keys=0, out=FAKE, lse=FAKE, ws=FAKE,
            nbytes=None):
    c = cache() if c is None else c
    nbytes = nsa.workspace_size(p, nsa.OP_PREFILL_Q8) if nbytes is None else nbytes
    return L.nsa_prefill_q8(ctypes.byref(p), ctypes.byref(c), q, N, cu, lens, keys, out, lse, ws,
                            nbytes, None)


P = nsa.params(2, 1000, 16, 2, 64)


@pytest.mark.parametrize("call", (append, decode, prefill))
def test_cache_and_parameters_are_checked(call):
    for field in ("k_pages", "v_pages", "k_scale", "v_scale", "page_table"):
        assert call(P, cache(**{field: None})) == 1
        assert field in detail()
    assert call(P, cache(num_pages=0)) == 1
    assert call(P, cache(k_pages=264)) == 1 and "aligned" in detail()
    assert call(P, cache(v_pages=264)) == 1 and "aligned" in detail()
    for page in (0, 8, 24, 48, 256):
        bad = nsa.params(2, 1000, 16, 2, 64, sel_block=page)
        n = ctypes.c_size_t()
        assert L.nsa_workspace_size(ctypes.byref(bad), nsa.OP_DECODE_Q8, ctypes.byref(n)) == 2
        kw = {} if call is append else {"nbytes": 0}
        assert call(bad, **kw) == 2 and "pages" in detail()
    for bad in (nsa.params(2, 1000, 15, 2, 64), nsa.params(0, 1000, 16, 2, 64),
                nsa.params(2, 1000, 16, 2, 96)):
        assert call(bad, **({} if call is append else {"nbytes": 0})) in (1, 2)


def test_longest_sequence():
    """T up to 2^30 is taken, and no more (positions, and what lies past them, are ints)."""
    n = ctypes.c_size_t()
    for T, want in ((1 << 30, 0), ((1 << 30) + 1, 2)):
        p = nsa.params(1, T, 1, 1, 64)
        for op in (nsa.OP_DECODE_Q8, nsa.OP_PREFILL_Q8):
            assert L.nsa_workspace_size(ctypes.byref(p), op, ctypes.byref(n)) == want


def test_append_refusals():
    assert append(P, k=None) == 1 and append(P, v=None) == 1 and append(P, pos=None) == 1
    assert append(P, N=3) == 1 and "cu_new" in detail()  # one token per sequence: N == B
    assert append(P, N=-1, cu=FAKE) == 1
    assert append(P, N=0, cu=FAKE) == 0                 # nothing to write, nothing launched
    assert append(P, q=FAKE) == 1 and append(P, q_out=FAKE) == 1
    assert append(P, k_out=FAKE) == 1 and append(P, v_out=FAKE) == 1
    for kw in (dict(k=ODD), dict(v=ODD), dict(q=ODD, q_out=FAKE), dict(q=FAKE, q_out=ODD),
               dict(k_out=ODD, v_out=FAKE), dict(k_out=FAKE, v_out=ODD)):
        assert append(P, **kw) == 1 and "aligned" in detail()
    for dim in (0, 8, 24, 65, 80):
        assert append(P, turn=rope(dim=dim)) == 2 and "multiple of 16" in detail()
    assert append(P, turn=rope(style=2)) == 1 and "style" in detail()
    for bad in (rope(table=None), rope(table=264), rope(length=0)):
        assert append(P, turn=bad) == 1 and "table" in detail()


def test_attention_refusals():
    for call in (decode, prefill):
        for kw in (dict(q=None), dict(lens=None), dict(out=None)):
            assert call(P, **kw) == 1
        assert call(P, q=ODD) == 1 and call(P, out=ODD) == 1
        assert call(P, ws=None) == 1 and call(P, ws=ODD) == 1
        op = nsa.OP_DECODE_Q8 if call is decode else nsa.OP_PREFILL_Q8
        assert call(P, nbytes=nsa.workspace_size(P, op) - 1) == 3
        assert call(P, keys=3) == 1 and call(P, keys=-1) == 1
    assert decode(P, keys=2, sel=None) == 1 and "sel_idx" in detail()
    assert prefill(P, keys=2) == 1
    assert prefill(P, N=3, cu=None) == 1 and "cu_q" in detail()
    assert prefill(P, N=-1) == 1
    assert prefill(P, N=2 * 1000 + 1) == 1
    assert prefill(P, N=0) == 0


def test_wrapper_refusals_on_cpu_tensors():
    pages = torch.zeros(4, 2, 64, 64, dtype=torch.uint8).view(torch.float8_e4m3fn)
    sc = torch.ones(4, 2)
    with pytest.raises(ValueError, match="CUDA"):
        nsa.Q8Cache(pages, pages, sc, sc, torch.zeros(2, 16, dtype=torch.int32))


def test_reference_e4m3_is_the_type():
    """Every code decodes to itself; values between two codes go to the nearer,
    halfway ones to the even mantissa (checked against the type's own cast)."""
    codes = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).float().double()
    fine = codes[torch.isfinite(codes)]
    assert torch.equal(q8_ref.e4m3(fine), fine)
    v = torch.unique(fine)
    mid = (v[1:] + v[:-1]) / 2
    x = torch.cat((mid, mid * (1 + 2.0 ** -20), mid * (1 - 2.0 ** -20)))
    x = x[x.abs() <= 448]
    assert torch.equal(q8_ref.e4m3(x), x.float().to(torch.float8_e4m3fn).double())


def test_reference_scale():
    for a, s in ((0.0, 2.0 ** -126), (448.0, 1.0), (448.1, 2.0), (1.75, 2.0 ** -8), (1.0, 2.0 ** -8),
                 (1.76, 2.0 ** -7), (3.0e38, 2.0 ** 120)):
        assert q8_ref.need(a) == s, a


def test_reference_attention_closed_forms():
    """Equal keys give the mean of the values; one key gives its value; the
    reference agrees with torch's masked softmax."""
    g = torch.Generator().manual_seed(0)
    page, d, Hkv, G, n = 16, 64, 2, 3, 37
    pages = lambda: torch.randn(4, Hkv, page, d, generator=g).to(torch.float8_e4m3fn)  # noqa: E731
    k, v = pages(), pages()
    ks, vs = torch.rand(4, Hkv, generator=g) + 0.5, torch.rand(4, Hkv, generator=g) + 0.5
    table = torch.tensor([[2, 0, 3]], dtype=torch.int32)
    q = torch.randn(5, Hkv * G, d, generator=g)
    cu = torch.tensor([0, 5], dtype=torch.int32)
    lens = torch.tensor([n], dtype=torch.int32)
    out, lse, A, B = q8_ref.attend(q, k, v, ks, vs, table, lens, page, cu)
    kk = (k.float().double() * ks.double()[..., None, None])[table[0].long()].transpose(0, 1).reshape(Hkv, -1, d)[:, :n]
    vv = (v.float().double() * vs.double()[..., None, None])[table[0].long()].transpose(0, 1).reshape(Hkv, -1, d)[:, :n]
    z = torch.einsum("nhgd,hkd->nhgk", q.view(5, Hkv, G, d).double(), kk.double()) / math.sqrt(d)
    hide = torch.arange(n)[None] > (n - 5 + torch.arange(5))[:, None]
    z = z.masked_fill(hide[:, None, None], -math.inf)
    want = torch.einsum("nhgk,hkd->nhgd", z.softmax(-1), vv.double()).reshape(5, -1, d)
    torch.testing.assert_close(out, want, rtol=1e-12, atol=1e-12)
    torch.testing.assert_close(lse, z.logsumexp(-1).reshape(5, -1), rtol=1e-12, atol=1e-12)
    # a window of one: the query's own value; zero queries: the mean of the listed block
    one, _, _, _ = q8_ref.attend(q, k, v, ks, vs, table, lens, page, cu, keys="window", window=1)
    torch.testing.assert_close(one[4, 0], vv[0, n - 1].double())
    sel = torch.tensor([[[1, 1], [1, -1]]], dtype=torch.int32)
    mean, _, _, _ = q8_ref.attend(torch.zeros(1, Hkv * G, d), k, v, ks, vs, table, lens, page,
                                  keys="blocks", sel=sel)
    torch.testing.assert_close(mean[0, 0], vv[0, 16:32].double().mean(0))
