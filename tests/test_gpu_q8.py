"""The 8-bit paged cache on the GPU against the 64-bit definitions of
tests/q8_ref.py: append with rotation, single-token attention, chunks, and a
serving loop of them together."""
import math

import pytest
import torch

from tests import q8_ref as ref

pytestmark = pytest.mark.gpu
nsa = pytest.importorskip("dynamic_block_sparse_nsa_b200.nsa")
BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(autouse=True)
def clean_error_word(cuda_ok):
    yield
    nsa.nsa_check()  # no test leaves a device error behind


def gen(seed):
    return torch.Generator().manual_seed(seed)


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def random_cache(p, lens, seed, extra=3, spread=1.0):
    """A cache whose sequences' pages lie scattered in the pool; slots that no
    token lives in hold arbitrary codes, the NaN code among them."""
    g = gen(seed)
    wide = -(-p.T // p.sel_block)
    count = [-(-n // p.sel_block) for n in lens]
    P = sum(count) + extra
    order = torch.randperm(P, generator=g).to(torch.int32)
    table = torch.full((p.B, wide), -1, dtype=torch.int32)  # unused entries are no pages
    at = 0
    for b, c in enumerate(count):
        table[b, :c] = order[at:at + c]
        at += c

    def pool():
        x = torch.randn(P, p.Hkv, p.sel_block, p.d, generator=g)
        s = torch.exp2(torch.randint(-2, 3, (P, p.Hkv), generator=g).float() * spread - 5)
        s *= 1 + torch.rand(P, p.Hkv, generator=g)  # attention takes any positive scale
        codes = (x / s[..., None, None]).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        dead = torch.ones(P, p.sel_block, dtype=torch.bool)
        for b, n in enumerate(lens):
            for j in range(count[b]):
                dead[table[b, j], :max(0, min(p.sel_block, n - j * p.sel_block))] = False
        noise = torch.randint(0, 256, codes.shape, generator=g, dtype=torch.uint8)
        noise[..., ::3] = 0x7f
        codes = torch.where(dead[:, None, :, None], noise, codes)
        return codes.view(torch.float8_e4m3fn).cuda(), s.cuda()

    k, ks = pool()
    v, vs = pool()
    return nsa.Q8Cache(k, v, ks, vs, table.cuda())


def check_attention(got, p, q, cache, lens, cu=None, keys="all", sel=None, scale=None):
    out, lse = got
    want, wlse, A, B = ref.attend(q, cache.k_pages, cache.v_pages, cache.k_scale, cache.v_scale,
                                  cache.page_table, lens, p.sel_block, cu, keys, p.window, sel,
                                  scale)
    t_out, t_lse = ref.bounds(want, wlse, A, B, p.torch_dtype, max(1, int(lens.max())))
    rows = torch.isfinite(want).all(-1).all(-1)
    out, lse = out.double().cpu(), lse.double().cpu()
    err = (out - want).abs()
    assert (err <= t_out)[rows].all(), (float((err / t_out)[rows].max()), float(err[rows].max()))
    empty = torch.isinf(wlse) & rows[:, None]
    assert (lse[empty] == -math.inf).all()
    fine = ~empty & rows[:, None]
    assert ((lse - wlse).abs() <= t_lse)[fine].all(), float(((lse - wlse).abs() / t_lse)[fine].max())


# ---- append -----------------------------------------------------------------

def check_append(p, cache, k, v, pos, cu, rope, style, q=None, steps=1):
    before = [t.clone() for t in (cache.k_pages, cache.v_pages, cache.k_scale, cache.v_scale)]
    want = ref.append(k, v, pos.cpu(), None if cu is None else cu.cpu(), before[:2], before[2:],
                      cache.page_table, p.sel_block, rope, style)
    q_out, k_out, v_out = nsa.nsa_append_q8(p, k, v, pos, cache, cu_new=cu, q=q, rope=rope,
                                            rope_style=style, want_kv=True)
    nsa.nsa_check()
    table = cache.page_table.cpu()
    for (name, codes, scale, x, slack), pages, sc, held in zip(
            want, (cache.k_pages, cache.v_pages), (cache.k_scale, cache.v_scale), (k_out, v_out)):
        got, gs = ref.decode(pages), sc.cpu().double()
        if name == "v" or rope is None:  # nothing is computed before the codes
            assert torch.equal(got.nan_to_num(nan=999.0), codes.nan_to_num(nan=999.0)), name
            assert torch.equal(gs, scale), name
        for b in range(p.B):
            lo, hi = ref.tokens(cu, b)
            for r in range(lo, hi):
                t = int(pos[b]) + r - lo
                pid, slot = int(table[b, t // p.sel_block]), t % p.sel_block
                s = gs[pid][:, None]
                stored = got[pid, :, slot]
                fine = torch.isfinite(x[r])
                assert torch.equal(torch.isnan(stored), ~fine), name
                err = (stored * s - x[r]).abs()[fine]
                half = (ref.step_of(stored.nan_to_num()) / 2 * s)[fine]
                assert (err <= half * (1 + 2.0 ** -20) + slack[r][fine]).all(), name
                # the rows as held, rounded to dtype (exact in both: 4 significant bits)
                assert torch.equal(held[r].cpu().double().nan_to_num(nan=999.0),
                                   (stored * s).nan_to_num(nan=999.0)), name
        if name == "k" and rope is not None:
            # a scale may differ where the rotated maximum lies on a power of two
            same = gs == scale
            assert ((gs == scale) | (gs == 2 * scale) | (2 * gs == scale)).all()
            assert same.double().mean() > 0.99 or same.numel() < 100
    if q is not None and rope is not None:
        for b in range(p.B):
            lo, hi = ref.tokens(cu, b)
            if hi == lo:
                continue
            at = torch.arange(int(pos[b]), int(pos[b]) + hi - lo)
            x = q[lo:hi].cpu().double()
            y = ref.turned(x, rope, at, style)
            lim = 2.0 ** -21 * (x.abs().amax(-1, keepdim=True) * 2)
            lim = lim + y.abs() * (2.0 ** -8 if p.torch_dtype == BF16 else 2.0 ** -24)
            assert ((q_out[lo:hi].cpu().double() - y).abs() <= lim).all()
    return q_out, k_out, v_out


APPENDS = [
    # B, Hq, Hkv, d, page, dtype, rot, style, past, new
    (1, 4, 1, 128, 64, BF16, 128, "half", [0], [1]),
    (1, 4, 2, 128, 64, BF16, 128, "half", [0], [200]),
    (3, 6, 3, 64, 16, F32, 32, "pairs", [5, 0, 47], [40, 1, 17]),
    (2, 5, 5, 128, 32, BF16, 64, "pairs", [31, 64], [2, 65]),
    (4, 8, 1, 128, 128, F32, 128, "half", [100, 0, 127, 1], [0, 300, 2, 1]),
    (2, 2, 2, 64, 64, BF16, 16, "half", [63, 3], [129, 61]),
    (2, 7, 1, 64, 128, BF16, 64, "half", [0, 200], [128, 57]),
    (2, 3, 3, 64, 32, F32, 48, "pairs", [1, 0], [31, 32]),
]


@pytest.mark.parametrize("case", APPENDS, ids=lambda c: f"B{c[0]}_d{c[3]}_page{c[4]}_{c[7]}")
@pytest.mark.parametrize("big", (1.0, 300.0))
def test_append_matches_the_definition(case, big):
    """Chunks into new and part-filled pages, whose scales stay (big = 1) or grow."""
    B, Hq, Hkv, d, page, dt, rot, style, past, new = case
    T = max(a + n for a, n in zip(past, new))
    p = nsa.params(B, T, Hq, Hkv, d, sel_block=page, dtype=dt)
    cache = random_cache(p, [a + n for a, n in zip(past, new)], 1, spread=2.0)
    # a part-filled page's scale is a power of two in a cache that appends wrote
    for sc in (cache.k_scale, cache.v_scale):
        sc.copy_(torch.exp2(torch.floor(torch.log2(sc))))
    g = gen(2)
    N = sum(new)
    k = (torch.randn(N, Hkv, d, generator=g) * big).to(dt).cuda()
    v = (torch.randn(N, Hkv, d, generator=g) * big).to(dt).cuda()
    q = torch.randn(N, Hq, d, generator=g).to(dt).cuda()
    cu = i32([0] + torch.tensor(new).cumsum(0).tolist())
    check_append(p, cache, k, v, i32(past), cu, nsa.rope_table(T, rot), style, q)


@pytest.mark.parametrize("dt", (BF16, F32))
@pytest.mark.parametrize("d,page,style", ((128, 64, "half"), (64, 16, "pairs")))
def test_append_one_token_per_sequence(dt, d, page, style):
    past = [0, 1, page - 1, page, 3 * page + 7]
    T = 5 * page
    p = nsa.params(5, T, 12, 3, d, sel_block=page, dtype=dt)
    cache = random_cache(p, [a + 1 for a in past], 3)
    for sc in (cache.k_scale, cache.v_scale):
        sc.copy_(torch.exp2(torch.floor(torch.log2(sc))))
    g = gen(4)
    make = lambda h: torch.randn(5, h, d, generator=g).to(dt).cuda()  # noqa: E731
    k, v, q = make(3) * 50, make(3) * 0.01, make(12)
    check_append(p, cache, k, v, i32(past), None, nsa.rope_table(T, d), style, q)
    # the same through offsets
    again = random_cache(p, [a + 1 for a in past], 3)
    for sc in (again.k_scale, again.v_scale):
        sc.copy_(torch.exp2(torch.floor(torch.log2(sc))))
    nsa.nsa_append_q8(p, k, v, i32(past), again, cu_new=i32(list(range(6))),
                      rope=nsa.rope_table(T, d), rope_style=style)
    for a, b in ((cache.k_pages, again.k_pages), (cache.v_pages, again.v_pages)):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    assert torch.equal(cache.k_scale, again.k_scale) and torch.equal(cache.v_scale, again.v_scale)


def test_append_without_rotation_zero_and_non_finite():
    """No rotation: codes are exact. A head of zeros takes the smallest scale;
    NaN and infinities become NaN and do not set the scale; the largest and
    smallest magnitudes stay in range."""
    p = nsa.params(1, 64, 2, 2, 64, sel_block=16, dtype=F32)
    cache = random_cache(p, [64], 5)
    k = torch.randn(40, 2, 64, generator=gen(6))
    k[:16, 0] = 0.0
    k[3, 1, 5], k[4, 1, 6], k[5, 1, 7] = math.nan, math.inf, -math.inf
    k[17, 0, 0] = 3.0e38
    k[32:, 0] *= 1e-38
    k[33:, 1] = math.nan
    v = k.flip(0).contiguous()
    check_append(p, cache, k.cuda(), v.cuda(), i32([0]), i32([0, 40]), None, "half")


def test_append_token_by_token_equals_one_call():
    """Values of equal magnitude: a page grown token by token holds what one
    call writes; and calls repeat bit for bit."""
    p = nsa.params(1, 256, 4, 2, 128, sel_block=64)
    sign = torch.randint(0, 2, (150, 2, 128), generator=gen(7)).float() * 2 - 1
    k = (sign * torch.exp2(torch.randint(-3, 1, (150, 2, 128), generator=gen(8)).float())).to(BF16)
    k[..., 0] = 1.0  # every token's largest magnitude
    k = k.cuda()
    table = i32([[2, 0, 3, 1]])
    one, steps = nsa.q8_cache(p, 4, table), nsa.q8_cache(p, 4, table)
    nsa.nsa_append_q8(p, k, k, i32([0]), one, cu_new=i32([0, 150]))
    for t in range(150):
        nsa.nsa_append_q8(p, k[t:t + 1], k[t:t + 1], i32([t]), steps)
    live = [(2, 64), (0, 64), (3, 22)]
    for a, b in ((one.k_pages, steps.k_pages), (one.v_pages, steps.v_pages)):
        for pid, n in live:
            assert torch.equal(a.view(torch.uint8)[pid, :, :n], b.view(torch.uint8)[pid, :, :n])
    assert torch.equal(one.k_scale, steps.k_scale)


@pytest.mark.parametrize("dt", (BF16, F32))
def test_append_long_call_equals_short_ones(dt):
    """A call whose query rows have a launch of their own, against calls that do not."""
    N, cut = 2500, 1280  # (the cut between two pages)
    p = nsa.params(1, N, 64, 1, 128, dtype=dt)
    table = torch.randperm(40, generator=gen(81)).to(torch.int32)[None].cuda()
    rope = nsa.rope_table(N, 128)
    g = gen(82)
    k, v = (torch.randn(N, 1, 128, generator=g).to(dt).cuda() for _ in range(2))
    q = torch.randn(N, 64, 128, generator=g).to(dt).cuda()
    one, two = nsa.q8_cache(p, 40, table), nsa.q8_cache(p, 40, table)
    whole = nsa.nsa_append_q8(p, k, v, i32([0]), one, i32([0, N]), q, rope, want_kv=True)
    for lo, hi in ((0, cut), (cut, N)):
        part = nsa.nsa_append_q8(p, k[lo:hi], v[lo:hi], i32([lo]), two, i32([0, hi - lo]), q[lo:hi],
                                 rope, want_kv=True)
        nsa.nsa_check()
        for x, y in zip(whole, part):
            assert torch.equal(x[lo:hi], y)
    for x, y in ((one.k_pages, two.k_pages), (one.v_pages, two.v_pages)):
        assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))
    assert torch.equal(one.k_scale, two.k_scale) and torch.equal(one.v_scale, two.v_scale)
    turned = ref.turned(q.cpu().double(), rope, torch.arange(N), "half")
    lim = 2.0 ** -20 * q.abs().max().item() + turned.abs() * (2.0 ** -8 if dt == BF16 else 2.0 ** -24)
    assert ((whole[0].cpu().double() - turned).abs() <= lim).all()


def test_append_many_sequences():
    """More sequences than a block's threads, many without new tokens."""
    B = 700
    g = gen(13)
    past = torch.randint(0, 70, (B,), generator=g).tolist()
    new = (torch.randint(0, 40, (B,), generator=g) * (torch.rand(B, generator=g) < 0.3)).tolist()
    p = nsa.params(B, 128, 2, 1, 64, sel_block=32, dtype=BF16)
    cache = random_cache(p, [a + n for a, n in zip(past, new)], 14)
    for sc in (cache.k_scale, cache.v_scale):
        sc.copy_(torch.exp2(torch.floor(torch.log2(sc))))
    N = sum(new)
    k, v = (torch.randn(N, 1, 64, generator=g).to(BF16).cuda() for _ in range(2))
    q = torch.randn(N, 2, 64, generator=g).to(BF16).cuda()
    cu = i32([0] + torch.tensor(new).cumsum(0).tolist())
    check_append(p, cache, k, v, i32(past), cu, nsa.rope_table(128, 64), "half", q)


def test_append_padded_rows_and_other_pages_stay():
    """Rows behind the last sequence are ignored; pages of no new token keep
    their bytes; q_out may be q."""
    p = nsa.params(2, 100, 4, 1, 64, sel_block=32, dtype=BF16)
    cache = random_cache(p, [100, 70], 9)
    before = [t.clone() for t in (cache.k_pages, cache.v_pages, cache.k_scale)]
    k = (torch.randn(20, 1, 64, generator=gen(10)) * 1e-3).to(BF16).cuda()  # no scale grows
    q = torch.randn(20, 4, 64, generator=gen(11)).to(BF16).cuda()
    keep = q.clone()
    cu = i32([0, 9, 12])
    q_out, k_out, _ = nsa.nsa_append_q8(p, k, k, i32([60, 33]), cache, cu_new=cu, q=q, q_out=q,
                                        rope=nsa.rope_table(100, 64), want_kv=True)
    nsa.nsa_check()
    assert q_out is q and torch.equal(q[12:], keep[12:]) and not torch.equal(q[:12], keep[:12])
    touched = {int(cache.page_table[0, 1]), int(cache.page_table[0, 2]), int(cache.page_table[1, 1])}
    for pid in set(range(before[0].shape[0])) - touched:
        assert torch.equal(cache.k_pages.view(torch.uint8)[pid], before[0].view(torch.uint8)[pid])
        assert torch.equal(cache.v_pages.view(torch.uint8)[pid], before[1].view(torch.uint8)[pid])
    later = cache.page_table[1, 1]  # sequence 1 wrote slots 1 .. 3 of it
    if torch.equal(cache.k_scale[later], before[2][later]):
        assert torch.equal(cache.k_pages.view(torch.uint8)[later, :, 4:],
                           before[0].view(torch.uint8)[later, :, 4:])


def test_append_reports_bad_positions_pages_and_offsets():
    p = nsa.params(3, 64, 2, 1, 64, sel_block=16, dtype=F32)
    rope = nsa.rope_table(32, 64)
    k = torch.randn(6, 1, 64, generator=gen(12)).cuda()

    def refused(pos, cu, table=None, turn=None):
        cache = nsa.q8_cache(p, 4, i32([[0, 1, 2, 3]] * 3) if table is None else table)
        nsa.nsa_append_q8(p, k if cu is not None else k[:3], k if cu is not None else k[:3],
                          i32(pos), cache, cu_new=None if cu is None else i32(cu), rope=turn)
        with pytest.raises(nsa.NsaError) as e:
            nsa.nsa_check()
        assert e.value.status == 1
        return cache, str(e.value)

    cache, text = refused([-1, 64, 70], None)
    assert "position" in text and not cache.k_pages.view(torch.uint8).any()
    cache, text = refused([63, -5, 40], [0, 2, 4, 6], turn=rope)  # 40 is past the table of 32
    assert "position" in text and not cache.k_pages.view(torch.uint8).any()
    cache, text = refused([0, 0, 0], [0, 9, 4, 2])
    assert "offsets" in text
    cache, text = refused([0, 0, 0], None, table=i32([[-1, 0, 0, 0], [4, 0, 0, 0], [99, 0, 0, 0]]))
    assert "page" in text and not cache.k_pages.view(torch.uint8).any()


def turned_fp32(x, table, positions, style):
    """x fp32 [N, H, d] rotated in fp32, each product and each sum rounded."""
    t = table[positions]
    c, s, half = t[:, 0, None], t[:, 1, None], t.shape[-1]
    i = torch.arange(half, device=x.device)
    a, b = (i, i + half) if style == "half" else (2 * i, 2 * i + 1)
    y = x.clone()
    xa_c, xb_s, xb_c, xa_s = x[..., a] * c, x[..., b] * s, x[..., b] * c, x[..., a] * s
    y[..., a] = xa_c - xb_s
    y[..., b] = xb_c + xa_s
    return y


@pytest.mark.parametrize("dt", (BF16, F32))
@pytest.mark.parametrize("style,d,rot", (("half", 128, 128), ("pairs", 128, 64), ("half", 64, 32), ("pairs", 64, 64)))
def test_append_rotation_is_that_of_rounded_products(dt, style, d, rot):
    """Queries, key codes and scales bit for bit, of chunks (with the query rows in the
    pages' launch and in one of their own) and of one token a sequence."""
    page, Hq, Hkv = 64, 16, 2
    for B, n in ((1, 128), (2, 2304), (40, 1)):
        T = 4000
        p = nsa.params(B, T, Hq, Hkv, d, sel_block=page, dtype=dt)
        wide = -(-T // page)
        cache = nsa.q8_cache(p, B * wide, torch.arange(B * wide, dtype=torch.int32, device="cuda").view(B, wide))
        g = gen(150 + n)
        k = (torch.randn(B * n, Hkv, d, generator=g) * 37).to(dt).cuda()
        q = torch.randn(B * n, Hq, d, generator=g).to(dt).cuda()
        rope = nsa.rope_table(T, rot)
        past = [page * (b % 20) for b in range(B)]  # each begins a page
        at = torch.tensor([past[b] + i for b in range(B) for i in range(n)]).cuda()
        cu = None if n == 1 else i32([n * b for b in range(B + 1)])
        q_out, _, _ = nsa.nsa_append_q8(p, k, k, i32(past), cache, cu_new=cu, q=q, rope=rope, rope_style=style)
        nsa.nsa_check()
        assert torch.equal(q_out, turned_fp32(q.float(), rope, at, style).to(dt))
        want = turned_fp32(k.float(), rope, at, style).view(B, n, Hkv, d)
        for b in range(B):
            for j in range(0, n, page):
                x = want[b, j:j + page]
                pid = int(cache.page_table[b, (past[b] + j) // page])
                for h in range(Hkv):
                    s = ref.need(float(x[:, h].abs().max()))
                    assert float(cache.k_scale[pid, h]) == s
                    codes = (x[:, h] / s).to(torch.float8_e4m3fn).view(torch.uint8)
                    assert torch.equal(cache.k_pages.view(torch.uint8)[pid, h, :len(x)], codes)


@pytest.mark.parametrize("offsets", (False, True))
def test_append_recodes_zeros_of_any_scale(offsets):
    """Stale slots of a page begun anew: zeros stay zeros under every scale, and
    others become NaN where the new one cannot hold them, up to 2^246 below."""
    p = nsa.params(2, 64, 2, 2, 64, sel_block=32, dtype=F32)
    for old in (2.0 ** -126, 1.0, 8.0, 2.0 ** 100, 2.0 ** 120):
        for new in (0.0, 2.0 ** -100, 1.0, 2.0 ** 127):
            cache = random_cache(p, [0, 0], 160, extra=4)
            cache.page_table.copy_(i32([[0, 1], [2, 3]]))
            codes = torch.randint(0, 256, cache.k_pages.shape, generator=gen(161), dtype=torch.uint8)
            codes[..., ::4] = 0
            codes[..., 1::4] = 0x80
            for t in (cache.k_pages, cache.v_pages):
                t.view(torch.uint8).copy_(codes)
            cache.k_scale.fill_(old)
            cache.v_scale.fill_(old)
            k = torch.full((2, 2, 64), new, device="cuda")
            check_append(p, cache, k, k, i32([0, 32]), i32([0, 1, 2]) if offsets else None, None, "half")


# ---- attention: single tokens ---------------------------------------------------

DECODES = [
    # Hq, Hkv, d, page, dtype, lens
    (16, 1, 128, 64, BF16, [1, 2, 31, 32, 33, 63, 64, 65, 0, 500]),
    (64, 4, 128, 64, BF16, [1000, 3, 700]),
    (8, 8, 128, 128, BF16, [129, 700]),
    (40, 8, 64, 16, F32, [333, 0, 17, 1, 16]),
    (6, 2, 128, 32, F32, [257, 31]),
    (20, 1, 64, 64, BF16, [130, 5]),        # more than 16 heads to a KV head
    (34, 2, 128, 16, F32, [77, 48]),
    (5, 1, 64, 128, F32, [400]),
    (4, 4, 64, 32, BF16, [90, 1, 64]),
]


@pytest.mark.parametrize("case", DECODES, ids=lambda c: f"h{c[0]}_{c[1]}_d{c[2]}_page{c[3]}")
@pytest.mark.parametrize("keys", ("all", "window", "blocks"))
def test_decode_matches_the_definition(case, keys):
    Hq, Hkv, d, page, dt, lens = case
    B, T = len(lens), max(lens) + 5
    g = gen(20)
    for window, n in ((1, 1), (37, 3), (64, 9), (10000, 40)) if keys != "all" else ((1, 1),):
        p = nsa.params(B, T, Hq, Hkv, d, sel_block=page, dtype=dt, window=window, top_n=n)
        cache = random_cache(p, lens, 21)
        q = torch.randn(B, Hq, d, generator=g).to(dt).cuda()
        sel = None
        if keys == "blocks":  # any order, repeated, negative and past the end
            sel = torch.randint(-2, -(-T // page) + 2, (B, Hkv, n), generator=g).to(torch.int32)
        got = nsa.nsa_decode_q8(p, q, cache, i32(lens), keys=keys,
                                sel_idx=None if sel is None else sel.cuda())
        nsa.nsa_check()
        check_attention(got, p, q, cache, i32(lens), None, keys, sel)


def test_decode_many_sequences_and_long_ones():
    """Units that span blocks, warps and both; more tiles than a block plans."""
    for B, Hq, Hkv, lens in ((1, 16, 1, [20000]), (1200, 2, 1, None), (37, 8, 2, None)):
        if lens is None:
            lens = torch.randint(0, 90, (B,), generator=gen(22)).tolist()
        p = nsa.params(B, max(lens), Hq, Hkv, 128, sel_block=64)
        cache = random_cache(p, lens, 23)
        q = torch.randn(B, Hq, 128, generator=gen(24)).to(BF16).cuda()
        got = nsa.nsa_decode_q8(p, q, cache, i32(lens))
        nsa.nsa_check()
        check_attention(got, p, q, cache, i32(lens))


@pytest.mark.parametrize("longest", (300, 1400, 2000))
def test_decode_lengths_far_apart_in_few_chunks(longest):
    """Whole units to a block, as many each or by their chunks: most lengths are
    short, empty ones among them, and the long ones lie together."""
    B = 70
    lens = [(b * 7) % 9 for b in range(B)]
    lens[20:24] = [longest, longest - 63, longest // 2, 64]
    for Hq, Hkv, dt, page in ((12, 3, BF16, 64), (8, 1, F32, 16), (40, 1, BF16, 32)):
        p = nsa.params(B, longest, Hq, Hkv, 64, dtype=dt, sel_block=page, window=longest - 100)
        cache = random_cache(p, lens, 71)
        q = torch.randn(B, Hq, 64, generator=gen(72)).to(dt).cuda()
        n = torch.tensor(lens, dtype=torch.int32)
        for keys in ("all", "window"):
            got = nsa.nsa_decode_q8(p, q, cache, n.cuda(), keys=keys)
            nsa.nsa_check()
            check_attention(got, p, q, cache, n, keys=keys)


def test_decode_far_positions():
    """The window of a long sequence: pages before it are never looked up."""
    L = 300001
    p = nsa.params(1, L + 63, 16, 2, 64, sel_block=64, dtype=F32, window=150)
    small = random_cache(nsa.params(1, 256, 16, 2, 64, sel_block=64, dtype=F32), [256], 33, extra=0)
    table = torch.full((1, -(-p.T // 64)), -1, dtype=torch.int32)
    first = (L - 150) // 64
    table[0, first:first + 4] = small.page_table[0].cpu()
    cache = nsa.Q8Cache(small.k_pages, small.v_pages, small.k_scale, small.v_scale, table.cuda())
    q = torch.randn(1, 16, 64, generator=gen(34)).cuda()
    got = nsa.nsa_decode_q8(p, q, cache, i32([L]), keys="window")
    nsa.nsa_check()
    check_attention(got, p, q, cache, i32([L]), keys="window")


@pytest.mark.parametrize("dt,d,page", ((BF16, 128, 64), (F32, 64, 16), (BF16, 64, 128)), ids=str)
def test_longest_sequence(dt, d, page):
    """2^30 tokens, on few pages that repeat: listed blocks, the last among them, beside
    absent ones and one whose number is no page; and a window at the end."""
    T, n = 1 << 30, (1 << 30) // page
    small = random_cache(nsa.params(1, 4 * page, 4, 1, d, sel_block=page, dtype=dt), [4 * page], 110)
    order = small.page_table[0].cpu()
    table = order.repeat(n // 4)[None].contiguous()
    table[0, 7] = -5
    far = nsa.Q8Cache(small.k_pages, small.v_pages, small.k_scale, small.v_scale, table.cuda())
    q = torch.randn(1, 4, d, generator=gen(111)).to(dt).cuda()

    def near(blocks):
        t = table[:, blocks].to(torch.int32).contiguous().cuda()
        return nsa.Q8Cache(small.k_pages, small.v_pages, small.k_scale, small.v_scale, t)

    for sel in ([n - 1, -1, -1, -1, -1, -1], [-1, 5, n - 1, n, -7, n - 3], [-1, 2, -1, -1, 7, -1]):
        p = nsa.params(1, T, 4, 1, d, sel_block=page, dtype=dt, top_n=6)
        got = nsa.nsa_decode_q8(p, q, far, i32([T]), keys="blocks", sel_idx=i32([[sel]]))
        if 7 in sel:
            with pytest.raises(nsa.NsaError, match="page"):
                nsa.nsa_check()
        nsa.nsa_check()
        live = [b for b in sel if 0 <= b < n and b != 7]
        p = nsa.params(1, len(live) * page, 4, 1, d, sel_block=page, dtype=dt)
        check_attention(got, p, q, near(live), i32([len(live) * page]))
    p = nsa.params(1, T, 1, 1, d, sel_block=page, dtype=dt, window=2 * page + 3)
    q = torch.randn(40, 1, d, generator=gen(112)).to(dt).cuda()
    got = nsa.nsa_prefill_q8(p, q, far, i32([T]), i32([0, 40]), keys="window")
    nsa.nsa_check()
    blocks = list(range(n - 2 - -(-48 // page), n))
    pn = nsa.params(1, len(blocks) * page, 1, 1, d, sel_block=page, dtype=dt, window=2 * page + 3)
    assert len(blocks) * page >= 2 * page + 3 + 40
    check_attention(got, pn, q, near(blocks), i32([len(blocks) * page]), i32([0, 40]).cpu(), "window")
    last = q[-1:].contiguous()
    got = nsa.nsa_decode_q8(p, last, far, i32([T]), keys="window")
    nsa.nsa_check()
    check_attention(got, pn, last, near(blocks), i32([len(blocks) * page]), None, "window")


def test_pool_beyond_32_bit_offsets():
    """Pages whose bytes lie past 2^31 of the pool: appended and attended to."""
    Hkv, page, d = 4, 64, 128
    P = (1 << 31) // (Hkv * page * d) + 40
    for new, dt in ((130, BF16), (1, F32)):
        p = nsa.params(1, 192, 16, Hkv, d, sel_block=page, dtype=dt)
        table = i32([[P - 1, P - 9, P - 4]])
        pools = [torch.empty(P, Hkv, page, d, dtype=torch.uint8, device="cuda") for _ in range(2)]
        pools = [x.view(torch.float8_e4m3fn) for x in pools]
        sc = [torch.ones(P, Hkv, device="cuda") for _ in range(2)]
        cache = nsa.Q8Cache(*pools, *sc, table)
        k = torch.randn(new, Hkv, d, generator=gen(35)).to(dt).cuda()
        q = torch.randn(new, 16, d, generator=gen(36)).to(dt).cuda()
        cu = i32([0, new])
        nsa.nsa_append_q8(p, k, k, i32([0]), cache, cu_new=cu if new > 1 else None)
        lens = i32([new])
        near = nsa.Q8Cache(*[x.view(torch.uint8)[P - 16:].clone().view(torch.float8_e4m3fn) for x in pools],
                           *[x[P - 16:].clone() for x in sc], table - (P - 16))
        check_attention(nsa.nsa_prefill_q8(p, q, cache, lens, cu), p, q, near, lens, cu.cpu())
        last = q[-1:].contiguous()
        check_attention(nsa.nsa_decode_q8(p, last, cache, lens), p, last, near, lens)
        nsa.nsa_check()
        del cache, near, pools
        torch.cuda.empty_cache()


def test_decode_scales_far_apart():
    """Pages whose value scales differ by up to 2^200, with the large ones hardly
    attended: their products leave fp16's and fp32's ranges on the way."""
    p = nsa.params(1, 256, 4, 1, 64, sel_block=64, dtype=F32)
    for big, order in ((2.0 ** 90, [0, 1, 2, 3]), (2.0 ** 90, [3, 2, 1, 0]), (2.0 ** 20, [1, 3, 0, 2])):
        cache = random_cache(p, [256], 25, extra=0)
        k = torch.full((4, 1, 64, 64), 1.0)
        k[1] = -1.0                                   # page 1: scores far below the others'
        cache.k_pages.copy_(k.to(torch.float8_e4m3fn))
        cache.k_scale.fill_(1.0)
        cache.v_scale.copy_(torch.tensor([[1.0], [big], [2.0 ** -100], [2.0 ** -126]]))
        cache.page_table.copy_(i32([order]))
        q = torch.full((1, 4, 64), 6.0).cuda()        # e^(-96): 2^-138 of the others
        got = nsa.nsa_decode_q8(p, q, cache, i32([256]))
        nsa.nsa_check()
        check_attention(got, p, q, cache, i32([256]))


@pytest.mark.parametrize("dt", (BF16, F32))
def test_negative_softmax_scale(dt):
    p = nsa.params(1, 200, 16, 1, 128, sel_block=64, dtype=dt, softmax_scale=-0.125)
    cache = random_cache(p, [200], 37)
    q = torch.randn(20, 16, 128, generator=gen(38)).to(dt).cuda()
    lens, cu = i32([200]), i32([0, 20])
    check_attention(nsa.nsa_prefill_q8(p, q, cache, lens, cu), p, q, cache, lens, cu.cpu(),
                    scale=-0.125)
    last = q[-1:].contiguous()
    check_attention(nsa.nsa_decode_q8(p, last, cache, lens), p, last, cache, lens, scale=-0.125)
    nsa.nsa_check()


def test_decode_softmax_scale_and_extreme_scores():
    p = nsa.params(2, 100, 8, 2, 64, sel_block=32, dtype=F32, softmax_scale=0.5)
    cache = random_cache(p, [100, 50], 26)
    q = torch.randn(2, 8, 64, generator=gen(27))
    q[0] *= 1e-3
    q[1] *= 4.0
    got = nsa.nsa_decode_q8(p, q.cuda(), cache, i32([100, 50]))
    check_attention(got, p, q, cache, i32([100, 50]), scale=0.5)
    q[0], q[1] = 1e30, 0.0  # finite scores beyond any exponent: the largest key wins
    cache.k_scale.fill_(1.0)
    out, lse = nsa.nsa_decode_q8(p, q.cuda(), cache, i32([100, 50]))
    nsa.nsa_check()
    assert torch.isfinite(out).all() and torch.isfinite(lse).all()


def test_decode_non_finite_components():
    """A NaN key or value reaches the queries that attend to it and no others."""
    p = nsa.params(2, 128, 4, 2, 64, sel_block=32, dtype=BF16, window=40, top_n=1)
    cache = random_cache(p, [128, 128], 28)
    q = torch.randn(2, 4, 64, generator=gen(29)).to(BF16).cuda()
    base = nsa.nsa_decode_q8(p, q, cache, i32([128, 128]), keys="window")[0]
    pid = int(cache.page_table[0, 2])  # positions 64 .. 95: 88 on are in the window
    cache.k_pages.view(torch.uint8)[pid, 0, 10] = 0x7f
    cache.v_pages.view(torch.uint8)[pid, 1, 23, 7] = 0xff
    out = nsa.nsa_decode_q8(p, q, cache, i32([128, 128]), keys="window")[0]
    assert torch.equal(out, base)
    cache.v_pages.view(torch.uint8)[pid, 1, 24, 7] = 0xff
    out = nsa.nsa_decode_q8(p, q, cache, i32([128, 128]), keys="window")[0]
    bad = torch.isnan(out)
    assert bad[0, 2:, 7].all() and int(bad.sum()) == 2
    cache.k_pages.view(torch.uint8)[pid, 0, 30] = 0x7f
    out, lse = nsa.nsa_decode_q8(p, q, cache, i32([128, 128]), keys="window")
    assert torch.isnan(out[0, :2]).all() and torch.isnan(lse[0, :2]).all()
    assert torch.isfinite(out[1]).all()
    qn = q.clone()
    qn[1, 0, 0] = math.nan
    qn[1, 1, 0] = math.inf
    out = nsa.nsa_decode_q8(p, qn, cache, i32([128, 128]))[0]
    assert torch.isnan(out[1, 0]).all() and torch.isfinite(out[1, 2:]).all()


def test_attention_reports_bad_lengths_pages_and_offsets():
    p = nsa.params(3, 128, 4, 1, 64, sel_block=32, dtype=BF16)
    cache = random_cache(p, [128, 100, 64], 30)
    q = torch.randn(3, 4, 64, generator=gen(31)).to(BF16).cuda()
    out, lse = nsa.nsa_decode_q8(p, q, cache, i32([128, 129, -1]))
    with pytest.raises(nsa.NsaError, match="length"):
        nsa.nsa_check()
    assert not out[1:].any() and (lse[1:] == -math.inf).all() and torch.isfinite(out[0]).all()
    check_attention((out[:1], lse[:1]), nsa.params(1, 128, 4, 1, 64, sel_block=32), q[:1],
                    nsa.Q8Cache(cache.k_pages, cache.v_pages, cache.k_scale, cache.v_scale,
                                cache.page_table[:1].contiguous()), i32([128]))
    # pages outside the pool are left out
    cache.page_table[0, 1] = 9999
    cache.page_table[1, 0] = -3
    got = nsa.nsa_decode_q8(p, q, cache, i32([128, 100, 64]))
    with pytest.raises(nsa.NsaError, match="page"):
        nsa.nsa_check()
    check_attention(got, p, q, cache, i32([128, 100, 64]))
    # offsets past the rows: that sequence is not written; more queries than tokens: zeros
    cache = random_cache(p, [128, 100, 64], 30)
    q = torch.randn(12, 4, 64, generator=gen(32)).to(BF16).cuda()
    out = torch.full_like(q, 7.0)
    cu = i32([0, 4, 6, 40])
    _, lse = nsa.nsa_prefill_q8(p, q, cache, i32([128, 1, 64]), cu, out=out)
    with pytest.raises(nsa.NsaError, match="length"):
        nsa.nsa_check()
    assert not out[4:6].any() and (lse[4:6] == -math.inf).all() and (out[6:] == 7.0).all()
    assert torch.isfinite(out[:4]).all() and not (out[:4] == 7.0).all(-1).any()
    nsa.nsa_prefill_q8(p, q, cache, i32([128, 100, 64]), cu)
    with pytest.raises(nsa.NsaError, match="offsets"):
        nsa.nsa_check()


# ---- attention: chunks ------------------------------------------------------------

PREFILLS = [
    # Hq, Hkv, d, page, dtype, lens, new
    (16, 1, 128, 64, BF16, [70], [70]),
    (64, 4, 128, 64, BF16, [300, 129], [130, 5]),
    (8, 2, 128, 128, BF16, [257, 1, 40], [100, 1, 0]),
    (10, 2, 64, 16, F32, [60, 33], [33, 33]),
    (6, 6, 128, 32, F32, [64, 90], [20, 3]),
    (20, 1, 64, 64, BF16, [77], [9]),
    (32, 8, 128, 16, BF16, [150, 17], [80, 17]),
    (7, 1, 128, 32, BF16, [200], [61]),
    (4, 1, 64, 128, F32, [131], [131]),
]


@pytest.mark.parametrize("case", PREFILLS, ids=lambda c: f"h{c[0]}_{c[1]}_d{c[2]}_page{c[3]}")
@pytest.mark.parametrize("keys", ("all", "window"))
def test_prefill_matches_the_definition(case, keys):
    Hq, Hkv, d, page, dt, lens, new = case
    N = sum(new) + 3  # rows behind the last sequence
    for window in (1, 20, 64) if keys == "window" else (1,):
        p = nsa.params(len(lens), max(lens) + 20, Hq, Hkv, d, sel_block=page, dtype=dt,
                       window=window)
        cache = random_cache(p, lens, 40)
        q = torch.randn(N, Hq, d, generator=gen(41)).to(dt).cuda()
        cu = i32([0] + torch.tensor(new).cumsum(0).tolist())
        out = torch.full_like(q, 5.0)
        lse = torch.full((N, Hq), 5.0, device="cuda")
        nsa.nsa_prefill_q8(p, q, cache, i32(lens), cu, keys=keys, out=out, lse=lse)
        nsa.nsa_check()
        assert (out[-3:] == 5.0).all() and (lse[-3:] == 5.0).all()
        check_attention((out, lse), p, q, cache, i32(lens), cu.cpu(), keys)


@pytest.mark.parametrize("past,new,keys", (
    ([100, 0, 7, 1900], [650] * 4, "all"),
    ([100, 0, 7, 1900], [650] * 4, "window"),
    ([577], [2600], "all"),
    ([0] * 4, [1040, 260, 520, 780], "all"),
    ([1500 + 90 * b for b in range(24)], [1 + b % 7 for b in range(24)], "all"),
), ids=str)
def test_prefill_repeats_its_bits(past, new, keys):
    """Many calls that fill the machine, each with the first one's bits. (A slot that
    was copied into while its codes were still being read showed in one call of 50.)"""
    B, N = len(new), sum(new)
    lens = [a + n for a, n in zip(past, new)]
    p = nsa.params(B, max(lens), 64, 4, 128, sel_block=64, window=200)
    cache = random_cache(p, lens, 46, extra=0, spread=0.0)
    q = torch.randn(N, 64, 128, generator=gen(47)).to(BF16).cuda()
    cu = i32([0] + torch.tensor(new).cumsum(0).tolist())
    L, ws = i32(lens), nsa.workspace(p, nsa.OP_PREFILL_Q8)
    first = nsa.nsa_prefill_q8(p, q, cache, L, cu, keys=keys, ws=ws)
    differ = 0
    for _ in range(150):
        got = nsa.nsa_prefill_q8(p, q, cache, L, cu, keys=keys, ws=ws)
        differ += not (torch.equal(got[0], first[0]) and torch.equal(got[1], first[1]))
    nsa.nsa_check()
    assert differ == 0


@pytest.mark.parametrize("Hq,Hkv,lens,new", (
    (16, 1, [9000], [4]),                      # one unit over every block
    (16, 2, [70] * 200, [2] * 200),            # many units of one chunk
    (8, 1, [60, 1] * 600, [9, 1] * 600),       # more sequences than the plan's threads
    (300, 1, [140, 40], [3, 5]),               # a token's heads fill a tile
    (3, 1, [700, 259, 5], [700, 131, 5]),      # tokens that straddle tiles
))
def test_prefill_many_and_long(Hq, Hkv, lens, new):
    p = nsa.params(len(lens), max(lens) + 3, Hq, Hkv, 128, sel_block=64)
    cache = random_cache(p, lens, 47)
    N = sum(new)
    q = torch.randn(N, Hq, 128, generator=gen(48)).to(BF16).cuda()
    cu = i32([0] + torch.tensor(new).cumsum(0).tolist())
    got = nsa.nsa_prefill_q8(p, q, cache, i32(lens), cu)
    nsa.nsa_check()
    check_attention(got, p, q, cache, i32(lens), cu.cpu())
    again = nsa.nsa_prefill_q8(p, q, cache, i32(lens), cu)
    assert torch.equal(got[0], again[0]) and torch.equal(got[1], again[1])


def test_prefill_scales_far_apart():
    """Value scales that differ by 2^150 between a tile's pages (tensor memory)."""
    p = nsa.params(1, 256, 16, 1, 128, sel_block=32)
    for order in (list(range(8)), list(range(7, -1, -1))):
        cache = random_cache(p, [256], 49, extra=0)
        s = torch.exp2(torch.tensor([0.0, 20.0, -100.0, 3.0, 50.0, -126.0, -50.0, 1.0]))[:, None]
        cache.v_scale.copy_(s)
        cache.page_table.copy_(i32([order]))
        q = torch.randn(40, 16, 128, generator=gen(50)).to(BF16).cuda()
        cu = i32([0, 40])
        got = nsa.nsa_prefill_q8(p, q, cache, i32([256]), cu)
        nsa.nsa_check()
        check_attention(got, p, q, cache, i32([256]), cu.cpu())


def test_prefill_rows_equal_single_tokens():
    """A chunk's rows agree with the same queries one at a time (fp32)."""
    p = nsa.params(1, 90, 6, 2, 128, sel_block=32, dtype=F32)
    cache = random_cache(p, [90], 42)
    q = torch.randn(12, 6, 128, generator=gen(43)).cuda()
    out, lse = nsa.nsa_prefill_q8(p, q, cache, i32([90]), i32([0, 12]))
    for i in range(12):
        o, s = nsa.nsa_decode_q8(p, q[i:i + 1], cache, i32([79 + i]))
        torch.testing.assert_close(o[0], out[i], rtol=2e-5, atol=2e-5)
        torch.testing.assert_close(s[0], lse[i], rtol=2e-5, atol=2e-5)


@pytest.mark.parametrize("dt,d,page", ((BF16, 128, 64), (BF16, 128, 32), (F32, 64, 16), (BF16, 64, 128)))
def test_pages_before_the_window_are_not_looked_up(dt, d, page):
    lens = torch.tensor([1000, 333, 5], dtype=torch.int32)
    new = [40, 33, 5]
    cu = torch.tensor([0, 40, 73, 78], dtype=torch.int32)
    p = nsa.params(3, 1024, 8, 2, d, dtype=dt, sel_block=page, window=150)
    cache = random_cache(p, lens.tolist(), 61)
    table = cache.page_table.cpu()
    g = gen(62)
    for count in (1, 2):  # single tokens, then chunks of queries
        gone = table.clone()
        for b in range(3):
            first = int(lens[b]) - (1 if count == 1 else new[b])  # the first query's position
            gone[b, :max(0, first + 1 - 150) // page] = (-1, 1 << 30)[b % 2]
        less = nsa.Q8Cache(cache.k_pages, cache.v_pages, cache.k_scale, cache.v_scale, gone.cuda())
        q = torch.randn(3 if count == 1 else 78, 8, d, generator=g).to(dt).cuda()
        if count == 1:
            got = nsa.nsa_decode_q8(p, q, less, lens.cuda(), keys="window")
        else:
            got = nsa.nsa_prefill_q8(p, q, less, lens.cuda(), cu.cuda(), keys="window")
        nsa.nsa_check()
        check_attention(got, p, q, cache, lens, None if count == 1 else cu, "window")


@pytest.mark.parametrize("dt,d,Hq", ((BF16, 128, 16), (F32, 64, 4), (BF16, 128, 2)))
def test_prefill_nan_values_reach_later_queries_only(dt, d, Hq):
    p = nsa.params(1, 200, Hq, 1, d, sel_block=64, dtype=dt, window=30)
    for keys in ("all", "window"):
        cache = random_cache(p, [200], 44)
        q = torch.randn(100, Hq, d, generator=gen(45)).to(dt).cuda()
        base = nsa.nsa_prefill_q8(p, q, cache, i32([200]), i32([0, 100]), keys=keys)[0]
        for pos, dim in ((150, 3), (161, 3), (128, d - 1)):
            pid = int(cache.page_table[0, pos // 64])
            cache.v_pages.view(torch.uint8)[pid, 0, pos % 64, dim] = 0x7f
        pid = int(cache.page_table[0, 190 // 64])
        cache.k_pages.view(torch.uint8)[pid, 0, 190 % 64, 0] = 0x7f
        out = nsa.nsa_prefill_q8(p, q, cache, i32([200]), i32([0, 100]), keys=keys)[0]
        nsa.nsa_check()
        t = 100 + torch.arange(100)
        last = 200 if keys == "all" else 30
        sees = lambda x: (t >= x) & (t < x + last)  # noqa: E731
        want = torch.zeros(100, Hq, d, dtype=torch.bool)
        want[sees(150) | sees(161), :, 3] = True
        want[sees(128), :, d - 1] = True
        want[sees(190)] = True
        assert torch.equal(torch.isnan(out).cpu(), want)
        clean = ~want.cuda()
        assert torch.equal(out[clean], base[clean])


def test_prefill_nan_values_in_many_short_sequences():
    """Marks of NaN values in units of one and two tile halves that follow one another."""
    B, Hq, d = 120, 16, 128
    new = [(5, 31, 40, 7)[b % 4] for b in range(B)]
    lens = [50 + 3 * b for b in range(B)]
    cu = [sum(new[:b]) for b in range(B + 1)]
    p = nsa.params(B, 512, Hq, 2, d, sel_block=64)
    cache = random_cache(p, lens, 63)
    q = torch.randn(cu[-1], Hq, d, generator=gen(64)).bfloat16().cuda()
    base = nsa.nsa_prefill_q8(p, q, cache, i32(lens), i32(cu))[0]
    want = torch.zeros(cu[-1], Hq, d, dtype=torch.bool)
    table, codes = cache.page_table.cpu(), cache.v_pages.view(torch.uint8)
    for b in range(B):
        for h in range(2):
            pos, dim = lens[b] - 1 - (b + h) % new[b], (7 * b + h) % d
            codes[int(table[b, pos // 64]), h, pos % 64, dim] = 0x7f
            first = cu[b] + pos - (lens[b] - new[b])
            want[first:cu[b + 1], 8 * h:8 * h + 8, dim] = True
    for _ in range(3):
        out = nsa.nsa_prefill_q8(p, q, cache, i32(lens), i32(cu))[0]
        nsa.nsa_check()
        assert torch.equal(torch.isnan(out).cpu(), want)
        assert torch.equal(out[~want.cuda()], base[~want.cuda()])


def nan_marks(p, cache, lens, new, at, dims):
    """NaN value codes at positions at[b] of each sequence, component dims[b], in both
    their tables' pages; the elements [N, Hq, d] of a chunk call that they reach."""
    G, table = p.Hq // p.Hkv, cache.page_table.cpu()
    codes = cache.v_pages.view(torch.uint8)
    want = torch.zeros(sum(new), p.Hq, p.d, dtype=torch.bool)
    first = 0
    for b, n in enumerate(new):
        h = b % p.Hkv
        codes[int(table[b, at[b] // p.sel_block]), h, at[b] % p.sel_block, dims[b]] = 0x7f
        sees = max(0, at[b] - (lens[b] - n))  # the first query that sees it
        want[first + sees:first + n, h * G:(h + 1) * G, dims[b]] = True
        first += n
    return want


@pytest.mark.parametrize("page", (32, 64, 128))
def test_prefill_nan_values_of_drafts(page):
    """Marks of NaN values where both tile halves share a unit's keys: few queries a
    sequence, warps without rows, several chunks, units cut between blocks."""
    B = 40
    new = [(2, 6, 1, 5, 4, 6)[b % 6] for b in range(B)]
    lens = [300 + 41 * b for b in range(B)]
    cu = [sum(new[:b]) for b in range(B + 1)]
    p = nsa.params(B, 2048, 16, 1, 128, sel_block=page)
    assert 32 * B <= cu[-1] * 16 <= 128 * B
    cache = random_cache(p, lens, 130)
    q = torch.randn(cu[-1], 16, 128, generator=gen(131)).to(BF16).cuda()
    base = nsa.nsa_prefill_q8(p, q, cache, i32(lens), i32(cu))
    nsa.nsa_check()
    check_attention(base, p, q, cache, i32(lens), i32(cu).cpu())
    # among the new tokens, in the chunk before them, and far before them
    for at in ([lens[b] - 1 - b % new[b] for b in range(B)],
               [lens[b] - new[b] - 1 - b % 100 for b in range(B)], [7 * b for b in range(B)]):
        want = nan_marks(p, cache, lens, new, at, [(11 * b) % 128 for b in range(B)])
        for _ in range(3):
            out, lse = nsa.nsa_prefill_q8(p, q, cache, i32(lens), i32(cu))
            nsa.nsa_check()
            assert torch.equal(torch.isnan(out).cpu(), want)
            assert torch.equal(out[~want.cuda()], base[0][~want.cuda()]) and torch.equal(lse, base[1])
        cache = random_cache(p, lens, 130)


@pytest.mark.parametrize("keys", ("all", "window"))
def test_prefill_shared_units_among_others(keys):
    """Units that the tile halves share between units of two halves of several chunks
    and units of one chunk, in one call; with NaN values in every sequence's last chunk."""
    new = [2, 20, 3, 1, 12, 2, 2, 9, 1, 1, 4, 2, 1, 3, 2, 1, 2, 1, 1, 2]
    lens = [1500, 1400, 100, 9, 777, 2900, 50, 640, 1, 130, 2048, 300, 260, 3, 1023, 64, 513, 128, 2, 2000]
    B, N = len(new), sum(new)
    cu = [sum(new[:b]) for b in range(B + 1)]
    p = nsa.params(B, 3000, 32, 2, 128, sel_block=64, window=600)
    assert 32 * B <= N * 16 <= 128 * B and max(new) * 16 > 256
    cache = random_cache(p, lens, 132)
    q = torch.randn(N, 32, 128, generator=gen(133)).to(BF16).cuda()
    base = nsa.nsa_prefill_q8(p, q, cache, i32(lens), i32(cu), keys=keys)
    nsa.nsa_check()
    check_attention(base, p, q, cache, i32(lens), i32(cu).cpu(), keys)
    want = nan_marks(p, cache, lens, new, [n - 1 - b % m for b, (n, m) in enumerate(zip(lens, new))],
                     [(5 * b) % 128 for b in range(B)])
    for _ in range(3):
        out, lse = nsa.nsa_prefill_q8(p, q, cache, i32(lens), i32(cu), keys=keys)
        nsa.nsa_check()
        assert torch.equal(torch.isnan(out).cpu(), want)
        assert torch.equal(out[~want.cuda()], base[0][~want.cuda()]) and torch.equal(lse, base[1])


@pytest.mark.parametrize("dt", (BF16, F32))
@pytest.mark.parametrize("B,Hq,Hkv,page,longest", ((3, 40, 2, 64, 700), (1200, 2, 1, 32, 90), (9, 8, 8, 16, 300)))
def test_prefill_without_offsets_equals_decode(dt, B, Hq, Hkv, page, longest):
    lens = torch.randint(0, longest + 1, (B,), generator=gen(134)).tolist()
    for d in (64, 128):
        p = nsa.params(B, longest, Hq, Hkv, d, sel_block=page, dtype=dt, window=70)
        cache = random_cache(p, lens, 135)
        q = torch.randn(B, Hq, d, generator=gen(136)).to(dt).cuda()
        for keys in ("all", "window"):
            one = nsa.nsa_decode_q8(p, q, cache, i32(lens), keys=keys)
            two = nsa.nsa_prefill_q8(p, q, cache, i32(lens), keys=keys)
            nsa.nsa_check()
            assert torch.equal(one[0], two[0]) and torch.equal(one[1], two[1])
        check_attention(one, p, q, cache, i32(lens), keys="window")


@pytest.mark.parametrize("dt,Hq,Hkv,page,N", (
    (BF16, 64, 4, 64, 2600),   # query rows in a launch of their own; tensor memory
    (BF16, 16, 1, 32, 24),     # few queries a sequence
    (BF16, 8, 2, 16, 150),     # not the tensor memory's
    (F32, 6, 3, 64, 90),
), ids=str)
def test_captured_chunks_serve_other_lengths(dt, Hq, Hkv, page, N):
    """One graph of an append and two attention calls over chunks, replayed with other
    offsets, lengths and positions in the same tensors: the bits of eager calls."""
    B, T, d = 4, 3200, 128
    p = nsa.params(B, T, Hq, Hkv, d, sel_block=page, dtype=dt, window=200)
    rope = nsa.rope_table(T, d)
    table = torch.randperm(B * T // page, generator=gen(140)).view(B, -1).to(torch.int32).cuda()
    g = gen(141)

    def filled():
        c = nsa.q8_cache(p, B * T // page, table)
        for t, seed in ((c.k_pages, 142), (c.v_pages, 143)):
            x = torch.randn(t.shape, generator=torch.Generator("cuda").manual_seed(seed), device="cuda")
            t.copy_((x * 64).to(torch.float8_e4m3fn))
        c.k_scale.fill_(2.0 ** -6)
        c.v_scale.fill_(2.0 ** -6)
        return c

    q, k, v = (torch.randn(N, h, d, generator=g).to(dt).cuda() for h in (Hq, Hkv, Hkv))
    pos, lens = torch.zeros(B, dtype=torch.int32, device="cuda"), torch.zeros(B, dtype=torch.int32, device="cuda")
    cu = torch.zeros(B + 1, dtype=torch.int32, device="cuda")
    q_rot = torch.empty_like(q)
    outs = [(torch.empty_like(q), torch.empty(N, Hq, device="cuda")) for _ in range(2)]
    ws = nsa.workspace(p, nsa.OP_PREFILL_Q8)

    def step(c, qr, o):
        nsa.nsa_append_q8(p, k, v, pos, c, cu_new=cu, q=q, rope=rope, q_out=qr)
        for keys, (out, lse) in zip(("all", "window"), o):
            nsa.nsa_prefill_q8(p, qr, c, lens, cu, keys=keys, out=out, lse=lse, ws=ws)

    def shape(shares, past):
        new = [int(N * s) for s in shares]
        cu.copy_(i32([sum(new[:b]) for b in range(B + 1)]))
        pos.copy_(i32(past))
        lens.copy_(i32([a + n for a, n in zip(past, new)]))

    cache = filled()
    shape((0.25, 0.25, 0.25, 0.25), [100, 0, 7, 1900])
    step(cache, q_rot, outs)  # (loads the kernels)
    nsa.nsa_check()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step(cache, q_rot, outs)
    for shares, past in (((0.25, 0.25, 0.25, 0.25), [100, 0, 7, 1900]), ((0.9, 0.05, 0.0, 0.0), [400, 3000, 5, 0]),
                         ((0.0, 0.0, 1.0, 0.0), [9, 9, 577, 9]), ((0.4, 0.1, 0.2, 0.3), [0, 0, 0, 0])):
        shape(shares, past)
        fresh, other = filled(), torch.full_like(q, 3.0)
        want = [(torch.full_like(q, 3.0), torch.full((N, Hq), 3.0, device="cuda")) for _ in range(2)]
        step(fresh, other, want)
        kept = filled()
        for a, b in ((cache.k_pages, kept.k_pages), (cache.v_pages, kept.v_pages),
                     (cache.k_scale, kept.k_scale), (cache.v_scale, kept.v_scale)):
            a.copy_(b)
        q_rot.fill_(3.0)
        for out, lse in outs:
            out.fill_(3.0)
            lse.fill_(3.0)
        graph.replay()
        nsa.nsa_check()
        for a, b in ((cache.k_pages, fresh.k_pages), (cache.v_pages, fresh.v_pages)):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
        assert torch.equal(cache.k_scale, fresh.k_scale) and torch.equal(cache.v_scale, fresh.v_scale)
        assert torch.equal(q_rot, other)
        for a, b in zip(outs, want):
            assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("dt,d,page,G", ((BF16, 128, 64, 16), (BF16, 64, 16, 4), (F32, 64, 32, 4), (F32, 128, 128, 3)), ids=str)
def test_queries_with_infinite_components(dt, d, page, G):
    """Every score of such a query is infinite or NaN, and so its softmax NaN, whatever
    the scores' signs; its neighbours keep theirs, and without keys it has 0 and -inf."""
    p = nsa.params(3, 200, G, 1, d, sel_block=page, dtype=dt, window=150)
    cache = random_cache(p, [200, 150, 0], 170)
    codes = cache.k_pages.view(torch.uint8)
    codes[..., 5] = 0x38 | 0x80  # component 5 of every key is negative
    codes[..., 6] = 0x38         # component 6 positive
    for bad in ({5: math.inf}, {6: -math.inf}, {5: -math.inf}, {5: math.inf, 6: -math.inf}, {7: math.nan}):
        n = 40
        q = torch.randn(2 * n, G, d, generator=gen(171)).to(dt)
        clean = q.clone().cuda()
        for r, h in ((0, 0), (17, G - 1), (n + 3, 1)):
            for e, x in bad.items():
                q[r, h, e] = x
        q, lens, cu = q.cuda(), i32([200, 150, 0]), i32([0, n, 2 * n, 2 * n])
        hit = torch.zeros(2 * n, G, dtype=torch.bool)
        hit[0, 0] = hit[17, G - 1] = hit[n + 3, 1] = True
        for keys in ("all", "window"):
            want = nsa.nsa_prefill_q8(p, clean, cache, lens, cu, keys=keys)
            out, lse = nsa.nsa_prefill_q8(p, q, cache, lens, cu, keys=keys)
            nsa.nsa_check()
            assert torch.equal(torch.isnan(out).all(-1).cpu(), hit) and torch.equal(torch.isnan(lse).cpu(), hit)
            assert torch.equal(out[~hit.cuda()], want[0][~hit.cuda()])
            assert torch.equal(lse[~hit.cuda()], want[1][~hit.cuda()])
            one = q[[0, n + 3, 0]].contiguous()
            out, lse = nsa.nsa_decode_q8(p, one, cache, lens, keys=keys)
            nsa.nsa_check()
            assert torch.isnan(out[0, 0]).all() and torch.isnan(out[1, 1]).all()
            assert torch.isnan(lse[0, 0]) and torch.isnan(lse[1, 1])
            assert torch.isfinite(out[0, 1:]).all() and torch.isfinite(out[1, 2:]).all()
            assert not out[2].any() and (lse[2] == -math.inf).all()


# ---- value scales that are none of a query's own ------------------------------------

def outlier_cache(p, lens, seed, at, ratio, held=True):
    """random_cache with scales alike, but for the page of sequence 0's token `at`: its
    value scale covers values `ratio` times the others', its codes are what is left of
    the values under it. That token has the largest code everywhere, unless it was
    written over since (held False: the scale stays)."""
    cache = random_cache(p, lens, seed, extra=0, spread=0.0)
    pid, slot = int(cache.page_table[0, at // p.sel_block]), at % p.sel_block
    codes = (cache.v_pages[pid].float() / ratio).to(torch.float8_e4m3fn).view(torch.uint8)
    codes[:, slot] = 0x7e if held else 0
    cache.v_pages.view(torch.uint8)[pid] = codes
    cache.v_scale[pid] *= ratio
    return cache


OUTLIERS = ((BF16, 128, 64), (BF16, 128, 32), (BF16, 64, 16), (F32, 64, 16), (F32, 128, 128))


@pytest.mark.parametrize("dt,d,page", OUTLIERS, ids=str)
@pytest.mark.parametrize("ratio", (2.0 ** 7, 2.0 ** 10, 2.0 ** 12, 2.0 ** 16, 2.0 ** 24, 2.0 ** 40, 2.0 ** 100))
def test_decode_unseen_outlier_values(dt, d, page, ratio):
    """A value that a query does not see, in a page of which it sees other tokens, takes
    nothing from the query's sums, however large: a token before the window, one
    written over since, and one behind the sequence's end."""
    p = nsa.params(1, 1000, 16, 1, d, sel_block=page, dtype=dt, window=501)
    q = torch.randn(1, 16, d, generator=gen(91)).to(dt).cuda()
    lens = i32([1000])
    first = 1000 - 501
    for at, held, keys in (((first // page) * page, True, "window"), (999, False, "all"),
                           (5, False, "all"), (700, False, "window")):
        cache = outlier_cache(p, [1000], 92, at, ratio, held)
        got = nsa.nsa_decode_q8(p, q, cache, lens, keys=keys)
        nsa.nsa_check()
        check_attention(got, p, q, cache, lens, None, keys)
    lens = i32([990])  # tokens 990 .. 999 were drafts, refused since
    cache = outlier_cache(p, [1000], 92, 990 + 5, ratio)
    got = nsa.nsa_decode_q8(p, q, cache, lens)
    nsa.nsa_check()
    check_attention(got, p, q, cache, lens)
    # a listed block whose scale is none of its codes', before and behind others
    p = nsa.params(1, 1000, 16, 1, d, sel_block=page, dtype=dt, top_n=5)
    cache = outlier_cache(p, [1000], 92, 3 * page, ratio, False)
    for sel in ([3, 0, 1, -1, 6], [0, 1, 6, 2, 3]):
        got = nsa.nsa_decode_q8(p, q, cache, i32([1000]), keys="blocks", sel_idx=i32([[sel]]))
        nsa.nsa_check()
        check_attention(got, p, q, cache, i32([1000]), None, "blocks", torch.tensor([[sel]]))


@pytest.mark.parametrize("dt,d,page", OUTLIERS, ids=str)
@pytest.mark.parametrize("ratio", (2.0 ** 7, 2.0 ** 10, 2.0 ** 12, 2.0 ** 16, 2.0 ** 24, 2.0 ** 40, 2.0 ** 100))
def test_prefill_unseen_outlier_values(dt, d, page, ratio):
    """The same for chunks: queries before the outlier's token, and those whose window
    has left it, keep their sums; the others have its value."""
    p = nsa.params(1, 700, 16, 1, d, sel_block=page, dtype=dt, window=130)
    n = 300
    q = torch.randn(n, 16, d, generator=gen(93)).to(dt).cuda()
    lens, cu = i32([700]), i32([0, n])
    for at, held in ((640, True), (699, True), (405, True), (500, False)):
        cache = outlier_cache(p, [700], 94, at, ratio, held)
        for keys in ("all", "window"):
            got = nsa.nsa_prefill_q8(p, q, cache, lens, cu, keys=keys)
            nsa.nsa_check()
            check_attention(got, p, q, cache, lens, cu.cpu(), keys)


@pytest.mark.parametrize("dt,d,page,Hq,Hkv", ((BF16, 128, 64, 40, 2), (BF16, 128, 32, 6, 2), (F32, 128, 16, 6, 2),
                                              (BF16, 64, 128, 20, 1)), ids=str)
def test_nan_values_among_scales_far_apart(dt, d, page, Hq, Hkv):
    """NaN values in pages of scales 2^-120 to 2^110: the rows that see them, no others;
    pages of zeros of any scale, and rows whose keys are all in such pages."""
    lens, new = [500, 333, 700], [90, 20, 60]
    p = nsa.params(3, 720, Hq, Hkv, d, sel_block=page, dtype=dt, window=140)
    N, g = sum(new), gen(99)
    cache = random_cache(p, lens, 100, spread=0.0)
    pages = cache.v_scale.shape[0]
    cache.v_scale.copy_(torch.exp2(torch.randint(-120, 111, (pages, Hkv), generator=g).float()))
    zero = torch.rand(pages, Hkv, generator=g) < 0.4
    table = cache.page_table.cpu()
    last = [int(x) for x in table[1] if x >= 0]
    zero[last] = True                       # sequence 1 has nothing but zeros
    live = cache.v_pages.view(torch.uint8)
    live.copy_(torch.where(zero[..., None, None].cuda(), 0, live))
    q = torch.randn(N, Hq, d, generator=g).to(dt).cuda()
    cu = i32([0, 90, 110, 170])
    for keys in ("all", "window"):
        got = nsa.nsa_prefill_q8(p, q, cache, i32(lens), cu, keys=keys)
        nsa.nsa_check()
        want, wlse, A, B = ref.attend(q, cache.k_pages, cache.v_pages, cache.k_scale, cache.v_scale,
                                      cache.page_table, i32(lens), page, cu.cpu(), keys, p.window)
        t_out, t_lse = ref.bounds(want, wlse, A, B, dt, 700)
        # (beside the relative bound: a weight's last place next to the row's largest
        # product, 2^-21 of it a key where codes may be as small as here)
        t_out = t_out + 700 * 2.0 ** -21 * A.amax(-1, keepdim=True)
        assert ((got[0].double().cpu() - want).abs() <= t_out).all()
        assert ((got[1].double().cpu() - wlse).abs() <= t_lse).all()
        assert not got[0][90:110].any()
    base = nsa.nsa_prefill_q8(p, q, cache, i32(lens), cu)
    want = nan_marks(p, cache, lens, new, [470, 320, 100], [3, 5, 7])
    out, lse = nsa.nsa_prefill_q8(p, q, cache, i32(lens), cu)
    nsa.nsa_check()
    assert torch.equal(torch.isnan(out).cpu(), want) and torch.equal(lse, base[1])
    # (a code less may change the units that sums are held in)
    scale = base[0].abs().amax(-1, keepdim=True).expand_as(out)[~want.cuda()].double()
    assert ((out - base[0]).abs()[~want.cuda()].double() <= scale * 2.0 ** -7).all()


def test_prefill_drafts_unseen_outlier_values():
    """Few queries a sequence over many keys, where both tile halves share the keys."""
    B, new = 20, 4
    lens = [600 + 37 * b for b in range(B)]
    p = nsa.params(B, 1400, 16, 1, 128, sel_block=64)
    q = torch.randn(B * new, 16, 128, generator=gen(95)).to(BF16).cuda()
    cu = i32([new * b for b in range(B + 1)])
    for ratio in (2.0 ** 24, 2.0 ** 60):
        cache = random_cache(p, lens, 96, extra=0, spread=0.0)
        codes, table = cache.v_pages.view(torch.uint8), cache.page_table.cpu()
        for b in range(B):  # some page's scale is that of a token written over since,
            pid = int(table[b, b % 9])
            codes[pid] = 0
            cache.v_scale[pid] *= ratio
            pid = int(table[b, (lens[b] - 1) // 64])  # or of the last draft
            few = (cache.v_pages[pid].float() / ratio).to(torch.float8_e4m3fn).view(torch.uint8)
            few[:, (lens[b] - 1) % 64] = 0x7e
            codes[pid] = few
            cache.v_scale[pid] *= ratio
        got = nsa.nsa_prefill_q8(p, q, cache, i32(lens), cu)
        nsa.nsa_check()
        check_attention(got, p, q, cache, i32(lens), cu.cpu())


@pytest.mark.parametrize("dt,d,page", OUTLIERS, ids=str)
def test_outlier_in_one_channel(dt, d, page):
    """A value that is seen, far above the others in one channel: the other channels
    have its key's weight's share, and at most 2^-33 of the largest product of a weight
    and a value for each key besides (a weight's last place beside that product)."""
    p = nsa.params(1, 700, 16, 1, d, sel_block=page, dtype=dt)
    n = 40
    q = torch.randn(n, 16, d, generator=gen(97)).to(dt).cuda()
    lens, cu = i32([700]), i32([0, n])
    for ratio in (2.0 ** 6, 2.0 ** 12, 2.0 ** 20):
        cache = outlier_cache(p, [700], 98, 300, ratio)
        pid = int(cache.page_table[0, 300 // page])
        cache.v_pages.view(torch.uint8)[pid, :, 300 % page, 1:] = 0
        got = nsa.nsa_prefill_q8(p, q, cache, lens, cu)
        nsa.nsa_check()
        want, wlse, A, B = ref.attend(q, cache.k_pages, cache.v_pages, cache.k_scale,
                                      cache.v_scale, cache.page_table, lens, page, cu.cpu())
        t_out, t_lse = ref.bounds(want, wlse, A, B, dt, 700)
        t_out = t_out + 700 * 2.0 ** -33 * A.amax(-1, keepdim=True)
        err = (got[0].double().cpu() - want).abs()
        assert (err <= t_out).all(), float((err / t_out).max())
        assert ((got[1].double().cpu() - wlse).abs() <= t_lse).all()


# ---- together -----------------------------------------------------------------------

@pytest.mark.parametrize("dt", (BF16, F32))
def test_serving_loop(dt):
    """A prompt appended and attended in chunks, then tokens one at a time, with
    the window and the selected blocks joined through lse: each step equals
    attention over the cache it stands on, and the same steps replayed from CUDA
    graphs give the same bits."""
    B, Hq, Hkv, d, page = 2, 8, 2, 128, 64
    prompts, steps, T = [150, 83], 6, 256
    p = nsa.params(B, T, Hq, Hkv, d, sel_block=page, dtype=dt, window=48, top_n=2)
    rope = nsa.rope_table(T, d)
    table = torch.randperm(2 * 4, generator=gen(50)).view(2, 4).to(torch.int32).cuda()
    cache = nsa.q8_cache(p, 8, table)
    g = gen(51)

    def fresh(n):
        return [torch.randn(n, h, d, generator=g).to(dt).cuda() for h in (Hq, Hkv, Hkv)]

    done = [0, 0]
    for chunk in (64, 100):
        new = [min(chunk, n - x) for n, x in zip(prompts, done)]
        q, k, v = fresh(sum(new))
        cu = i32([0, new[0], sum(new)])
        q_rot, _, _ = nsa.nsa_append_q8(p, k, v, i32(done), cache, cu_new=cu, q=q, rope=rope)
        done = [x + n for x, n in zip(done, new)]
        got = nsa.nsa_prefill_q8(p, q_rot, cache, i32(done), cu)
        nsa.nsa_check()
        check_attention(got, p, q_rot, cache, i32(done), cu.cpu())
    assert done == prompts

    q, k, v = fresh(B)
    pos, lens = i32(done), i32([x + 1 for x in done])
    sel = i32([[[0, 2], [0, 1]], [[0, 1], [1, -1]]])
    ws = nsa.workspace(p, nsa.OP_DECODE_Q8)
    q_rot = torch.empty_like(q)
    bufs = {n: (torch.empty_like(q), torch.empty(B, Hq, device="cuda"))
            for n in ("all", "window", "blocks")}

    def step():
        nsa.nsa_append_q8(p, k, v, pos, cache, q=q, q_out=q_rot, rope=rope)
        for name, (o, s) in bufs.items():
            nsa.nsa_decode_q8(p, q_rot, cache, lens, keys=name, out=o, lse=s, ws=ws,
                              sel_idx=sel if name == "blocks" else None)

    start = [t.clone() for t in (cache.k_pages, cache.v_pages, cache.k_scale, cache.v_scale)]
    inputs, eager = [], []
    for i in range(steps):
        for dst, src in zip((q, k, v), fresh(B)):
            dst.copy_(src)
        inputs.append([t.clone() for t in (q, k, v)])
        step()
        nsa.nsa_check()
        for name, got in bufs.items():
            check_attention(got, p, q_rot, cache, lens, None, name, sel.cpu())
        eager.append([t.clone() for pair in bufs.values() for t in pair])
        pos += 1
        lens += 1
    for dst, src in zip((cache.k_pages, cache.v_pages, cache.k_scale, cache.v_scale), start):
        dst.copy_(src)
    pos -= steps
    lens -= steps
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for dst, src in zip((q, k, v), inputs[0]):
            dst.copy_(src)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step()
    for i in range(steps):
        for dst, src in zip((q, k, v), inputs[i]):
            dst.copy_(src)
        graph.replay()
        for got, want in zip([t for pair in bufs.values() for t in pair], eager[i]):
            assert torch.equal(got, want)
        pos += 1
        lens += 1
    nsa.nsa_check()


def test_two_streams_with_their_own_workspaces():
    p = nsa.params(4, 3000, 16, 1, 128, sel_block=64)
    lens = [3000, 1, 700, 2048]
    cache = random_cache(p, lens, 60)
    qs = [torch.randn(4, 16, 128, generator=gen(61 + i)).to(BF16).cuda() for i in range(2)]
    want = [nsa.nsa_decode_q8(p, q, cache, i32(lens)) for q in qs]
    L = i32(lens)
    streams = [torch.cuda.Stream() for _ in qs]
    wss = [nsa.workspace(p, nsa.OP_DECODE_Q8) for _ in qs]
    outs = [[(torch.empty_like(q), torch.empty(4, 16, device="cuda")) for _ in range(20)] for q in qs]
    torch.cuda.synchronize()
    for r in range(20):
        for q, s, w, o in zip(qs, streams, wss, outs):
            nsa.nsa_decode_q8(p, q, cache, L, out=o[r][0], lse=o[r][1], ws=w, stream=s)
    torch.cuda.synchronize()
    for o, (out, lse) in zip(outs, want):
        for a, b in o:
            assert torch.equal(a, out) and torch.equal(b, lse)
    nsa.nsa_check()


def test_two_streams_of_chunks():
    """Chunks of two caches at once, on streams and workspaces of their own, between
    appends of one and the other: the bits of one stream alone."""
    T, new = 2400, [400, 300, 500]
    p = nsa.params(3, T, 64, 4, 128, sel_block=64)
    rope, N = nsa.rope_table(T, 128), sum(new)
    past, cu = i32([1900, 0, 1000]), i32([0, 400, 700, 1200])
    lens = i32([2300, 300, 1500])
    parts = []
    for x in range(2):
        g = gen(190 + x)
        q, k, v = (torch.randn(N, h, 128, generator=g).to(BF16).cuda() for h in (64, 4, 4))
        parts.append((random_cache(p, [2300, 300, 1500], 192 + x), q, k, v, nsa.workspace(p, nsa.OP_PREFILL_Q8),
                      torch.cuda.Stream()))

    def run(part, stream):
        cache, q, k, v, ws, _ = part
        rot, _, _ = nsa.nsa_append_q8(p, k, v, past, cache, cu_new=cu, q=q, rope=rope, stream=stream)
        return nsa.nsa_prefill_q8(p, rot, cache, lens, cu, ws=ws, stream=stream)

    want = [run(part, None) for part in parts]
    torch.cuda.synchronize()
    got = [[run(part, part[-1]) for part in parts] for _ in range(30)]
    torch.cuda.synchronize()
    nsa.nsa_check()
    for pair in got:
        for (out, lse), (o, s) in zip(pair, want):
            assert torch.equal(out, o) and torch.equal(lse, s)


def test_a_given_stream_owns_what_a_call_makes(monkeypatch):
    """As tests/test_gpu_nsa.py's: outputs and workspaces made for a call on a stream."""
    from tests.test_gpu_nsa import _owner
    made, empty = [], torch.empty

    def spy(*a, **kw):
        made.append(empty(*a, **kw))
        return made[-1]

    p = nsa.params(2, 256, 16, 1, 128, sel_block=64)
    q = torch.randn(6, 16, 128, generator=gen(120)).to(BF16).cuda()
    k, v = (torch.randn(6, 1, 128, generator=gen(121 + i)).to(BF16).cuda() for i in range(2))
    lens, cu, rope = i32([200, 99]), i32([0, 4, 6]), nsa.rope_table(256, 128)
    first = q[:2].contiguous()
    side = torch.cuda.Stream()
    calls = {
        "append": lambda c, s: nsa.nsa_append_q8(p, k, v, i32([196, 97]), c, cu_new=cu, q=q, rope=rope,
                                                 want_kv=True, stream=s),
        "decode": lambda c, s: nsa.nsa_decode_q8(p, first, c, lens, stream=s),
        "prefill": lambda c, s: nsa.nsa_prefill_q8(p, q, c, lens, cu, stream=s),
    }
    for name, call in calls.items():
        want = call(random_cache(p, [200, 99], 122), None)
        cache = random_cache(p, [200, 99], 122)
        torch.cuda.synchronize()
        made.clear()
        monkeypatch.setattr(torch, "empty", spy)
        got = call(cache, side)
        monkeypatch.setattr(torch, "empty", empty)
        torch.cuda.synchronize()
        assert len(made) == 3 and all(_owner(t) == side.cuda_stream for t in made), name
        for a, b in zip(got, want):
            assert torch.equal(a, b), name
    nsa.nsa_check()


def test_cache_tensors_set_anew():
    """An assigned tensor is the one that calls use; one that does not fit is refused."""
    p = nsa.params(2, 100, 4, 2, 64, sel_block=32)
    cache, other = random_cache(p, [100, 50], 180), random_cache(p, [100, 50], 181)
    assert cache.k_pages.shape == other.k_pages.shape
    q = torch.randn(2, 4, 64, generator=gen(182)).to(BF16).cuda()
    lens = i32([100, 50])
    want = nsa.nsa_decode_q8(p, q, other, lens)
    for name in ("page_table", "k_pages", "v_pages", "k_scale", "v_scale"):
        setattr(cache, name, getattr(other, name))
        assert getattr(cache, name) is getattr(other, name)
    got = nsa.nsa_decode_q8(p, q, cache, lens)
    nsa.nsa_check()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    for name, bad, text in (("page_table", i32([1, 2]), "page_table"), ("k_scale", other.k_scale[:1], "k_scale"),
                            ("v_pages", other.v_pages.float(), "v_pages")):
        with pytest.raises(ValueError, match=text):
            setattr(cache, name, bad)
        assert getattr(cache, name) is getattr(other, name)
    cache.page_table = i32([[0, 1, 2, 3, 4]] * 2)  # more pages than the parameters have
    with pytest.raises(ValueError, match="page_table"):
        nsa.nsa_decode_q8(p, q, cache, lens)


def test_wrapper_refusals():
    p = nsa.params(2, 100, 4, 2, 64, sel_block=32)
    cache = random_cache(p, [100, 50], 70)
    q = torch.zeros(2, 4, 64, dtype=BF16, device="cuda")
    lens = i32([100, 50])
    with pytest.raises(ValueError, match="keys"):
        nsa.nsa_decode_q8(p, q, cache, lens, keys="some")
    with pytest.raises(ValueError, match="q must be"):
        nsa.nsa_decode_q8(p, q.float(), cache, lens)
    with pytest.raises(ValueError, match="q must be"):
        nsa.nsa_decode_q8(p, q[:1], cache, lens)
    with pytest.raises(ValueError, match="contiguous"):
        nsa.nsa_decode_q8(p, q.transpose(0, 1), cache, lens)
    with pytest.raises(ValueError, match="pages are"):
        nsa.nsa_decode_q8(nsa.params(2, 100, 4, 2, 64, sel_block=64), q, cache, lens)
    with pytest.raises(ValueError, match="page_table"):
        nsa.nsa_decode_q8(nsa.params(2, 200, 4, 2, 64, sel_block=32), q, cache, lens)
    with pytest.raises(ValueError, match="sel_idx must be"):
        nsa.nsa_decode_q8(p, q, cache, lens, keys="blocks", sel_idx=i32([[1]]))
    with pytest.raises(nsa.NsaError, match="sel_idx"):
        nsa.nsa_decode_q8(p, q, cache, lens, keys="blocks")
    with pytest.raises(ValueError, match="rope_style"):
        nsa.nsa_append_q8(p, q[:, :2].contiguous(), q[:, :2].contiguous(), lens, cache,
                          rope=nsa.rope_table(100, 64), rope_style="other")
    with pytest.raises(ValueError, match="pos must be"):
        nsa.nsa_append_q8(p, q[:, :2].contiguous(), q[:, :2].contiguous(), lens[:1], cache)
