"""What is measured of the 8-bit paged KV cache: the append with the position
rotation on the way, attention of single tokens over the cache, and attention
of chunks of tokens over it.

``run`` computes each operator in its plain form (elementary torch operations,
fp32) while ``own`` is false, and calls the library while it is true.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
E4M3 = torch.float8_e4m3fn


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def _append(name, B, new, past, Hq, Hkv, d, page, dtype, rot, style, ragged=False):
    return dict(name=name, op="append", B=B, new=new, past=past, Hq=Hq, Hkv=Hkv, d=d, page=page,
                dtype=dtype, rot=rot, style=style, ragged=ragged)


def _decode(name, B, L, Hq, Hkv, d, page, dtype, keys, window=0, n=0, ragged=False):
    return dict(name=name, op="decode", B=B, L=L, Hq=Hq, Hkv=Hkv, d=d, page=page, dtype=dtype,
                keys=keys, window=window, n=n, ragged=ragged)


def _prefill(name, B, new, L, Hq, Hkv, d, page, dtype, keys, window=0, ragged=False):
    return dict(name=name, op="prefill", B=B, new=new, L=L, Hq=Hq, Hkv=Hkv, d=d, page=page,
                dtype=dtype, keys=keys, window=window, ragged=ragged)


def listed():
    return [
        # one token for each of 32 sequences: the append of a decode step
        _append("append_step_b32", 32, 1, 4999, 64, 4, 128, 64, "bf16", 128, "half"),
        # the keys and values of a whole 8192-token prompt
        _append("append_prompt_8192", 1, 8192, 0, 64, 4, 128, 64, "bf16", 128, "half"),
        # chunks of several requests, from inside their pages on; fp32, part of the head rotated
        _append("append_chunks_f32", 11, 701, 333, 12, 3, 64, 32, "f32", 32, "pairs", True),
        # a short chat: one sequence, where latency counts
        _decode("decode_b1_l1000", 1, 1000, 64, 4, 128, 64, "bf16", "all"),
        # the long-context decode shape: 32 sequences of 65536 tokens
        _decode("decode_b32_l65536", 32, 65536, 64, 4, 128, 64, "bf16", "all"),
        # ragged requests, an empty slot among them, five heads per KV head; fp32, small pages
        _decode("decode_ragged_f32", 24, 9001, 40, 8, 64, 16, "f32", "all", ragged=True),
        # the selected branch: 16 listed blocks of 64 for each sequence and KV head
        _decode("decode_blocks_b32", 32, 65536, 64, 4, 128, 64, "bf16", "blocks", n=16),
        # a sliding-window layer over ragged requests
        _decode("decode_window_b64", 64, 20011, 32, 8, 128, 64, "bf16", "window", window=512,
                ragged=True),
        # a 2048-token chunk of a long prompt
        _prefill("prefill_chunk_2048", 1, 2048, 16384, 64, 4, 128, 64, "bf16", "all"),
        # several requests' chunks in one call
        _prefill("prefill_ragged", 5, 997, 4001, 32, 8, 128, 64, "bf16", "all", ragged=True),
        # a windowed layer's prompt; fp32
        _prefill("prefill_window_f32", 1, 1500, 1500, 8, 2, 64, 32, "f32", "window", window=512),
        # four draft tokens of each of 16 sequences, checked at once
        _prefill("prefill_drafts", 16, 4, 8191, 64, 4, 128, 64, "bf16", "all"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    d = rng.choice((64, 128, 128))
    page = rng.choice((16, 32, 64, 64, 64, 128))
    Hkv = rng.choice((1, 2, 3, 4, 8))
    G = rng.choice((1, 2, 4, 5, 7, 8, 16, 16, 20))
    dtype = rng.choice(("bf16", "bf16", "bf16", "f32"))
    ragged = rng.random() < 0.5
    shape = dict(Hq=Hkv * G, Hkv=Hkv, d=d, page=page, dtype=dtype, ragged=ragged)
    op = rng.choice(("append", "decode", "decode", "prefill"))
    if op == "append":
        B = _log(rng, 1, 64)
        new = 1 if rng.random() < 0.4 else _log(rng, 1, max(1, min(8192, 16384 // B)))
        return dict(op=op, B=B, new=new, past=rng.choice((0, _log(rng, 1, 20000))),
                    rot=16 * rng.randint(1, d // 16), style=rng.choice(("half", "pairs")), **shape)
    if op == "decode":
        B = _log(rng, 1, 64)
        L = _log(rng, rng.choice((1, 200, 200)), min(100000, (1 << 22) // (B * Hkv)))
        keys = rng.choice(("all", "window", "blocks"))
        return dict(op=op, B=B, L=L, keys=keys, window=_log(rng, 1, 4096) if keys == "window" else 0,
                    n=_log(rng, 1, 32) if keys == "blocks" else 0, **shape)
    B = _log(rng, 1, 16)
    new = _log(rng, 1, 2048)
    most = (1 << 29) // (B * Hkv * G * new)  # scores of the plain form
    new = min(new, max(1, most))
    L = new + _log(rng, 1, max(1, min(32768, most)))
    keys = rng.choice(("all", "all", "window"))
    return dict(op=op, B=B, new=new, L=L, keys=keys,
                window=_log(rng, 1, 4096) if keys == "window" else 0, **shape)


# ---------------------------------------------------------------------------
# sizes that follow from a case
# ---------------------------------------------------------------------------

def _spread(most, B, ragged, least):
    """B lengths up to `most`: all of them `most`, or spread over [least, most]."""
    if not ragged or B == 1:
        return [most] * B
    got = [least + int((most - least) * ((0.31 + 0.6180339887 * b) % 1.0)) for b in range(B)]
    got[B // 2], got[-1] = least, most
    return got


def _sizes(c):
    """(tokens in the cache, new tokens) of each sequence after the call."""
    if c["op"] == "decode":
        lens = _spread(c["L"], c["B"], c["ragged"], 0)
        return lens, [1] * c["B"]
    new = _spread(c["new"], c["B"], c["ragged"], 0 if c["op"] == "append" else 1)
    if c["op"] == "append":
        past = _spread(c["past"], c["B"], c["ragged"], 0)
        return [p + n for p, n in zip(past, new)], new
    past = _spread(c["L"] - c["new"], c["B"], c["ragged"], 0)
    return [p + n for p, n in zip(past, new)], new


def _first_key(c, position):
    return max(0, position - c["window"] + 1) if c["keys"] == "window" else 0


def work(c):
    lens, new = _sizes(c)
    es = 2 if c["dtype"] == "bf16" else 4
    Hq, Hkv, d, page = c["Hq"], c["Hkv"], c["d"], c["page"]
    if c["op"] == "append":
        N = sum(new)
        pages = sum(-(-m // page) - (m - n) // page for m, n in zip(lens, new) if n)
        # k, v, q and the table rows in; codes, scales, q_out, k_out, v_out out
        return {"bytes": N * ((Hq + 2 * Hkv) * d * es * 2 + 2 * Hkv * d + c["rot"] * 4)
                + pages * (2 * Hkv * 4 + 4), "flops": N * (Hq + Hkv) * c["rot"] * 3}
    tokens, seen, rows = 0, 0, sum(new)
    for m, n in zip(lens, new):
        if c["op"] == "decode" and c["keys"] == "blocks":
            tokens += min(m, c["n"] * page)
            seen += min(m, c["n"] * page)
        elif m:
            tokens += m - _first_key(c, m - n)
            if c["keys"] == "window":
                # positions m - n .. m - 1, each with min(position + 1, window) keys
                w = c["window"]
                full = min(n, max(0, m - w))
                part = n - full
                seen += full * w + part * (m - n) + part * (part + 1) // 2
            else:
                seen += n * (m - n) + n * (n + 1) // 2
    moved = tokens * 2 * Hkv * d + -(-tokens // page) * (8 * Hkv + 4)
    return {"bytes": moved + rows * Hq * (2 * d * es + 4), "flops": 4 * seen * Hq * d}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def prepare(c, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed)
    dt = DTYPES[c["dtype"]]
    B, Hq, Hkv, d, page = c["B"], c["Hq"], c["Hkv"], c["d"], c["page"]
    lens, new = _sizes(c)
    T = max(1, max(lens))
    wide = -(-T // page)

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device=dev).to(dt)

    def ints(v):
        return torch.tensor(v, dtype=torch.int32, device=dev)

    def pool():
        """Codes and scales of random pages: normal components, some channels
        larger than others, magnitudes that differ from page to page."""
        codes = torch.empty(pages, Hkv, page, d, dtype=torch.uint8, device=dev)
        scales = torch.empty(pages, Hkv, dtype=torch.float32, device=dev)
        gain = torch.exp(0.4 * torch.randn(Hkv, 1, d, generator=gen, device=dev))
        step = max(1, (1 << 27) // (Hkv * page * d))
        for at in range(0, pages, step):
            n = min(step, pages - at)
            x = torch.randn(n, Hkv, page, d, generator=gen, device=dev)
            x *= gain * torch.exp(0.3 * torch.randn(n, Hkv, 1, 1, generator=gen, device=dev))
            s = _power_of_two(x.abs().amax(dim=(2, 3)))
            codes[at:at + n] = (x / s[..., None, None]).to(E4M3).view(torch.uint8)
            scales[at:at + n] = s
        return codes.view(E4M3), scales

    # every sequence's pages lie scattered in the pool; an append needs its tail pages only
    first = [(m - n) // page if c["op"] == "append" else 0 for m, n in zip(lens, new)]
    count = [-(-m // page) - f for m, f in zip(lens, first)]
    pages = sum(count) + 3
    order = torch.randperm(pages, generator=gen, device=dev).to(torch.int32)
    table = torch.zeros(B, wide, dtype=torch.int32, device=dev)
    at = 0
    for b in range(B):
        table[b, first[b]:first[b] + count[b]] = order[at:at + count[b]]
        at += count[b]
    k_pages, k_scale = pool()
    v_pages, v_scale = pool()
    starts = [0]
    for n in new:
        starts.append(starts[-1] + n)
    N = starts[-1]
    state = dict(case=c, T=T, k_pages=k_pages, v_pages=v_pages, k_scale=k_scale, v_scale=v_scale,
                 table=table, lens=ints(lens), new=max(new), q=normal(N, Hq, d),
                 cu=None if c["op"] == "decode" or new == [1] * B else ints(starts))
    if c["op"] == "append":
        rot = c["rot"]
        freq = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device=dev) / rot)
        angle = torch.arange(T, dtype=torch.float64, device=dev)[:, None] * freq
        state.update(k=normal(N, Hkv, d) * 2, v=normal(N, Hkv, d),
                     pos=ints([m - n for m, n in zip(lens, new)]),
                     rope=torch.stack((angle.cos(), angle.sin()), dim=1).float().contiguous())
    if c["op"] == "decode" and c["keys"] == "blocks":
        # block 0 and n - 1 others in ascending order, -1 past them, as a selection writes them
        have = -(-state["lens"].long() // page)
        x = torch.rand(B, Hkv, max(wide, c["n"]), generator=gen, device=dev)
        at = torch.arange(x.shape[2], device=dev)
        x[..., 0] = 2.0
        x = torch.where(at < have[:, None, None], x, -1.0)
        top = x.topk(c["n"], dim=2)
        none = x.shape[2]
        pick = torch.where(top.values >= 0, top.indices, none).sort(dim=2).values
        state["sel"] = torch.where(pick < none, pick, -1).to(torch.int32).contiguous()
    return state


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------

def _power_of_two(a):
    """The smallest power of two s (at least 2^-126) with a <= 448 s."""
    part, e = torch.frexp(a)  # 448 = 0.875 * 2^9
    e = torch.where(a > 0, e - 9 + (part > 0.875), -126).clamp(min=-126)
    return torch.ldexp(torch.ones_like(a), e)


def _rotate(x, rope, style):
    """x [N, H, d] fp32 with its first components rotated by rope [N, 2, rot / 2]."""
    cos, sin = rope[:, 0, None], rope[:, 1, None]
    half = cos.shape[-1]
    y = x.clone()
    if style == "half":
        a, b = x[..., :half], x[..., half:2 * half]
        y[..., :half], y[..., half:2 * half] = a * cos - b * sin, b * cos + a * sin
    else:
        a, b = x[..., 0:2 * half:2], x[..., 1:2 * half:2]
        y[..., 0:2 * half:2], y[..., 1:2 * half:2] = a * cos - b * sin, b * cos + a * sin
    return y


def _rows(s, N):
    """Sequence and index within it of each of the call's N tokens."""
    t = torch.arange(N, device=s["table"].device)
    if s["cu"] is None:
        return t, torch.zeros_like(t)
    b = (t[:, None] >= s["cu"][None, 1:]).sum(1)
    return b, t - s["cu"][b]


def _write(pages, scales, x, pid, slot):
    """Puts rows x [N, Hkv, d] into slots of pages, in place; returns them as stored."""
    P, Hkv = scales.shape
    top = torch.zeros_like(scales).index_reduce_(0, pid, x.abs().amax(-1), "amax")
    hit = torch.zeros(P, dtype=torch.bool, device=x.device).index_fill_(0, pid, True)
    begun = torch.zeros(P, dtype=torch.int32, device=x.device)
    begun = begun.index_reduce_(0, pid, (slot == 0).int(), "amax") > 0
    need = _power_of_two(top)
    s = torch.where(begun[:, None], need, torch.maximum(scales, need))
    s = torch.where(hit[:, None], s, scales)
    pages.copy_((pages.float() * (scales / s)[..., None, None]).to(E4M3))
    scales.copy_(s)
    codes = (x / s[pid][..., None]).to(E4M3)
    pages.view(torch.uint8)[pid, :, slot] = codes.view(torch.uint8)
    return codes.float() * s[pid][..., None]


def _append_plain(s):
    c = s["case"]
    dt = DTYPES[c["dtype"]]
    b, i = _rows(s, s["k"].shape[0])
    at = s["pos"][b] + i
    pid, slot = s["table"][b, at // c["page"]].long(), at % c["page"]
    turn = s["rope"][at]
    q_out = _rotate(s["q"].float(), turn, c["style"]).to(dt)
    k_out = _write(s["k_pages"], s["k_scale"], _rotate(s["k"].float(), turn, c["style"]), pid, slot)
    v_out = _write(s["v_pages"], s["v_scale"], s["v"].float(), pid, slot)
    return q_out, k_out.to(dt), v_out.to(dt)


def _read(pages, scales, pid, head):
    x = pages.view(torch.uint8)[pid, head].view(E4M3).float()
    return x * scales[pid, head][..., None, None]


def _attend(s, q, n, lens):
    """q [B, rows, Hq, d] fp32, row i of sequence b at position lens[b] - n[b] + i."""
    c = s["case"]
    B, R, Hq, d = q.shape
    Hkv, page, dev = c["Hkv"], c["page"], q.device
    at = lens.long()[:, None] - n[:, None] + torch.arange(R, device=dev)  # positions of the rows
    wide = s["table"].shape[1]
    if c["keys"] == "blocks":
        block = s["sel"].long()
    elif c["keys"] == "window":
        from_ = (at[:, 0] - c["window"] + 1).clamp(min=0) // page
        count = min(wide, (c["window"] + R - 2) // page + 2)
        block = from_[:, None, None] + torch.arange(count, device=dev)
        block = torch.where(block < wide, block, -1).expand(B, Hkv, count)
    else:
        block = torch.arange(wide, device=dev).expand(B, Hkv, wide)
    pid = s["table"].long().gather(1, block.clamp(min=0).reshape(B, -1)).reshape(block.shape)
    head = torch.arange(Hkv, device=dev)[None, :, None]
    k = _read(s["k_pages"], s["k_scale"], pid, head).reshape(B, Hkv, -1, d)
    v = _read(s["v_pages"], s["v_scale"], pid, head).reshape(B, Hkv, -1, d)
    key = block[..., None] * page + torch.arange(page, device=dev)
    key = torch.where(block[..., None] >= 0, key, 1 << 40).reshape(B, Hkv, 1, -1)
    row = at[:, None, :, None]
    seen = key <= row
    if c["keys"] == "window":
        seen = seen & (key > row - c["window"])
    # rows [B, Hkv, R * G], the group's heads of a token side by side
    G = Hq // Hkv
    q = q.reshape(B, R, Hkv, G, d).transpose(1, 2).reshape(B, Hkv, R * G, d)
    seen = seen[:, :, :, None].expand(B, Hkv, R, G, seen.shape[-1]).reshape(B, Hkv, R * G, -1)
    z = q @ k.transpose(2, 3)
    z *= 1.0 / math.sqrt(d)
    z.masked_fill_(~seen, -math.inf)
    top = z.amax(-1, keepdim=True)
    base = torch.where(top > -math.inf, top, 0.0)
    e = z.sub_(base).exp_()
    total = e.sum(-1, keepdim=True)
    out = (e @ v) / torch.where(total > 0, total, 1.0)
    lse = (base + total.log())[..., 0]
    out = out.reshape(B, Hkv, R, G, d).transpose(1, 2).reshape(B, R, Hq, d)
    return out, lse.reshape(B, Hkv, R, G).transpose(1, 2).reshape(B, R, Hq)


def _attend_plain(s):
    c = s["case"]
    dt = DTYPES[c["dtype"]]
    N, B, R = s["q"].shape[0], c["B"], s["new"]
    if s["cu"] is None:
        n = torch.ones_like(s["lens"], dtype=torch.int64)
        out, lse = _attend(s, s["q"].float().view(B, 1, c["Hq"], c["d"]), n, s["lens"])
        return out[:, 0].to(dt), lse[:, 0]
    cu = s["cu"].long()
    b, i = _rows(s, N)
    pick = (cu[:-1, None] + torch.arange(R, device=cu.device)).clamp(max=N - 1)
    out, lse = _attend(s, s["q"].float()[pick], cu[1:] - cu[:-1], s["lens"])
    return out[b, i].to(dt), lse[b, i]


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def run(s):
    c = s["case"]
    if own:
        from dynamic_block_sparse_nsa_b200 import nsa
        if "p" not in s:  # a program keeps its parameters, cache handle and workspace
            s["p"] = nsa.params(c["B"], s["T"], c["Hq"], c["Hkv"], c["d"], sel_block=c["page"],
                                top_n=c.get("n") or 1, window=c.get("window") or 1,
                                dtype=DTYPES[c["dtype"]])
            s["cache"] = nsa.Q8Cache(s["k_pages"], s["v_pages"], s["k_scale"], s["v_scale"],
                                     s["table"])
            if c["op"] != "append":
                s["ws"] = nsa.workspace(s["p"], nsa.OP_DECODE_Q8 if c["op"] == "decode"
                                        else nsa.OP_PREFILL_Q8)
        if c["op"] == "append":
            rows = nsa.nsa_append_q8(s["p"], s["k"], s["v"], s["pos"], s["cache"], cu_new=s["cu"],
                                     q=s["q"], rope=s["rope"], rope_style=c["style"], want_kv=True)
        elif c["op"] == "decode":
            return nsa.nsa_decode_q8(s["p"], s["q"], s["cache"], s["lens"], keys=c["keys"],
                                     sel_idx=s.get("sel"), ws=s["ws"])
        else:
            return nsa.nsa_prefill_q8(s["p"], s["q"], s["cache"], s["lens"], s["cu"],
                                      keys=c["keys"], ws=s["ws"])
    elif c["op"] == "append":
        rows = _append_plain(s)
    else:
        return _attend_plain(s)
    # the rows as stored, and the cache: its codes stand for code * scale
    return rows + (s["k_pages"], s["v_pages"], s["k_scale"], s["v_scale"])


# ---------------------------------------------------------------------------
# from the definition, in 64 bits
# ---------------------------------------------------------------------------

def exact(c, seed):
    def append(s):
        lens, new = _sizes(c)
        page, Hkv, dt = c["page"], c["Hkv"], torch.float64
        table, rope = s["table"].cpu(), s["rope"].to(dt)
        position = torch.cat([torch.arange(m - n, m) for m, n in zip(lens, new)]).to(rope.device)
        half = c["rot"] // 2
        first = torch.arange(half) if c["style"] == "half" else 2 * torch.arange(half)
        second = first + (half if c["style"] == "half" else 1)
        unit = torch.complex(rope[position, 0], rope[position, 1])[:, None]

        def turned(x):
            x = x.to(dt)
            z = torch.complex(x[..., first], x[..., second]) * unit
            x[..., first], x[..., second] = z.real, z.imag
            return x

        got = {"q": turned(s["q"])}
        for name, x in (("k", turned(s["k"])), ("v", s["v"].to(dt))):
            codes, scale = s[name + "_pages"].to(dt), s[name + "_scale"].to(dt)
            held = torch.empty_like(x)
            row = 0
            for b in range(c["B"]):
                at = lens[b] - new[b]
                while at < lens[b]:
                    j, slot = at // page, at % page
                    m = min(page - slot, lens[b] - at)
                    pid = int(table[b, j])
                    rows = x[row:row + m].transpose(0, 1)  # [Hkv, m, d]
                    biggest = rows.abs().amax(dim=(1, 2))
                    need = torch.exp2(torch.ceil(torch.log2(biggest / 448.0)).clamp(min=-126.0))
                    need = torch.where(biggest > 448.0 * need, 2 * need, need)
                    was = scale[pid]
                    now = need if slot == 0 else torch.maximum(was, need)
                    codes[pid] = (codes[pid] * (was / now)[:, None, None]).float().to(E4M3).to(dt)
                    put = (rows / now[:, None, None]).float().to(E4M3).to(dt)
                    codes[pid][:, slot:slot + m] = put
                    scale[pid] = now
                    held[row:row + m] = (put * now[:, None, None]).transpose(0, 1)
                    row, at = row + m, at + m
            got[name], got[name + "_pages"], got[name + "_scale"] = held, codes, scale
        return tuple(got[n] for n in ("q", "k", "v", "k_pages", "v_pages", "k_scale", "v_scale"))

    def attend(s):
        lens, new = _sizes(c)
        dt, page, d, Hkv = torch.float64, c["page"], c["d"], c["Hkv"]
        G = c["Hq"] // Hkv
        out = torch.zeros_like(s["q"], dtype=dt)
        lse = torch.full(s["q"].shape[:2], -math.inf, dtype=dt, device=s["q"].device)
        row = 0
        for b, (m, n) in enumerate(zip(lens, new)):
            rows, row = slice(row, row + n), row + n
            if m == 0:
                continue
            pid = s["table"][b, :-(-m // page)].long()
            position = torch.arange(m - n, m, device=out.device)
            key = torch.arange(m, device=out.device)
            for g in range(Hkv):
                k = s["k_pages"].view(torch.uint8)[pid, g].view(E4M3)
                v = s["v_pages"].view(torch.uint8)[pid, g].view(E4M3)
                k = (k.to(dt) * s["k_scale"][pid, g].to(dt)[:, None, None]).reshape(-1, d)[:m]
                v = (v.to(dt) * s["v_scale"][pid, g].to(dt)[:, None, None]).reshape(-1, d)[:m]
                hide = key[None] > position[:, None]
                if c["keys"] == "window":
                    hide = hide | (key[None] <= position[:, None] - c["window"])
                if c["keys"] == "blocks":
                    listed_ = s["sel"][b, g]
                    hide = hide | ~(key[:, None] // page == listed_[None]).any(1)[None]
                for h in range(g * G, (g + 1) * G):
                    z = s["q"][rows, h].to(dt) @ k.T / math.sqrt(d)
                    z = z.masked_fill(hide, -math.inf)
                    lse[rows, h] = torch.logsumexp(z, dim=1)
                    out[rows, h] = torch.softmax(z, dim=1).nan_to_num() @ v
        return out, lse

    s = prepare(c, seed)
    return append(s) if c["op"] == "append" else attend(s)
