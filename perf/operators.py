"""What is measured of the paged latent cache: the rotation, the append, the
read-back, and the two attentions that read the cache.

A latent row holds 512 latent dims and 64 rotary dims. A bf16 page stores
rows of 576 bf16 values; an e4m3 page stores rows of 656 bytes: 512 e4m3
codes, four fp32 scales (one per 128 dims, powers of two) and 64 bf16 values.
"""
import math
import random

import torch

own = False

LATENT, ROT, ROW = 512, 64, 576
GROUP, ROW_BYTES = 128, 656


# ---------------------------------------------------------------- cases
def listed():
    return [
        # one decode step's queries, 128 heads, rotary dims at the end of the head
        dict(name="rope_decode", op="rope", T=32, H=128, D=576, off=512, layout="interleaved", dtype="bf16", factor=1.0),
        # a prefill chunk's indexer queries: 64 of 128 dims in the half layout, a table scaled for 1M tokens
        dict(name="rope_prefill_half", op="rope", T=8192, H=64, D=128, off=0, layout="half", dtype="bf16", factor=8.0),
        # one decode step's tokens into e4m3 pages, two of them padding
        dict(name="append_decode_e4m3", op="append", T=32, page=64, pages=600, fp8=True, skip=2),
        # a long prefill chunk into e4m3 pages
        dict(name="append_prefill_e4m3", op="append", T=16384, page=64, pages=300, fp8=True, skip=0),
        # a short context read back from bf16 pages
        dict(name="read_short_bf16", op="read", B=3, len=1021, page=16, fp8=False),
        # a batch's cached contexts expanded for a chunked prefill
        dict(name="read_long_e4m3", op="read", B=16, len=8192, page=64, fp8=True),
        # the smallest decode: one sequence, few heads, a short context
        dict(name="decode_small_bf16", op="decode", B=1, Q=1, H=8, len=200, page=16, fp8=False, gate=False),
        # a ragged decode batch at the model's 128 heads, idle slots among it
        dict(name="decode_batch_bf16", op="decode", B=32, Q=1, H=128, len=8192, page=64, fp8=False, gate=True),
        # the same batch with e4m3 pages
        dict(name="decode_batch_e4m3", op="decode", B=32, Q=1, H=128, len=8192, page=64, fp8=True, gate=True),
        # few long sequences, heads split over eight devices, one draft token
        dict(name="decode_long_e4m3", op="decode", B=4, Q=2, H=16, len=131071, page=128, fp8=True, gate=False),
        # one query's 256 selected rows, few heads
        dict(name="sparse_small_e4m3", op="sparse", B=1, H=8, k=256, page=64, pages=64, gate=False),
        # the decode step's 2048 selected rows per query at 128 heads
        dict(name="sparse_batch_e4m3", op="sparse", B=32, H=128, k=2048, page=64, pages=2048, gate=True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rope", "append", "read", "decode", "decode", "sparse"])
    page = rng.choice([16, 32, 64, 128])
    if op == "rope":
        H = _log(rng, 1, 128)
        D = rng.choice([64, 128, 192, 576])
        return dict(op="rope", T=_log(rng, 1, max(1, min(8192, 67108864 // (H * D)))), H=H, D=D,
                    off=rng.choice([0, D - 64]), layout=rng.choice(["interleaved", "half"]),
                    dtype=rng.choice(["bf16", "bf16", "f32"]), factor=rng.choice([1.0, 8.0, 40.0]))
    if op == "append":
        T = _log(rng, 1, 16384)
        return dict(op="append", T=T, page=page, pages=T // page + 1 + rng.randint(1, 40), fp8=rng.random() < 0.7,
                    skip=rng.randint(0, min(3, T - 1)))
    if op == "read":
        B = _log(rng, 1, 16)
        return dict(op="read", B=B, len=_log(rng, 1, 8192), page=page, fp8=rng.random() < 0.7)
    if op == "decode":
        B, H = _log(rng, 1, 48), _log(rng, 1, 128)
        Q = rng.choice([1, 1, 1, 2, 4])
        most = min(131071, 32 * 8192 * 128 // (B * max(64, H * Q)))
        return dict(op="decode", B=B, Q=Q, H=H, len=_log(rng, Q, most), page=page, fp8=rng.random() < 0.5,
                    gate=rng.random() < 0.5)
    B = _log(rng, 1, 32)
    k = _log(rng, 1, 2048)
    return dict(op="sparse", B=B, H=_log(rng, 1, 128), k=k, page=page, pages=k // page + 1 + rng.randint(1, 1000),
                gate=rng.random() < 0.5)


def _lengths(case):
    """Context lengths of the case's sequences: the longest, an idle slot (0), a first token, the rest spread."""
    r = random.Random(case["B"] * 1000003 + case["len"])
    Q = case.get("Q", 1)
    fixed = [case["len"], 0, Q]
    return [fixed[b] if b < 3 else r.randint(max(Q, case["len"] // 2), case["len"]) for b in range(case["B"])]


def work(case):
    op = case["op"]
    row = ROW_BYTES if case.get("fp8", True) else ROW * 2
    if op == "rope":
        n = case["T"] * case["H"] * case["D"] * (2 if case["dtype"] == "bf16" else 4)
        return dict(bytes=2 * n + case["T"] * 8 + ROT * 4, flops=case["T"] * case["H"] * ROT * 3)
    if op == "append":
        T = case["T"] - case["skip"]
        return dict(bytes=T * (ROW * 2 + row) + case["T"] * 16, flops=T * ROW * 3)
    if op == "read":
        n = sum(_lengths(case))
        return dict(bytes=n * (row + ROW * 2), flops=n * LATENT)
    if op == "decode":
        rows, n = case["B"] * case["Q"] * case["H"], sum(_lengths(case))
        b = n * row + rows * (ROW * 2 + LATENT * 2 + 4 + (LATENT * 2 if case["gate"] else 0))
        return dict(bytes=b, flops=2 * case["Q"] * case["H"] * n * (ROW + LATENT))
    rows = case["B"] * case["H"]
    total = case["pages"] * case["page"]
    seen = total * (1 - (1 - min(1.0, case["k"] / total)) ** case["B"])  # distinct rows of random selections
    b = seen * row + case["B"] * case["k"] * 4 + rows * (ROW * 2 + LATENT * 2 + 4 + (LATENT * 2 if case["gate"] else 0))
    return dict(bytes=int(b), flops=2 * rows * case["k"] * (ROW + LATENT))


# ---------------------------------------------------------------- inputs
def _frequencies(factor, device):
    """64-bit rotary frequencies; factor > 1: the low ones divided by it, a ramp between (long contexts)."""
    i = torch.arange(ROT // 2, dtype=torch.float64, device=device)
    f = 10000.0 ** (-2.0 * i / ROT)
    if factor > 1:
        ramp = ((i - 10.0) / 13.0).clamp(0, 1)
        f = f * (1 - ramp) + f / factor * ramp
    return f


def _scales(y):
    """The power-of-two scale of each group of 128: the least 2^e >= amax / 448 (1 for an all-zero group)."""
    amax = y.abs().amax(dim=-1)
    m, e = torch.frexp(amax)
    e = e - 9 + (m > 0.875).to(e.dtype)
    s = torch.ldexp(torch.ones_like(amax), e.clamp(min=-100))
    return torch.where(amax > 0, s, torch.ones_like(s))


def _pack(rows):
    """fp32 latent rows [R, 576] -> e4m3 row bytes [R, 656]."""
    y = rows[:, :LATENT].reshape(-1, LATENT // GROUP, GROUP)
    s = _scales(y)
    codes = (y / s[..., None]).to(torch.float8_e4m3fn).view(torch.uint8).reshape(-1, LATENT)
    rot = rows[:, LATENT:].to(torch.bfloat16).contiguous().view(torch.uint8)
    return torch.cat([codes, s.contiguous().view(torch.uint8), rot], dim=1)


def _unpack(b):
    """e4m3 row bytes [..., 656] -> fp32 latent rows [..., 576]."""
    codes = b[..., :LATENT].view(torch.float8_e4m3fn).float()
    s = b[..., LATENT:LATENT + 16].contiguous().view(torch.float32)
    rot = b[..., LATENT + 16:].contiguous().view(torch.bfloat16).float()
    lat = codes.unflatten(-1, (LATENT // GROUP, GROUP)) * s[..., None]
    return torch.cat([lat.flatten(-2), rot], dim=-1)


def _pool(pages, page, fp8, g):
    """A cache whose every row holds a token: latent values after a norm, tokens of unlike size."""
    n = pages * page
    x = torch.randn(n, ROW, generator=g, device="cuda")
    x *= 0.5 + torch.rand(n, 1, generator=g, device="cuda")
    x = x.to(torch.bfloat16)
    return (_pack(x.float()) if fp8 else x).view(pages, page, -1)


def prepare(case, seed):
    st = _inputs(case, seed)
    if own and case["op"] != "rope":
        # a serving loop keeps one workspace for its calls
        from lightning_indexer_cross_b200 import ops
        need = 256
        if case["op"] == "decode":
            need = ops.latent_decode_workspace_size(case["B"], case["Q"], case["H"], st["table"].shape[1] * case["page"])
        if case["op"] == "sparse":
            need = ops.latent_sparse_workspace_size(case["B"], case["H"], case["k"])
        st["ws"] = ops.new_workspace(need, "cuda")
    return st


def _inputs(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    op, st = case["op"], dict(case)

    def randn(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    if op == "rope":
        dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
        st["x"] = randn(case["T"], case["H"], case["D"]).to(dt)
        st["pos"] = torch.randint(0, 1 << 20, (case["T"],), generator=g, device="cuda")
        st["freq"] = _frequencies(case["factor"], "cuda")
        st["mscale"] = 0.1 * math.log(case["factor"]) + 1.0
        return st
    if op == "append":
        st["cache"] = _pool(case["pages"], case["page"], case["fp8"], g)
        n = case["pages"] * case["page"]
        slots = torch.randperm(n, generator=g, device="cuda")[:case["T"]]
        slots[case["T"] - case["skip"]:] = -1  # padding at the end of the batch
        st["slots"] = slots
        st["pos"] = torch.randint(0, 1 << 20, (case["T"],), generator=g, device="cuda")
        st["kv"] = randn(case["T"], ROW).to(torch.bfloat16)
        st["freq"] = _frequencies(1.0, "cuda")
        return st
    if op == "sparse":
        st["cache"] = _pool(case["pages"], case["page"], True, g)
        n = case["pages"] * case["page"]
        pick = torch.rand(case["B"], n, generator=g, device="cuda").argsort(dim=1)[:, :case["k"]]
        pick = pick.to(torch.int32).contiguous()
        if case["B"] > 1:
            pick[1, case["k"] // 2:] = -1  # a context shorter than the selection
        st["slots"] = pick
        st["q"] = randn(case["B"], case["H"], ROW).to(torch.bfloat16)
    else:
        lens = _lengths(case)
        need = [-(-n // case["page"]) for n in lens]
        width = max(1, max(need))
        pages = sum(need) + 3
        st["cache"] = _pool(pages, case["page"], case["fp8"], g)
        perm = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
        table = torch.zeros(case["B"], width, dtype=torch.int32, device="cuda")
        at = 0
        for b, n in enumerate(need):
            table[b, :n] = perm[at:at + n]
            at += n
        st["table"] = table
        if op == "read":
            cu = [0]
            for n in lens:
                cu.append(cu[-1] + n)
            st["cu"] = torch.tensor(cu, dtype=torch.int64, device="cuda")
            st["out"] = randn(cu[-1] + 5, ROW).to(torch.bfloat16)  # five rows behind the last sequence
            return st
        st["lens"] = torch.tensor(lens, dtype=torch.int64, device="cuda")
        st["q"] = randn(case["B"], case["Q"], case["H"], ROW).to(torch.bfloat16)
    st["sink"] = randn(case["H"]) * 0.5
    st["gate"] = randn(*st["q"].shape[:-1], LATENT).to(torch.bfloat16) if case["gate"] else None
    return st


# ---------------------------------------------------------------- one pass
def _rotate(x, pos, freq, layout, mscale):
    """fp32 x [..., 64] with pos broadcastable to its leading dims; angles in 64 bits."""
    a = pos.double()[..., None] * freq
    c, s = (a.cos() * mscale).float(), (a.sin() * mscale).float()
    if layout == "half":
        u, v = x[..., :ROT // 2], x[..., ROT // 2:]
        return torch.cat([u * c - v * s, u * s + v * c], dim=-1)
    u, v = x[..., 0::2], x[..., 1::2]
    return torch.stack([u * c - v * s, u * s + v * c], dim=-1).flatten(-2)


def _attend(q, kv, valid, sink, gate, sm_scale):
    """q [B, R, 576] fp32 rows, kv [B, N, 576] fp32, valid [B, R, N] or [B, 1, N]; sink [R], gate [B, R, 512] or None."""
    z = torch.bmm(q, kv.transpose(1, 2)) * sm_scale
    z = z.masked_fill(~valid, float("-inf"))
    m = torch.maximum(z.amax(dim=-1), sink)
    p = torch.exp(z - m[..., None])
    den = p.sum(dim=-1) + torch.exp(sink - m)
    o = torch.bmm(p, kv[..., :LATENT]) / den[..., None]
    if gate is not None:
        o = o * torch.sigmoid(gate.float())
    return o, m + torch.log(den)


def _views(cache, fp8):
    """The cache's parts as the values they stand for, without a copy."""
    if not fp8:
        return cache
    return (cache[..., :LATENT].view(torch.float8_e4m3fn), cache[..., LATENT:LATENT + 16].view(torch.float32),
            cache[..., LATENT + 16:].view(torch.bfloat16))


def run(st):
    op = st["op"]
    if own:
        from lightning_indexer_cross_b200 import ops
        ws = st.get("ws")
        if op == "rope":
            return ops.rope(st["x"], st["pos"], st["freq"], rot_off=st["off"], layout=st["layout"],
                            mscale=st["mscale"])
        if op == "append":
            ops.latent_append(st["kv"], st["slots"], st["cache"], pos=st["pos"], freq=st["freq"], workspace=ws)
            return _views(st["cache"], st["fp8"])
        if op == "read":
            return ops.latent_read(st["cache"], st["table"], st["cu"], st["out"], workspace=ws)
        if op == "decode":
            return ops.latent_decode(st["q"], st["cache"], st["table"], st["lens"], sink=st["sink"], gate=st["gate"],
                                     workspace=ws)
        return ops.latent_sparse_decode(st["q"], st["cache"], st["slots"], sink=st["sink"], gate=st["gate"],
                                        workspace=ws)
    if op == "rope":
        x, off = st["x"], st["off"]
        y = _rotate(x[..., off:off + ROT].float(), st["pos"][:, None], st["freq"], st["layout"], st["mscale"])
        return torch.cat([x[..., :off], y.to(x.dtype), x[..., off + ROT:]], dim=-1)
    if op == "append":
        keep = st["slots"] >= 0
        x = st["kv"][keep].float()
        x = torch.cat([x[:, :LATENT], _rotate(x[:, LATENT:], st["pos"][keep], st["freq"], "interleaved", 1.0)], dim=1)
        flat = st["cache"].view(-1, st["cache"].shape[-1])
        flat[st["slots"][keep]] = _pack(x) if st["fp8"] else x.to(torch.bfloat16)
        return _views(st["cache"], st["fp8"])
    flat = st["cache"].view(-1, st["cache"].shape[-1])
    if op == "read":
        rows, cu = st["out"].shape[0], st["cu"]
        r = torch.arange(rows, device="cuda")
        b = (torch.searchsorted(cu, r, right=True) - 1).clamp(max=st["table"].shape[0] - 1)
        p = r - cu[b]
        inside = r < cu[-1]
        p = torch.where(inside, p, torch.zeros_like(p))
        src = flat[st["table"][b, p // st["page"]].long() * st["page"] + p % st["page"]]
        got = (_unpack(src) if st["fp8"] else src).to(torch.bfloat16)
        st["out"].copy_(torch.where(inside[:, None], got, st["out"]))
        return st["out"]
    if op == "decode":
        B, Q, H, _ = st["q"].shape
        p = torch.arange(st["table"].shape[1] * st["page"], device="cuda")
        rows = st["table"][:, p // st["page"]].long() * st["page"] + p % st["page"]
        kv = flat[rows]
        kv = _unpack(kv) if st["fp8"] else kv.float()
        # token j of Q sees the positions before len - (Q - 1 - j)
        last = st["lens"][:, None] - (Q - 1 - torch.arange(Q, device="cuda"))
        valid = (p < last[..., None]).repeat_interleave(H, dim=1)
        gate = None if st["gate"] is None else st["gate"].view(B, Q * H, LATENT)
        o, lse = _attend(st["q"].view(B, Q * H, ROW).float(), kv, valid, st["sink"].repeat(Q), gate, ROW ** -0.5)
        return o.to(torch.bfloat16).view(B, Q, H, LATENT), lse.view(B, Q, H)
    at = st["slots"].long()
    kv = _unpack(flat[at.clamp(min=0)])
    o, lse = _attend(st["q"].float(), kv, (at >= 0)[:, None], st["sink"], st["gate"], ROW ** -0.5)
    return o.to(torch.bfloat16), lse


# ---------------------------------------------------------------- the definition in 64 bits
def exact(case, seed):
    st = _inputs(case, seed)
    op = case["op"]

    def turn(x, pos, layout, mscale):
        # x + iy -> (x + iy) e^{i pos freq}
        half = ROT // 2
        z = torch.complex(x[..., :half], x[..., half:]) if layout == "half" else \
            torch.complex(x[..., 0::2].contiguous(), x[..., 1::2].contiguous())
        z = z * torch.polar(torch.full_like(st["freq"], mscale).expand(*pos.shape, -1).contiguous(),
                            pos.double()[..., None] * st["freq"])
        return torch.cat([z.real, z.imag], dim=-1) if layout == "half" else \
            torch.stack([z.real, z.imag], dim=-1).reshape(x.shape)

    def decode(b):
        if not case.get("fp8", True):
            return b.double()
        c = b[:, :LATENT].to(torch.int64)
        e, f = (c >> 3) & 15, (c & 7).double()
        v = torch.where(e > 0, (1 + f / 8) * torch.exp2((e - 7).double()), f / 512)
        v = torch.where(c >= 128, -v, v)
        s = b[:, LATENT:LATENT + 16].contiguous().view(torch.float32).double()
        return torch.cat([v * s.repeat_interleave(GROUP, dim=1),
                          b[:, LATENT + 16:].contiguous().view(torch.bfloat16).double()], dim=1)

    if op == "rope":
        y = st["x"].double()
        off = case["off"]
        y[..., off:off + ROT] = turn(y[..., off:off + ROT].clone(), st["pos"][:, None], case["layout"], st["mscale"])
        return y
    flat = st["cache"].view(-1, st["cache"].shape[-1])
    if op == "append":
        T = case["T"] - case["skip"]
        at = st["slots"][:T]
        x = st["kv"][:T].double()
        rot = turn(x[:, LATENT:].clone(), st["pos"][:T], "interleaved", 1.0)
        if not case["fp8"]:
            all_rows = flat.double()
            all_rows[at] = torch.cat([x[:, :LATENT], rot], dim=1)
            return all_rows.view(st["cache"].shape)
        parts = [v.reshape(-1, v.shape[-1]).double() for v in _views(st["cache"], True)]
        y = x[:, :LATENT].reshape(T, LATENT // GROUP, GROUP)
        amax = y.abs().amax(dim=-1)
        s = torch.exp2(torch.ceil(torch.log2(amax / 448)))
        v = y / s[..., None]
        step = torch.exp2(torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6))) - 3)
        v = torch.round(v / step) * step
        for part, new in zip(parts, (v.reshape(T, LATENT), s, rot)):
            part[at] = new
        return tuple(p.view(*st["cache"].shape[:2], -1) for p in parts)
    if op == "read":
        out = st["out"].double()
        lens = _lengths(case)
        at = 0
        for b, n in enumerate(lens):
            p = torch.arange(n, device="cuda")
            src = flat[st["table"][b].long()[p // case["page"]] * case["page"] + p % case["page"]]
            out[at:at + n] = decode(src)
            at += n
        return out
    B, H = case["B"], case["H"]
    Q = case.get("Q", 1)
    outs, lses = [], []
    for b in range(B):
        if op == "decode":
            n = int(st["lens"][b])
            p = torch.arange(n, device="cuda")
            at = st["table"][b].long()[p // case["page"]] * case["page"] + p % case["page"]
        else:
            at = st["slots"][b].long()
            at = at[at >= 0]
            n = at.numel()
        kv = decode(flat[at])
        for j in range(Q):
            seen = kv[:max(0, n - (Q - 1 - j))]
            q = (st["q"][b, j] if op == "decode" else st["q"][b]).double()
            z = torch.cat([st["sink"].double()[:, None], q @ seen.T / math.sqrt(ROW)], dim=1)
            lse = torch.logsumexp(z, dim=1)
            o = torch.exp(z[:, 1:] - lse[:, None]) @ seen[:, :LATENT]
            if st["gate"] is not None:
                o = o / (1 + torch.exp(-(st["gate"][b, j] if op == "decode" else st["gate"][b]).double()))
            outs.append(o)
            lses.append(lse)
    shape = (B, Q, H) if op == "decode" else (B, H)
    return torch.stack(outs).view(*shape, LATENT), torch.stack(lses).view(shape)
