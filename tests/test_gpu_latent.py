"""GPU parity of the paged latent cache (ic_rope, ic_latent_append,
ic_latent_read, ic_latent_decode, ic_latent_sparse_decode) against the float64
oracle.

Tolerances, from the arithmetic (u = half a step of the stored type: 2^-8 for
bf16, 2^-24 for fp32, relative to the value):
  rotation   The reduced angle is rounded to 32 bits (at most pi 2^-24) and its
             sine and cosine are off by at most 2 units of 2^-24, so each is off
             by less than 2^-21; with the three 32-bit roundings of u c - v s the
             result is off by at most 2^-20 mscale (|u| + |v|), plus u |y|.
  e4m3 rows  codes and scales are exact; the read-back is exact.
  attention  36 MMA steps of 16 dims, each off by at most two steps of 2^-23 of
             what the running sum can reach (sum |q k|), put a logit off by
             dz < 2^-16 reach; the exponent's argument and ex2 add 2^-20 (1 +
             reach). A weight is rounded to bf16 (2^-8 of it), the n / 16
             accumulation steps add n 2^-26, the gate's sigmoid 2^-20. So
             |out - exact| <= mass (2^-8 + 2 dz' + n 2^-26 + 2^-20) + u |exact|,
             dz' = 2^-16 reach + 2^-20 (1 + reach), and
             |lse - exact| <= 2 dz' + 2^-20 (1 + |lse|).
"""
import numpy as np
import pytest
import torch

from oracle import latent_oracle as L

pytestmark = pytest.mark.gpu

U = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


@pytest.fixture(scope="module")
def ops(cuda_dev):
    from lightning_indexer_cross_b200 import ops
    return ops


def f64(t):
    return t.detach().cpu().double().numpy()


def status_of(ops, ws):
    from lightning_indexer_cross_b200 import _abi
    return _abi.ic_last_device_status(ops._ptr(ws), ops._stream_ptr())


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def check_rotation(got, x, pos, freq, off, layout, mscale=1.0, transpose=False):
    want = L.rope(x, pos.cpu().numpy(), f64(freq), off, layout, mscale, transpose)
    n, u = freq.numel(), U[got.dtype]
    xf, g = np.abs(f64(x)), f64(got)
    a = np.arange(n) * (2 if layout == "interleaved" else 1) + off
    b = a + (1 if layout == "interleaved" else n)
    lim = np.zeros_like(g)
    lim[..., a] = lim[..., b] = 2.0 ** -20 * mscale * (xf[..., a] + xf[..., b])
    lim[..., a] += u * np.abs(want[..., a]) * 1.001
    lim[..., b] += u * np.abs(want[..., b]) * 1.001
    assert np.all(np.abs(g - want) <= lim), np.abs(g - want).max()  # other dims: bit for bit


# ---------------------------------------------------------------- rotation
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("layout", ["interleaved", "half"])
@pytest.mark.parametrize("T,H,D,off,rot", [(1, 1, 64, 0, 64), (3, 5, 576, 512, 64), (37, 2, 128, 0, 64), (5, 3, 96, 16, 32),
                                           (7, 3, 67, 1, 66), (2, 130, 10, 3, 6), (700, 1, 64, 0, 64), (3, 2, 1024, 0, 1024)])
def test_rope(ops, dtype, layout, T, H, D, off, rot):
    g = gen(T * D)
    x = torch.randn(T, H, D, generator=g, device="cuda").to(dtype)
    pos = torch.randint(0, 1 << 20, (T,), generator=g, device="cuda")
    pos[0] = 0
    freq, _ = ops.rope_frequencies(rot)
    y = ops.rope(x, pos, freq, rot_off=off, layout=layout, mscale=1.25)
    check_rotation(y, x, pos, freq, off, layout, 1.25)
    z = ops.rope(x, pos, freq, rot_off=off, layout=layout, mscale=1.25, transpose=True)
    check_rotation(z, x, pos, freq, off, layout, 1.25, transpose=True)
    w = x.clone()
    assert ops.rope(w, pos, freq, rot_off=off, layout=layout, mscale=1.25, out=w) is w
    assert torch.equal(w, y)


@pytest.mark.parametrize("layout", ["interleaved", "half"])
def test_rope_strided_and_far_positions(ops, layout):
    g = gen(5)
    freq, m = ops.rope_frequencies(64, 10000.0, {"type": "yarn", "factor": 40, "original_length": 4096})
    pos = torch.tensor([-3, (1 << 31) + 5, 1 << 40, 0, 999983, -(1 << 33)], device="cuda")
    wide = torch.randn(6, 3 * 200 + 40, generator=g, device="cuda").to(torch.bfloat16)
    views = [wide[:, 8:608].view(6, 3, 200),                         # part of a wider projection
             wide[:, 3:603].view(6, 3, 200),                         # the same, unaligned
             torch.randn(3, 6, 200, generator=g, device="cuda").to(torch.bfloat16).transpose(0, 1),  # heads first
             wide[:, :200].unsqueeze(1).expand(6, 3, 200)]           # heads that share one row
    for x in views:
        y = ops.rope(x, pos, freq, rot_off=72, layout=layout, mscale=m)
        check_rotation(y, x, pos, freq, 72, layout, m)
    out = torch.zeros(3, 6, 200, dtype=torch.bfloat16, device="cuda")
    ops.rope(views[0], pos, freq, rot_off=72, layout=layout, mscale=m, out=out.transpose(0, 1))
    assert torch.equal(out.transpose(0, 1), ops.rope(views[0], pos, freq, rot_off=72, layout=layout, mscale=m))


def test_rope_rotates_in_place_a_part_of_a_wider_tensor(ops):
    g = gen(6)
    freq, _ = ops.rope_frequencies(64)
    whole = torch.randn(9, 4, 192, generator=g, device="cuda").to(torch.bfloat16)
    pos = torch.arange(9, device="cuda")
    want = ops.rope(whole, pos, freq, rot_off=128)
    part = whole[..., 128:]
    ops.rope(part, pos, freq, out=part)
    assert torch.equal(whole, want)
    assert ops.rope(whole[:0], pos[:0], freq).shape == (0, 4, 192)


def test_rope_refuses(ops):
    freq, _ = ops.rope_frequencies(64)
    x = torch.zeros(4, 2, 128, dtype=torch.bfloat16, device="cuda")
    pos = torch.zeros(4, dtype=torch.int64, device="cuda")
    bad = [dict(pos=pos.int()), dict(pos=pos[:3]), dict(freq=freq.float()), dict(rot_off=65), dict(rot_off=-1),
           dict(layout="other"), dict(x=x.half()), dict(x=x[..., ::2]), dict(x=x[0]), dict(pos=pos.cpu()),
           dict(out=torch.zeros(4, 1, 128, dtype=torch.bfloat16, device="cuda").expand(4, 2, 128)),
           dict(out=x.float())]
    for kw in bad:
        args = dict(x=x, pos=pos, freq=freq)
        args.update(kw)
        with pytest.raises((ValueError, RuntimeError)):
            ops.rope(**args)


# ---------------------------------------------------------------- append and read-back
def parts(cache):
    return cache[..., :512], cache[..., 512:528].contiguous().view(torch.float32), \
        cache[..., 528:].contiguous().view(torch.bfloat16)


@pytest.mark.parametrize("layout", ["interleaved", "half"])
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("T,page,pages", [(1, 16, 1), (9, 32, 5), (100, 48, 4), (333, 64, 7)])
def test_append(ops, layout, fp8, T, page, pages):
    g = gen(T)
    cache = ops.new_latent_cache(pages, page, fp8)
    cache.view(torch.uint8).random_(generator=g)
    before = cache.clone()
    wide = torch.randn(T, 600, generator=g, device="cuda").to(torch.bfloat16)
    kv = wide[:, 16:592]
    kv[0, :128] = 0
    if T > 3:
        kv[1] *= 1e-30
        kv[2, 3], kv[2, 200], kv[2, 300] = float("inf"), float("nan"), float("-inf")
        kv[3] *= 1e30
    slots = torch.randperm(pages * page, generator=g, device="cuda")[:T]
    if T > 5:
        slots[4] = -1
    pos = torch.randint(0, 1 << 20, (T,), generator=g, device="cuda")
    freq, _ = ops.rope_frequencies(64)
    ws = ops.latent_append(kv, slots, cache, pos=pos, freq=freq, layout=layout)
    assert status_of(ops, ws) == 0
    keep = slots >= 0
    at = slots[keep]
    mask = torch.ones(pages * page, dtype=torch.bool, device="cuda")
    mask[at] = False
    flat, old = cache.view(torch.uint8).view(pages * page, -1), before.view(torch.uint8).view(pages * page, -1)
    assert torch.equal(flat[mask], old[mask])
    rows = cache.view(pages * page, -1)[at]
    x = kv[keep]
    rot = rows[:, 512:] if not fp8 else parts(rows)[2]
    check_rotation(rot[:, None], x[:, None, 512:], pos[keep], freq, 0, layout)
    if not fp8:
        assert torch.equal(rows[:, :512].contiguous().view(torch.int16), x[:, :512].contiguous().view(torch.int16))
        return
    codes, scale, _ = parts(rows)
    xc = x.cpu().double()
    xc = torch.where(torch.isinf(xc), torch.sign(xc) * 1e300, xc)  # stored as +-448 scale
    want_s = L.pow2_scale(f64(x)[:, :512].reshape(-1, 4, 128))
    assert np.array_equal(f64(scale), want_s)
    q = np.clip(xc[:, :512].numpy() / np.repeat(want_s, 128, axis=1), -448, 448)
    nan = np.isnan(q)
    got = codes.cpu().numpy()
    from oracle.cache_append_oracle import encode_e4m3
    want = encode_e4m3(np.where(nan, 0.0, q))
    same = (got == want) | ((got & 0x7f == 0) & (want & 0x7f == 0))
    assert np.all(same[~nan]) and np.all((got & 0x7f)[nan] == 0x7f)


def test_append_without_rotation_and_into_spaced_pages(ops):
    g = gen(3)
    for fp8 in (False, True):
        big = ops.new_latent_cache(5, 40, fp8)
        big.view(torch.uint8).random_(generator=g)
        cache = big[:, :32]  # pages 40 rows apart
        before = big.clone()
        kv = torch.randn(4, 576, generator=g, device="cuda").to(torch.bfloat16)
        slots = torch.tensor([0, 4 * 32 + 31, 32, 95], device="cuda")
        ws = ops.latent_append(kv, slots, cache)
        assert status_of(ops, ws) == 0
        got = cache[slots // 32, slots % 32]
        rot = parts(got)[2] if fp8 else got[:, 512:]
        assert torch.equal(rot, kv[:, 512:])
        before[:, :32][slots // 32, slots % 32] = got
        assert torch.equal(big.view(torch.uint8), before.view(torch.uint8))


def test_append_records_slots_outside(ops):
    from lightning_indexer_cross_b200 import _abi
    cache = ops.new_latent_cache(2, 16, True)
    kv = torch.ones(3, 576, dtype=torch.bfloat16, device="cuda")
    for bad in (32, -2, 1 << 40, -(1 << 62)):
        cache.zero_()
        ws = ops.latent_append(kv, torch.tensor([bad, 5, -1], device="cuda"), cache)
        assert status_of(ops, ws) == _abi.IC_ERR_BAD_INDEX
        assert cache[0, 5].any() and not cache[0, :5].any() and not cache[0, 6:].any() and not cache[1].any()
    with pytest.raises(ValueError):
        ops.latent_append(kv, torch.zeros(3, dtype=torch.int32, device="cuda"), cache)
    with pytest.raises(ValueError):
        ops.latent_append(kv, torch.zeros(3, dtype=torch.int64, device="cuda"), cache, pos=torch.zeros(3, dtype=torch.int64, device="cuda"))
    with pytest.raises(RuntimeError):
        ops.latent_append(kv, torch.zeros(3, dtype=torch.int64, device="cuda"), ops.new_latent_cache(2, 24, True))
    assert ops.latent_append(kv[:0], torch.zeros(0, dtype=torch.int64, device="cuda"), cache).numel() >= 4


def random_cache(ops, pages, page, fp8, g):
    cache = ops.new_latent_cache(pages, page, fp8)
    n = pages * page
    x = torch.randn(n, 576, generator=g, device="cuda") * (0.5 + torch.rand(n, 1, generator=g, device="cuda"))
    ops.latent_append(x.to(torch.bfloat16), torch.arange(n, device="cuda"), cache)
    return cache


def paged(lens, page, g, spare=3, extra=2):
    """(block table, pages): the sequences' pages in random order; entries behind a sequence's last page are invalid."""
    need = [-(-max(n, 0) // page) for n in lens]
    pages = sum(need) + spare
    perm = torch.randperm(pages, generator=g, device="cuda").int()
    table = torch.full((len(lens), max(need) + extra), -7, dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = perm[at:at + n]
        at += n
    return table, pages


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("lens,page", [([1], 16), ([0, 5, 0, 33, 1], 16), ([100, 0, 64], 64), ([17] * 40, 32), ([0, 0], 16)])
def test_read(ops, fp8, lens, page):
    g = gen(len(lens))
    table, pages = paged(lens, page, g)
    cache = random_cache(ops, pages, page, fp8, g)
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    out = torch.randn(cu[-1] + 6, 576, generator=g, device="cuda").to(torch.bfloat16)
    want = f64(out)
    rows = L.cache_rows(cache)
    for b, n in enumerate(lens):
        p = np.arange(n)
        want[cu[b]:cu[b + 1]] = rows[f64(table)[b].astype(int)[p // page] * page + p % page]
    ws = ops.new_workspace(256, "cuda")
    ops.latent_read(cache, table, torch.tensor(cu, device="cuda"), out, workspace=ws)
    assert status_of(ops, ws) == 0
    assert np.array_equal(f64(out), want)


def test_read_records_bad_pages_and_lengths(ops):
    from lightning_indexer_cross_b200 import _abi
    g = gen(1)
    cache = random_cache(ops, 3, 16, True, g)
    rows = L.cache_rows(cache)
    table = torch.tensor([[2, 3], [1, -1]], dtype=torch.int32, device="cuda")
    out = torch.full((50, 576), 7.0, dtype=torch.bfloat16, device="cuda")
    ws = ops.new_workspace(256, "cuda")
    ops.latent_read(cache, table, torch.tensor([0, 20, 30], device="cuda"), out, workspace=ws)
    assert status_of(ops, ws) == _abi.IC_ERR_BAD_INDEX
    o = f64(out)
    assert np.array_equal(o[:16], rows[32:48]) and not o[16:20].any()
    assert np.array_equal(o[20:30], rows[16:26]) and np.all(o[30:] == 7)
    guard = torch.full((40, 576), 7.0, dtype=torch.bfloat16, device="cuda")
    ws.zero_()
    ops.latent_read(cache, table[1:], torch.tensor([0, 64], device="cuda"), guard[:20], workspace=ws)  # cu past out and table
    assert status_of(ops, ws) == _abi.IC_ERR_BAD_INDEX
    o = f64(guard)
    assert np.array_equal(o[:16], rows[16:32]) and not o[16:20].any() and np.all(o[20:] == 7)


def test_read_rounds_foreign_scales(ops):
    """Scales that are no power of two: code * scale, rounded once to bf16."""
    g = gen(2)
    cache = random_cache(ops, 1, 16, True, g)
    cache[..., 512:528] = (torch.rand(1, 16, 4, generator=g, device="cuda") + 0.1).view(torch.uint8)
    out = torch.zeros(16, 576, dtype=torch.bfloat16, device="cuda")
    ops.latent_read(cache, torch.zeros(1, 1, dtype=torch.int32, device="cuda"), torch.tensor([0, 16], device="cuda"), out)
    want = torch.from_numpy(L.cache_rows(cache).astype(np.float32)).to(torch.bfloat16)  # an exact product in 32 bits
    assert torch.equal(out.cpu(), want)


# ---------------------------------------------------------------- attention
def check_attention(out, lse, want, n, sum_u=0.0):
    o, s, mass, reach = want
    g, u = f64(out), U[out.dtype]
    dz = 2.0 ** -16 * reach + 2.0 ** -20 * (1 + reach)
    lim = mass * (2.0 ** -8 + 2 * dz[..., None] + n * 2.0 ** -26 + 2.0 ** -20) + u * np.abs(o)
    err = np.abs(g - o)
    assert np.all(err <= lim), (err.max(), (err / np.maximum(lim, 1e-300)).max())
    if lse is not None:
        ls = f64(lse)
        none = np.isneginf(s)
        assert np.array_equal(none, np.isneginf(ls))
        d = np.abs(np.where(none, 0, ls) - np.where(none, 0, s))
        assert np.all(d <= sum_u + 2 * dz + 2.0 ** -20 * (1 + np.abs(np.where(none, 0, s)))), d.max()


def queries(shape, g):
    return torch.randn(*shape, 576, generator=g, device="cuda").to(torch.bfloat16)


DECODE = [
    # lens, Q, H, page
    ([1], 1, 1, 16), ([0], 1, 3, 16), ([63], 1, 64, 16), ([64], 1, 8, 64), ([65, 0, 1], 1, 65, 32),
    ([200, 131, 7, 0, 64], 1, 128, 48), ([300, 2, 1, 0], 4, 5, 16), ([1000, 513], 2, 128, 64),
    ([5000], 1, 16, 128), ([4097, 1], 3, 33, 64), ([130] * 70, 1, 16, 16),
    # a dozen tiles and more in every share, and shares that pass from one sequence to the next, and over a short one
    ([61000, 0, 70, 64064], 1, 4, 64), ([9000, 3, 11111], 2, 64, 32), ([640] * 300, 1, 2, 16),
]


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("lens,Q,H,page", DECODE)
def test_decode(ops, fp8, lens, Q, H, page):
    g = gen(sum(lens) + H)
    B = len(lens)
    table, pages = paged(lens, page, g)
    cache = random_cache(ops, pages, page, fp8, g)
    q = queries((B, Q, H), g)
    ln = torch.tensor(lens, device="cuda")
    # rows behind a sequence's end hold anything
    for b, n in enumerate(lens):
        if n % page:
            cache.view(torch.uint8)[table[b, n // page].long(), n % page:] = 0xff  # NaN codes, scales and values
    sink = torch.randn(H, generator=g, device="cuda")
    gate = torch.randn(B, Q, H, 512, generator=g, device="cuda").to(torch.bfloat16)
    clean = torch.nan_to_num(cache) if not fp8 else cache
    with np.errstate(invalid="ignore"):
        want = L.decode(q, clean, table, lens, sink, gate)
        plain = L.decode(q, clean, table, lens, None, None, 0.11)
    ws = ops.new_workspace(ops.latent_decode_workspace_size(B, Q, H, table.shape[1] * page), "cuda")
    out, lse = ops.latent_decode(q, cache, table, ln, sink=sink, gate=gate, workspace=ws)
    assert status_of(ops, ws) == 0
    check_attention(out, lse, want, max(lens))
    again, lse2 = ops.latent_decode(q, cache, table, ln, sink=sink, gate=gate, workspace=ws)
    assert torch.equal(out, again) and torch.equal(lse, lse2)  # no order of work shows
    out, lse = ops.latent_decode(q, cache, table, ln, sm_scale=0.11, out_dtype=torch.float32)
    check_attention(out, lse, plain, max(lens))
    if Q == 1:
        flat, _ = ops.latent_decode(q[:, 0], cache, table, ln, sm_scale=0.11, out_dtype=torch.float32, want_lse=False)
        assert torch.equal(flat, out[:, 0])


@pytest.mark.parametrize("fp8", [False, True])
def test_decode_moves_its_reference(ops, fp8):
    """Logits that grow along the context: the running maximum moves again and again, by less and by more than the
    threshold, and the early weights vanish."""
    g = gen(8)
    lens, H, page = [900, 640], 20, 64
    table, pages = paged(lens, page, g)
    cache = ops.new_latent_cache(pages, page, fp8)
    d = torch.randn(576, generator=g, device="cuda")
    for b, n in enumerate(lens):
        ramp = torch.linspace(0, 12 if b == 0 else -12, n, device="cuda")[:, None]
        x = (d * ramp * 0.1 + 0.3 * torch.randn(n, 576, generator=g, device="cuda")).to(torch.bfloat16)
        p = torch.arange(n, device="cuda")
        ops.latent_append(x, table[b, p // page].long() * page + p % page, cache)
    q = (d + 0.2 * torch.randn(2, 1, H, 576, generator=g, device="cuda")).to(torch.bfloat16)
    want = L.decode(q, cache, table, lens, None, None, 1.0)
    out, lse = ops.latent_decode(q, cache, table, torch.tensor(lens, device="cuda"), sm_scale=1.0, out_dtype=torch.float32)
    check_attention(out, lse, want, max(lens))


@pytest.mark.parametrize("fp8", [False, True])
def test_decode_records_bad_pages_and_lengths(ops, fp8):
    from lightning_indexer_cross_b200 import _abi
    g = gen(9)
    cache = random_cache(ops, 6, 16, fp8, g)
    table = torch.tensor([[0, 6, 2, 3], [4, -1, 1, 5], [5, 4, 3, 2]], dtype=torch.int32, device="cuda")
    lens = [50, 64, 1000]
    q = queries((3, 1, 7), g)
    ws = ops.new_workspace(ops.latent_decode_workspace_size(3, 1, 7, 64), "cuda")
    out, lse = ops.latent_decode(q, cache, table, torch.tensor(lens, device="cuda"), workspace=ws)
    assert status_of(ops, ws) == _abi.IC_ERR_BAD_INDEX
    check_attention(out, lse, L.decode(q, cache, table, lens), 64)
    ws.zero_()
    out, lse = ops.latent_decode(q, cache, table[2:].expand(3, 4).contiguous(), torch.tensor([-5, 64, 3], device="cuda"), workspace=ws)
    assert status_of(ops, ws) == _abi.IC_ERR_BAD_INDEX
    check_attention(out, lse, L.decode(q, cache, table[2:].expand(3, 4), [0, 64, 3]), 64)


def test_decode_refuses(ops):
    cache = ops.new_latent_cache(4, 16)
    q = torch.zeros(2, 8, 576, dtype=torch.bfloat16, device="cuda")
    table, lens = torch.zeros(2, 2, dtype=torch.int32, device="cuda"), torch.zeros(2, dtype=torch.int64, device="cuda")
    args = dict(q=q, cache=cache, block_table=table, lens=lens)
    for kw in (dict(q=q.float()), dict(q=q[..., :512]), dict(q=q[:1]), dict(cache=cache.float()), dict(cache=cache[0]),
               dict(block_table=table.long()), dict(block_table=table[:1]), dict(lens=lens.int()), dict(lens=lens.cpu()),
               dict(sink=torch.zeros(7, device="cuda")), dict(gate=torch.zeros(2, 8, 512, device="cuda")),
               dict(sm_scale=0.0), dict(out_dtype=torch.float16), dict(workspace=torch.zeros(64, dtype=torch.uint8, device="cuda"))):
        with pytest.raises((ValueError, RuntimeError)):
            ops.latent_decode(**{**args, **kw})


SPARSE = [(150, 2, 1000, 64), (1, 1, 1, 16), (2, 8, 63, 16), (3, 128, 64, 64), (1, 65, 257, 32), (4, 16, 2048, 64), (40, 3, 100, 48)]


@pytest.mark.parametrize("B,H,k,page", SPARSE)
def test_sparse(ops, B, H, k, page):
    g = gen(B * k)
    pages = 2 * k // page + 2
    cache = random_cache(ops, pages, page, True, g)
    slots = torch.randint(0, pages * page, (B, k), generator=g, device="cuda").int()  # the same slot twice among them
    if k > 2:
        slots[0, k // 3:2 * k // 3] = -1
    if B > 1:
        slots[1] = -1
    if B > 2:
        slots[2, 1:] = -1
    q = queries((B, H), g)
    sink = torch.randn(H, generator=g, device="cuda")
    gate = torch.randn(B, H, 512, generator=g, device="cuda").to(torch.bfloat16)
    ws = ops.new_workspace(ops.latent_sparse_workspace_size(B, H, k), "cuda")
    out, lse = ops.latent_sparse_decode(q, cache, slots, sink=sink, gate=gate, workspace=ws)
    assert status_of(ops, ws) == 0
    check_attention(out, lse, L.sparse(q, cache, slots, sink, gate), k)
    out, lse = ops.latent_sparse_decode(q, cache, slots, out_dtype=torch.float32)
    check_attention(out, lse, L.sparse(q, cache, slots), k)


def test_sparse_records_slots_outside(ops):
    from lightning_indexer_cross_b200 import _abi
    g = gen(4)
    cache = random_cache(ops, 3, 16, True, g)
    slots = torch.tensor([[0, 48, -2, 47, (1 << 31) - 1, -(1 << 31), -1]], dtype=torch.int32, device="cuda")
    q = queries((1, 5), g)
    ws = ops.new_workspace(ops.latent_sparse_workspace_size(1, 5, 7), "cuda")
    out, lse = ops.latent_sparse_decode(q, cache, slots, workspace=ws)
    assert status_of(ops, ws) == _abi.IC_ERR_BAD_INDEX
    check_attention(out, lse, L.sparse(q, cache, slots), 7)
    with pytest.raises(ValueError):
        ops.latent_sparse_decode(q, ops.new_latent_cache(3, 16), slots)


# ---------------------------------------------------------------- in use
@pytest.mark.parametrize("fp8", [False, True])
def test_far_pages(ops, fp8):
    """Byte offsets past 32 bits."""
    g = gen(10)
    page = 64
    pages = (5 << 30) // (page * (656 if fp8 else 1152))
    cache = torch.empty((pages, page, 656 if fp8 else 576), dtype=torch.uint8 if fp8 else torch.bfloat16, device="cuda")
    table = torch.tensor([[pages - 1, 0, pages - 2]], dtype=torch.int32, device="cuda")
    p = torch.arange(150, device="cuda")
    slots = table[0, p // page].long() * page + p % page
    kv = torch.randn(150, 576, generator=g, device="cuda").to(torch.bfloat16)
    ops.latent_append(kv, slots, cache)
    small = cache[[pages - 1, 0, pages - 2]]
    small_table = torch.arange(3, dtype=torch.int32, device="cuda")[None]
    out = torch.zeros(150, 576, dtype=torch.bfloat16, device="cuda")
    ops.latent_read(cache, table, torch.tensor([0, 150], device="cuda"), out)
    assert np.array_equal(f64(out), L.cache_rows(small)[:150])
    q = queries((1, 1, 9), g)
    o, s = ops.latent_decode(q, cache, table, torch.tensor([150], device="cuda"))
    check_attention(o, s, L.decode(q, small, small_table, [150]), 150)
    if fp8:
        o, s = ops.latent_sparse_decode(q[0], cache, slots[None, ::2].int())
        check_attention(o, s, L.sparse(q[0], small, p[None, ::2].int()), 75)


@pytest.mark.parametrize("fp8", [False, True])
def test_decode_steps_with_the_indexers_selection(ops, fp8):
    """Several decode steps of a small model's layer: rotate, append, attend densely, then to a top-k's positions."""
    g = gen(11)
    B, H, page, k = 3, 16, 16, 24
    start = [30, 0, 47]
    table, pages = paged([n + 4 for n in start], page, g)
    cache = ops.new_latent_cache(pages, page, fp8)
    freq, m = ops.rope_frequencies(64)
    for b, n in enumerate(start):
        if n:
            p = torch.arange(n, device="cuda")
            ops.latent_append(torch.randn(n, 576, generator=g, device="cuda").to(torch.bfloat16),
                              table[b, p // page].long() * page + p % page, cache, pos=p, freq=freq, mscale=m)
    for step in range(3):
        pos = torch.tensor([n + step for n in start], device="cuda")
        kv = torch.randn(B, 576, generator=g, device="cuda").to(torch.bfloat16)
        q = ops.rope(queries((B, H), g), pos, freq, rot_off=512, mscale=m)
        slots = ops.slots_of(pos[:, None].int(), table, page)[:, 0].long()
        ops.latent_append(kv, slots, cache, pos=pos, freq=freq, mscale=m)
        lens = [n + step + 1 for n in start]
        out, lse = ops.latent_decode(q, cache, table, torch.tensor(lens, device="cuda"))
        check_attention(out, lse, tuple(x[:, 0] for x in L.decode(q[:, None], cache, table, lens)), max(lens))
        scores = torch.rand(B, max(lens), generator=g, device="cuda")
        idx = ops.topk(scores, k, n_valid=torch.tensor(lens, dtype=torch.int32, device="cuda"))
        idx = idx[0] if isinstance(idx, tuple) else idx
        at = ops.slots_of(idx, table, page)
        want = L.sparse(q, cache, at)
        if fp8:
            out, lse = ops.latent_sparse_decode(q, cache, at)
        else:
            out, lse = ops.sparse_mla_decode(q, cache.view(1, -1, 576), at, torch.full((H,), -float("inf"), device="cuda"))
        # the bf16 kernel sums the weights as rounded to bf16, each off by at most 2^-8 of itself: so is the sum, and its
        # logarithm by at most -log(1 - 2^-8) < 2^-8 (1 + 2^-8)
        check_attention(out, lse, want, k, sum_u=0.0 if fp8 else 2.0 ** -8 * (1 + 2.0 ** -8))


def test_captured_graphs_and_side_streams(ops):
    """Two graphs that share a workspace, replayed as lengths and rows change, and a run on another stream."""
    g = gen(12)
    B, H, page = 3, 40, 16
    table, pages = paged([200, 200, 200], page, g)
    caches = [random_cache(ops, pages, page, fp8, g) for fp8 in (False, True)]
    q, lens = queries((B, 1, H), g), torch.tensor([5, 0, 100], device="cuda")
    kv = torch.randn(B, 576, generator=g, device="cuda").to(torch.bfloat16)
    slots, pos = torch.zeros(B, dtype=torch.int64, device="cuda"), torch.zeros(B, dtype=torch.int64, device="cuda")
    freq, _ = ops.rope_frequencies(64)
    ws = ops.new_workspace(ops.latent_decode_workspace_size(B, 1, H, table.shape[1] * page), "cuda")
    graphs, outs = [], []
    for c in caches:
        ops.latent_decode(q, c, table, lens, workspace=ws)
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            ops.latent_append(kv, slots, c, pos=pos, freq=freq, workspace=ws)
            outs.append(ops.latent_decode(q, c, table, lens, workspace=ws))
        graphs.append(gr)
    for step, ln in enumerate(([6, 1, 101], [150, 64, 200], [1, 0, 2])):
        lens.copy_(torch.tensor(ln))
        p = (lens - 1).clamp(min=0)
        pos.copy_(p)
        at = table.gather(1, (p // page)[:, None])[:, 0].long() * page + p % page
        slots.copy_(torch.where(lens > 0, at, torch.full_like(at, -1)))
        kv.copy_(torch.randn(B, 576, generator=g, device="cuda"))
        q.copy_(torch.randn(B, 1, H, 576, generator=g, device="cuda"))
        for gr, c, (out, lse) in zip(graphs, caches, outs):
            gr.replay()
            check_attention(out, lse, L.decode(q, c, table, ln), max(ln))
    assert status_of(ops, ws) == 0
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out, lse = ops.latent_decode(q, caches[1], table, lens, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(out, outs[1][0]) and torch.equal(lse, outs[1][1])


@pytest.mark.parametrize("page_gap", [0, 16])
def test_every_code_and_scale_is_widened(ops, page_gap):
    """Sequences of one row: the output is the row itself, whatever its codes and scales (powers of two near and far,
    and others). The weight 2^(z - max) is off from 1 by less than 2^-20, and so is the output."""
    scales = [1.0, 2.0 ** -100, 2.0 ** 7, 2.0 ** 8, 2.0 ** 100, 0.3, 1.5, 2.0 ** -126]
    n = len(scales)
    big = ops.new_latent_cache(n, 16 + page_gap, True)
    cache = big[:, :16]
    codes = torch.arange(256, dtype=torch.uint8, device="cuda")
    codes[codes & 0x7f == 0x7f] = 0  # NaN
    rows = cache[:, 3]
    rows[:, :512] = codes.repeat(2)
    rows[:, 512:528] = torch.tensor(scales, device="cuda")[:, None].repeat(1, 4).view(torch.uint8)
    want = f64(torch.from_numpy(L.unpack(rows).astype(np.float32)).to(torch.bfloat16))[:, :512]
    q = torch.zeros(n, 5, 576, dtype=torch.bfloat16, device="cuda")
    slots = torch.arange(n, device="cuda", dtype=torch.int32)[:, None] * 16 + 3
    first = cache.clone()
    first[:, 0] = rows
    table = torch.arange(n, device="cuda", dtype=torch.int32)[:, None]
    for out in (ops.latent_sparse_decode(q, cache, slots, out_dtype=torch.float32)[0],
                ops.latent_decode(q, first, table, torch.ones(n, dtype=torch.int64, device="cuda"), out_dtype=torch.float32)[0]):
        assert np.all(np.abs(f64(out) - want[:, None]) <= np.abs(want[:, None]) * 2.0 ** -18 + 2.0 ** -140)
    rows[0, 77] = 0x7f
    rows[1, 78] = 0xff
    out = ops.latent_sparse_decode(q, cache, slots)[0]
    assert out[:2].isnan().all() and not out[2:].isnan().any()


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("H", [16, 64, 128])
def test_a_wait_that_gives_up_is_recorded_and_the_next_call_is_right(ops, fp8, H):
    """With the wait limit at 0 a wait that is not satisfied at once gives up: the call returns, its status says so, and
    the next call with the default limit is right. (No GPU fault is involved: the host tells the waits to give up.)"""
    from lightning_indexer_cross_b200 import _abi
    g = gen(13)
    lens = [1500, 0, 700]
    table, pages = paged(lens, 64, g)
    cache = random_cache(ops, pages, 64, fp8, g)
    q, ln = queries((3, 1, H), g), torch.tensor(lens, device="cuda")
    ws = ops.new_workspace(ops.latent_decode_workspace_size(3, 1, H, table.shape[1] * 64), "cuda")
    default = _abi.ic_wait_limit_ns()
    try:
        _abi.ic_set_wait_limit_ns(0)
        ops.latent_decode(q, cache, table, ln, workspace=ws)
    finally:
        _abi.ic_set_wait_limit_ns(default)
    assert status_of(ops, ws) == _abi.IC_ERR_TIMEOUT
    out, lse = ops.latent_decode(q, cache, table, ln, workspace=ws)
    assert status_of(ops, ws) == 0
    check_attention(out, lse, L.decode(q, cache, table, lens), max(lens))


@pytest.mark.parametrize("H", [7, 40, 128])
def test_every_row_of_a_tile_is_widened_in_every_block_size(ops, H):
    """Queries of zeros weigh all rows alike, by exactly 1: the output is the mean of the rows, here of every code and
    of scales that are no powers of two beside such. n sums in 32 bits, each off by 2^-22 of the terms' magnitudes at
    most, and a division."""
    g = gen(H)
    n, page = 104, 16  # two tiles, the second ragged
    pages = n // page + 1
    cache = ops.new_latent_cache(pages, page, True)
    codes = torch.randint(0, 256, (pages, page, 512), generator=g, device="cuda").to(torch.uint8)
    codes[codes & 0x7f == 0x7f] = 0  # NaN
    cache[..., :512] = codes
    scales = torch.rand(pages, page, 4, generator=g, device="cuda") + 0.1
    scales[:, ::2] = 2.0 ** torch.randint(-3, 4, (pages, page // 2, 4), generator=g, device="cuda")
    cache[..., 512:528] = scales.view(torch.uint8)
    perm = torch.randperm(pages, generator=g, device="cuda").int()
    rows = torch.from_numpy(L.cache_rows(cache).astype(np.float32)).to(torch.bfloat16)  # [pages * page, 576]
    slots = (perm.long()[:, None] * page + torch.arange(page, device="cuda")).reshape(-1)[:n]
    v = f64(rows.reshape(-1, 576)[slots.cpu()])[:, :512]
    lim = np.abs(v).mean(0) * (n * 2.0 ** -22 + 2.0 ** -20)
    q = torch.zeros(2, H, 576, dtype=torch.bfloat16, device="cuda")
    dense, _ = ops.latent_decode(q, cache, perm[None].repeat(2, 1), torch.tensor([n, n], device="cuda"),
                                 out_dtype=torch.float32)
    sparse, _ = ops.latent_sparse_decode(q, cache, slots.int()[None].repeat(2, 1).contiguous(), out_dtype=torch.float32)
    for out in (dense, sparse):
        assert np.all(np.abs(f64(out) - v.mean(0)) <= lim)


def test_the_largest_values_stay_finite(ops):
    """Rows of the largest bf16, 255 * 2^120, alone, beside infinities and beside a NaN, and of the largest value that a
    code reaches: scales of 2^119 at most, and a read-back that is finite and no further off than that."""
    most = 448 * 2.0 ** 119
    kv = torch.full((4, 576), 255 * 2.0 ** 120, dtype=torch.float64)
    kv[1, 0], kv[1, 300] = float("inf"), float("-inf")
    kv[1, 301] = -255 * 2.0 ** 120
    kv[2, 5] = float("nan")
    kv[3] = most
    kv = kv.to(torch.bfloat16).cuda()
    cache = ops.new_latent_cache(1, 16, True)
    ws = ops.latent_append(kv, torch.arange(4, device="cuda"), cache)
    assert status_of(ops, ws) == 0
    assert np.all(f64(parts(cache[0, :4])[1]) == 2.0 ** 119)
    out = torch.zeros(4, 576, dtype=torch.bfloat16, device="cuda")
    ops.latent_read(cache, torch.zeros(1, 1, dtype=torch.int32, device="cuda"), torch.tensor([0, 4], device="cuda"), out)
    want = np.full((4, 512), most)
    want[1, 300] = want[1, 301] = -most
    want[2, 5] = np.nan
    assert np.array_equal(f64(out)[:, :512], want, equal_nan=True)
    assert torch.equal(out[:, 512:], kv[:, 512:])


@pytest.mark.parametrize("fp8", [False, True])
def test_append_of_one_row_whatever_its_stride(ops, fp8):
    """One token: the distance to a next row means nothing (a transposed column and a cut row have odd ones)."""
    g = gen(14)
    col = torch.randn(576, 1, generator=g, device="cuda").to(torch.bfloat16)
    wide = torch.zeros(1, 579, dtype=torch.bfloat16, device="cuda")
    wide[:, :576] = col.t()
    slot = torch.tensor([7], device="cuda")
    want = ops.new_latent_cache(1, 16, fp8)
    ops.latent_append(col.t().contiguous().view(576).view(1, 576), slot, want)
    assert want[0, 7].any()
    for kv in (col.t(), wide[:, :576]):
        cache = ops.new_latent_cache(1, 16, fp8)
        assert status_of(ops, ops.latent_append(kv, slot, cache)) == 0
        assert torch.equal(cache.view(torch.uint8), want.view(torch.uint8))


def test_read_of_an_empty_batch_leaves_every_row(ops):
    """No sequences: as for the other calls there is nothing to do, and the rows of out stay as they are."""
    cache = ops.new_latent_cache(2, 16, True)
    out = torch.full((5, 576), 7.0, dtype=torch.bfloat16, device="cuda")
    table, cu = torch.zeros(0, 3, dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int64, device="cuda")
    assert ops.latent_read(cache, table, cu, out) is out
    assert bool((out == 7).all())
    o, s = ops.latent_decode(torch.zeros(0, 8, 576, dtype=torch.bfloat16, device="cuda"), cache, table, cu[:0])
    assert o.shape == (0, 8, 512) and s.shape == (0, 8)


# ---------------------------------------------------------------- the rotation's grid
def rotated64(x, pos, freq, off, layout, mscale):
    """(y, limit) in 64 bits on the GPU, from the formula; the limit is the one of this file's head, 0 for copied dims."""
    n = freq.numel()
    a = torch.arange(n, device="cuda") * (2 if layout == "interleaved" else 1) + off
    b = a + (1 if layout == "interleaved" else n)
    angle = pos.double()[:, None, None] * freq
    c, s = mscale * angle.cos(), mscale * angle.sin()
    y = x.double()
    u, v = y[..., a], y[..., b]
    lim = torch.zeros_like(y)
    y[..., a], y[..., b] = u * c - v * s, u * s + v * c
    for d in (a, b):
        lim[..., d] = 2.0 ** -20 * mscale * (u.abs() + v.abs()) + U[x.dtype] * 1.001 * y[..., d].abs()
    return y, lim


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("layout", ["interleaved", "half"])
@pytest.mark.parametrize("T,H,D,off,rot", [
    (5, 128, 576, 512, 64),     # a decode step: blocks of 15 heads (fp32: 8), the last of 8
    (300, 131, 64, 0, 64),      # blocks of heads in place too, the last of 3
    (2401, 8, 576, 512, 64),    # two tokens a CTA, the last alone
    (8192, 64, 128, 0, 64),     # a prompt: four tokens a CTA, copies in several turns
    (4737, 128, 64, 0, 64),     # nothing copied: rotated words in several turns
    (3, 2, 16384, 16, 1024),    # one head's copies in several turns
    (40001, 1, 64, 0, 64),      # many tokens a CTA
    (230, 300, 70, 1, 66),      # unaligned: blocks of heads, and more than one token a CTA
])
def test_rope_in_every_shape_of_its_grid(ops, dtype, layout, T, H, D, off, rot):
    g = gen(T + H)
    x = torch.randn(T, H, D, generator=g, device="cuda").to(dtype)
    pos = torch.randint(0, 1 << 20, (T,), generator=g, device="cuda")
    freq, _ = ops.rope_frequencies(rot)
    want, lim = rotated64(x, pos, freq, off, layout, 1.25)
    y = ops.rope(x, pos, freq, rot_off=off, layout=layout, mscale=1.25)
    assert bool(((y.double() - want).abs() <= lim).all()), ((y.double() - want).abs() - lim).max().item()
    del want, lim
    w = x.clone()
    ops.rope(w, pos, freq, rot_off=off, layout=layout, mscale=1.25, out=w)
    assert torch.equal(w, y)
    heads_first = torch.empty(H, T, D, dtype=dtype, device="cuda").transpose(0, 1)
    ops.rope(x, pos, freq, rot_off=off, layout=layout, mscale=1.25, out=heads_first)
    assert torch.equal(heads_first, y)


@pytest.mark.parametrize("H", [16, 64, 128])
def test_a_sparse_wait_that_gives_up_is_recorded_and_the_next_call_is_right(ops, H):
    """The same for selected rows, in each block size: a ring of three descriptors, with the rows' places beside it."""
    from lightning_indexer_cross_b200 import _abi
    g = gen(15)
    B, k, page = 3, 700, 64
    cache = random_cache(ops, 40, page, True, g)
    slots = torch.randint(0, 40 * page, (B, k), generator=g, device="cuda").int()
    slots[1, 100:] = -1
    q = queries((B, H), g)
    ws = ops.new_workspace(ops.latent_sparse_workspace_size(B, H, k), "cuda")
    default = _abi.ic_wait_limit_ns()
    try:
        _abi.ic_set_wait_limit_ns(0)
        ops.latent_sparse_decode(q, cache, slots, workspace=ws)
    finally:
        _abi.ic_set_wait_limit_ns(default)
    assert status_of(ops, ws) == _abi.IC_ERR_TIMEOUT
    out, lse = ops.latent_sparse_decode(q, cache, slots, workspace=ws)
    assert status_of(ops, ws) == 0
    check_attention(out, lse, L.sparse(q, cache, slots), k)


@pytest.mark.parametrize("H", [16, 64, 96, 128])
@pytest.mark.parametrize("kind", ["bf16", "e4m3", "sparse"])
def test_calls_repeat_bit_for_bit_whatever_runs_beside_them(ops, kind, H):
    """Ragged sequences in each block size: right once, and then the same bits with a cold L2, a warm one, and a second
    call on another stream at the same time. (What a CTA tells the other one of its pair, a wait too few would show.)"""
    g = gen(16 + H)
    lens, page, k = [4000, 1, 0, 65, 2111, 1024, 777, 3333, 130, 64, 4001, 5], 32, 1100
    B = len(lens)
    table, pages = paged(lens, page, g)
    cache = random_cache(ops, pages, page, kind != "bf16", g)
    q, sink = queries((B, H), g), torch.randn(H, generator=g, device="cuda")
    gate = torch.randn(B, H, 512, generator=g, device="cuda").to(torch.bfloat16)
    if kind == "sparse":
        slots = torch.randint(0, pages * page, (B, k), generator=g, device="cuda").int()
        slots[3, 700:] = -1
        want = L.sparse(q, cache, slots, sink, gate)
        call = lambda **kw: ops.latent_sparse_decode(q, cache, slots, sink=sink, gate=gate, **kw)  # noqa: E731
    else:
        ln = torch.tensor(lens, device="cuda")
        want = tuple(x[:, 0] for x in L.decode(q[:, None], cache, table, lens, sink, gate[:, None]))
        call = lambda **kw: ops.latent_decode(q, cache, table, ln, sink=sink, gate=gate, **kw)  # noqa: E731
    out, lse = call()
    check_attention(out, lse, want, max(lens))
    side, big = torch.cuda.Stream(), torch.empty(64 << 20, dtype=torch.int32, device="cuda")
    for i in range(30):
        if i % 3 == 0:
            big.fill_(i)  # past what L2 holds
        side.wait_stream(torch.cuda.current_stream())
        beside = call(stream=side) if i % 3 == 2 else None
        got = call()
        torch.cuda.current_stream().wait_stream(side)
        for o, s in (got, beside or got):
            assert torch.equal(o, out) and torch.equal(s, lse), i


def test_the_bindings_functions_equal_the_tensor_front_end(ops):
    """The C calls through _abi, on raw pointers, against the same calls on tensors: rotation, append, read-back, dense
    and sparse attention, with every argument at a value of its own."""
    from lightning_indexer_cross_b200 import _abi
    g = gen(17)
    B, Q, H, page, k, T = 2, 2, 5, 32, 40, 50
    st = ops._stream_ptr()
    P = ops._ptr
    x = torch.randn(T, 3, 100, generator=g, device="cuda").to(torch.bfloat16)
    pos = torch.randint(0, 1 << 20, (T,), generator=g, device="cuda")
    freq, _ = ops.rope_frequencies(64)
    y = torch.empty(3, T, 100, dtype=torch.bfloat16, device="cuda")
    _abi.ic_rope(P(x), 300, 100, P(pos), P(freq), 1.5, _abi.IC_ROPE_HALF, 1, _abi.IC_BF16, T, 3, 100, 20, 64, P(y), 100,
                 T * 100, st)
    assert torch.equal(y.transpose(0, 1), ops.rope(x, pos, freq, rot_off=20, layout="half", mscale=1.5, transpose=True))
    kv = torch.randn(T, 600, generator=g, device="cuda").to(torch.bfloat16)[:, :576]
    slots = torch.randperm(3 * page, generator=g, device="cuda")[:T]
    table = torch.tensor([[2, 0, 9], [1, 2, 0]], dtype=torch.int32, device="cuda")[:, :2]
    lens, cu = torch.tensor([33, 60], device="cuda"), torch.tensor([0, 33, 93], device="cuda")
    q, sink = queries((B, Q, H), g), torch.randn(H, generator=g, device="cuda")
    gate = torch.randn(B, Q, H, 512, generator=g, device="cuda").to(torch.bfloat16)
    sel = torch.randint(0, 3 * page, (B, k), generator=g, device="cuda").int()
    ws = ops.new_workspace(max(_abi.ic_latent_decode_workspace_size(B, Q, H, 2 * page),
                               _abi.ic_latent_sparse_workspace_size(B, H, k), _abi.ic_latent_append_workspace_size(),
                               _abi.ic_latent_read_workspace_size()), "cuda")
    n = ws.numel()
    for fp8 in (False, True):
        code = _abi.IC_FP8_E4M3 if fp8 else _abi.IC_BF16
        big = [ops.new_latent_cache(4, page + 16, fp8) for _ in range(2)]
        a, b = (c[:3, :page] for c in big)
        stride = big[0].stride(0) * big[0].element_size()
        ops.latent_append(kv, slots, a, pos=pos, freq=freq, layout="half", mscale=0.5)
        _abi.ic_latent_append(P(kv), 600, P(slots), P(pos), P(freq), 0.5, _abi.IC_ROPE_HALF, T, code, P(b), 3, page, stride,
                              P(ws), n, st)
        assert torch.equal(big[0].view(torch.uint8), big[1].view(torch.uint8)) and a.any()
        want = ops.latent_read(a, table, cu, torch.zeros(95, 576, dtype=torch.bfloat16, device="cuda"))
        got = torch.zeros_like(want)
        _abi.ic_latent_read(P(b), code, 3, page, stride, P(table), 3, 2, P(cu), B, P(got), 95, P(ws), n, st)
        assert torch.equal(got, want) and want.any()
        out, lse = ops.latent_decode(q, a, table, lens, sink=sink, gate=gate, sm_scale=0.07, out_dtype=torch.float32)
        o, s = torch.empty_like(out), torch.empty_like(lse)
        _abi.ic_latent_decode(P(q), P(b), code, 3, page, stride, P(table), 3, 2, P(lens), P(sink), P(gate), 0.07, B, Q, H,
                              _abi.IC_F32, P(o), P(s), P(ws), n, st)
        assert torch.equal(o, out) and torch.equal(s, lse)
    out, lse = ops.latent_sparse_decode(q[:, 0].contiguous(), a, sel, sink=sink, gate=gate[:, 1].contiguous(), sm_scale=0.07)
    o, s = torch.empty_like(out), torch.empty_like(lse)
    q0, gate1 = q[:, 0].contiguous(), gate[:, 1].contiguous()
    _abi.ic_latent_sparse_decode(P(q0), P(b), 3, page, stride, P(sel), k, P(sink), P(gate1), 0.07, B, H, _abi.IC_BF16, P(o),
                                 P(s), P(ws), n, st)
    assert torch.equal(o, out) and torch.equal(s, lse)
    assert status_of(ops, ws) == 0


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("H", [9, 48, 100])
def test_decode_from_spaced_pages_and_a_cut_table(ops, fp8, H):
    """Pages some rows apart, a block table that is a part of a wider one, an odd page size, NaN in every row that holds
    no token."""
    g = gen(18)
    lens, Q, page = [333, 0, 81, 5], 2, 80
    need = [-(-n // page) for n in lens]
    big = ops.new_latent_cache(sum(need) + 1, page + 8, fp8)
    big.view(torch.uint8).fill_(0xff)
    cache = big[:, :page]
    wide = torch.full((len(lens), max(need) + 3), 1 << 30, dtype=torch.int32, device="cuda")
    table = wide[:, :max(need)]
    perm = torch.randperm(sum(need) + 1, generator=g, device="cuda").int()
    at = 0
    for b, n in enumerate(lens):
        table[b, :need[b]] = perm[at:at + need[b]]
        at += need[b]
        p = torch.arange(n, device="cuda")
        if n:
            kv = torch.randn(n, 576, generator=g, device="cuda").to(torch.bfloat16)
            ops.latent_append(kv, table[b].long()[p // page] * page + p % page, cache)
    q = queries((len(lens), Q, H), g)
    ws = ops.new_workspace(ops.latent_decode_workspace_size(len(lens), Q, H, table.shape[1] * page), "cuda")
    ws[256:] = 0xff  # partial results that nothing has written are NaN
    out, lse = ops.latent_decode(q, cache, table, torch.tensor(lens, device="cuda"), workspace=ws, out_dtype=torch.float32)
    assert status_of(ops, ws) == 0
    with np.errstate(invalid="ignore"):
        check_attention(out, lse, L.decode(q, cache, table, lens), max(lens))


@pytest.mark.parametrize("fp8", [False, True])
def test_shares_of_more_tiles_than_32_bits_divide(ops, fp8):
    """4300 sequences of 65536 rows that share their pages: 4.4 million tiles, whose shares are counted in 64 bits."""
    g = gen(19)
    B, H, page, pages = 4300, 2, 128, 512
    cache = random_cache(ops, pages, page, fp8, g)
    table = torch.stack([torch.randperm(pages, generator=g, device="cuda").int() for _ in range(4)]).repeat(B // 4, 1)
    q = queries((B, H), g)
    lens = torch.full((B,), pages * page, device="cuda")
    lens[3::11] -= 1
    out, lse = ops.latent_decode(q, cache, table, lens, out_dtype=torch.float32)
    some = [0, 3, 2147, B - 1]
    want = L.decode(q[some][:, None], cache, table[some], lens[some].tolist())
    check_attention(out[some], lse[some], tuple(x[:, 0] for x in want), pages * page)
