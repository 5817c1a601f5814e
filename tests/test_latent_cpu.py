"""The paged latent cache on the host: pins of its oracle against plain loops
and torch, the frequency tables, and the refusals of the entry points and of
the tensor front end (no GPU)."""
import ctypes
import math

import numpy as np
import pytest
import torch

from oracle import latent_oracle as L

INV = 1


@pytest.fixture(scope="module")
def abi():
    from lightning_indexer_cross_b200 import build
    build.build()
    from lightning_indexer_cross_b200 import _abi
    return _abi


@pytest.fixture(scope="module")
def ops(abi):
    from lightning_indexer_cross_b200 import ops
    return ops


def _fake(n=1 << 20):
    # host memory stands in for device pointers: validation must reject before any use
    buf = (ctypes.c_uint8 * n)()
    return ctypes.c_void_p(ctypes.addressof(buf) + (-ctypes.addressof(buf)) % 256), buf


# ---------------------------------------------------------------- oracle pins
@pytest.mark.parametrize("layout", ["interleaved", "half"])
def test_oracle_rope_equals_loops_and_keeps_the_norm(layout):
    rng = np.random.default_rng(0)
    x = rng.standard_normal((3, 2, 10))
    freq = np.array([1.0, 0.1, 0.01])
    pos = np.array([0, 5, 123456])
    y = L.rope(x, pos, freq, rot_off=2, layout=layout, mscale=1.5)
    for t in range(3):
        for h in range(2):
            for i in range(3):
                u, v = (2 + 2 * i, 3 + 2 * i) if layout == "interleaved" else (2 + i, 5 + i)
                a = pos[t] * freq[i]
                assert y[t, h, u] == pytest.approx(1.5 * (x[t, h, u] * math.cos(a) - x[t, h, v] * math.sin(a)), abs=1e-12)
                assert y[t, h, v] == pytest.approx(1.5 * (x[t, h, u] * math.sin(a) + x[t, h, v] * math.cos(a)), abs=1e-12)
    assert np.array_equal(y[..., [0, 1, 8, 9]], x[..., [0, 1, 8, 9]])
    np.testing.assert_allclose(L.rope(L.rope(x, pos, freq, 2, layout), pos, freq, 2, layout, transpose=True), x, atol=1e-12)


def test_oracle_rope_transpose_is_the_gradient_by_differences():
    rng = np.random.default_rng(1)
    x, g = rng.standard_normal((2, 1, 6)), rng.standard_normal((2, 1, 6))
    freq, pos = np.array([0.7, 0.2]), np.array([3, 11])
    f = lambda v: float((L.rope(v, pos, freq, 1, "half", 1.3) * g).sum())  # noqa: E731
    grad = L.rope(g, pos, freq, 1, "half", 1.3, transpose=True)
    # dims outside the rotation pass through, so their gradient does too
    for i in np.ndindex(x.shape):
        d = np.zeros_like(x)
        d[i] = 1e-4
        assert (f(x + d) - f(x - d)) / 2e-4 == pytest.approx(grad[i], abs=1e-9)


def test_oracle_scale_is_the_least_power_of_two():
    for amax, want in [(448.0, 1.0), (448.1, 2.0), (224.0, 0.5), (1.75, 2.0 ** -8), (1.76, 2.0 ** -7), (0.0, 1.0),
                       (2.0 ** -126, 2.0 ** -100)]:
        y = np.zeros((1, 128))
        y[0, 5] = -amax
        assert L.pow2_scale(y)[0] == want
    y = np.zeros((1, 128))
    y[0, 0], y[0, 1], y[0, 2] = np.inf, np.nan, 1.0
    assert L.pow2_scale(y)[0] == 2.0 ** -8


def test_oracle_pack_round_trip_is_torchs_cast():
    g = torch.Generator().manual_seed(2)
    x = (torch.randn(5, 576, generator=g) * torch.tensor([1e-3, 1, 30, 1e4, 0.0])[:, None]).to(torch.bfloat16)
    codes, s = L.pack(x)
    ref = (x[:, :512].float().view(5, 4, 128) / torch.from_numpy(s).float()[..., None]).to(torch.float8_e4m3fn)
    assert np.array_equal(codes, ref.view(torch.uint8).reshape(5, 512).numpy())
    raw = torch.zeros(5, 656, dtype=torch.uint8)
    raw[:, :512] = torch.from_numpy(codes)
    raw[:, 512:528] = torch.from_numpy(s.astype(np.float32)).view(torch.uint8)
    raw[:, 528:] = x[:, 512:].contiguous().view(torch.uint8)
    back = L.unpack(raw)
    assert np.array_equal(back[:, 512:], x[:, 512:].double().numpy())
    # at most half a step of e4m3 (2^-4 of the value), or half of its least step (2^-10) times the scale
    lim = np.maximum(np.abs(x[:, :512].double().numpy()) * 2.0 ** -4, np.repeat(s, 128, axis=1) * 2.0 ** -10)
    assert np.all(np.abs(back[:, :512] - x[:, :512].double().numpy()) <= lim)


def test_oracle_attention_equals_torch_softmax_and_handles_no_rows():
    g = torch.Generator().manual_seed(3)
    q, kv = torch.randn(4, 576, generator=g).double(), torch.randn(9, 576, generator=g).double()
    sink = torch.randn(4, generator=g).double()
    z = torch.cat([sink[:, None], q @ kv.T / 24.0], dim=1)
    ref = torch.softmax(z, dim=1)[:, 1:] @ kv[:, :512]
    out, lse, _, _ = L.attend(q.numpy(), kv.numpy(), sink.numpy())
    np.testing.assert_allclose(out, ref.numpy(), atol=1e-12)
    np.testing.assert_allclose(lse, torch.logsumexp(z, dim=1).numpy(), atol=1e-12)
    out, lse, _, _ = L.attend(q.numpy(), kv.numpy()[:0], sink.numpy())
    assert not out.any()
    np.testing.assert_allclose(lse, sink.numpy(), atol=1e-12)
    assert np.all(L.attend(q.numpy(), kv.numpy()[:0])[1] == -np.inf)


def test_oracle_decode_sees_the_positions_before_each_tokens_limit():
    g = torch.Generator().manual_seed(4)
    cache = torch.randn(5, 16, 576, generator=g).to(torch.bfloat16)
    q = torch.randn(1, 2, 1, 576, generator=g).to(torch.bfloat16)
    table = torch.tensor([[3, 0]], dtype=torch.int32)
    out, lse, _, _ = L.decode(q, cache, table, [20])
    rows = torch.cat([cache[3], cache[0]]).double().numpy()
    for j, n in ((0, 19), (1, 20)):
        o, s, _, _ = L.attend(q[0, j].double().numpy(), rows[:n])
        np.testing.assert_allclose(out[0, j], o, atol=1e-12)
        np.testing.assert_allclose(lse[0, j], s, atol=1e-12)


# ---------------------------------------------------------------- frequency tables
def test_rope_frequencies(ops):
    f, m = ops.rope_frequencies(64, 10000.0, device="cpu")
    assert f.dtype == torch.float64 and m == 1.0
    np.testing.assert_allclose(f.numpy(), [10000.0 ** (-2 * i / 64) for i in range(32)], rtol=1e-15)
    g, m = ops.rope_frequencies(64, 10000.0, {"type": "linear", "factor": 4}, device="cpu")
    assert torch.equal(g, f / 4) and m == 1.0
    y, m = ops.rope_frequencies(64, 10000.0, {"type": "yarn", "factor": 40, "original_length": 4096}, device="cpu")
    assert m == pytest.approx(0.1 * math.log(40) + 1)
    turns = f * 4096 / (2 * math.pi)
    fast, slow = turns > 40, turns < 0.8  # clear of the ramp's rounded ends
    assert fast.any() and slow.any()
    assert torch.equal(y[turns > 45], f[turns > 45])
    np.testing.assert_allclose(y[slow].numpy(), (f / 40)[slow].numpy(), rtol=1e-12)
    assert torch.all(y <= f) and torch.all(y >= f / 40 * (1 - 1e-12)) and torch.all(y[1:] < y[:-1])
    for bad in ({"type": "other", "factor": 2}, {"type": "linear", "factor": 0}):
        with pytest.raises(ValueError):
            ops.rope_frequencies(64, 10000.0, bad, device="cpu")
    with pytest.raises(ValueError):
        ops.rope_frequencies(63, device="cpu")


# ---------------------------------------------------------------- refusals of the C entries
def test_rope_rejects_bad_arguments(abi):
    p, keep = _fake()
    call = lambda **kw: abi._rope(*[kw.get(n, d) for n, d in [  # noqa: E731
        ("x", p), ("xts", 512), ("xhs", 128), ("pos", p), ("freq", p), ("m", 1.0), ("lay", 0), ("tr", 0),
        ("dt", abi.IC_BF16), ("T", 4), ("H", 4), ("D", 128), ("off", 64), ("rot", 64),
        ("out", ctypes.c_void_p(p.value + 65536)), ("yts", 512), ("yhs", 128), ("st", None)]])
    for kw in (dict(x=None), dict(pos=None), dict(freq=None), dict(out=None), dict(lay=2), dict(T=0), dict(H=0),
               dict(D=1), dict(rot=63), dict(rot=0), dict(off=65), dict(off=-1), dict(m=float("nan")), dict(xts=-1),
               dict(yhs=100), dict(yts=256), dict(yts=0), dict(H=65536), dict(x=ctypes.c_void_p(p.value + 1)),
               dict(out=p, yts=1024)):
        assert call(**kw) == abi.IC_ERR_INVALID_ARG, kw
    assert call(dt=abi.IC_FP8_E4M3) == abi.IC_ERR_UNSUPPORTED
    assert call(D=4096, rot=2048, off=0, xts=16384, xhs=4096, yts=16384, yhs=4096) == abi.IC_ERR_UNSUPPORTED


def test_latent_append_rejects_bad_arguments(abi):
    p, keep = _fake()
    call = lambda **kw: abi._lat_append(*[kw.get(n, d) for n, d in [  # noqa: E731
        ("kv", p), ("ks", 576), ("slots", p), ("pos", p), ("freq", p), ("m", 1.0), ("lay", 0), ("T", 4),
        ("dt", abi.IC_FP8_E4M3), ("c", p), ("P", 2), ("ps", 16), ("pst", 656 * 16), ("ws", p), ("wsb", 256),
        ("st", None)]])
    for kw in (dict(kv=None), dict(ks=575), dict(ks=580), dict(slots=None), dict(pos=None), dict(freq=None),
               dict(lay=7), dict(T=0), dict(c=None), dict(P=0), dict(ps=24), dict(ps=8), dict(ps=0),
               dict(pst=656 * 16 - 16), dict(pst=656 * 16 + 8), dict(ws=None), dict(wsb=8),
               dict(c=ctypes.c_void_p(p.value + 8)), dict(kv=ctypes.c_void_p(p.value + 2)), dict(m=float("inf")),
               dict(dt=abi.IC_BF16)):  # a bf16 page needs 1152 bytes a row
        assert call(**kw) == abi.IC_ERR_INVALID_ARG, kw
    assert call(dt=abi.IC_F32) == abi.IC_ERR_UNSUPPORTED
    assert abi.ic_latent_append_workspace_size() >= 4


def test_latent_read_rejects_bad_arguments(abi):
    p, keep = _fake()
    call = lambda **kw: abi._lat_read(*[kw.get(n, d) for n, d in [  # noqa: E731
        ("c", p), ("dt", abi.IC_BF16), ("P", 2), ("ps", 16), ("pst", 1152 * 16), ("tab", p), ("ts", 4), ("w", 4),
        ("cu", p), ("B", 2), ("out", p), ("R", 10), ("ws", p), ("wsb", 256), ("st", None)]])
    for kw in (dict(c=None), dict(tab=None), dict(cu=None), dict(out=None), dict(B=0), dict(w=0), dict(ts=3),
               dict(R=0), dict(ws=None), dict(wsb=4), dict(pst=1152), dict(out=ctypes.c_void_p(p.value + 8))):
        assert call(**kw) == abi.IC_ERR_INVALID_ARG, kw
    assert call(dt=abi.IC_F32) == abi.IC_ERR_UNSUPPORTED


def test_latent_decode_rejects_bad_arguments(abi):
    p, keep = _fake()
    need = abi.ic_latent_decode_workspace_size(2, 1, 8, 64)
    call = lambda **kw: abi._lat_decode(*[kw.get(n, d) for n, d in [  # noqa: E731
        ("q", p), ("c", p), ("dt", abi.IC_BF16), ("P", 4), ("ps", 16), ("pst", 1152 * 16), ("tab", p), ("ts", 4),
        ("w", 4), ("lens", p), ("sink", None), ("gate", None), ("sc", 0.04), ("B", 2), ("Q", 1), ("H", 8),
        ("od", abi.IC_BF16), ("out", p), ("lse", None), ("ws", p), ("wsb", need), ("st", None)]])
    for kw in (dict(q=None), dict(c=None), dict(tab=None), dict(lens=None), dict(out=None), dict(ws=None), dict(B=0),
               dict(Q=0), dict(H=0), dict(w=0), dict(ts=3), dict(sc=0.0), dict(sc=-1.0), dict(sc=float("nan")),
               dict(sc=float("inf")), dict(wsb=need - 1), dict(ps=20), dict(q=ctypes.c_void_p(p.value + 2)),
               dict(gate=ctypes.c_void_p(p.value + 8)), dict(w=1 << 28, ts=1 << 28)):
        assert call(**kw) == abi.IC_ERR_INVALID_ARG, kw
    assert call(od=abi.IC_FP8_E4M3) == abi.IC_ERR_UNSUPPORTED
    assert call(dt=abi.IC_F32) == abi.IC_ERR_UNSUPPORTED
    # the workspace holds two partial blocks a share, whatever the batch
    assert abi.ic_latent_decode_workspace_size(4096, 1, 128, 1 << 20) < 64 << 20


def test_latent_sparse_decode_rejects_bad_arguments(abi):
    p, keep = _fake()
    need = abi.ic_latent_sparse_workspace_size(2, 8, 100)
    call = lambda **kw: abi._lat_sparse(*[kw.get(n, d) for n, d in [  # noqa: E731
        ("q", p), ("c", p), ("P", 4), ("ps", 16), ("pst", 656 * 16), ("slots", p), ("k", 100), ("sink", None),
        ("gate", None), ("sc", 0.04), ("B", 2), ("H", 8), ("od", abi.IC_BF16), ("out", p), ("lse", None), ("ws", p),
        ("wsb", need), ("st", None)]])
    for kw in (dict(q=None), dict(c=None), dict(slots=None), dict(out=None), dict(ws=None), dict(k=0), dict(B=0),
               dict(H=0), dict(sc=0.0), dict(wsb=need - 1), dict(pst=656), dict(P=1 << 28)):
        assert call(**kw) == abi.IC_ERR_INVALID_ARG, kw
    assert call(od=abi.IC_FP8_E4M3) == abi.IC_ERR_UNSUPPORTED


# ---------------------------------------------------------------- refusals of the tensor front end
def test_ops_refuse_cpu_tensors(ops):
    cache = ops.new_latent_cache(2, 16, device="cpu")
    q = torch.zeros(1, 8, 576, dtype=torch.bfloat16)
    table, lens = torch.zeros(1, 2, dtype=torch.int32), torch.zeros(1, dtype=torch.int64)
    f, _ = ops.rope_frequencies(64, device="cpu")
    with pytest.raises(ValueError):
        ops.rope(q, lens, f)
    with pytest.raises(ValueError):
        ops.latent_append(torch.zeros(1, 576, dtype=torch.bfloat16), lens, cache)
    with pytest.raises(ValueError):
        ops.latent_read(cache, table, torch.zeros(2, dtype=torch.int64), torch.zeros(3, 576, dtype=torch.bfloat16))
    with pytest.raises(ValueError):
        ops.latent_decode(q, cache, table, lens)
    with pytest.raises(ValueError):
        ops.latent_sparse_decode(q, ops.new_latent_cache(2, 16, True, device="cpu"), torch.zeros(1, 4, dtype=torch.int32))


def test_slots_of_maps_positions_through_the_table(ops):
    table = torch.tensor([[7, 3, 5], [0, 1, 2]], dtype=torch.int32)
    idx = torch.tensor([[0, 15, 16, 40, -1], [33, -1, -1, 2, 31]], dtype=torch.int32)
    got = ops.slots_of(idx, table, 16)
    assert got.dtype == torch.int32
    assert got.tolist() == [[112, 127, 48, 88, -1], [33, -1, -1, 2, 31]]


def test_slots_of_gives_no_cached_slot_past_the_table_or_for_pages_below_zero(ops):
    table = torch.tensor([[7, -1]], dtype=torch.int32)
    none = 2 ** 31 - 1
    idx = torch.tensor([[15, 16, 31, 32, 2 ** 31 - 1, -1]], dtype=torch.int32)
    assert ops.slots_of(idx, table, 16).tolist() == [[127, none, none, none, none, -1]]
    with pytest.raises(ValueError):
        ops.slots_of(idx, table[:, :0], 16)


def test_slots_of_gives_no_cached_slot_for_pages_whose_slots_pass_32_bits(ops):
    """page * page_size + row is formed in 64 bits: an entry of the table that is too large becomes the slot that no
    cache has, never a slot of another page and never the padding -1."""
    none = 2 ** 31 - 1
    table = torch.tensor([[2 ** 25, 2 ** 26, 2 ** 26 + 3, 2 ** 26 - 1, 2 ** 31 - 1, 5]], dtype=torch.int32)
    idx = torch.tensor([[0, 63, 64, 127, 128, 129, 192, 255, 256, 319, 320, 383, -1]], dtype=torch.int32)
    got = ops.slots_of(idx, table, 64)
    assert got.dtype == torch.int32
    assert got.tolist() == [[none] * 10 + [320, 383, -1]]
    # the last page whose slots are all below it
    last = torch.tensor([[2 ** 25 - 2]], dtype=torch.int32)
    assert ops.slots_of(torch.tensor([[0, 63]], dtype=torch.int32), last, 64).tolist() == [[2 ** 31 - 128, 2 ** 31 - 65]]
    assert ops.slots_of(idx[:, :1], torch.tensor([[2 ** 28 + 3]], dtype=torch.int32), 16).tolist() == [[none]]


def test_oracle_scale_keeps_every_code_finite_in_bf16():
    """Up to the largest bf16, 255 * 2^120: a scale of 2^119 at most, as 256 * 2^120 = 2^128 would read back as
    infinite; what 448 * 2^119 does not reach is stored as that."""
    big = np.zeros((1, 576))
    big[0, :512] = 255 * 2.0 ** 120
    big[0, 1], big[0, 128] = np.inf, -np.inf
    big[0, 256:384] = -448 * 2.0 ** 119
    assert L.pow2_scale(big[:, :512].reshape(-1, 4, 128)).tolist() == [[2.0 ** 119] * 4]
    codes, s = L.pack(big)
    raw = np.zeros((1, 656), dtype=np.uint8)
    raw[:, :512] = codes
    raw[:, 512:528] = s.astype(np.float32).view(np.uint8)
    back = torch.from_numpy(L.unpack(raw).astype(np.float32)).to(torch.bfloat16).double().numpy()
    most = 448 * 2.0 ** 119
    assert np.all(back[0, :128] == most) and back[0, 128] == -most and np.all(back[0, 129:256] == most)
    assert np.all(back[0, 256:384] == -most) and np.all(back[0, 384:512] == most)


# ---------------------------------------------------------------- the binding's functions
def test_the_bindings_functions_raise_on_refusals(abi):
    """The five calls under the header's names: a null or bad argument is an ICError with its code."""
    p, keep = _fake()
    rope = [p, 512, 128, p, p, 1.0, 0, 0, abi.IC_BF16, 4, 4, 128, 64, 64, ctypes.c_void_p(p.value + 65536), 512, 128, None]
    append = [p, 576, p, p, p, 1.0, 0, 4, abi.IC_FP8_E4M3, p, 2, 16, 656 * 16, p, 256, None]
    read = [p, abi.IC_BF16, 2, 16, 1152 * 16, p, 4, 4, p, 2, p, 10, p, 256, None]
    decode = [p, p, abi.IC_BF16, 4, 16, 1152 * 16, p, 4, 4, p, None, None, 0.04, 2, 1, 8, abi.IC_BF16, p, None, p,
              abi.ic_latent_decode_workspace_size(2, 1, 8, 64), None]
    sparse = [p, p, 4, 16, 656 * 16, p, 100, None, None, 0.04, 2, 8, abi.IC_BF16, p, None, p,
              abi.ic_latent_sparse_workspace_size(2, 8, 100), None]
    for call, args, ws in ((abi.ic_rope, rope, None), (abi.ic_latent_append, append, -2), (abi.ic_latent_read, read, -2),
                           (abi.ic_latent_decode, decode, -2), (abi.ic_latent_sparse_decode, sparse, -2)):
        bad = [(0, None)] + ([(ws, 8)] if ws else [(5, float("nan"))])
        for i, v in bad:
            with pytest.raises(abi.ICError) as e:
                call(*(args[:i] + [v] + args[i:][1:]))
            assert e.value.code == abi.IC_ERR_INVALID_ARG and call.__name__ in str(e.value)
    for call, args, i in ((abi.ic_rope, rope, 8), (abi.ic_latent_append, append, 8), (abi.ic_latent_read, read, 1),
                          (abi.ic_latent_decode, decode, 2)):
        with pytest.raises(abi.ICError) as e:
            call(*(args[:i] + [7] + args[i + 1:]))
        assert e.value.code == abi.IC_ERR_UNSUPPORTED
    with pytest.raises(abi.ICError) as e:
        abi.ic_latent_sparse_decode(*(sparse[:12] + [7] + sparse[13:]))
    assert e.value.code == abi.IC_ERR_UNSUPPORTED
