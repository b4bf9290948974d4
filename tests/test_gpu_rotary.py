"""pkv_rotary and paged_kv_append_rotary on the GPU against the formula in 64 bits.

Tolerance, per element: the result is rounded once (half a step of the output
type relative to its value, or half a step of its smallest subnormal), and before
that the fp32 arithmetic is off by at most m (|x_a| + |x_b|) * 5e-7: the cosine
and sine by 2 pi 2^-26 (the reduced turns rounded to fp32), two fp32 steps of the
function and half a step of the magnitude, the products by half a step each."""
import numpy as np
import pytest
import torch

import oracle
import paged_kv_cache_367_b200 as pkv
from paged_kv_cache_367_b200 import workloads as W

pytestmark = pytest.mark.gpu

TORCH = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
HALF_SUBNORMAL = {"f32": 0.0, "f16": 2.0 ** -25, "bf16": 0.0, "e4m3": 2.0 ** -10}
HALF_STEP = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8, "e4m3": 2.0 ** -4}


def formula(x, pos, f, m, inter, transposed):
    """The rotated rows in fp64, and |x_a| + |x_b| of each element's pair."""
    x = x.detach().double().cpu().numpy()
    pos = np.asarray(pos.cpu().numpy(), np.longdouble)
    f = f.cpu().numpy()
    r = 2 * len(f)
    t = np.asarray(pos[:, None] * f[None, :].astype(np.longdouble), np.longdouble)
    c, s = np.cos(t).astype(np.float64)[:, None], np.sin(t).astype(np.float64)[:, None]
    if transposed:
        s = -s
    ia = np.arange(0, r, 2) if inter else np.arange(r // 2)
    ib = ia + 1 if inter else ia + r // 2
    y, size = x.copy(), np.zeros_like(x)
    a, b = x[..., ia], x[..., ib]
    y[..., ia] = m * (a * c - b * s)
    y[..., ib] = m * (b * c + a * s)
    size[..., ia] = size[..., ib] = np.abs(a) + np.abs(b)
    return y, size


def assert_rotated(got, want, size, m, dt):
    got = got.detach().double().cpu().numpy() if torch.is_tensor(got) else got
    tol = np.abs(want) * HALF_STEP[dt] * (1 + 1e-6) + HALF_SUBNORMAL[dt] + 5e-7 * m * size
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), (int(bad.sum()), np.abs(got - want)[bad].max())


def rows(T, heads, D, dt, gen, dev, fused):
    """Row tensors of the given head counts: slices of one tensor, or their own."""
    if fused:
        x = torch.randn((T, sum(heads), D), generator=gen, device=dev).to(TORCH[dt])
        return list(torch.split(x, heads, 1))
    return [torch.randn((T, h, D), generator=gen, device=dev).to(TORCH[dt]) for h in heads]


SIZES = [  # T, Hq, Hkv, D, rot
    (1, 32, 8, 128, 128), (1, 1, 1, 8, 2), (7, 5, 2, 72, 40), (33, 3, 1, 64, 22),
    (130, 12, 3, 96, 96), (257, 1, 1, 16, 16), (19, 8, 8, 256, 256), (5, 2, 1, 256, 2),
    (6, 1, 1, 512, 510), (3, 2, 1, 120, 48),
    (700, 40, 40, 128, 64), (2048, 1, 1, 64, 64),
]


@pytest.mark.parametrize("T,Hq,Hkv,D,rot", SIZES)
@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("inter", [False, True])
def test_rotary_matches_the_formula(cuda_dev, T, Hq, Hkv, D, rot, dt, inter):
    gen = torch.Generator(device=cuda_dev).manual_seed(T + D + rot)
    q, k = rows(T, [Hq, Hkv], D, dt, gen, cuda_dev, fused=T % 2 == 1)
    pos = torch.randint(0, 1 << 20, (T,), generator=gen, device=cuda_dev)
    f, _ = pkv.pkv_rotary_inv_freq(rot, device=cuda_dev)
    m, transposed = (1.25, True) if T % 3 == 0 else (1.0, False)
    flags = (pkv.PKV_ROTARY_INTERLEAVED if inter else 0) | \
        (pkv.PKV_ROTARY_TRANSPOSED if transposed else 0)
    qo, ko = torch.full_like(q, float("nan")), torch.full_like(k, float("nan"))
    qo, ko = qo.contiguous(), ko.contiguous()
    keep = q.clone(), k.clone()
    pkv.pkv_rotary(qo, q, pos, f, k_out=ko, key=k, magnitude=m, flags=flags)
    for got, x in ((qo, q), (ko, k)):
        want, size = formula(x, pos, f, m, inter, transposed)
        assert_rotated(got, want, size, m, dt)
        assert torch.equal(got[..., rot:], x[..., rot:])
    assert torch.equal(q, keep[0]) and torch.equal(k, keep[1])
    # In place (slices of the wider tensor), the same bits; then one side alone.
    pkv.pkv_rotary(q, q, pos, f, k_out=k, key=k, magnitude=m, flags=flags)
    assert torch.equal(q, qo) and torch.equal(k, ko)
    ko.fill_(float("nan"))
    pkv.pkv_rotary(None, None, pos, f, k_out=ko, key=keep[1], magnitude=m, flags=flags)
    assert torch.equal(ko, k)


@pytest.mark.parametrize("pad", [1, 4, 8])
def test_rotary_row_strides(cuda_dev, pad):
    """Rows with gaps between tokens (strides that are no multiple of a vector);
    what lies between the output rows stays as it was."""
    T, Hq, D = 9, 3, 64
    gen = torch.Generator(device=cuda_dev).manual_seed(pad)
    wide = torch.randn((T, Hq * D + pad), generator=gen, device=cuda_dev).to(torch.bfloat16)
    out = torch.full_like(wide, 7.0)
    q, qo = (x[:, :Hq * D].unflatten(1, (Hq, D)) for x in (wide, out))
    pos = torch.arange(T, device=cuda_dev)
    f, _ = pkv.pkv_rotary_inv_freq(D, device=cuda_dev)
    pkv.pkv_rotary(qo, q, pos, f)
    want, size = formula(q, pos, f, 1.0, False, False)
    assert_rotated(qo, want, size, 1.0, "bf16")
    assert torch.all(out[:, Hq * D:] == 7.0)


def test_rotary_broadcast_rows(cuda_dev):
    """One row at many positions (an input with a token stride of 0)."""
    gen = torch.Generator(device=cuda_dev).manual_seed(3)
    q = torch.randn((1, 4, 128), generator=gen, device=cuda_dev).expand(50, 4, 128)
    pos = torch.arange(50, device=cuda_dev) * 977
    f, _ = pkv.pkv_rotary_inv_freq(128, device=cuda_dev)
    out = torch.empty((50, 4, 128), device=cuda_dev)
    pkv.pkv_rotary(out, q, pos, f)
    want, size = formula(q, pos, f, 1.0, False, False)
    assert_rotated(out, want, size, 1.0, "f32")


@pytest.mark.parametrize("p", [0, -1, -12345, (1 << 31) - 1, 1 << 31, (1 << 33) + 5])
def test_rotary_far_and_negative_positions(cuda_dev, p):
    """The angle keeps its fp32 accuracy far out: position times frequency is
    reduced in fp64 (2^33 turns leave 2^-19 of one in 53 bits; counted here)."""
    gen = torch.Generator(device=cuda_dev).manual_seed(1)
    q = torch.randn((2, 2, 128), generator=gen, device=cuda_dev)
    pos = torch.tensor([p, p + 1], device=cuda_dev)
    f, _ = pkv.pkv_rotary_inv_freq(128, device=cuda_dev)
    out = torch.empty_like(q)
    pkv.pkv_rotary(out, q, pos, f)
    want, size = formula(q, pos, f, 1.0, False, False)
    # Two fp64 roundings of the turns (2^-52 of them together), times 2 pi.
    extra = 2 * np.pi * (abs(p) + 1) / (2 * np.pi) * 2.0 ** -52
    assert_rotated(out, want, size * (1 + extra / 5e-7), 1.0, "f32")
    if p == 0:
        assert torch.equal(out[0], q[0])


def test_rotary_non_finite_values_stay_in_their_pairs(cuda_dev):
    q = torch.ones((1, 1, 64), device=cuda_dev)
    q[0, 0, 3], q[0, 0, 40] = float("nan"), float("inf")
    f, _ = pkv.pkv_rotary_inv_freq(64, device=cuda_dev)
    out = torch.empty_like(q)
    pkv.pkv_rotary(out, q, torch.tensor([5], device=cuda_dev), f)
    bad = {i for i in range(64) if not torch.isfinite(out[0, 0, i])}
    assert bad == {3, 35, 8, 40}


@pytest.mark.parametrize("inter", [False, True])
def test_rotary_transposed_is_the_gradient(cuda_dev, inter):
    """Against the formula's gradient and against differences of the call itself."""
    T, H, D, rot, m = 6, 2, 32, 24, 1.5
    gen = torch.Generator(device=cuda_dev).manual_seed(11)
    x = torch.randn((T, H, D), generator=gen, device=cuda_dev)
    dy = torch.randn((T, H, D), generator=gen, device=cuda_dev)
    pos = torch.arange(T, device=cuda_dev) * 37
    f, _ = pkv.pkv_rotary_inv_freq(rot, device=cuda_dev)
    fl = pkv.PKV_ROTARY_INTERLEAVED if inter else 0
    dx = torch.empty_like(x)
    pkv.pkv_rotary(dx, dy, pos, f, magnitude=m, flags=fl | pkv.PKV_ROTARY_TRANSPOSED)
    # Autograd of the formula in 64 bits.
    x64 = x.double().requires_grad_()
    t = (pos.double()[:, None] * f)[:, None]
    a, b = ((x64[..., 0:rot:2], x64[..., 1:rot:2]) if inter
            else (x64[..., :rot // 2], x64[..., rot // 2:rot]))
    ya, yb = m * (a * t.cos() - b * t.sin()), m * (b * t.cos() + a * t.sin())
    y = torch.cat([torch.stack([ya, yb], -1).flatten(-2) if inter else torch.cat([ya, yb], -1),
                   x64[..., rot:]], -1)
    (y * dy.double()).sum().backward()
    _, size = formula(dy, pos, f, m, inter, True)
    assert_rotated(dx, x64.grad.cpu().numpy(), size, m, "f32")
    # The call is linear: its difference over a step of 1 in an element is exact
    # but for the roundings of two calls.
    base, moved = torch.empty_like(x), torch.empty_like(x)
    pkv.pkv_rotary(base, x, pos, f, magnitude=m, flags=fl)
    for e in (0, rot // 2, rot - 1, D - 1):
        step = x.clone()
        step[..., e] += 1.0
        pkv.pkv_rotary(moved, step, pos, f, magnitude=m, flags=fl)
        diff = ((moved.double() - base.double()) * dy.double()).sum(-1)
        # Two elements of y move; each call's are off by 18 (2^-24 + 5e-7) at most
        # (|y| <= m (|a| + |b|) <= 1.5 * 12), the step by 2^-24 * 6 * m, dx by
        # 5 m (2^-24 + 5e-7) * 2; |dy| <= 5.
        assert (diff - dx[..., e].double()).abs().max() <= 5 * (4 * 18 * 5.6e-7 + 1e-6) + 1e-5


# ------------------------------------------------------------------ append ----

def append_case(dev, T, Hq, Hkv, D, rot, bs, src, cache, seed, fused):
    rng = np.random.default_rng(seed)
    gen = torch.Generator(device=dev).manual_seed(seed)
    nb = -(-T // bs) + 3
    q, k, v = rows(T, [Hq, Hkv, Hkv], D, src, gen, dev, fused)
    kc, vc = (W._randn((nb, bs, Hkv, D), cache, gen, dev) for _ in range(2))
    slots = rng.choice(nb * bs, T, replace=False).astype(np.int64)
    slots[::5] = -1
    if T > 3:
        slots[3] = nb * bs            # one past the pool
    pos = torch.from_numpy(rng.integers(0, 1 << 20, T)).to(dev)
    f, _ = pkv.pkv_rotary_inv_freq(rot, device=dev)
    return q, k, v, kc, vc, slots, pos, f


def check_pool(pool, before, rows64, size, m, slots, cache, scale):
    """Written slots hold the rows (within the tolerance), all others their bytes."""
    nb, bs = pool.shape[:2]
    got, old = W.host(pool), before
    flat = lambda x: x.reshape(nb * bs, *x.shape[2:])
    got, old = flat(got), flat(old)
    kept = [t for t, s in enumerate(slots) if 0 <= s < nb * bs]
    rest = np.ones(nb * bs, bool)
    rest[slots[kept]] = False
    assert np.array_equal(got[rest].view(np.uint8), old[rest].view(np.uint8))
    new = pool.reshape(nb * bs, *pool.shape[2:])[torch.from_numpy(slots[kept]).to(pool.device)]
    want = rows64[kept] / scale
    if cache == "e4m3":
        new = new.view(torch.float8_e4m3fn).float()
        want = np.clip(want, -448, 448)
    assert_rotated(new, want, size[kept] / scale, m, cache)


@pytest.mark.parametrize("T,Hq,Hkv,D,rot,bs", [
    (1, 32, 8, 128, 128, 16), (50, 4, 3, 128, 64, 16), (23, 2, 1, 72, 40, 8), (9, 3, 2, 64, 6, 32),
    (400, 8, 8, 64, 64, 16), (65, 1, 1, 256, 256, 8), (12, 0, 2, 128, 128, 16),
])
@pytest.mark.parametrize("src,cache", [("f32", "f32"), ("f16", "f16"), ("bf16", "bf16"),
                                       ("f32", "e4m3"), ("f16", "e4m3"), ("bf16", "e4m3")])
@pytest.mark.parametrize("inter", [False, True])
def test_append_rotary_matches_the_formula(cuda_dev, T, Hq, Hkv, D, rot, bs, src, cache, inter):
    m = 1.125
    q, k, v, kc, vc, slots, pos, f = append_case(cuda_dev, T, Hq, Hkv, D, rot, bs, src, cache,
                                                 T + D, fused=T % 2 == 0)
    k_before, v_before = W.host(kc).copy(), W.host(vc).copy()
    sc = [float(x.float().abs().amax()) / 300.0 for x in (k, v)]
    scale = [torch.tensor([x], dtype=torch.float32, device=cuda_dev) for x in sc]
    sc = [x.item() for x in scale]
    if cache != "e4m3":
        sc = [1.0, 1.0]
    qo = torch.full(q.shape, float("nan"), dtype=q.dtype, device=cuda_dev) if Hq else None
    pkv.paged_kv_append_rotary(qo, q if Hq else None, k, v, kc, vc,
                               torch.from_numpy(slots).to(cuda_dev), pos, f, magnitude=m,
                               k_scale=scale[0], v_scale=scale[1],
                               flags=pkv.PKV_ROTARY_INTERLEAVED if inter else 0)
    if Hq:
        want, size = formula(q, pos, f, m, inter, False)
        assert_rotated(qo, want, size, m, src)
        assert torch.equal(qo[..., rot:], q[..., rot:])
    want, size = formula(k, pos, f, m, inter, False)
    check_pool(kc, k_before, want, size, m, slots, cache, sc[0])
    # The values: what paged_kv_append writes, byte for byte.
    vh, kh = v_before.copy(), k_before.copy()
    oracle.append(W.host(k), W.host(v), kh, vh, slots, num_kv_heads=Hkv, head_dim=D,
                  block_size=bs, num_blocks=kc.shape[0], src_dtype=src, cache_dtype=cache,
                  k_scale=sc[0], v_scale=sc[1])
    assert np.array_equal(W.host(vc).view(np.uint8), vh.view(np.uint8))
    # Past rot_dim the keys too.
    assert np.array_equal(W.host(kc)[..., rot:], kh[..., rot:], equal_nan=cache != "bf16")


def test_append_rotary_saturates(cuda_dev):
    k = torch.full((1, 1, 64), 1e6, device=cuda_dev)
    kc = torch.zeros((1, 8, 1, 64), dtype=torch.uint8, device=cuda_dev)
    vc = torch.zeros_like(kc)
    one = torch.ones(1, device=cuda_dev)
    f, _ = pkv.pkv_rotary_inv_freq(64, device=cuda_dev)
    pkv.paged_kv_append_rotary(None, None, k, -k, kc, vc, torch.tensor([2], device=cuda_dev),
                               torch.tensor([0], device=cuda_dev), f, k_scale=one, v_scale=one)
    assert torch.all(kc.view(8, 64)[2] == 0x7E) and torch.all(vc.view(8, 64)[2] == 0xFE)
    assert kc.sum().item() == 64 * 0x7E


@pytest.mark.parametrize("scale", [1.0, 0.011160714, 0.0371, 3.0, 1e-30, 1e30, 2e-39, -0.25, 0.0,
                                   float("inf")])
@pytest.mark.parametrize("D", [64, 72])
def test_append_rotary_codes_are_those_of_append(cuda_dev, scale, D):
    """Values (and keys at position 0) over the whole range of codes, at ties, one
    step beside them, and at zeros, infinities and NaN: the bytes paged_kv_append
    stores."""
    sc = torch.tensor([scale], dtype=torch.float32, device=cuda_dev)
    gen = torch.Generator(device=cuda_dev).manual_seed(9)
    T, Hkv, bs = 4096, 1, 16
    u = torch.randn((T // 2, D), generator=gen, device=cuda_dev)
    u = u * torch.exp2(torch.randint(-14, 10, (T // 2, 1), generator=gen, device=cuda_dev).float())
    codes = torch.arange(256, device=cuda_dev, dtype=torch.int32).to(torch.uint8)
    e = codes.view(torch.float8_e4m3fn).float()
    e = torch.sort(e[torch.isfinite(e)]).values
    ties = torch.cat([e, (e[1:] + e[:-1]) / 2])
    near = torch.cat([ties * (1 + k * 2.0 ** -23) for k in range(-3, 4)])
    special = torch.tensor([0.0, -0.0, float("inf"), float("-inf"), float("nan"), 1e38, -1e38,
                            1e-38, 1e-45, -1e-45], device=cuda_dev)
    pool_of = torch.cat([near, special])
    pick = torch.randint(0, len(pool_of), (T // 2, D), generator=gen, device=cuda_dev)
    v = (torch.cat([u, pool_of[pick]]) * sc if 0 < abs(scale) < 1e35 else
         torch.cat([u, pool_of[pick]])).view(T, 1, D).contiguous()
    k = torch.where(torch.isfinite(v) & (v != 0), v, torch.ones_like(v))
    kc, vc, kw, vw = (torch.zeros((T // bs, bs, Hkv, D), dtype=torch.uint8, device=cuda_dev)
                      for _ in range(4))
    slots = torch.arange(T, device=cuda_dev)
    f, _ = pkv.pkv_rotary_inv_freq(D, device=cuda_dev)
    pkv.paged_kv_append(k, v, kw, vw, slots, k_scale=sc, v_scale=sc)
    pkv.paged_kv_append_rotary(None, None, k, v, kc, vc, slots, torch.zeros_like(slots), f,
                               k_scale=sc, v_scale=sc)
    assert torch.equal(vc, vw)
    assert torch.equal(kc, kw)


def test_append_rotary_queries_in_place_and_zero_tokens(cuda_dev):
    q, k, v, kc, vc, slots, pos, f = append_case(cuda_dev, 20, 4, 2, 128, 128, 16, "bf16", "bf16",
                                                 5, fused=True)
    s = torch.from_numpy(slots).to(cuda_dev)
    qo = torch.empty(q.shape, dtype=q.dtype, device=cuda_dev)
    pkv.paged_kv_append_rotary(qo, q, k, v, kc, vc, s, pos, f)
    first = kc.clone(), vc.clone()
    kv = k.clone(), v.clone()
    pkv.paged_kv_append_rotary(q, q, k, v, kc, vc, s, pos, f)
    assert torch.equal(q, qo) and torch.equal(kc, first[0]) and torch.equal(vc, first[1])
    assert torch.equal(k, kv[0]) and torch.equal(v, kv[1])    # the slices beside q are kept
    pkv.paged_kv_append_rotary(q[:0], q[:0], k[:0], v[:0], kc, vc, s[:0], pos[:0], f)
    assert torch.equal(kc, first[0])


def test_append_rotary_into_a_pool_past_32_bit_offsets(cuda_dev):
    """Slots whose element offsets pass 2^31 (and byte offsets 2^32)."""
    Hkv, D, bs = 8, 128, 16
    nb = (1 << 31) // (bs * Hkv * D) + 8
    kc = torch.zeros((nb, bs, Hkv, D), dtype=torch.bfloat16, device=cuda_dev)
    vc = torch.zeros_like(kc)
    k = torch.randn((2, Hkv, D), device=cuda_dev).to(torch.bfloat16)
    slots = torch.tensor([nb * bs - 1, 0], device=cuda_dev)
    f, _ = pkv.pkv_rotary_inv_freq(D, device=cuda_dev)
    zero = torch.zeros(2, dtype=torch.int64, device=cuda_dev)
    pkv.paged_kv_append_rotary(None, None, k, k, kc, vc, slots, zero, f)
    assert torch.equal(kc[-1, -1], k[0]) and torch.equal(vc[-1, -1], k[0])
    assert torch.equal(kc[0, 0], k[1])
    assert int(torch.count_nonzero(kc[:, 0, 0, 0])) + int(torch.count_nonzero(kc[-1, -1])) <= 1 + Hkv * D


@pytest.mark.parametrize("early", [False, True])
def test_step_on_a_rotated_cache(cuda_dev, early):
    """A serving step as it is run: keys rotated into the cache, the queries
    rotated, the decode over it; captured into a graph, replayed with new inputs,
    and equal to the eager calls. With the early-starting decode the queries are
    rotated by a launch of their own before the append."""
    cfg = W.CONFIGS["gqa70b"].replace(num_seqs=9, lens=("uniform", 20, 700), partition_size=128,
                                      seed=77)
    wl = W.make_workload(cfg, device=cuda_dev)
    S, Hq, Hkv, D = cfg.num_seqs, cfg.num_heads, cfg.num_kv_heads, cfg.head_dim
    bt, lens, slots = (torch.from_numpy(x).to(cuda_dev) for x in
                       (wl.block_table, wl.seq_lens, wl.slot_mapping))
    pos = lens.long() - 1
    f, m = pkv.pkv_rotary_inv_freq(D, scaling=pkv.PKV_ROTARY_SCALE_RAMP, factor=4.0,
                                   trained_len=512, device=cuda_dev)
    ws = torch.empty(pkv.paged_attention_workspace_size(S, Hq, Hkv, D, wl.max_seq_len, 128),
                     dtype=torch.uint8, device=cuda_dev)
    qkv = torch.empty((S, Hq + 2 * Hkv, D), dtype=torch.bfloat16, device=cuda_dev)
    q, k, v = torch.split(qkv, [Hq, Hkv, Hkv], 1)
    qo, out = torch.empty((2, S, Hq, D), dtype=torch.bfloat16, device=cuda_dev)

    def step():
        if early:
            pkv.pkv_rotary(qo, q, pos, f, magnitude=m)
            pkv.paged_kv_append_rotary(None, None, k, v, wl.k_cache, wl.v_cache, slots, pos, f,
                                       magnitude=m)
        else:
            pkv.paged_kv_append_rotary(qo, q, k, v, wl.k_cache, wl.v_cache, slots, pos, f,
                                       magnitude=m)
        pkv.paged_attention_decode(out, qo, wl.k_cache, wl.v_cache, bt, lens,
                                   max_seq_len=wl.max_seq_len, scale=cfg.scale,
                                   partition_size=128, workspace=ws,
                                   flags=pkv.PKV_DECODE_EARLY_START if early else 0)

    def draw(seed):
        gen = torch.Generator(device=cuda_dev).manual_seed(seed)
        qkv.copy_(torch.randn(qkv.shape, generator=gen, device=cuda_dev))

    side = torch.cuda.Stream()
    draw(1)
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):        # the current stream, not the default one
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for seed in (2, 3):
        draw(seed)
        out.fill_(float("nan"))
        graph.replay()
        got = out.clone()
        kc, vc = W.host(wl.k_cache).copy(), W.host(wl.v_cache).copy()
        want, _ = oracle.decode(W.host(qo), kc, vc, wl.block_table, wl.seq_lens, num_heads=Hq,
                                num_kv_heads=Hkv, head_dim=D, block_size=cfg.block_size,
                                scale=cfg.scale, q_dtype="bf16", cache_dtype="bf16")
        err = np.abs(got.double().cpu().numpy() - want)
        assert err.max() <= 1e-2 and err.mean() <= 1e-3
        wq, size = formula(q, pos, f, m, False, False)
        assert_rotated(qo, wq, size, m, "bf16")
        wk, size = formula(k, pos, f, m, False, False)
        rows_ = wl.k_cache.view(-1, Hkv, D)[slots]
        assert_rotated(rows_, wk, size, m, "bf16")
        step()
        assert torch.equal(out, got)


@pytest.mark.parametrize("D", [16, 32, 512])
@pytest.mark.parametrize("inter", [False, True])
def test_rotary_one_head_at_many_positions(cuda_dev, D, inter):
    """A block of as many tokens as it can hold: its table of cosines and sines takes
    all of the shared memory that needs no opt-in."""
    T = 148 * 8 * (4096 // D) + 777
    gen = torch.Generator(device=cuda_dev).manual_seed(D)
    q = torch.randn((T, 1, D), generator=gen, device=cuda_dev).to(torch.bfloat16)
    pos = torch.randint(0, 1 << 20, (T,), generator=gen, device=cuda_dev)
    f, _ = pkv.pkv_rotary_inv_freq(D, device=cuda_dev)
    out = torch.full_like(q, float("nan"))
    pkv.pkv_rotary(out, q, pos, f, flags=pkv.PKV_ROTARY_INTERLEAVED if inter else 0)
    assert torch.isfinite(out).all()
    some = torch.cat([torch.arange(800), torch.randint(0, T, (4000,)), torch.arange(T - 800, T)]).cuda()
    want, size = formula(q[some], pos[some], f, 1.0, inter, False)
    assert_rotated(out[some], want, size, 1.0, "bf16")


@pytest.mark.parametrize("p", [1, 3, 1000, (1 << 20) + 1, 1 << 40, -(1 << 52)])
def test_rotary_angle_bound(cuda_dev, p):
    """The stated bound of the angle, 2^-26 + |p f| 2^-53 turns, in fp32: a unit vector
    moves by 2 pi times that, and by three fp32 steps of sine, cosine and products."""
    f, _ = pkv.pkv_rotary_inv_freq(64, device=cuda_dev)
    x = torch.zeros((1, 1, 64), device=cuda_dev)
    x[..., :32] = 1.0
    out = torch.empty_like(x)
    pkv.pkv_rotary(out, x, torch.tensor([p], device=cuda_dev), f)
    with_f = f.cpu().numpy().astype(np.longdouble)
    t = np.asarray([p], np.longdouble) * with_f
    bound = 2 * np.pi * (2.0 ** -26 + np.abs(t) * 2.0 ** -53) + 3 * 2.0 ** -23
    # The reference's own reduction: a 64-bit mantissa of |t|.
    bound += np.abs(t) * 2.0 ** -63
    got = out.cpu().numpy().astype(np.longdouble)[0, 0]
    assert (np.abs(got[:32] - np.cos(t)) <= bound).all()
    assert (np.abs(got[32:] - np.sin(t)) <= bound).all()
