"""Rotary positions without a GPU: the frequency tables of pkv_rotary_inv_freq
against their formulas and closed forms, and the arguments that pkv_rotary and
paged_kv_append_rotary refuse on the host (nothing is enqueued)."""
import math

import numpy as np
import pytest
import torch

import paged_kv_cache_367_b200 as pkv

OK, ENULL, ESHAPE, EDTYPE, EUNSUP, EALIGN = 0, -1, -2, -3, -4, -7
F32, F16, BF16, FP8 = 0, 1, 2, 3
A = 1 << 20          # a fake, aligned "device" address; never dereferenced
NONE, LINEAR, BASE, RAMP, BANDED = range(5)


@pytest.fixture(scope="module")
def lib():
    from paged_kv_cache_367_b200 import build
    build.build()
    return pkv.load_library()


def plain(rot, base=10000.0):
    return base ** (-2.0 * np.arange(rot // 2) / rot)


@pytest.mark.parametrize("rot", [2, 64, 128, 256])
@pytest.mark.parametrize("base", [10000.0, 500000.0])
def test_unscaled_and_linear_frequencies(lib, rot, base):
    f, m = pkv.pkv_rotary_inv_freq(rot, base=base)
    assert f.dtype == torch.float64 and f.shape == (rot // 2,) and m == 1.0
    assert f[0].item() == 1.0
    np.testing.assert_allclose(f.numpy(), plain(rot, base), rtol=1e-14)
    f, m = pkv.pkv_rotary_inv_freq(rot, base=base, scaling=LINEAR, factor=4.0)
    np.testing.assert_allclose(f.numpy(), plain(rot, base) / 4.0, rtol=1e-14)
    assert m == 1.0


def test_base_scaling_keeps_the_fastest_pair_and_divides_the_slowest(lib):
    f, m = pkv.pkv_rotary_inv_freq(128, scaling=BASE, factor=8.0)
    assert f[0].item() == 1.0 and m == 1.0
    np.testing.assert_allclose(f[-1].item(), plain(128)[-1] / 8.0, rtol=1e-12)
    assert np.all(np.diff(f.numpy()) < 0)


def test_ramp_scaling(lib):
    rot, L, factor = 128, 8192.0, 8.0
    f, m = pkv.pkv_rotary_inv_freq(rot, scaling=RAMP, factor=factor, trained_len=L)
    assert m == pytest.approx(0.1 * math.log(factor) + 1.0, rel=1e-7)
    turns = L * plain(rot) / (2 * math.pi)
    ratio = f.numpy() / plain(rot)
    first = int(np.argmax(turns < 32.0))     # first pair below 32 turns
    last = int(np.argmax(turns < 1.0))       # first pair below one turn
    np.testing.assert_allclose(ratio[:first], 1.0, rtol=1e-14)
    np.testing.assert_allclose(ratio[last:], 1.0 / factor, rtol=1e-14)
    mid = np.arange(first - 1, last + 1)     # the ramp's ends are the pairs around them
    np.testing.assert_allclose(ratio[mid], 1 - (mid - mid[0]) / (mid[-1] - mid[0]) * (1 - 1 / factor),
                               rtol=1e-12)
    f1, m1 = pkv.pkv_rotary_inv_freq(rot, scaling=RAMP, factor=1.0, trained_len=L)
    assert m1 == 1.0
    np.testing.assert_allclose(f1.numpy(), plain(rot), rtol=1e-14)


def test_banded_scaling(lib):
    rot, L, factor = 128, 8192.0, 8.0
    f, m = pkv.pkv_rotary_inv_freq(rot, base=500000.0, scaling=BANDED, factor=factor,
                                   trained_len=L, low=1.0, high=4.0)
    assert m == 1.0
    p = plain(rot, 500000.0)
    for i, w in enumerate(2 * math.pi / p):  # by wavelength
        if w < L / 4.0:
            want = p[i]
        elif w > L / 1.0:
            want = p[i] / factor
        else:
            s = (L / w - 1.0) / 3.0
            want = (1 - s) * p[i] / factor + s * p[i]
        assert f[i].item() == pytest.approx(want, rel=1e-13)


@pytest.mark.parametrize("kw", [
    dict(rot_dim=0), dict(rot_dim=-2), dict(rot_dim=7), dict(rot_dim=514), dict(base=1.0),
    dict(base=float("nan")), dict(base=float("inf")), dict(scaling=LINEAR, factor=0.0),
    dict(scaling=LINEAR, factor=float("nan")), dict(scaling=BASE, factor=2.0, rot_dim=2),
    dict(scaling=RAMP, factor=2.0), dict(scaling=RAMP, factor=2.0, trained_len=64, low=2, high=1),
    dict(scaling=BANDED, factor=2.0, trained_len=64, low=0.0),
    dict(scaling=BANDED, factor=2.0, trained_len=-1), dict(scaling=5), dict(scaling=-1),
])
def test_inv_freq_refusals(lib, kw):
    kw = dict(dict(rot_dim=64), **kw)
    with pytest.raises(pkv.PagedKVError):
        pkv.pkv_rotary_inv_freq(kw.pop("rot_dim"), **kw)


def rotary(lib, **kw):
    a = dict(q_out=A, query=A, k_out=A, key=A, positions=A, inv_freq=A, magnitude=1.0,
             num_tokens=4, num_heads=8, num_kv_heads=2, head_dim=128, rot_dim=128,
             q_stride=1024, q_out_stride=1024, k_stride=256, k_out_stride=256, dtype=BF16,
             flags=0, stream=None)
    a.update(kw)
    return lib.pkv_rotary(*a.values())


@pytest.mark.parametrize("kw,code", [
    (dict(num_tokens=0, query=None), OK), (dict(num_heads=0, num_kv_heads=0, key=None), OK),
    (dict(q_out=None), ENULL), (dict(key=None), ENULL), (dict(positions=None), ENULL),
    (dict(inv_freq=None), ENULL), (dict(num_tokens=-1), ESHAPE), (dict(num_heads=-1), ESHAPE),
    (dict(head_dim=100), ESHAPE), (dict(head_dim=0), ESHAPE), (dict(rot_dim=0), ESHAPE),
    (dict(rot_dim=63), ESHAPE), (dict(rot_dim=130), ESHAPE), (dict(magnitude=float("inf")), ESHAPE),
    (dict(flags=4), ESHAPE), (dict(q_stride=-8), ESHAPE), (dict(q_out_stride=1016), ESHAPE),
    (dict(k_out_stride=255), ESHAPE), (dict(q_stride=2048), ESHAPE),   # in place, other stride
    (dict(num_heads=4093, q_out_stride=1 << 20, q_stride=1 << 20), ESHAPE),
    (dict(head_dim=520, rot_dim=64, q_out_stride=8192, q_stride=8192, k_stride=2048,
          k_out_stride=2048), EUNSUP),
    (dict(dtype=FP8), EDTYPE), (dict(dtype=9), EDTYPE), (dict(query=A + 8, q_out=A + 8), EALIGN),
    (dict(positions=A + 4), EALIGN), (dict(inv_freq=A + 4), EALIGN),
])
def test_rotary_rejects_bad_arguments(lib, kw, code):
    assert rotary(lib, **kw) == code


def append_rotary(lib, **kw):
    a = dict(q_out=A, query=A, key=A, value=A, k_cache=A, v_cache=A, slot_mapping=A, positions=A,
             inv_freq=A, magnitude=1.0, num_tokens=4, num_heads=8, num_kv_heads=2, head_dim=128,
             rot_dim=64, block_size=16, num_blocks=10, q_stride=1024, q_out_stride=1024,
             k_stride=256, v_stride=256, src_dtype=BF16, cache_dtype=BF16, k_scale=A, v_scale=A,
             flags=0, stream=None)
    a.update(kw)
    return lib.paged_kv_append_rotary(*a.values())


@pytest.mark.parametrize("kw,code", [
    (dict(num_tokens=0, key=None), OK), (dict(key=None), ENULL), (dict(value=None), ENULL),
    (dict(query=None), ENULL), (dict(k_cache=None), ENULL), (dict(slot_mapping=None), ENULL),
    (dict(cache_dtype=FP8, v_scale=None), ENULL), (dict(num_kv_heads=0), ESHAPE),
    (dict(block_size=0), ESHAPE), (dict(num_blocks=0), ESHAPE),
    (dict(num_blocks=1 << 62, block_size=16), ESHAPE), (dict(rot_dim=3), ESHAPE),
    (dict(flags=2), ESHAPE), (dict(q_out_stride=1000), ESHAPE), (dict(v_stride=-1), ESHAPE),
    (dict(src_dtype=F32), EDTYPE), (dict(src_dtype=FP8, cache_dtype=FP8), EDTYPE),
    (dict(cache_dtype=F16), EDTYPE), (dict(key=A + 2), EALIGN), (dict(v_cache=A + 8), EALIGN),
    (dict(slot_mapping=A + 4), EALIGN), (dict(head_dim=520, rot_dim=64, q_out_stride=8192,
                                                       q_stride=8192), EUNSUP),
])
def test_append_rotary_rejects_bad_arguments(lib, kw, code):
    assert append_rotary(lib, **kw) == code


def test_binding_refuses_what_the_pointers_cannot_say(lib):
    T, Hq, Hkv, D = 3, 4, 2, 64
    q, k = torch.zeros(T, Hq, D), torch.zeros(T, Hkv, D)
    pos = torch.zeros(T, dtype=torch.int64)
    f, _ = pkv.pkv_rotary_inv_freq(D)
    pool = torch.zeros(2, 8, Hkv, D)
    slots = torch.zeros(T, dtype=torch.int64)

    def rot(q_out=q, query=q, positions=pos, inv_freq=f, **kw):
        pkv.pkv_rotary(q_out, query, positions, inv_freq, stream=0, **kw)

    with pytest.raises(ValueError):          # not on a GPU
        rot()
    with pytest.raises(ValueError):
        rot(q_out=None)
    with pytest.raises(ValueError):
        rot(query=None, q_out=None)
    with pytest.raises(ValueError):
        rot(key=k)
    with pytest.raises(ValueError):
        rot(q_out=torch.zeros(T, Hq + 1, D))
    with pytest.raises(TypeError):
        rot(q_out=q.half())
    with pytest.raises(ValueError):          # heads of a token apart
        rot(q_out=torch.zeros(T, Hq, 2 * D)[..., :D])
    with pytest.raises(ValueError):
        rot(positions=pos.int())
    with pytest.raises(ValueError):
        rot(positions=pos[:2])
    with pytest.raises(ValueError):
        rot(inv_freq=f.float())

    def app(key=k, value=k, k_cache=pool, v_cache=pool, slot_mapping=slots, **kw):
        pkv.paged_kv_append_rotary(q, q, key, value, k_cache, v_cache, slot_mapping, pos, f,
                                   stream=0, **kw)

    with pytest.raises(ValueError):
        app()
    with pytest.raises(ValueError):
        app(value=torch.zeros(T, Hkv + 1, D))
    with pytest.raises(ValueError):
        app(k_cache=torch.zeros(2, 8, Hkv, D + 8))
    with pytest.raises(ValueError):
        app(v_cache=torch.zeros(3, 8, Hkv, D))
    with pytest.raises(ValueError):
        app(k_cache=torch.zeros(2, Hkv, 8, D).transpose(1, 2))
    with pytest.raises(ValueError):
        app(slot_mapping=slots[:1])
    with pytest.raises(TypeError):
        app(k_scale=torch.ones(1, dtype=torch.float64))


@pytest.mark.parametrize("big", [1 << 31, (1 << 32) + 3])
def test_binding_refuses_sizes_past_32_bits(lib, big):
    """They would reach the library without their upper bits: 3 rows rotated of 2^32 + 3."""
    D = 64
    rows = torch.zeros(1, 2, D).expand(big, 2, D)
    pos = torch.zeros(1, dtype=torch.int64).expand(big)
    pool = torch.zeros(2, 8, 2, D)
    f, _ = pkv.pkv_rotary_inv_freq(D)
    with pytest.raises(ValueError, match="32 bits"):
        pkv.pkv_rotary(rows, rows, pos, f, stream=0)
    with pytest.raises(ValueError, match="32 bits"):
        pkv.paged_kv_append_rotary(None, None, rows, rows, pool, pool, pos, pos, f, stream=0)
    with pytest.raises(ValueError, match="32 bits"):
        pkv.pkv_rotary_inv_freq(big)


@pytest.mark.parametrize("scale", ["k_scale", "v_scale"])
def test_append_rotary_rejects_a_misaligned_scale(lib, scale):
    assert append_rotary(lib, cache_dtype=FP8, **{scale: A + 2}) == EALIGN
