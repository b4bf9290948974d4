"""paged_cross_attention without a GPU: the arguments it refuses on the host, and the
workspace it asks for."""
import pytest
import torch

import paged_kv_cache_367_b200 as pkv

OK, ENULL, ESHAPE, EDTYPE, EUNSUP, EWS, EALIGN = 0, -1, -2, -3, -4, -5, -7
F32, F16, BF16, FP8 = 0, 1, 2, 3
A = 1 << 20          # a fake, aligned "device" address; never dereferenced


@pytest.fixture(scope="module")
def lib():
    from paged_kv_cache_367_b200 import build
    build.build()
    return pkv.load_library()


def cross(lib, **kw):
    a = dict(out=A, query=A, k_cache=A, v_cache=A, block_table=A, seq_lens=A, query_start=A,
             num_seqs=2, num_q_tokens=10, max_q_len=8, num_heads=8, num_kv_heads=2, head_dim=128,
             block_size=16, max_blocks_per_seq=8, num_blocks=100, max_seq_len=100, scale=0.1,
             q_dtype=BF16, cache_dtype=BF16, k_scale=A, v_scale=A, workspace=None,
             workspace_bytes=0, stream=None)
    a.update(kw)
    return lib.paged_cross_attention(*a.values())


@pytest.mark.parametrize("kw,code", [
    (dict(num_seqs=0), OK), (dict(num_q_tokens=0, out=None), OK), (dict(max_q_len=0), OK),
    (dict(out=None), ENULL), (dict(query_start=None), ENULL), (dict(seq_lens=None), ENULL),
    (dict(cache_dtype=FP8, k_scale=None), ENULL), (dict(cache_dtype=FP8, v_scale=None), ENULL),
    (dict(num_heads=6, num_kv_heads=4), ESHAPE), (dict(num_kv_heads=0), ESHAPE),
    (dict(num_seqs=-1), ESHAPE), (dict(num_seqs=70000), ESHAPE), (dict(num_q_tokens=-1), ESHAPE),
    (dict(max_q_len=-1), ESHAPE), (dict(max_seq_len=-1), ESHAPE), (dict(num_blocks=0), ESHAPE),
    (dict(num_blocks=1 << 31), ESHAPE), (dict(max_blocks_per_seq=0), ESHAPE),
    (dict(scale=float("nan")), ESHAPE), (dict(scale=float("inf")), ESHAPE),
    (dict(scale=0.0), ESHAPE), (dict(scale=-0.1), ESHAPE),
    (dict(num_seqs=65535, num_kv_heads=65535, num_heads=65535, num_q_tokens=1 << 30,
          max_q_len=1 << 30), ESHAPE),
    (dict(head_dim=96), EUNSUP), (dict(head_dim=256), EUNSUP), (dict(block_size=4), EUNSUP),
    (dict(block_size=64), EUNSUP), (dict(q_dtype=F32, cache_dtype=F32), EDTYPE),
    (dict(cache_dtype=F16), EDTYPE), (dict(q_dtype=FP8, cache_dtype=FP8), EDTYPE),
    (dict(query=A + 8), EALIGN), (dict(v_cache=A + 4), EALIGN), (dict(query_start=A + 2), EALIGN),
    (dict(cache_dtype=FP8, k_scale=A + 1), EALIGN),
    (dict(max_seq_len=100000), EWS),
    (dict(max_seq_len=100000, workspace=A, workspace_bytes=100), EWS),
    (dict(max_seq_len=100000, workspace=A + 16, workspace_bytes=1 << 40), EALIGN),
])
def test_cross_rejects_bad_arguments(lib, kw, code):
    assert cross(lib, **kw) == code


def test_workspace_size(lib):
    def ws(*sizes, dt=torch.bfloat16):
        return pkv.paged_cross_attention_workspace_size(*sizes, dt)

    assert ws(8, 0, 1, 16, 16, 64, 1000) == 0 and ws(0, 8, 1, 16, 16, 64, 1000) == 0
    assert ws(8, 8 * 100, 100, 16, 16, 64, 64) == 0       # one piece, no copies of rows
    need = ws(1, 4, 4, 8, 2, 128, 65536)
    assert need % 256 == 0 and need >= 4 * 8 * (128 + 1) * 4 * 2
    assert cross(lib, num_seqs=1, num_q_tokens=4, max_q_len=4, max_seq_len=65536, workspace=A,
                 workspace_bytes=need - 1) == EWS
    # max_q_len beyond the rows there are changes nothing.
    assert ws(1, 4, 4000, 8, 2, 128, 65536) == need
    assert ws(64, 64 * 1024, 1024, 64, 8, 128, 65536) == 0   # plenty of units
    assert ws(-1, 8, 1, 16, 16, 64, 1000) == 0
    assert ws(8, 8, 1, 16, 16, 96, 1000) == 0
    assert ws(8, 8, 1, 15, 4, 64, 1000) == 0
    assert ws(8, 8, 1, 16, 16, 64, 1000, dt=torch.float32) == 0
    assert ws(1, 1 << 24, 1, 64, 8, 128, 1 << 20) <= 161 << 20    # rows of no sequence
    assert ws(60000, 60000, 1, 64, 8, 64, 64) <= 161 << 20
    for seqs in (1, 3, 8, 30):
        for q in (1, 7, 16, 100, 129, 700):
            for heads, kv in ((8, 8), (32, 8), (16, 1), (12, 2), (64, 4)):
                assert ws(seqs, seqs * q, q, heads, kv, 128, 1 << 20) <= 161 << 20


def test_binding_refuses_what_the_pointers_cannot_say(lib):
    bf = torch.bfloat16
    q = torch.zeros(4, 8, 64, dtype=bf)
    pool = torch.zeros(6, 16, 2, 64, dtype=bf)
    bt = torch.zeros(2, 3, dtype=torch.int32)
    ln = torch.zeros(2, dtype=torch.int32)
    qs = torch.zeros(3, dtype=torch.int32)

    def call(out=q, query=q, k_cache=pool, v_cache=pool, block_table=bt, seq_lens=ln,
             query_start=qs, **kw):
        pkv.paged_cross_attention(out, query, k_cache, v_cache, block_table, seq_lens,
                                  query_start, max_q_len=2, max_seq_len=48, scale=0.1, stream=0,
                                  **kw)

    with pytest.raises(ValueError):                      # not on a GPU
        call()
    with pytest.raises(ValueError):
        call(out=q[:3])
    with pytest.raises(ValueError):
        call(out=q.half())
    with pytest.raises(ValueError):
        call(query=torch.zeros(4, 16, 64, dtype=bf)[:, ::2])
    with pytest.raises(ValueError):
        call(k_cache=pool[..., :32], v_cache=pool[..., :32])
    with pytest.raises(ValueError):
        call(v_cache=pool[:3])
    with pytest.raises(ValueError):
        call(block_table=bt.long())
    with pytest.raises(ValueError):
        call(seq_lens=ln.long())
    with pytest.raises(ValueError):
        call(seq_lens=ln[:1])
    with pytest.raises(ValueError):
        call(query_start=qs[:2])
    with pytest.raises(TypeError):
        call(k_scale=torch.ones(1, dtype=torch.float16))


def test_binding_refuses_a_workspace_that_is_not_dense(lib):
    """Its bytes are counted from its elements: a broadcast one holds fewer."""
    bf = torch.bfloat16
    q = torch.zeros(4, 8, 64, dtype=bf)
    pool = torch.zeros(6, 16, 2, 64, dtype=bf)
    for ws in (torch.zeros(1, dtype=torch.uint8).expand(1 << 30),
               torch.zeros(64, 2, dtype=torch.uint8)[:, 0]):
        with pytest.raises(ValueError, match="workspace"):
            pkv.paged_cross_attention(q, q, pool, pool, torch.zeros(2, 3, dtype=torch.int32),
                                      torch.zeros(2, dtype=torch.int32),
                                      torch.zeros(3, dtype=torch.int32), max_q_len=2,
                                      max_seq_len=48, scale=0.1, workspace=ws, stream=0)


@pytest.mark.parametrize("big", [1 << 32, (1 << 32) + 5, 1 << 31, -(1 << 31) - 1])
def test_binding_refuses_sizes_past_32_bits(lib, big):
    """They would reach the library without their upper bits (a length bound of 2^32
    as 0)."""
    bf = torch.bfloat16
    q = torch.zeros(4, 8, 64, dtype=bf)
    pool = torch.zeros(6, 16, 2, 64, dtype=bf)
    for kw in (dict(max_q_len=big, max_seq_len=48), dict(max_q_len=2, max_seq_len=big)):
        with pytest.raises(ValueError, match="32 bits"):
            pkv.paged_cross_attention(q, q, pool, pool, torch.zeros(2, 3, dtype=torch.int32),
                                      torch.zeros(2, dtype=torch.int32),
                                      torch.zeros(3, dtype=torch.int32), scale=0.1, stream=0, **kw)
    sizes = (2, 10, 8, 8, 2, 128, 100)
    for i in range(len(sizes)):
        with pytest.raises(ValueError, match="32 bits"):
            pkv.paged_cross_attention_workspace_size(*sizes[:i], big, *sizes[i + 1:], bf)
    if big > 0:
        rows = torch.zeros(1, 8, 64, dtype=bf).expand(big, 8, 64)
        with pytest.raises(ValueError, match="32 bits"):
            pkv.paged_cross_attention(rows, rows, pool, pool, torch.zeros(2, 3, dtype=torch.int32),
                                      torch.zeros(2, dtype=torch.int32),
                                      torch.zeros(3, dtype=torch.int32), max_q_len=2,
                                      max_seq_len=48, scale=0.1, stream=0)
