"""Pins of the cache oracle (CPU): the quantiser, the layout, and the operators'
definitions against independent statements of them."""
import numpy as np
import pytest
import torch

from oracle import cache as C


def test_quantise_hand_worked():
    """64 channels 0..15 four times each: zero 0, scale 1, the codes themselves;
    shifted and scaled by powers of two the codes stay."""
    x = np.tile(np.arange(16.0), 4).astype(np.float32)
    code, scale, zero = C.quantise(x[None])
    assert scale[0, 0] == 1 and zero[0, 0] == 0 and np.array_equal(code[0], x)
    code, scale, zero = C.quantise((x * 4 - 8)[None])
    assert scale[0, 0] == 4 and zero[0, 0] == -8 and np.array_equal(code[0], x)
    assert np.array_equal(C.held((x * 4 - 8)[None])[0], x * 4 - 8)


def test_quantise_error_is_half_a_step():
    """Every value is held to half a step of its group, plus what rounding the
    scale (2^-9 of it, over 15 steps) and, for float32 inputs, the zero
    (2^-9 of it) moves."""
    rng = np.random.default_rng(0)
    x = (rng.standard_normal((50, 128)) * 3 + 1).astype(np.float32)
    _, scale, zero = C.quantise(x)
    err = np.abs(C.held(x) - x).reshape(50, 2, 64)
    assert np.all(err <= (scale * (0.5 + 15 * 2.0 ** -8) + np.abs(zero) * 2.0 ** -8)[..., None])


@pytest.mark.parametrize("x,want", [
    (np.full(64, 7.25, np.float32), 7.25),                       # constant: the zero alone
    (np.full(64, 1e-42, np.float32), C.bf16(np.float32(1e-42)).item()),  # a range too small for a scale
    (np.zeros(64, np.float32), 0.0),
])
def test_quantise_constant_groups(x, want):
    assert np.all(C.held(x[None]) == want)


@pytest.mark.parametrize("bad", [np.nan, np.inf, -np.inf, 3e38])
def test_quantise_not_finite_reads_back_nan(bad):
    x = np.linspace(-3e38, 0, 128).astype(np.float32)[::-1].copy()
    x[:64] = 1.0
    x[100] = bad
    assert np.all(np.isnan(C.held(x[None])[0, 64:])) and np.all(C.held(x[None])[0, :64] == 1.0)


@pytest.mark.parametrize("D", [64, 128])
def test_layout_is_a_bijection(D):
    """Setting one byte of the codes changes two channels of one token, and every
    byte is used."""
    base = np.zeros(72 * D, np.uint8)
    base[64 * D:] = np.tile(torch.tensor([1.0, 0.0]).bfloat16().view(torch.uint8).numpy(), 2 * D)
    seen = set()
    for byte in range(0, 64 * D, 37):
        t = base.copy()
        t[byte] = 0x21
        hits = [(n, *np.argwhere(x)[i], x[tuple(np.argwhere(x)[i])]) for n, x in enumerate(C.tile_values(t))
                for i in range(len(np.argwhere(x)))]
        assert len(hits) == 2 and hits[0][:2] == hits[1][:2] and hits[1][2] == hits[0][2] + 1
        assert [h[3] for h in hits] == [1, 2] and hits[0][0] == (byte >= 32 * D)
        seen.add(hits[0][:3])
    assert len(seen) == len(range(0, 64 * D, 37))


def _filled(rng, B, n, Hk, D, bs, P):
    cache = C.new_cache(B * P + 2, Hk, D, bs)
    table = rng.permutation(B * P + 2)[:B * P].reshape(B, P)
    k, v = (rng.standard_normal((B, n, Hk, D)).astype(np.float32) for _ in "kv")
    C.write(cache, k, v, table, np.zeros(B, int))
    return cache, table, k, v


def test_attention_over_all_blocks_is_causal_sdpa():
    rng = np.random.default_rng(1)
    B, n, T, H, Hk, D, bs = 2, 150, 7, 6, 2, 64, 64
    cache, table, k, v = _filled(rng, B, n, Hk, D, bs, 3)
    q = rng.standard_normal((B, T, H, D))
    o, _, _ = C.attn(cache, q, table, np.full(B, n - T))
    kk, vv = (torch.from_numpy(C.held(x)).permute(0, 2, 1, 3).repeat_interleave(H // Hk, 1) for x in (k, v))
    mask = torch.arange(n)[None] <= torch.arange(n - T, n)[:, None]
    ref = torch.nn.functional.scaled_dot_product_attention(torch.from_numpy(q).permute(0, 2, 1, 3), kk, vv, mask)
    assert np.allclose(o, ref.permute(0, 2, 1, 3).numpy(), atol=1e-12)


def test_read_gives_what_was_written_and_sums():
    rng = np.random.default_rng(2)
    cache, table, k, v = _filled(rng, 2, 130, 3, 64, 64, 3)
    rk, rv = C.read(cache, table, np.array([0, 5]), 125)
    assert np.array_equal(rk[1], C.held(k)[1, 5:]) and np.array_equal(rv[0], C.held(v)[0, :125])
    assert np.allclose(cache["k_sum"][table[1, 1]], C.held(k)[1, 64:128].sum(0))
    assert np.allclose(cache["k_sum"][table[1, 2]], C.held(k)[1, 128:].sum(0))


def test_block_topk_against_numpy():
    rng = np.random.default_rng(3)
    B, T, H, Hk, D, bs, P = 2, 3, 4, 2, 64, 64, 9
    k_sum = rng.standard_normal((B * P, Hk, D)).astype(np.float32).astype(np.float64)
    table = rng.permutation(B * P).reshape(B, P)
    q = rng.standard_normal((B, T, H, D))
    idx, _ = C.block_topk(q, k_sum, table, np.array([500, 40]), 4, bs)
    s = np.einsum("bthd,bjhd->bhj", q.reshape(B, T, Hk, 2, D).sum(3), k_sum[table])[0] / np.r_[[bs] * 7, 503 - 448, 1]
    for h in range(Hk):
        assert list(idx[0, h]) == sorted(np.argsort(-s[h, :8])[:4])
    assert idx[1].tolist() == [[0, -1, -1, -1]] * 2  # 43 tokens: one block
    forced, _ = C.block_topk(q, k_sum, table, np.array([510, 40]), 2, bs, force_diag=True)
    assert forced[0].tolist() == [[7, 8]] * 2  # tokens 510..512 lie in blocks 7 and 8


def test_block_topk_order_of_forced_and_special_scores():
    """Forced blocks, then NaN, then +inf, then the rest; equal ones by their number."""
    k_sum = np.ones((8, 1, 64))
    k_sum[1], k_sum[3], k_sum[4], k_sum[6] = np.inf, np.nan, np.nan, -np.inf
    table, q = np.arange(8)[None], np.ones((1, 1, 1, 64))
    for topk, plain, forced in ((1, [3], [7]), (2, [3, 4], [3, 7]), (3, [1, 3, 4], [3, 4, 7]), (4, [0, 1, 3, 4], [1, 3, 4, 7]),
                                (7, [0, 1, 2, 3, 4, 5, 7], [0, 1, 2, 3, 4, 5, 7])):
        for force, want in ((False, plain), (True, forced)):
            idx, _ = C.block_topk(q, k_sum, table, np.array([511]), topk, 64, force_diag=force)
            assert idx.tolist() == [[want]], (topk, force)


def test_block_topk_forces_nothing_without_new_tokens():
    """A sequence of a padded batch that brings no token has scores of 0 throughout: its first blocks."""
    table, q = np.arange(4)[None], np.ones((1, 1, 1, 64))
    idx, _ = C.block_topk(q, np.ones((4, 1, 64)), table, np.array([200]), 2, 64, np.array([0]), force_diag=True)
    assert idx.tolist() == [[[0, 1]]]


@pytest.mark.parametrize("D", [64, 128])
def test_layout_uses_every_code_scale_and_zero_once(D):
    """Each of the 128 D four-bit places belongs to one channel of one token, keys in the first half, the low four bits
    to even channels; so does each scale and zero to one group. Places are numbered in base 16, a digit at a time."""
    one = torch.tensor([1.0, 0.0]).bfloat16().view(torch.uint8).numpy()
    place = np.zeros((2, 64, D), np.int64)
    for digit in range(4):
        n = np.arange(128 * D) >> (4 * digit) & 15
        tile = np.r_[(n[0::2] | n[1::2] << 4).astype(np.uint8), np.tile(one, 2 * D)]
        place += np.stack(C.tile_values(tile)).astype(np.int64) << (4 * digit)
    assert np.array_equal(np.sort(place.reshape(-1)), np.arange(128 * D))
    assert (place[0] < 64 * D).all() and (place % 2 == np.arange(D) % 2).all()
    groups = 2 * D  # of keys and values; their numbers are bfloat16 values
    for codes, pair in ((0x00, lambda i: (0, i)), (0x11, lambda i: (i, 0))):
        sz = torch.tensor([pair(i) for i in range(groups)]).bfloat16().view(torch.uint8).numpy().reshape(-1)
        v = np.stack(C.tile_values(np.r_[np.full(64 * D, codes, np.uint8), sz])).reshape(2, 64, D // 64, 64)
        assert (v == v[..., :1]).all() and np.array_equal(v[..., 0].reshape(-1), np.arange(groups))
