"""GPU parity of the 4-bit key/value cache with the float64 oracle.

Every cache starts with bytes of 0xff: an unwritten scale or zero is then a
NaN, so whatever reads a token that it should not shows in the result.

Tolerances, from the arithmetic (u = 2^-24 a float32 rounding):
* codes, scales and zeros are defined by float32 steps: equal bit for bit; what
  is read back is one float32 rounding of zero + scale code, and one to bf16
  (half a step: 2^-8 relative) for bf16.
* k_sum adds scale code and zero of at most block_size keys in float32: at most
  block_size + 8 roundings, each at most u times the sum of |zero| + |scale code|
  (the oracle's attn says why that is at most |value| + 2.3 times its group's largest).
* selection: dot products in float64 rounded once: index lists equal wherever no
  two different float32 scores are within a rounding of each other, which the
  random inputs avoid; exact ties are tested with equal blocks.
* attention, per output element, with A = the sum of p (|zero| + |scale code|), the
  size of what the weights multiply, L = the largest sum |q k| scale of a row:
    a score is off by at most (D + 8) u L (a float32 dot product, its scaling
    and the exponential's argument), for float32 queries also by 2^-21 L (two
    float16 parts of each query element leave 2^-22 of it), so a weight by that
    and 2^-22 (the exponential) relative, and the weight's share in the sum by
    twice that;
    bf16: a weight times its scale is rounded to float16, 2^-11 relative;
    f32: to two float16 parts, 2^-22;
    the sums add n tokens in steps of 32 or more, each step two to four matrix
    products (a truncation each, 2 u), then the warps and the parts of a row:
    (n / 4 + 64) u at most; the output's own rounding: 2^-8 (bf16), 2^-24 (f32).
  These are bounds of the worst case. That float32 queries keep float32's accuracy
  is tested beside a float32 evaluation of the formula on the same values.
"""
import numpy as np
import pytest
import torch

from oracle import cache as C

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
U = 2.0 ** -24


@pytest.fixture(scope="module")
def bsa():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a CUDA device")
    import block_sparse_attention_19_b200 as m

    yield m
    assert m.bsa_device_error() == 0


def host(t):
    return t.double().cpu().numpy()


def dev(a, dtype=torch.int32):
    return torch.as_tensor(np.ascontiguousarray(a)).to("cuda", dtype)


class Both:
    """A cache on the GPU and in the oracle, with the same page table."""

    def __init__(self, bsa, rng, B, P, Hk, D, bs, spare=3, absent=()):
        self.bsa, self.bs, self.D, self.Hk = bsa, bs, D, Hk
        self.pages = B * P + spare
        self.table = rng.permutation(self.pages)[:B * P].reshape(B, P).astype(np.int64)
        for b, j, bad in absent:
            self.table[b, j] = bad
        self.ref = C.new_cache(self.pages, Hk, D, bs)
        self.cache, self.k_sum = bsa.bsa_cache_alloc(self.pages, Hk, D, bs)
        self.cache.fill_(0xFF)
        self.k_sum.fill_(float("nan"))
        self.tab = dev(self.table)

    def write(self, k, v, start, count=None):
        C.write(self.ref, host(k), host(v), self.table, start, count)
        self.bsa.bsa_cache_write(k, v, self.cache, self.k_sum, self.tab, dev(start), self.bs,
                                 count=None if count is None else dev(count))

    def check(self):
        """The whole cache and all sums against the oracle."""
        want_k, want_v = (self.ref["kv"][i].reshape(-1, 64, self.D) for i in range(2))
        tiles = self.cache.cpu().numpy().reshape(-1, 72 * self.D)
        for i, t in enumerate(tiles):
            k, v = C.tile_values(t)
            assert np.array_equal(k, want_k[i], equal_nan=True), f"keys of tile {i}"
            assert np.array_equal(v, want_v[i], equal_nan=True), f"values of tile {i}"
        got, want = host(self.k_sum), self.ref["k_sum"]
        assert np.array_equal(np.isnan(got), np.isnan(want))
        v = np.abs(np.nan_to_num(self.ref["kv"][0]))
        size = (v + 2.3 * np.repeat(v.reshape(*v.shape[:-1], -1, 64).max(-1), 64, -1)).sum(2)
        assert np.all((np.abs(got - want) <= (self.bs + 8) * U * size)[~np.isnan(want)])


def randn(rng, *shape, dtype="bf16", scale=1.0, offset=None):
    x = rng.standard_normal(shape) * scale
    return torch.as_tensor(x if offset is None else x + offset).to("cuda", DT[dtype])


WRITES = [  # (B, T, Hk, D, bs, P, dtype, start, count)
    (1, 1, 1, 64, 64, 1, "bf16", [0], None),
    (1, 1, 2, 128, 64, 2, "bf16", [64], None),
    (2, 1, 3, 128, 128, 2, "f32", [63, 128], None),
    (3, 5, 2, 64, 64, 3, "bf16", [61, 0, 126], [5, 0, 3]),
    (2, 67, 2, 128, 64, 3, "bf16", [0, 61], [67, 66]),
    (2, 130, 1, 64, 256, 2, "f32", [255, 131], [130, 125]),
    (1, 200, 3, 128, 128, 2, "f32", [1], None),
    (2, 192, 1, 128, 64, 3, "bf16", [0, 0], [192, 1]),
    (1, 300, 2, 64, 256, 2, "bf16", [212], None),
    (2, 9, 1, 64, 64, 2, "bf16", [-3, 120], [9, 20]),  # an empty sequence; a count past T, rows past the last block
]


@pytest.mark.parametrize("case", WRITES, ids=lambda c: "B{}T{}Hk{}D{}bs{}P{}{}".format(*c[:7]))
def test_write(bsa, case):
    B, T, Hk, D, bs, P, dtype, start, count = case
    rng = np.random.default_rng(B * 1000 + T)
    both = Both(bsa, rng, B, P, Hk, D, bs)
    old = max(max(start), 1)
    offset = rng.standard_normal(D) * 3
    for b, s in enumerate(start):  # the tokens before, so that the sums have their rows
        if s > 0:
            x = randn(rng, B, old, Hk, D, dtype=dtype, offset=offset)
            n = np.zeros(B, int)
            n[b] = s
            both.write(x, randn(rng, B, old, Hk, D, dtype=dtype), np.zeros(B, int), n)
    k, v = randn(rng, B, T, Hk, D, dtype=dtype, offset=offset), randn(rng, B, T, Hk, D, dtype=dtype, scale=0.01)
    if count is not None:  # rows behind a sequence's tokens are not looked at
        for b, c in enumerate(count):
            k[b, c:], v[b, c:] = float("nan"), float("inf")
    both.write(k, v, np.array(start), None if count is None else np.array(count))
    both.check()


@pytest.mark.parametrize("rows", [20, 64])  # some of a tile, and a tile of new rows only
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_write_special_groups(bsa, dtype, rows):
    """Constant groups, tiny ranges, huge values, and groups that are not finite."""
    rng = np.random.default_rng(5)
    both = Both(bsa, rng, 1, 1, 2, 128, 64)
    k = randn(rng, 1, rows, 2, 128, dtype="f32")
    k[0, 0] = 7.25
    k[0, 1] = 1e-42
    k[0, 2] *= 1e30
    k[0, 3] *= 1e-30
    k[0, 4, 0, 5] = float("nan")
    k[0, 5, 1, 70] = float("inf")
    k[0, 6, 0, 127] = -float("inf")
    k[0, 7, 0, :2] = torch.tensor([3e38, -3e38])
    k[0, 8] *= 1e-39
    k[0, 9] = k[0, 9] * 1e-3 + 1000
    k[0, 10] = -0.0
    k[0, 11] = torch.linspace(1.0, 1.0 + 2.0 ** -7, 128, device="cuda")
    k = k.to(DT[dtype])
    both.write(k, k.flip(1).contiguous(), np.array([0]))
    both.check()


def test_write_token_by_token_equals_at_once_and_rewrites_leave_no_trace(bsa):
    rng = np.random.default_rng(6)
    B, n, Hk, D, bs = 2, 140, 2, 128, 128
    k, v = randn(rng, B, n, Hk, D), randn(rng, B, n, Hk, D)
    one, many = Both(bsa, rng, B, 2, Hk, D, bs), None
    one.write(k, v, np.array([0, 0]))
    many = Both(bsa, np.random.default_rng(0), B, 2, Hk, D, bs)
    many.table, many.tab = one.table, one.tab
    t = 0
    for step in (1, 62, 1, 1, 30, 1, 33, 1, 10):
        # drafted tokens that are rejected: written, then written over
        d = randn(rng, B, 4, Hk, D, scale=5)
        many.write(d, d, np.array([t, t]))
        many.write(k[:, t:t + step].contiguous(), v[:, t:t + step].contiguous(), np.array([t, t]))
        t += step
    assert t == n
    # the drafts that lie behind the last token: only the rows up to it have to agree
    for x, y in zip(one.bsa.bsa_cache_read(one.cache, one.tab, dev([0, 0]), n, bs),
                    bsa.bsa_cache_read(many.cache, many.tab, dev([0, 0]), n, bs)):
        assert torch.equal(x, y)
    pages = torch.as_tensor(one.table.reshape(-1))
    assert torch.equal(one.k_sum[pages], many.k_sum[pages])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("D,bs,start,T,count", [(64, 64, [0, 3, 100], 70, [70, 0, 33]), (128, 128, [127, 1, 255], 1, None),
                                                (128, 256, [5, 17, 64], 129, [128, 129, 1])])
def test_read(bsa, D, bs, start, T, count, dtype):
    rng = np.random.default_rng(7)
    Hk, B, P = 3, 3, 256 // bs + 1
    both = Both(bsa, rng, B, P, Hk, D, bs, absent=[(0, P - 1, -1), (1, 0, 10 ** 6)])
    both.write(randn(rng, B, 256, Hk, D, offset=2), randn(rng, B, 256, Hk, D), np.zeros(B, int))
    cnt = None if count is None else np.array(count)
    k_out, v_out = randn(rng, B, T, Hk, D, dtype=dtype), randn(rng, B, T, Hk, D, dtype=dtype)
    want = C.read(both.ref, both.table, np.array(start), T, cnt, host(k_out), host(v_out))
    got = bsa.bsa_cache_read(both.cache, both.tab, dev(start), T, bs, count=None if count is None else dev(cnt),
                             k_out=k_out, v_out=v_out)
    for g, w in zip(got, want):
        w = torch.as_tensor(w).float().to(DT[dtype])
        assert torch.equal(torch.nan_to_num(g.cpu(), nan=77.0), torch.nan_to_num(w, nan=77.0))
    fresh = bsa.bsa_cache_read(both.cache, both.tab, dev(start), T, bs, count=None if count is None else dev(cnt),
                               dtype=DT[dtype])
    zero = C.read(both.ref, both.table, np.array(start), T, cnt)
    assert torch.equal(torch.nan_to_num(fresh[0].cpu(), nan=77.0),
                       torch.nan_to_num(torch.as_tensor(zero[0]).float().to(DT[dtype]), nan=77.0))


TOPK = [  # (B, T, H, Hk, D, bs, P, topk, dtype, start, count, force)
    (1, 1, 1, 1, 64, 64, 1, 1, "bf16", [0], None, False),
    (2, 1, 4, 2, 128, 64, 9, 4, "bf16", [511, 300], None, False),
    (3, 3, 6, 2, 64, 128, 20, 7, "f32", [2500, 0, 60], [3, 0, 1], True),
    (1, 5, 8, 8, 128, 256, 33, 33, "bf16", [8100], None, False),
    (2, 2, 5, 1, 128, 64, 700, 100, "bf16", [44000, 9000], None, True),
    (1, 1, 2, 2, 64, 64, 5000, 750, "f32", [319999], None, False),
    (2, 4, 3, 3, 64, 64, 40, 60, "bf16", [-1, 2000], None, False),  # topk above the blocks; an empty sequence
    (9, 1, 16, 16, 128, 128, 130, 19, "bf16", [16500, 127, 128, 129, 1, 0, 5000, 12345, 16639], None, True),
]


@pytest.mark.parametrize("case", TOPK, ids=lambda c: "B{}T{}H{}Hk{}D{}bs{}P{}k{}{}".format(*c[:9]))
def test_block_topk(bsa, case):
    B, T, H, Hk, D, bs, P, topk, dtype, start, count, force = case
    rng = np.random.default_rng(8 + P)
    pages = B * P + 2
    table = rng.permutation(pages)[:B * P].reshape(B, P)
    if P > 30:
        table[0, 7], table[-1, 20] = -1, pages
    k_sum = torch.as_tensor(rng.standard_normal((pages, Hk, D)) * bs).float().cuda()
    if P > 8:  # equal blocks: ties at every place, and signed zeros
        k_sum[dev(table[:, 3], torch.long)] = k_sum[dev(table[:, 1], torch.long)]
        k_sum[dev(table[0, 4:6], torch.long)] = 0.0
    q = randn(rng, B, T, H, D, dtype=dtype)
    if count is not None:
        for b, c in enumerate(count):
            q[b, c:] = float("nan")
    cnt = None if count is None else np.array(count)
    want, _ = C.block_topk(host(torch.nan_to_num(q)), host(k_sum), table, np.array(start), topk, bs, cnt, force)
    flags = bsa.BSA_FLAG_CAUSAL | bsa.BSA_FLAG_FORCE_DIAG if force else 0
    got = bsa.bsa_cache_block_topk(q, k_sum, dev(table), dev(start), topk, bs, count=None if cnt is None else dev(cnt),
                                   flags=flags)
    assert np.array_equal(got.cpu().numpy(), want)


def test_block_topk_ties_and_special_scores(bsa):
    """All blocks equal: the first topk. Infinite, NaN and negative sums keep the lists well formed."""
    B, P, Hk, D, bs, topk = 2, 300, 2, 64, 64, 37
    k_sum = torch.ones(B * P, Hk, D, device="cuda")
    table = torch.arange(B * P, dtype=torch.int32, device="cuda").view(B, P)
    q = torch.ones(B, 1, Hk, D, device="cuda")
    start = dev([P * bs - 1, 100 * bs - 1])
    got = bsa.bsa_cache_block_topk(q, k_sum, table, start, topk, bs)
    assert torch.equal(got, torch.arange(topk, dtype=torch.int32, device="cuda").expand(B, Hk, topk))
    k_sum[5], k_sum[9], k_sum[11] = float("nan"), float("inf"), -float("inf")
    k_sum[20:60] = -1.0
    got = bsa.bsa_cache_block_topk(q, k_sum, table, start, 3, bs)
    assert got[0].tolist() == [[0, 5, 9]] * Hk  # NaN, inf, and the first of the equal rest
    got = bsa.bsa_cache_block_topk(q, k_sum, table, start, 299, bs)
    assert got[0, 0].tolist() == [j for j in range(300) if j != 11]


def check_attn(got, ref, size, logit, n, D, dtype, live):
    err = np.abs(host(got) - ref)[live]
    f32 = dtype == "f32"
    delta = ((D + 8) * U + (2.0 ** -21 if f32 else 0)) * logit[..., None] + 2.0 ** -22
    tol = (2.0 ** -24 if f32 else 2.0 ** -8) * np.abs(ref) + (
        (2.0 ** -22 if f32 else 2.0 ** -11) + 2 * delta + (n / 4 + 64) * U) * size
    assert not np.isnan(err).any()
    assert np.all(err <= tol[live]), f"off by {(err / np.maximum(tol[live], 1e-300)).max():.3g} of the tolerance"


ATTN = [  # (B, T, H, Hk, D, bs, P, dtype, start, count, topk)
    (1, 1, 1, 1, 64, 64, 1, "bf16", [0], None, 0),
    (1, 1, 1, 1, 128, 64, 1, "f32", [0], None, 0),
    (2, 1, 4, 2, 128, 64, 3, "bf16", [63, 64], None, 0),
    (2, 1, 16, 2, 128, 128, 3, "bf16", [300, 17], None, 0),
    (1, 1, 8, 8, 64, 64, 40, "bf16", [2500], None, 0),
    (3, 2, 6, 2, 64, 64, 5, "f32", [255, 0, 100], [2, 2, 1], 0),
    (3, 5, 12, 4, 128, 64, 6, "bf16", [300, 62, 0], [5, 0, 3], 0),
    (2, 3, 32, 2, 128, 128, 4, "bf16", [500, 126], None, 0),      # 48 query rows of a key head
    (1, 17, 5, 1, 64, 64, 5, "bf16", [250], None, 0),             # 85 rows, odd
    (1, 9, 16, 1, 128, 64, 4, "f32", [200], None, 0),
    (2, 1, 8, 2, 128, 64, 20, "bf16", [1279, 600], None, 6),
    (2, 4, 4, 4, 64, 128, 12, "f32", [1500, 1], [4, 1], 5),
    (1, 2, 10, 2, 128, 256, 8, "bf16", [2000], None, 3),
    (4, 1, 4, 1, 64, 256, 6, "bf16", [1400, 0, 255, 256], None, 4),
    (2, 6, 3, 3, 128, 64, 4, "bf16", [-1, 252], [6, 6], 0),       # an empty sequence; tokens past the last block
]


def idx_rows(rng, B, Hk, topk, table, start, count, T, bs):
    """Rows of distinct ascending blocks with the newest among them, padded with -1."""
    idx = np.full((B, Hk, topk), -1, np.int32)
    P = table.shape[1]
    for b in range(B):
        n = min(max(start[b], 0) + (T if count is None else count[b]), P * bs)
        blocks = max(1, -(-n // bs))
        for h in range(Hk):
            some = rng.permutation(blocks - 1)[:topk - 1] if blocks > 1 else np.zeros(0, int)
            row = np.sort(np.r_[some, blocks - 1])
            idx[b, h, :len(row)] = row
    return idx


@pytest.mark.parametrize("case", ATTN, ids=lambda c: "B{}T{}H{}Hk{}D{}bs{}P{}{}k{}".format(*c[:8], c[10]))
def test_attn(bsa, case):
    B, T, H, Hk, D, bs, P, dtype, start, count, topk = case
    rng = np.random.default_rng(H * 100 + P)
    both = Both(bsa, rng, B, P, Hk, D, bs)
    n = [min(max(s, 0) + T, P * bs) for s in start]  # tokens of each sequence
    k, v = randn(rng, B, max(n), Hk, D, offset=rng.standard_normal(D)), randn(rng, B, max(n), Hk, D)
    both.write(k, v, np.zeros(B, int), np.array(n))
    q, out = randn(rng, B, T, H, D, dtype=dtype, scale=1.5), randn(rng, B, T, H, D, dtype=dtype)
    cnt = None if count is None else np.array(count)
    if count is not None:
        for b, c in enumerate(count):
            q[b, c:] = float("nan")
    idx = idx_rows(rng, B, Hk, topk, both.table, start, count, T, bs) if topk else None
    before = host(out)
    ref, size, logit = C.attn(both.ref, host(q), both.table, np.array(start), idx, count=cnt, out=before)
    got = bsa.bsa_cache_attn(q, both.cache, both.tab, dev(start), bs, idx=None if idx is None else dev(idx),
                             count=None if cnt is None else dev(cnt), out=out)
    assert got is out
    live = np.ones((B, T, H), bool)
    for b in range(B):
        c = 0 if start[b] < 0 else T if count is None else min(count[b], T)
        live[b, c:] = False
        assert np.array_equal(host(got)[b, c:], before[b, c:])  # rows that no token has stay
    check_attn(got, ref, size, logit, max(n), D, dtype, live)


def test_attn_rows_that_see_nothing_are_zero(bsa):
    """All blocks of a row absent, an index row of -1, an index beyond the table, and blocks after the row's position."""
    rng = np.random.default_rng(12)
    B, H, Hk, D, bs, P = 3, 4, 2, 64, 64, 3
    both = Both(bsa, rng, B, P, Hk, D, bs, absent=[(0, 0, -1), (0, 1, 99999), (0, 2, -7)])
    x = randn(rng, B, 192, Hk, D)
    both.write(x, x, np.zeros(B, int))
    q = randn(rng, B, 2, H, D)
    start = dev([150, 150, 62])
    o = bsa.bsa_cache_attn(q, both.cache, both.tab, start, bs)
    assert torch.equal(o[0], torch.zeros_like(o[0])) and bool((o[1:] != 0).any(-1).all())
    idx = torch.full((B, Hk, 2), -1, dtype=torch.int32, device="cuda")
    idx[1, 1, 0] = 3        # past the table
    idx[2, :, 0] = 1        # tokens 64..: token 0 of the step (position 62) and 1 (63) see none
    o = bsa.bsa_cache_attn(q, both.cache, both.tab, start, bs, idx=idx)
    assert torch.equal(o, torch.zeros_like(o))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_attn_absent_blocks_and_unsorted_lists(bsa, dtype):
    rng = np.random.default_rng(13)
    B, H, Hk, D, bs, P = 2, 6, 2, 128, 64, 8
    both = Both(bsa, rng, B, P, Hk, D, bs, absent=[(0, 2, -1), (1, 0, -5), (1, 7, 10 ** 6)])
    x, y = randn(rng, B, 512, Hk, D), randn(rng, B, 512, Hk, D)
    both.write(x, y, np.zeros(B, int))
    q = randn(rng, B, 3, H, D, dtype=dtype)
    start = np.array([500, 400])
    ref, size, logit = C.attn(both.ref, host(q), both.table, start)
    live = np.ones((B, 3, H), bool)
    check_attn(bsa.bsa_cache_attn(q, both.cache, both.tab, dev(start), bs), ref, size, logit, 512, D, dtype, live)
    idx = np.array([[[7, 0, 2, 5], [1, -1, 6, 4]], [[5, 0, 1, -1], [-1, 3, -1, 2]]])
    ref, size, logit = C.attn(both.ref, host(q), both.table, start, idx)
    check_attn(bsa.bsa_cache_attn(q, both.cache, both.tab, dev(start), bs, idx=dev(idx)), ref, size, logit, 512, D,
               dtype, live)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("q_scale,k_scale,v_scale", [(40.0, 1.0, 1.0), (1e-20, 1.0, 1.0), (1.0, 1e-12, 1e-12),
                                                     (1e-8, 1e9, 1e9), (1.0, 1.0, 0.0)])
def test_attn_magnitudes(bsa, dtype, q_scale, k_scale, v_scale):
    """Sharp and flat softmax, and values from 1e-12 to 1e9 (zero included)."""
    rng = np.random.default_rng(14)
    B, H, Hk, D, bs, P = 2, 8, 2, 128, 64, 10
    both = Both(bsa, rng, B, P, Hk, D, bs)
    both.write(randn(rng, B, 640, Hk, D, scale=k_scale), randn(rng, B, 640, Hk, D, scale=v_scale), np.zeros(B, int))
    q = randn(rng, B, 2, H, D, dtype=dtype, scale=q_scale)
    start = np.array([630, 77])
    ref, size, logit = C.attn(both.ref, host(q), both.table, start)
    got = bsa.bsa_cache_attn(q, both.cache, both.tab, dev(start), bs)
    check_attn(got, ref, size, logit, 640, D, dtype, np.ones((B, 2, H), bool))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_attn_values_of_very_different_sizes(bsa, dtype):
    """Tokens whose values differ by 2^40 from each other, the large ones with small weights and late."""
    rng = np.random.default_rng(15)
    B, H, Hk, D, bs, P = 1, 4, 1, 64, 64, 6
    both = Both(bsa, rng, B, P, Hk, D, bs)
    v = torch.randn(B, 384, Hk, D, device="cuda") * torch.exp2(torch.randint(-20, 20, (B, 384, 1, 1), device="cuda"))
    k = randn(rng, B, 384, Hk, D)
    both.write(k, v.bfloat16(), np.zeros(B, int))
    q = randn(rng, B, 1, H, D, dtype=dtype, scale=4.0)
    ref, size, logit = C.attn(both.ref, host(q), both.table, np.array([383]))
    check_attn(bsa.bsa_cache_attn(q, both.cache, both.tab, dev([383]), bs), ref, size, logit, 384, D, dtype,
               np.ones((B, 1, H), bool))


def _formula(q, kk, vv, dtype):
    """softmax(q k / sqrt(D)) v of one row of each head: q [H, D], k and v [n, H, D]."""
    x = torch.einsum("hd,nhd->hn", q.to(dtype), kk.to(dtype)) / q.shape[-1] ** 0.5
    return torch.einsum("hn,nhd->hd", x.softmax(-1), vv.to(dtype))


@pytest.mark.parametrize("G", [1, 4, 7])
@pytest.mark.parametrize("D", [64, 128])
def test_attn_float32_queries_keep_float32(bsa, D, G):
    """Long rows, whose result is much smaller than what is summed: the error
    against 64 bits is at most four times that of the formula in float32."""
    g = torch.Generator(device="cuda").manual_seed(5)
    Hk, bs, n = 2, 64, 6000
    cache, k_sum = bsa.bsa_cache_alloc(96, Hk, D, bs)
    table, zero = torch.randperm(96, generator=g, device="cuda").int().view(1, -1), dev([0])
    k, v = (torch.randn(1, n, Hk, D, generator=g, device="cuda") for _ in "kv")
    bsa.bsa_cache_write(k + torch.randn(D, generator=g, device="cuda"), v, cache, k_sum, table, zero, bs)
    kk, vv = bsa.bsa_cache_read(cache, table, zero, n, bs, dtype=torch.float32)
    kk, vv = (x[0].repeat_interleave(G, 1) for x in (kk, vv))
    q = torch.randn(1, 1, Hk * G, D, generator=g, device="cuda") * 1.5
    got = bsa.bsa_cache_attn(q, cache, table, dev([n - 1]), bs)[0, 0]
    ref = _formula(q[0, 0], kk, vv, torch.float64)
    err = lambda x: float((x.double() - ref).norm() / ref.norm())  # noqa: E731
    assert err(got) <= 4 * err(_formula(q[0, 0], kk, vv, torch.float32)), err(got)


def test_attn_long_rows_do_not_drift(bsa):
    """bf16: a whole unit of 131072 tokens on one CTA (more units than CTAs), where
    sums kept in the matrix unit would lose a part in 100: the relative error
    stays at the output's rounding (2^-9 on average, and the weights' 2^-12)."""
    g = torch.Generator(device="cuda").manual_seed(6)
    B, Hk, D, bs, n = 40, 16, 64, 256, 131072
    P = n // bs
    cache, k_sum = bsa.bsa_cache_alloc(P, Hk, D, bs)
    table = torch.arange(P, device="cuda", dtype=torch.int32)
    k, v = (torch.randn(1, n, Hk, D, generator=g, device="cuda").bfloat16() for _ in "kv")
    bsa.bsa_cache_write(k, v, cache, k_sum, table.view(1, -1), dev([0]), bs)
    kk, vv = bsa.bsa_cache_read(cache, table.view(1, -1), dev([0]), n, bs, dtype=torch.float32)
    for G, T in ((1, 1), (4, 3)):  # the kernel of few rows, and of many
        q = torch.randn(1, T, Hk * G, D, generator=g, device="cuda").bfloat16()
        o = bsa.bsa_cache_attn(q.expand(B, -1, -1, -1).contiguous(), cache, table.expand(B, -1).contiguous(),
                               dev([n - T] * B), bs)
        assert torch.equal(o, o[:1].expand_as(o)) or float((o - o[:1]).abs().max()) <= 2.0 ** -7 * float(o.abs().max())
        for h in (0, Hk * G - 1):
            x = kk[0, :, h // G].double() @ q[0, T - 1, h].double() / D ** 0.5
            ref = x.softmax(0) @ vv[0, :, h // G].double()
            err = float((o[0, T - 1, h].double() - ref).norm() / ref.norm())
            assert err <= 2.0 ** -8, err


def test_attn_nan_and_infinite_tokens_show_only_where_seen(bsa):
    rng = np.random.default_rng(16)
    both = Both(bsa, rng, 1, 2, 2, 64, 64)
    k, v = randn(rng, 1, 128, 2, 64), randn(rng, 1, 128, 2, 64)
    v[0, 100, 0, 3], k[0, 120, 1, 9] = float("inf"), float("nan")
    both.write(k, v, np.array([0]))
    q = randn(rng, 1, 1, 4, 64)
    for pos, bad in ((99, []), (100, [0, 1]), (119, [0, 1]), (120, [0, 1, 2, 3])):
        o = bsa.bsa_cache_attn(q, both.cache, both.tab, dev([pos]), 64)
        assert [h for h in range(4) if torch.isnan(o[0, 0, h]).any()] == bad, pos


@pytest.mark.parametrize("D", [64, 128])
def test_attn_of_many_rows_with_a_nan_among_the_new_tokens(bsa, D):
    """The rows before a token that is not finite do not see it; those from it on do."""
    rng = np.random.default_rng(21)
    T, H, Hk, n = 12, 8, 2, 200
    both = Both(bsa, rng, 1, 4, Hk, D, 64)
    k, v = randn(rng, 1, n, Hk, D), randn(rng, 1, n, Hk, D)
    v[0, n - 5, 0] = float("nan")
    k[0, n - 3, 1, 0] = float("inf")
    both.write(k, v, np.array([0]))
    q = randn(rng, 1, T, H, D)
    start = np.array([n - T])
    o = bsa.bsa_cache_attn(q, both.cache, both.tab, dev(start), 64)
    bad = torch.isnan(o[0].float()).any(-1).cpu().numpy()
    assert np.array_equal(bad[:, :4], np.arange(T)[:, None].repeat(4, 1) >= T - 5)
    assert np.array_equal(bad[:, 4:], np.arange(T)[:, None].repeat(4, 1) >= T - 3)
    kv = {**both.ref, "kv": np.nan_to_num(both.ref["kv"])}
    ref, size, logit = C.attn(kv, host(q), both.table, start)
    check_attn(torch.nan_to_num(o), ref, size, logit, n, D, "bf16", ~bad[None])


FORMS = [("bf16", 1, 1), ("bf16", 4, 2), ("bf16", 4, 3), ("bf16", 8, 5), ("f32", 4, 1), ("f32", 4, 2)]  # type, G, T


@pytest.mark.parametrize("dtype,G,T", FORMS, ids=lambda x: str(x))
@pytest.mark.parametrize("D", [64, 128])
def test_attn_queries_that_are_not_finite(bsa, D, dtype, G, T):
    """A row with an infinity, a NaN or an element of 2^117 and above gives NaN, also where all its scores would be
    -inf; the others know nothing of it, and neither does a row that sees no token."""
    rng = np.random.default_rng(23)
    Hk, n = 5, 150
    both = Both(bsa, rng, 1, 3, Hk, D, 64)
    k, v = randn(rng, 1, n, Hk, D, offset=-8.0), randn(rng, 1, n, Hk, D)
    both.write(k, v, np.array([0]))
    q = randn(rng, 1, T, Hk * G, D, dtype=dtype)
    clean, start = q.clone(), np.array([n - T])
    bad = np.zeros((1, T, Hk * G), bool)
    for i, x in enumerate((float("inf"), -float("inf"), float("nan"), 2.0 ** 117)):
        q[0, T - 1, i * G, 7 * i] = x
        bad[0, T - 1, i * G] = True
    o = bsa.bsa_cache_attn(q, both.cache, both.tab, dev(start), 64)
    assert torch.isnan(o[torch.as_tensor(bad, device="cuda")]).all()
    ref, size, logit = C.attn(both.ref, host(clean), both.table, start)
    check_attn(torch.nan_to_num(o), ref, size, logit, n, D, dtype, ~bad)
    idx = torch.full((1, Hk, 1), -1, dtype=torch.int32, device="cuda")
    assert not bsa.bsa_cache_attn(q, both.cache, both.tab, dev(start), 64, idx=idx).any()


@pytest.mark.parametrize("dtype,G,T", FORMS, ids=lambda x: str(x))
def test_attn_scores_far_below_zero(bsa, dtype, G, T):
    """Scores of -2^113 (i + 1): all weight is on token 0. Weight 1 in float16 (2^-11 at most), the output's rounding
    (2^-9) and float32 sums stay below 2^-8 of |zero| + 15 scale."""
    rng = np.random.default_rng(24)
    D, Hk, n = 64, 2, 200
    both = Both(bsa, rng, 1, 4, Hk, D, 64)
    k = torch.arange(1, n + 1, device="cuda", dtype=torch.float32).view(1, n, 1, 1).expand(1, n, Hk, D) * -2.0 ** 50
    v = randn(rng, 1, n, Hk, D)
    both.write(k.bfloat16().contiguous(), v, np.array([0]))
    q = torch.full((1, T, Hk * G, D), 2.0 ** 60, device="cuda", dtype=DT[dtype])
    o = bsa.bsa_cache_attn(q, both.cache, both.tab, dev([n - T]), 64)
    _, held = bsa.bsa_cache_read(both.cache, both.tab, dev([0]), n, 64, dtype=torch.float32)
    want = held[0, 0].repeat_interleave(G, 0).expand(T, -1, -1)
    size = 2 * held[0, 0].abs().amax(-1).repeat_interleave(G, 0).view(1, -1, 1)
    assert ((o[0].float() - want).abs() <= 2.0 ** -8 * size).all()


def test_attn_long_ragged_batch(bsa):
    """Many sequences of very different lengths against the float64 formula on what is read back."""
    g = torch.Generator(device="cuda").manual_seed(3)
    B, H, Hk, D, bs, P = 37, 8, 2, 128, 64, 90
    cache, k_sum = bsa.bsa_cache_alloc(B * P, Hk, D, bs)
    cache.fill_(0xFF)
    table = torch.randperm(B * P, generator=g, device="cuda").int().view(B, P)
    n = (torch.rand(B, generator=g, device="cuda") ** 3 * P * bs).int().clamp(min=1)
    n[5], n[6], n[7] = P * bs, 1, 64
    k, v = (torch.randn(B, P * bs, Hk, D, generator=g, device="cuda").bfloat16() for _ in "kv")
    zero = torch.zeros_like(n)
    bsa.bsa_cache_write(k, v, cache, k_sum, table, zero, bs, count=n)
    q = torch.randn(B, 1, H, D, generator=g, device="cuda").bfloat16() * 2
    o = bsa.bsa_cache_attn(q, cache, table, n - 1, bs)
    kk, vv = bsa.bsa_cache_read(cache, table, zero, P * bs, bs, dtype=torch.float32, count=n)
    for b in range(B):
        x = torch.einsum("gjd,njd->gjn", q[b, 0].double().view(Hk, 4, D).transpose(0, 1), kk[b, :n[b]].double()) / D ** 0.5
        w = x.softmax(-1)
        ref = torch.einsum("gjn,njd->gjd", w, vv[b, :n[b]].double()).transpose(0, 1).reshape(H, D)
        parts = vv[b, :n[b]].double().abs().view(-1, Hk, 2, 64)
        parts = (parts + 2.3 * parts.amax(-1, keepdim=True)).view(-1, Hk, D)
        size = torch.einsum("gjn,njd->gjd", w, parts).transpose(0, 1).reshape(H, D)
        # a read-back value is a float32 rounding of the cache's; logits here stay below 60
        tol = 2.0 ** -8 * ref.abs() + (2.0 ** -11 + 2 * (D + 8) * U * 60 + (P * bs / 4 + 64) * U) * size
        assert bool(((o[b, 0].double() - ref).abs() <= tol).all()), b


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_generation_step_by_step(bsa, dtype):
    """Write, select and attend as a generating model does: a prompt, single tokens
    and drafts, against the oracle at each step; then the same steps without
    selection, and the separate calls against the joined one."""
    rng = np.random.default_rng(17)
    B, H, Hk, D, bs, P, topk = 3, 6, 2, 64, 64, 8, 3
    both = Both(bsa, rng, B, P, Hk, D, bs)
    other, other_sum = both.cache.clone(), both.k_sum.clone()
    pos = np.zeros(B, int)
    for T, count, force in ((150, [150, 1, 77], True), (1, None, True), (1, None, False), (4, [4, 0, 2], True),
                            (1, None, True), (130, [0, 130, 100], False)):
        q, k, v = (randn(rng, B, T, n, D, dtype=dtype) for n in (H, Hk, Hk))
        cnt = None if count is None else np.array(count)
        c_dev, s_dev = None if cnt is None else dev(cnt), dev(pos)
        flags = bsa.BSA_FLAG_CAUSAL | bsa.BSA_FLAG_FORCE_DIAG if force else 0
        got = bsa.bsa_cache_forward(q, k, v, both.cache, both.k_sum, both.tab, s_dev, bs, topk, count=c_dev, flags=flags)
        C.write(both.ref, host(k), host(v), both.table, pos, cnt)
        idx = bsa.bsa_cache_block_topk(q, both.k_sum, both.tab, s_dev, topk, bs, count=c_dev, flags=flags)
        want, _ = C.block_topk(host(q), host(both.k_sum), both.table, pos, topk, bs, cnt, force)
        assert np.array_equal(idx.cpu().numpy(), want)
        live = np.arange(T)[None] < (np.full(B, T) if cnt is None else cnt)[:, None]
        live = np.broadcast_to(live[..., None], (B, T, H))
        ref, size, logit = C.attn(both.ref, host(q), both.table, pos, want, count=cnt)
        check_attn(got, ref, size, logit, P * bs, D, dtype, live)
        dense = bsa.bsa_cache_forward(q, k, v, other, other_sum, both.tab, s_dev, bs, count=c_dev)
        ref, size, logit = C.attn(both.ref, host(q), both.table, pos, count=cnt)
        check_attn(dense, ref, size, logit, P * bs, D, dtype, live)
        apart = bsa.bsa_cache_attn(q, both.cache, both.tab, s_dev, bs, idx=idx, count=c_dev)
        assert torch.equal(apart, got) and torch.equal(both.cache, other)
        pos = pos + (T if cnt is None else cnt)
    both.check()


def test_prompt_through_the_cache_agrees_with_the_prefill_path(bsa):
    """Keys and values written and read back feed bsa_forward; the last block's
    queries through the cache see the same tokens as its causal form does."""
    g = torch.Generator(device="cuda").manual_seed(4)
    N, H, D, bs = 1024, 4, 128, 128
    q, k, v = (torch.randn(1, N, H, D, generator=g, device="cuda").bfloat16() for _ in "qkv")
    cache, k_sum = bsa.bsa_cache_alloc(N // bs, H, D, bs)
    table, zero = torch.arange(N // bs, device="cuda", dtype=torch.int32).view(1, -1), dev([0])
    bsa.bsa_cache_write(k, v, cache, k_sum, table, zero, bs)
    kk, vv = bsa.bsa_cache_read(cache, table, zero, N, bs)
    full = bsa.bsa_forward(q, kk, vv, bs, 1.0, flags=bsa.BSA_FLAG_CAUSAL)
    step = bsa.bsa_cache_attn(q[:, -bs:].contiguous(), cache, table, dev([N - bs]), bs)
    # the prefill path rounds keys, values and weights to bf16 (2^-8 each): a loose check that the rows are the same ones
    assert float((full[:, -bs:].float() - step.float()).norm() / step.float().norm()) < 3 * 2.0 ** -8


def test_captured_step_follows_the_device_lengths(bsa):
    rng = np.random.default_rng(18)
    B, H, Hk, D, bs, P, topk = 2, 4, 2, 128, 64, 5, 2
    caches = [bsa.bsa_cache_alloc(B * P, Hk, D, bs) for _ in range(2)]
    for c, s in caches:
        c.fill_(0xFF)
        s.fill_(float("nan"))
    table = dev(rng.permutation(B * P).reshape(B, P))
    x = [[randn(rng, B, 1, n, D) for n in (H, Hk, Hk)] for _ in range(150)]
    q, k, v = (t.clone() for t in x[0])
    start, out = dev([0, 100]), torch.empty_like(q)
    ws = torch.empty(bsa.bsa_cache_forward_workspace_bytes(B, 1, H, Hk, D, topk), dtype=torch.uint8, device="cuda")
    pre = [randn(rng, B, 100, Hk, D) for _ in "kv"]
    for c, s in caches:
        bsa.bsa_cache_write(*pre, c, s, table, dev([0, 0]), bs, count=dev([0, 100]))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graphs = []
    with torch.cuda.stream(side):
        bsa.bsa_cache_forward(q, k, v, *caches[0], table, start, bs, topk, workspace=ws, out=out)  # warm-up
        for kk in (topk, 0):  # two graphs that share a workspace
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=side):
                bsa.bsa_cache_forward(q, k, v, *caches[0], table, start, bs, kk, workspace=ws, out=out)
            graphs.append(g)
    torch.cuda.current_stream().wait_stream(side)
    for t in range(150):
        for a, b in zip((q, k, v), x[t]):
            a.copy_(b)
        start.copy_(dev([t, 100 + t]))
        graphs[t % 2].replay()
        want = bsa.bsa_cache_forward(*x[t], *caches[1], table, dev([t, 100 + t]), bs, (topk, 0)[t % 2])
        assert torch.equal(out, want), t
    assert torch.equal(caches[0][0], caches[1][0])


def test_steps_on_two_streams_at_once(bsa):
    rng = np.random.default_rng(19)
    B, H, Hk, D, bs, P = 4, 8, 2, 128, 64, 40
    both = Both(bsa, rng, B, P, Hk, D, bs)
    n = P * bs - 1
    x, y = randn(rng, B, n, Hk, D), randn(rng, B, n, Hk, D)
    bsa.bsa_cache_write(x, y, both.cache, both.k_sum, both.tab, dev([0] * B), bs)
    qs = [randn(rng, B, 1, H, D) for _ in range(6)]
    start = dev([n - 1, 700, 5, 64])
    want = [bsa.bsa_cache_attn(q, both.cache, both.tab, start, bs) for q in qs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [None] * 6
    for r in range(3):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                got[2 * r + i] = bsa.bsa_cache_attn(qs[2 * r + i], both.cache, both.tab, start, bs)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_cache_past_32_bit_offsets(bsa):
    """Pages beyond 2^32 bytes of the cache and 2^31 elements of the sums."""
    Hk, D, bs = 16, 128, 256
    pages = 9000  # 9000 * 16 * 36864 bytes = 5.3 GB
    cache = torch.zeros(pages, Hk, bs // 64, 72 * D, dtype=torch.uint8, device="cuda")
    k_sum = torch.zeros(pages, Hk, D, device="cuda")
    rng = np.random.default_rng(20)
    k, v = randn(rng, 1, 300, Hk, D), randn(rng, 1, 300, Hk, D)
    table = dev([[pages - 1, pages - 3]])
    bsa.bsa_cache_write(k, v, cache, k_sum, table, dev([0]), bs)
    kk, vv = bsa.bsa_cache_read(cache, table, dev([0]), 300, bs)
    assert torch.equal(kk, torch.as_tensor(C.held(host(k))).bfloat16().cuda())
    assert torch.equal(vv, torch.as_tensor(C.held(host(v))).bfloat16().cuda())
    q = randn(rng, 1, 1, Hk, D)
    o = bsa.bsa_cache_attn(q, cache, table, dev([299]), bs)
    near = bsa.bsa_cache_alloc(2, Hk, D, bs)
    low = dev([[1, 0]])
    bsa.bsa_cache_write(k, v, *near, low, dev([0]), bs)
    assert torch.equal(o, bsa.bsa_cache_attn(q, near[0], low, dev([299]), bs))
    a = bsa.bsa_cache_block_topk(q, k_sum, table, dev([299]), 1, bs)
    assert torch.equal(a, bsa.bsa_cache_block_topk(q, near[1], low, dev([299]), 1, bs))


@pytest.mark.parametrize("count", [None, [1, 2]])
def test_rows_without_a_token_are_zeros_where_the_call_makes_the_tensor(bsa, count):
    """A negative start makes a sequence empty, with count or without: its rows are no leftovers of other tensors."""
    rng = np.random.default_rng(25)
    B, T, H, Hk, D, bs = 2, 2, 4, 2, 64, 64
    both = Both(bsa, rng, B, 2, Hk, D, bs)
    x, q = randn(rng, B, T, Hk, D), randn(rng, B, T, H, D)
    start, cnt = dev([-1, 0]), None if count is None else dev(count)

    def litter():
        """Freed memory of the sizes to come, full of NaN."""
        for n in (H, Hk, Hk):
            torch.full((B, T, n, D), float("nan"), device="cuda", dtype=torch.bfloat16)

    litter()
    o = bsa.bsa_cache_forward(q, x, x, both.cache, both.k_sum, both.tab, start, bs, count=cnt)
    assert not o[0].any() and bool(o[1].any())
    litter()
    o = bsa.bsa_cache_attn(q, both.cache, both.tab, start, bs, count=cnt)
    assert not o[0].any() and bool(o[1].any())
    litter()
    k, v = bsa.bsa_cache_read(both.cache, both.tab, start, T, bs, count=cnt)
    assert not k[0].any() and not v[0].any() and bool(k[1].any())


@pytest.mark.parametrize("P", [12, 300])
def test_block_topk_forced_blocks_rank_above_scores_that_are_not_finite(bsa, P):
    """Older blocks with NaN or infinite sums do not push out the blocks of the new tokens."""
    Hk, D, bs, T = 2, 64, 64, 3
    k_sum = torch.randn(P, Hk, D, device="cuda", generator=torch.Generator(device="cuda").manual_seed(7))
    k_sum[1:8:2], k_sum[2], k_sum[6] = float("nan"), float("inf"), -float("inf")
    table, start = np.arange(P)[None], np.array([(P - 1) * bs - 1])  # new tokens in the last two blocks
    q = torch.ones(1, T, Hk, D, device="cuda")
    for topk in (1, 2, 3, 6, 7, P - 1, P):
        for flags in (0, bsa.BSA_FLAG_CAUSAL | bsa.BSA_FLAG_FORCE_DIAG):
            with np.errstate(invalid="ignore"):
                want, _ = C.block_topk(host(q), host(k_sum), table, start, topk, bs, force_diag=bool(flags))
            got = bsa.bsa_cache_block_topk(q, k_sum, dev(table), dev(start), topk, bs, flags=flags)
            assert np.array_equal(got.cpu().numpy(), want), (topk, flags)
            assert not flags or set(range(P - 2, P)[:topk]) <= set(got[0, 0].tolist())


@pytest.mark.parametrize("P", [4, 400])
def test_block_topk_forces_nothing_without_new_tokens(bsa, P):
    Hk, D, bs, B = 2, 64, 64, 3
    k_sum = torch.ones(B * P, Hk, D, device="cuda")
    table, q = np.arange(B * P).reshape(B, P), torch.ones(B, 2, Hk, D, device="cuda")
    start, count = np.array([(P - 1) * bs + 8, (P - 1) * bs, (P - 1) * bs + 8]), np.array([0, 0, 2])
    want, _ = C.block_topk(host(q), host(k_sum), table, start, 2, bs, count, force_diag=True)
    got = bsa.bsa_cache_block_topk(q, k_sum, dev(table), dev(start), 2, bs, count=dev(count),
                                   flags=bsa.BSA_FLAG_CAUSAL | bsa.BSA_FLAG_FORCE_DIAG)
    assert np.array_equal(got.cpu().numpy(), want)
    assert got[0].tolist() == [[0, 1]] * Hk and got[2].tolist() == [[0, P - 1]] * Hk


@pytest.mark.parametrize("dtype,G,T", FORMS, ids=lambda x: str(x))
@pytest.mark.parametrize("D", [64, 128])
def test_attn_large_queries_times_a_large_scale(bsa, D, dtype, G, T):
    """A row whose element times scale leaves what a score can be made of gives NaN, never the zeros of a row that sees
    nothing, however its scores' signs fall; half the rows are ordinary ones and know nothing of it."""
    rng = np.random.default_rng(26)
    Hk, n, scale = 2, 150, 2.0 ** 12
    both = Both(bsa, rng, 1, 3, Hk, D, 64)
    k, v = randn(rng, 1, n, Hk, D, offset=-8.0), randn(rng, 1, n, Hk, D)
    both.write(k, v, np.array([0]))
    q = randn(rng, 1, T, Hk * G, D, dtype=dtype, scale=2.0 ** -14)
    start, bad = np.array([n - T]), np.zeros((1, T, Hk * G), bool)
    q[0, T - 1, :G] = 2.0 ** 112  # (times 2^12 log2(e) beyond 2^120)
    bad[0, T - 1, :G] = True
    o = bsa.bsa_cache_attn(q, both.cache, both.tab, dev(start), 64, scale=scale)
    assert torch.isnan(o[torch.as_tensor(bad, device="cuda")]).all()
    ref, size, logit = C.attn(both.ref, np.where(bad[..., None], 0, host(q)), both.table, start, scale=scale)
    check_attn(torch.nan_to_num(o), ref, size, logit, n, D, dtype, ~bad)


@pytest.mark.parametrize("dtype,G,T", FORMS, ids=lambda x: str(x))
@pytest.mark.parametrize("D", [64, 128])
def test_attn_values_of_every_size(bsa, D, dtype, G, T):
    """Values whose scales lie between 2^-122 and 2^97, the accuracy relative to them throughout."""
    rng = np.random.default_rng(27)
    Hk, n = 2, 200
    k, v = randn(rng, 1, n, Hk, D, offset=1), torch.as_tensor(rng.standard_normal((1, n, Hk, D)), device="cuda").float()
    q, start = randn(rng, 1, T, Hk * G, D, dtype=dtype, scale=1.5), np.array([n - T])
    for v_scale in (1e-36, 1e-31, 1e-26, 1e-22, 1e-18, 1e20, 1e30):
        both = Both(bsa, rng, 1, 4, Hk, D, 64)
        both.write(k, (v * v_scale).bfloat16(), np.array([0]))
        ref, size, logit = C.attn(both.ref, host(q), both.table, start)
        o = bsa.bsa_cache_attn(q, both.cache, both.tab, dev(start), 64)
        check_attn(o, ref, size, logit, n, D, dtype, np.ones((1, T, Hk * G), bool))


@pytest.mark.parametrize("dtype,G,T", FORMS, ids=lambda x: str(x))
def test_attn_value_groups_of_different_sizes(bsa, dtype, G, T):
    """The two groups of 64 channels differ by powers of two: each keeps its own accuracy."""
    rng = np.random.default_rng(28)
    D, Hk, n = 128, 2, 300
    k, v = randn(rng, 1, n, Hk, D, offset=1), torch.as_tensor(rng.standard_normal((1, n, Hk, D)), device="cuda").float()
    q, start = randn(rng, 1, T, Hk * G, D, dtype=dtype, scale=1.5), np.array([n - T])
    for e in (-100, -30, -20, -10, 10, 20, 30, 100):
        both = Both(bsa, rng, 1, 5, Hk, D, 64)
        x = v * 2.0 ** (-e // 2)
        x[..., 64:] *= 2.0 ** e
        both.write(k, x.bfloat16(), np.array([0]))
        ref, size, logit = C.attn(both.ref, host(q), both.table, start)
        o = bsa.bsa_cache_attn(q, both.cache, both.tab, dev(start), 64)
        check_attn(o, ref, size, logit, n, D, dtype, np.ones((1, T, Hk * G), bool))


@pytest.mark.parametrize("G", [1, 7])
@pytest.mark.parametrize("e", [-30, -20, 20, 30])
def test_attn_float32_groups_keep_float32(bsa, G, e):
    """Beside a group that is 2^30 times larger or smaller: the criterion of the test of float32 queries, by group."""
    g = torch.Generator(device="cuda").manual_seed(8)
    Hk, D, bs, n = 2, 128, 64, 6000
    cache, k_sum = bsa.bsa_cache_alloc(94, Hk, D, bs)
    table, zero = torch.randperm(94, generator=g, device="cuda").int().view(1, -1), dev([0])
    k, v = (torch.randn(1, n, Hk, D, generator=g, device="cuda") for _ in "kv")
    v[..., 64:] *= 2.0 ** e
    bsa.bsa_cache_write(k, v, cache, k_sum, table, zero, bs)
    kk, vv = bsa.bsa_cache_read(cache, table, zero, n, bs, dtype=torch.float32)
    kk, vv = (x[0].repeat_interleave(G, 1) for x in (kk, vv))
    q = torch.randn(1, 1, Hk * G, D, generator=g, device="cuda") * 1.5
    got = bsa.bsa_cache_attn(q, cache, table, dev([n - 1]), bs)[0, 0]
    ref, plain = _formula(q[0, 0], kk, vv, torch.float64), _formula(q[0, 0], kk, vv, torch.float32)
    for part in (slice(0, 64), slice(64, 128)):
        err = lambda x: float((x[:, part].double() - ref[:, part]).norm() / ref[:, part].norm())  # noqa: E731
        assert err(got) <= 4 * err(plain), (part, err(got), err(plain))


@pytest.mark.parametrize("dtype,G,T", FORMS, ids=lambda x: str(x))
@pytest.mark.parametrize("D", [64, 128])
def test_attn_groups_of_one_large_value(bsa, D, dtype, G, T):
    """A group of equal values has scale 0 and says nothing of how far weights may grow: values of 1e25 throughout, and
    (D = 128) beside ordinary ones, with sharp scores that rise along the sequence."""
    rng = np.random.default_rng(29)
    Hk, n = 2, 400
    k = randn(rng, 1, n, Hk, D, offset=np.linspace(0, 1, n)[:, None, None])
    q, start = randn(rng, 1, T, Hk * G, D, dtype=dtype, scale=3, offset=1), np.array([n - T])
    both = Both(bsa, rng, 1, 7, Hk, D, 64)
    v = randn(rng, 1, n, Hk, D)
    v[..., :64] = 1e25
    both.write(k, v, np.array([0]))
    ref, size, logit = C.attn(both.ref, host(q), both.table, start)
    o = bsa.bsa_cache_attn(q, both.cache, both.tab, dev(start), 64)
    check_attn(o, ref, size, logit, n, D, dtype, np.ones((1, T, Hk * G), bool))


@pytest.mark.parametrize("dtype,G,T", FORMS, ids=lambda x: str(x))
@pytest.mark.parametrize("rise", [0.3, -0.3])
def test_attn_scores_that_rise_as_the_values_shrink(bsa, dtype, G, T, rise):
    """Scores from 0 to 75 (or back), and values that shrink (grow) as their weights grow (shrink): the weights'
    references and the groups' factors move far apart."""
    rng = np.random.default_rng(30)
    D, Hk, n = 128, 1, 250
    i = torch.arange(n, device="cuda", dtype=torch.float32) if rise > 0 else torch.arange(n, 0, -1, device="cuda").float()
    k = torch.zeros(1, n, Hk, D, device="cuda")
    k[0, :, 0, 0] = i
    v = torch.as_tensor(rng.standard_normal((1, n, Hk, D)), device="cuda").float()
    v *= torch.exp(-abs(rise) * i + 20).view(1, n, 1, 1)
    q = torch.zeros(1, T, Hk * G, D, device="cuda", dtype=DT[dtype])
    q[..., 0] = 0.3 * D ** 0.5
    q[:, :, 1:, 0] *= 0.5
    both = Both(bsa, rng, 1, 4, Hk, D, 64)
    both.write(k, v, np.array([0]))
    start = np.array([n - T])
    ref, size, logit = C.attn(both.ref, host(q), both.table, start)
    o = bsa.bsa_cache_attn(q, both.cache, both.tab, dev(start), 64)
    check_attn(o, ref, size, logit, n, D, dtype, np.ones((1, T, Hk * G), bool))


@pytest.mark.parametrize("G,T", [(1, 1), (4, 1), (8, 1), (4, 3)])
@pytest.mark.parametrize("D", [64, 128])
def test_attn_long_rows_stay_at_the_outputs_rounding(bsa, D, G, T):
    """131072 tokens on one CTA (more units than CTAs). Beside the output's rounding, which the float32 formula rounded
    once has too: the weights' rounding to float16 (2^-12 on average, independent, so 2^-12 of the result), and what
    sums in the matrix unit lose, up to 2^-23 of them at each step: over 32 steps of a growing sum 2^-20 of it on
    average, a quarter of 32 2^-23, of a sum of the size of the values' zeros."""
    g = torch.Generator(device="cuda").manual_seed(9)
    B, Hk, bs, n = 40, 16, 256, 131072
    P = n // bs
    cache, k_sum = bsa.bsa_cache_alloc(P, Hk, D, bs)
    table = torch.arange(P, device="cuda", dtype=torch.int32)
    k, v = (torch.randn(1, n, Hk, D, generator=g, device="cuda").bfloat16() for _ in "kv")
    bsa.bsa_cache_write(k, v, cache, k_sum, table.view(1, -1), dev([0]), bs)
    kk, vv = bsa.bsa_cache_read(cache, table.view(1, -1), dev([0]), n, bs, dtype=torch.float32)
    q = torch.randn(1, T, Hk * G, D, generator=g, device="cuda").bfloat16()
    o = bsa.bsa_cache_attn(q.expand(B, -1, -1, -1).contiguous(), cache, table.expand(B, -1).contiguous(),
                           dev([n - T] * B), bs)
    total = np.zeros(2)
    for h in range(Hk):
        x = kk[0, :, h].double() @ q[0, T - 1, h * G].double() / D ** 0.5
        p = x.softmax(0)
        ref = p @ vv[0, :, h].double()
        plain = ((kk[0, :, h] @ q[0, T - 1, h * G].float() / D ** 0.5).softmax(0) @ vv[0, :, h]).bfloat16()
        zeros = (p @ vv[0, :, h].double().view(n, -1, 64).abs().amax(-1)).repeat_interleave(64)
        err = lambda y: float((y.double() - ref).norm() / ref.norm())  # noqa: E731
        total += err(o[0, T - 1, h * G]), err(plain) + 2.0 ** -12 + 2.0 ** -20 * float(zeros.norm() / ref.norm())
    assert total[0] <= total[1], total / Hk


@pytest.mark.parametrize("dtype,D,G", [("bf16", 64, 2), ("bf16", 128, 40), ("bf16", 128, 5), ("f32", 128, 1)])
@pytest.mark.parametrize("B", [2800, 4096])
def test_attn_thousands_of_sequences(bsa, dtype, D, G, B):
    """Up to the most sequences that a call takes, some of them empty, against the formula in 64 bits on what is read
    back (its float32 rounding of the values, and the tolerance of the long ragged batch, whose logits stay below 60)."""
    g = torch.Generator(device="cuda").manual_seed(10)
    bs, P, most = 64, 3, 150
    cache, k_sum = bsa.bsa_cache_alloc(B * P, 1, D, bs)
    cache.fill_(0xFF)
    table = torch.randperm(B * P, generator=g, device="cuda").int().view(B, P)
    n = torch.randint(1, most + 1, (B,), generator=g, device="cuda").int()
    k, v = (torch.randn(B, most, 1, D, generator=g, device="cuda").to(DT[dtype]) for _ in "kv")
    zero = torch.zeros_like(n)
    bsa.bsa_cache_write(k, v, cache, k_sum, table, zero, bs, count=n)
    q = torch.randn(B, 1, G, D, generator=g, device="cuda").to(DT[dtype])
    start = n - 1
    start[::7] = -1
    out = torch.full_like(q, 7.0)
    ws = torch.empty(bsa.bsa_cache_attn_workspace_bytes(B, 1, G, 1, D), dtype=torch.uint8, device="cuda")
    o = bsa.bsa_cache_attn(q, cache, table, start, bs, workspace=ws, out=out)
    assert bool((o[::7] == 7).all())
    kk, vv = (x[:, :, 0].double() for x in bsa.bsa_cache_read(cache, table, zero, most, bs, dtype=torch.float32, count=n))
    seen = torch.arange(most, device="cuda") < n[:, None]
    x = torch.einsum("bgd,bnd->bgn", q[:, 0].double(), kk) / D ** 0.5
    w = torch.where(seen[:, None], x, -torch.inf).softmax(-1)
    parts = vv.abs().view(B, most, -1, 64)
    parts = (parts + 2.3 * parts.amax(-1, keepdim=True)).view(B, most, D)
    ref, size = (torch.einsum("bgn,bnd->bgd", w, y) for y in (vv, parts))
    f32 = dtype == "f32"
    tol = (2.0 ** -24 if f32 else 2.0 ** -8) * ref.abs() + (
        (2.0 ** -22 if f32 else 2.0 ** -11) + 2 * ((D + 8) * U + (2.0 ** -21 if f32 else 0)) * 60 + (most / 4 + 64) * U) * size
    live = torch.arange(B, device="cuda") % 7 != 0
    assert bool(((o[:, 0].double() - ref).abs() <= tol)[live].all())
    if B == 2800 and G == 40:
        # A CTA has four tiles of 9216 bytes, 30720 of operands, 44800 of sequences, some 4 KB of static memory and 1 KB
        # reserved: an SM's 228 KB hold one, not two. The work, a tile and four more for a unit that begins, is cut for
        # that many CTAs; its piece for each stands first in the workspace.
        tiles = ((start[live] + 64) // 64 + 4).sum().item()
        sms = torch.cuda.get_device_properties(0).multi_processor_count
        assert ws[:4].view(torch.int32).item() == -(-tiles // sms)


def test_block_topk_past_2_31_elements_of_the_sums(bsa):
    Hk, D, bs, P, topk = 16, 128, 64, 300, 40
    g = torch.Generator(device="cuda").manual_seed(11)
    low = torch.randn(P, Hk, D, generator=g, device="cuda") * bs
    q, start = torch.randn(1, 1, Hk, D, generator=g, device="cuda"), dev([P * bs - 1])
    here = torch.arange(P, device="cuda", dtype=torch.int32)[None]
    want = bsa.bsa_cache_block_topk(q, low, here, start, topk, bs)
    pages = (1 << 20) + P  # of 2048 sums each
    k_sum = torch.zeros(pages, Hk, D, device="cuda")
    k_sum[-P:] = low
    assert torch.equal(bsa.bsa_cache_block_topk(q, k_sum, here + pages - P, start, topk, bs), want)


@pytest.mark.parametrize("B,Hk", [(1, 1), (3, 7)])
def test_block_topk_of_the_longest_rows(bsa, B, Hk):
    """49152 blocks, the most that a call takes: one CTA an SM, clusters of eight."""
    D, bs, P = 64, 64, 49152
    g = torch.Generator(device="cuda").manual_seed(12)
    k_sum = torch.randn(P, Hk, D, generator=g, device="cuda")
    table = torch.stack([torch.randperm(P, generator=g, device="cuda") for _ in range(B)]).int()
    q = torch.randn(B, 1, Hk, D, generator=g, device="cuda")
    start = dev([P * bs - 1, P * bs // 2, 700][:B])
    for topk in (1, 3000, 20000):
        got = bsa.bsa_cache_block_topk(q, k_sum, table, start, topk, bs)
        want, _ = C.block_topk(host(q), host(k_sum), table.cpu().numpy(), start.cpu().numpy(), topk, bs)
        assert np.array_equal(got.cpu().numpy(), want)
