"""What the cache's entry points refuse, on the host before any device work (CPU)."""
import ctypes

import pytest
import torch

A = 0x10000  # an aligned stand-in for a device pointer: never read here


@pytest.fixture(scope="module")
def bsa():
    from conftest import build_library

    build_library()
    import block_sparse_attention_19_b200 as m

    return m


def _ptr(x):
    return ctypes.c_void_p(x)


def _write(bsa, k=A, v=A, cache=A, k_sum=A, table=A, start=A, count=A, B=2, T=3, Hk=2, D=64, bs=64, pages=8, blocks=4,
           dt=1):
    return bsa.lib.bsa_cache_write(*map(_ptr, (k, v, cache, k_sum, table, start, count)), B, T, Hk, D, bs, pages,
                                   blocks, dt, _ptr(0))


def _read(bsa, cache=A, table=A, start=A, count=A, k=A + 0x100, v=A + 0x200, B=2, T=3, Hk=2, D=64, bs=64, pages=8, blocks=4, dt=1):
    return bsa.lib.bsa_cache_read(*map(_ptr, (cache, table, start, count, k, v)), B, T, Hk, D, bs, pages, blocks, dt,
                                  _ptr(0))


def _topk(bsa, q=A, k_sum=A, table=A, start=A, count=A, idx=A, B=2, T=3, H=4, Hk=2, D=64, bs=64, pages=8, blocks=4,
          topk=2, dt=1, flags=0):
    return bsa.lib.bsa_cache_block_topk(*map(_ptr, (q, k_sum, table, start, count, idx)), B, T, H, Hk, D, bs, pages,
                                        blocks, topk, dt, flags, _ptr(0))


def _attn(bsa, q=A, cache=A, table=A, start=A, count=A, idx=A, o=A + 0x100, B=2, T=3, H=4, Hk=2, D=64, bs=64, pages=8,
          blocks=4, topk=2, scale=0.125, dt=1, ws=A + 0x1000, wsb=1 << 30):
    return bsa.lib.bsa_cache_attn(*map(_ptr, (q, cache, table, start, count, idx, o)), B, T, H, Hk, D, bs, pages, blocks,
                                  topk, scale, dt, _ptr(ws), wsb, _ptr(0))


def _forward(bsa, q=A, k=A, v=A, cache=A, k_sum=A, table=A, start=A, count=A, o=A + 0x100, B=2, T=3, H=4, Hk=2, D=64,
             bs=64, pages=8, blocks=4, topk=2, dt=1, flags=0, ws=A + 0x1000, wsb=1 << 30):
    return bsa.lib.bsa_cache_forward(*map(_ptr, (q, k, v, cache, k_sum, table, start, count, o)), B, T, H, Hk, D, bs,
                                     pages, blocks, topk, dt, flags, _ptr(ws), wsb, _ptr(0))


CALLS = dict(write=_write, read=_read, topk=_topk, attn=_attn, forward=_forward)
COMMON = [
    (dict(table=0), 1), (dict(start=0), 1), (dict(table=A + 2), 3), (dict(start=A + 1), 3), (dict(count=A + 3), 3),
    (dict(B=0), 1), (dict(T=0), 1), (dict(T=-1), 1), (dict(Hk=0), 1), (dict(D=96), 2), (dict(D=32), 2),
    (dict(bs=32), 2), (dict(bs=100), 2), (dict(pages=0), 1), (dict(blocks=0), 1), (dict(blocks=1 << 25), 2),
    (dict(dt=2), 2), (dict(dt=9), 2), (dict(B=1 << 25), 2), (dict(T=1 << 29, B=1 << 3), 2),
]


@pytest.mark.parametrize("call", CALLS)
@pytest.mark.parametrize("kw,status", COMMON)
def test_common_refusals(bsa, call, kw, status):
    assert CALLS[call](bsa, **kw) == status
    assert bsa.lib.bsa_last_error_detail() != b""


@pytest.mark.parametrize("call,kw,status", [
    ("write", dict(k=0), 1), ("write", dict(v=A + 8), 3), ("write", dict(cache=0), 1), ("write", dict(k_sum=A + 4), 3),
    ("read", dict(cache=A + 8), 3), ("read", dict(k=0), 1), ("read", dict(v=A + 8), 3),
    ("read", dict(k=A), 1), ("read", dict(v=A), 1), ("read", dict(k=A + 0x200), 1),
    ("topk", dict(q=0), 1), ("topk", dict(idx=0), 1), ("topk", dict(idx=A + 2), 3), ("topk", dict(topk=0), 1),
    ("topk", dict(H=3), 1), ("topk", dict(flags=4), 2), ("topk", dict(flags=2), 1), ("topk", dict(flags=8), 1),
    ("topk", dict(flags=0x100), 2), ("topk", dict(blocks=49153), 2),
    ("attn", dict(q=0), 1), ("attn", dict(o=A), 1), ("attn", dict(o=A + 8), 3), ("attn", dict(topk=0), 1),
    ("attn", dict(scale=0.0), 1), ("attn", dict(scale=float("nan")), 1), ("attn", dict(scale=float("inf")), 1),
    ("attn", dict(H=5), 1), ("attn", dict(ws=0), 4), ("attn", dict(wsb=8), 4), ("attn", dict(ws=A + 8), 3),
    ("attn", dict(idx=A + 1), 3), ("attn", dict(B=4097), 2), ("forward", dict(B=4097), 2),
    ("forward", dict(q=0), 1), ("forward", dict(k=0), 1), ("forward", dict(o=A), 1), ("forward", dict(topk=-1), 1),
    ("forward", dict(flags=4), 2), ("forward", dict(flags=2), 1), ("forward", dict(ws=0), 4),
    ("forward", dict(wsb=64), 4), ("forward", dict(ws=A + 16), 3), ("forward", dict(blocks=49153), 2),
    ("forward", dict(H=5), 1),
])
def test_own_refusals(bsa, call, kw, status):
    assert CALLS[call](bsa, **kw) == status


def test_sizes(bsa):
    assert bsa.bsa_cache_bytes(10, 2, 128, 256) == 10 * 2 * 4 * 72 * 128
    assert bsa.bsa_cache_bytes(1 << 20, 16, 128, 256) == (1 << 20) * 16 * 4 * 72 * 128  # past 32 bits
    for bad in ((0, 2, 128, 64), (1, 0, 128, 64), (1, 1, 96, 64), (1, 1, 64, 96)):
        assert bsa.bsa_cache_bytes(*bad) == 0
    attn = bsa.bsa_cache_attn_workspace_bytes(2, 1, 8, 2, 128)
    assert attn > 0 and bsa.bsa_cache_attn_workspace_bytes(2, 1, 8, 3, 128) == 0
    a = lambda x: (x + 255) // 256 * 256  # noqa: E731
    assert bsa.bsa_cache_forward_workspace_bytes(2, 1, 8, 2, 128, 7) == a(2 * 2 * 7 * 4) + a(attn)
    assert bsa.bsa_cache_forward_workspace_bytes(2, 1, 8, 2, 128, 0) == a(attn)
    assert bsa.bsa_cache_forward_workspace_bytes(2, 1, 8, 2, 128, -1) == 0


def test_binding_refuses_before_the_device(bsa):
    """Shapes and types that do not fit each other would let a kernel read past a
    buffer: the binding refuses them before the device check."""
    B, T, H, Hk, D, bs = 2, 3, 4, 2, 64, 128
    q = torch.zeros(B, T, H, D, dtype=torch.bfloat16)
    k = torch.zeros(B, T, Hk, D, dtype=torch.bfloat16)
    cache, k_sum = bsa.bsa_cache_alloc(8, Hk, D, bs, device="cpu")
    table, start = torch.zeros(B, 4, dtype=torch.int32), torch.zeros(B, dtype=torch.int32)
    idx = torch.zeros(B, Hk, 2, dtype=torch.int32)
    bad = [
        lambda: bsa.bsa_cache_write(k, k[:, :2], cache, k_sum, table, start, bs),
        lambda: bsa.bsa_cache_write(k, k.float(), cache, k_sum, table, start, bs),
        lambda: bsa.bsa_cache_write(k, k, cache, k_sum, table, start, 64),                    # another block size
        lambda: bsa.bsa_cache_write(k, k, cache, k_sum[:4], table, start, bs),                # fewer sums than pages
        lambda: bsa.bsa_cache_write(k, k, cache.float(), k_sum, table, start, bs),
        lambda: bsa.bsa_cache_write(k, k, cache, k_sum.double(), table, start, bs),
        lambda: bsa.bsa_cache_write(k, k, cache, k_sum, table[:1], start, bs),
        lambda: bsa.bsa_cache_write(k, k, cache, k_sum, table.long(), start, bs),
        lambda: bsa.bsa_cache_write(k, k, cache, k_sum, table, start[:1], bs),
        lambda: bsa.bsa_cache_write(k, k, cache, k_sum, table, start, bs, count=start.long()),
        lambda: bsa.bsa_cache_write(k[..., :32], k[..., :32], cache, k_sum, table, start, bs),
        lambda: bsa.bsa_cache_read(cache, table, start, T, bs, k_out=q),
        lambda: bsa.bsa_cache_read(cache, table, start, T, bs, k_out=k, v_out=k.float()),
        lambda: bsa.bsa_cache_read(cache[..., :100], table, start, T, bs),
        lambda: bsa.bsa_cache_block_topk(q[..., :32], k_sum, table, start, 2, bs),
        lambda: bsa.bsa_cache_block_topk(q[:, :, :3], k_sum, table, start, 2, bs),
        lambda: bsa.bsa_cache_block_topk(q, k_sum, table, start, 2, bs, idx_out=idx[..., :1]),
        lambda: bsa.bsa_cache_block_topk(q, k_sum, table, start, 2, bs, idx_out=idx.long()),
        lambda: bsa.bsa_cache_attn(q, cache, table, start, bs, idx=idx[:1]),
        lambda: bsa.bsa_cache_attn(q, cache, table, start, bs, idx=idx.long()),
        lambda: bsa.bsa_cache_attn(q, cache, table, start, bs, out=q.float()),
        lambda: bsa.bsa_cache_attn(q, cache, table, start, 64),
        lambda: bsa.bsa_cache_forward(q, k, k, cache, k_sum, table, start, 64),
        lambda: bsa.bsa_cache_forward(q[:, :2], k, k, cache, k_sum, table, start, bs),
        lambda: bsa.bsa_cache_forward(q.float(), k, k, cache, k_sum, table, start, bs),
    ]
    for i, f in enumerate(bad):
        with pytest.raises((ValueError, TypeError)) as e:
            f()
        assert "CUDA tensor" not in str(e.value), (i, str(e.value))
    for f in (lambda: bsa.bsa_cache_write(k, k, cache, k_sum, table, start, bs),
              lambda: bsa.bsa_cache_read(cache, table, start, T, bs),
              lambda: bsa.bsa_cache_block_topk(q, k_sum, table, start, 2, bs),
              lambda: bsa.bsa_cache_attn(q, cache, table, start, bs, idx=idx),
              lambda: bsa.bsa_cache_forward(q, k, k, cache, k_sum, table, start, bs, 2)):
        with pytest.raises(ValueError, match="CUDA tensor"):
            f()
    with pytest.raises(ValueError):
        bsa.bsa_cache_alloc(8, 2, 96, 64, device="cpu")


@pytest.mark.parametrize("shape", [(2, 2, 0), (2, 0), ()])
def test_binding_refuses_an_empty_selection(bsa, shape):
    """idx without a block is not "all blocks", although its pointer is null."""
    q = torch.zeros(2, 1, 4, 64, dtype=torch.bfloat16)
    cache, _ = bsa.bsa_cache_alloc(8, 2, 64, 64, device="cpu")
    table, start = torch.zeros(2, 4, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="idx"):
        bsa.bsa_cache_attn(q, cache, table, start, 64, idx=torch.zeros(shape, dtype=torch.int32))


@pytest.mark.parametrize("shape", [(), (2,), (2, 4, 1)])
def test_binding_refuses_page_tables_of_other_dimensions(bsa, shape):
    x = torch.zeros(2, 1, 2, 64, dtype=torch.bfloat16)
    cache, k_sum = bsa.bsa_cache_alloc(8, 2, 64, 64, device="cpu")
    table, start = torch.zeros(shape, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    for call in (lambda: bsa.bsa_cache_write(x, x, cache, k_sum, table, start, 64),
                 lambda: bsa.bsa_cache_read(cache, table, start, 1, 64),
                 lambda: bsa.bsa_cache_block_topk(x, k_sum, table, start, 1, 64),
                 lambda: bsa.bsa_cache_attn(x, cache, table, start, 64),
                 lambda: bsa.bsa_cache_forward(x, x, x, cache, k_sum, table, start, 64)):
        with pytest.raises(ValueError, match="page_table"):
            call()


def test_workspace_sizes_belong_to_a_device(bsa, monkeypatch):
    """A size that was asked for on one device is not given for another with more SMs."""
    sms, current = {0: 100, 1: 148}, [0]

    class Device:
        def __init__(self, dev):
            self.dev = dev

        def __enter__(self):
            self.before, current[0] = current[0], self.dev

        def __exit__(self, *_):
            current[0] = self.before

    class Lib:
        @staticmethod
        def bsa_cache_attn_workspace_bytes(*sizes):
            return sms[current[0]] * sum(sizes)

        @staticmethod
        def bsa_cache_forward_workspace_bytes(*sizes):
            return sms[current[0]] * sum(sizes) + 1

    monkeypatch.setattr(torch.cuda, "device", Device)
    for name, sizes in (("bsa_cache_attn_workspace_bytes", (2, 1, 4, 2, 64)),
                        ("bsa_cache_forward_workspace_bytes", (2, 1, 4, 2, 64, 3))):
        assert bsa._workspace_bytes(0, name, *sizes) == getattr(bsa, name)(*sizes) > 0
    monkeypatch.setattr(bsa, "lib", Lib)
    for dev in (0, 1, 0):
        current[0] = dev
        assert bsa.bsa_cache_attn_workspace_bytes(1, 1, 4, 2, 64) == 72 * sms[dev]
        assert bsa.bsa_cache_forward_workspace_bytes(1, 1, 4, 2, 64, 3) == 75 * sms[dev] + 1
    current[0] = 0
    for dev in (0, 1, 0):  # what the calls allocate: the tensors' device counts, not the current one
        assert bsa._workspace_bytes(dev, "bsa_cache_attn_workspace_bytes", 1, 1, 4, 2, 64) == 72 * sms[dev]


@pytest.mark.parametrize("scale,status", [(3e38, 1), (-0.125, 1)])
def test_attention_refuses_scales_that_leave_float32(bsa, scale, status):
    assert _attn(bsa, scale=scale) == status
