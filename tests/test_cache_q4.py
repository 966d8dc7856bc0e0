"""The 4-bit paged cache: records written by attn_cache_store_q4 equal the
oracle's byte by byte, and attn_cache_load_q4 reads them back correctly rounded
(a code times a bf16 scale has at most 11 bits, so one rounding to bf16)."""
import ctypes

import numpy as np
import pytest
import torch

from oracle.serving import bf16_bits, bf16_value, q4_bytes, q4_quantise, q4_row, q4_write
from tests.helpers import check_canaries, guarded_empty


def rows(B, H, S, D, seed=0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(B, H, S, D, generator=g)
    return (x * torch.exp2(torch.randint(-6, 7, (B, H, S, 1), generator=g))).to(torch.bfloat16)


def store(k, v, slots, pages, page, strided=False):
    """The pool (numpy) after a store into one filled with 0xCC bytes."""
    import masked_attention_gb300 as M
    H, D = k.shape[1], k.shape[3]
    pool = guarded_empty((pages, H, q4_bytes(page, D)), torch.uint8)
    pool.fill_(0xCC)
    dk, dv = (x.cuda() for x in (k, v))
    if strided:   # [B, S, H, D] memory
        dk, dv = (x.transpose(1, 2).contiguous().transpose(1, 2) for x in (dk, dv))
    M.attn_cache_store_q4(dk, dv, torch.as_tensor(slots).cuda(), pool, page_size=page)
    check_canaries()
    return pool


def oracle_pool(k, v, slots, pages, page):
    B, H, S, D = k.shape
    pool = np.full((pages, H, q4_bytes(page, D)), 0xCC, np.uint8)
    kn, vn = k.double().numpy(), v.double().numpy()
    for n, slot in enumerate(np.asarray(slots).reshape(-1)):
        if 0 <= slot < pages * page:
            for h in range(H):
                q4_write(pool, int(slot), h, kn[n // S, h, n % S], vn[n // S, h, n % S], page)
    return pool


@pytest.mark.gpu
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("B,H,S", [(1, 1, 1), (3, 2, 5), (1, 3, 131), (17, 1, 1)])
def test_store_and_load(D, page, B, H, S):
    import masked_attention_gb300 as M
    rng = np.random.default_rng(B * S + D)
    pages = -(-B * S // page) + 2
    slots = rng.permutation(pages * page)[:B * S].astype(np.int64).reshape(B, S)
    if B * S > 3:   # places of a padded batch, and one past the pool
        slots.reshape(-1)[[1, -1]] = -1, pages * page
    k, v = rows(B, H, S, D, 1), rows(B, H, S, D, 2)
    for strided in (False, True):
        pool = store(k, v, slots, pages, page, strided)
        assert np.array_equal(pool.cpu().numpy(), oracle_pool(k, v, slots, pages, page))
    out = [guarded_empty((B, S, H, D), torch.bfloat16).transpose(1, 2) for _ in (0, 1)]
    M.attn_cache_load_q4(pool, torch.from_numpy(slots).cuda(), *out, page_size=page)
    check_canaries()
    host = pool.cpu().numpy()
    for n, slot in enumerate(slots.reshape(-1)):
        for h in range(H):
            for got, ref in zip(out, q4_row(host, int(slot), h, page, D)):
                got = got[n // S, h, n % S].float().cpu().numpy().astype(np.float64)
                assert np.array_equal(got, bf16_value(bf16_bits(ref)))


@pytest.mark.gpu
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("B,H,S", [(2, 8, 9), (1, 16, 40), (5, 1, 18), (3, 1, 17), (3, 5, 16),
                                   (40, 2, 3), (33, 1, 2), (2, 17, 6), (70, 4, 1), (1, 1, 700)])
def test_rows_that_fill_batches_and_that_do_not(D, B, H, S):
    """Tokens whose rows take whole batches, fractions of one, and batches that
    begin inside one token or sequence and end in another."""
    test_store_and_load(D, 16, B, H, S)


@pytest.mark.gpu
def test_half_aligned_rows():
    """Rows that start on 16 but not on 32 bytes (slices of an odd projection)."""
    import masked_attention_gb300 as M
    D, page, S = 128, 16, 21
    k, v = rows(1, 2, S, D, 8), rows(1, 2, S, D, 9)
    slots = np.random.default_rng(5).permutation(3 * page)[:S].astype(np.int64)
    ref = oracle_pool(k, v, slots, 3, page)
    for pad in (8, 24):
        dev = []
        for x in (k, v):
            wide = torch.full((1, S, 2, D + 8), 3.0, dtype=torch.bfloat16, device="cuda")
            buf = torch.full((wide.numel() + pad,), 3.0, dtype=torch.bfloat16, device="cuda")
            t = buf[pad:].view(wide.shape)[..., :D].transpose(1, 2)
            t.copy_(x.cuda())
            dev.append((t, buf))
        pool = torch.full(ref.shape, 0xCC, dtype=torch.uint8, device="cuda")
        ds = torch.from_numpy(slots).cuda()
        M.attn_cache_store_q4(dev[0][0], dev[1][0], ds, pool, page_size=page)
        assert np.array_equal(pool.cpu().numpy(), ref)
        plain = [torch.empty(1, 2, S, D, dtype=torch.bfloat16, device="cuda") for _ in (0, 1)]
        M.attn_cache_load_q4(pool, ds, *plain, page_size=page)
        M.attn_cache_load_q4(pool, ds, dev[0][0], dev[1][0], page_size=page)
        for (t, buf), x in zip(dev, plain):
            assert torch.equal(t, x)
            t.fill_(3.0)
            assert (buf == 3.0).all()   # nothing between the rows was touched


@pytest.mark.gpu
def test_values_at_the_edges():
    """Ties, tiny and huge magnitudes, signed zeros, infinities and NaN."""
    D, page = 64, 16
    k = rows(1, 1, 16, D, 3).float()
    k[0, 0, 0] = 0.0                                     # zero group: scale 0
    k[0, 0, 1] = -0.0
    k[0, 0, 2] = torch.arange(D) % 15 - 7.0              # codes themselves: scale 1
    k[0, 0, 3] = (torch.arange(D) % 15 - 7.0) / 2        # ties of scale 1 ...
    k[0, 0, 3, 0] = k[0, 0, 3, 32] = 7.0                 # ... set by one large channel
    k[0, 0, 4] *= 2.0 ** -120                            # scales near the smallest normal
    k[0, 0, 5] = 2.0 ** -133                             # subnormal channels and scale
    k[0, 0, 6] = 2.0 ** -131 * (torch.arange(D) % 7)
    k[0, 0, 7] = 3.3e38 * torch.sign(k[0, 0, 7])
    k[0, 0, 8, 5] = float("inf")
    k[0, 0, 9, 40] = float("nan")
    k[0, 0, 10, 3] = -float("inf")
    k[0, 0, 11, :32] = 1e-30
    k[0, 0, 11, 7] = 3e-30
    k = k.to(torch.bfloat16)
    v = k.flip(2)
    slots = np.arange(16, dtype=np.int64)
    pool = store(k, v, slots, 1, page)
    assert np.array_equal(pool.cpu().numpy(), oracle_pool(k, v, slots, 1, page))
    # and read back: subnormal scales, NaN groups
    import masked_attention_gb300 as M
    out = [torch.empty(1, 1, 16, D, dtype=torch.bfloat16, device="cuda") for _ in (0, 1)]
    M.attn_cache_load_q4(pool, torch.from_numpy(slots).cuda(), *out, page_size=page)
    for row in range(16):
        for got, ref in zip(out, q4_row(pool.cpu().numpy(), row, 0, page, D)):
            got = got[0, 0, row].double().cpu().numpy()
            assert np.array_equal(got, bf16_value(bf16_bits(ref)), equal_nan=True)


@pytest.mark.gpu
def test_every_quotient_near_a_tie():
    """Channels at and next to (c + 1/2) scale for many scales: the codes are
    the exact quotient's, ties to even."""
    scales = [1.0, 1.0078125, 1.3359375, 1.9921875, 0.01171875, 3.0]
    xs = []
    for s in scales:
        ties = (np.arange(-6, 6) + 0.5) * s
        near = bf16_value(bf16_bits(ties))
        step = 2.0 ** (np.floor(np.log2(np.abs(near))) - 7)
        row = np.concatenate([near, near + step, near - step])[:31]
        xs.append(np.concatenate([row, [7 * s]]))
    x = torch.tensor(np.stack(xs), dtype=torch.float32).to(torch.bfloat16).view(1, 1, -1, 64)
    slots = np.arange(x.shape[2], dtype=np.int64)
    assert np.array_equal(store(x, x, slots, 1, 16).cpu().numpy(), oracle_pool(x, x, slots, 1, 16))


@pytest.mark.gpu
def test_offsets_past_32_bits():
    """Records beyond 4 GiB of the pool."""
    import masked_attention_gb300 as M
    D, page, H = 128, 128, 4
    pages = (1 << 32) // (H * q4_bytes(page, D)) + 50
    pool = torch.empty(pages, H, q4_bytes(page, D), dtype=torch.uint8, device="cuda")
    slots = torch.tensor([pages * page - 1, 5, (pages - 20) * page + 3])
    k, v = rows(1, H, 3, D, 4), rows(1, H, 3, D, 5)
    M.attn_cache_store_q4(k.cuda(), v.cuda(), slots.cuda(), pool, page_size=page)
    ko, vo = (torch.empty(1, H, 3, D, dtype=torch.bfloat16, device="cuda") for _ in (0, 1))
    M.attn_cache_load_q4(pool, slots.cuda(), ko, vo, page_size=page)
    for x, o in ((k, ko), (v, vo)):
        n, bits = q4_quantise(x.double().numpy())
        ref = (n.astype(np.float64) - 8) * np.repeat(bf16_value(bits), 32, -1)
        assert np.array_equal(o.double().cpu().numpy(), bf16_value(bf16_bits(ref)))


@pytest.mark.gpu
def test_in_a_graph_on_another_stream():
    import masked_attention_gb300 as M
    D, page = 128, 32
    k, v = rows(2, 2, 20, D, 6), rows(2, 2, 20, D, 7)
    slots = np.random.default_rng(3).permutation(4 * page)[:40].astype(np.int64)
    ref = oracle_pool(k, v, slots, 4, page)
    pool = torch.full(ref.shape, 0xCC, dtype=torch.uint8, device="cuda")
    dk, dv, ds = k.cuda(), v.cuda(), torch.from_numpy(slots).cuda()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        M.attn_cache_store_q4(dk, dv, ds, pool, page_size=page)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        g.replay()
    s.synchronize()
    assert np.array_equal(pool.cpu().numpy(), ref)


def test_oracle_rounding():
    """bf16_bits against torch's rounding; codes of a row written out."""
    x = np.random.default_rng(0).normal(size=4000) * 2.0 ** np.random.default_rng(1).integers(
        -130, 120, 4000)
    x = x.astype(np.float32)
    ref = torch.from_numpy(x).to(torch.bfloat16).view(torch.int16).numpy().view(np.uint16)
    assert np.array_equal(bf16_bits(x.astype(np.float64)), ref)
    row = np.zeros(32)
    row[:5] = 7.0, -7.0, 2.5, 3.5, -0.5
    n, bits = q4_quantise(row[None])
    assert bits[0, 0] == 0x3f80 and n[0, :5].tolist() == [15, 1, 10, 12, 8]


def test_loads_into_broadcast_tensors_are_refused():
    import masked_attention_gb300 as M
    good = ctypes.byref(M.attn_view(0x1000, 4096, 1024, 128))
    for strides in ((0, 1024, 128), (4096, 0, 128), (4096, 1024, 0)):
        bad = ctypes.byref(M.attn_view(0x1000, *strides))
        for k, v in ((good, bad), (bad, good)):
            assert M.lib().attn_cache_load_q4(0x10000, 4, 16, 0x8000, k, v, 2, 2, 3, 128,
                                              None) == M.ATTN_ERR_INVALID_ARG


def test_refusals():
    import masked_attention_gb300 as M
    L = M.lib()

    def view(data=0x1000, strides=(4096, 1024, 128)):
        return ctypes.byref(M.attn_view(data, *strides))

    def both(k=None, v=None, slots=0x8000, pool=0x10000, pages=4, page=16, B=1, H=2, S=3, D=128):
        k, v = k or view(), v or view()
        a = L.attn_cache_store_q4(k, v, slots, pool, pages, page, B, H, S, D, None)
        b = L.attn_cache_load_q4(pool, pages, page, slots, k, v, B, H, S, D, None)
        assert a == b
        return a

    inv, uns, mis = M.ATTN_ERR_INVALID_ARG, M.ATTN_ERR_UNSUPPORTED, M.ATTN_ERR_MISALIGNED
    assert both(D=96) == both(page=8) == both(page=48) == both(page=256) == uns
    assert both(B=-1) == both(H=0) == both(S=-1) == both(pages=0) == inv
    assert both(slots=None) == both(pool=None) == both(k=view(None)) == inv
    assert both(k=view(strides=(0, -8, 8))) == inv
    assert both(k=view(0x1008)) == both(v=view(strides=(0, 1004, 128))) == mis
    assert both(slots=0x8004) == both(pool=0x10008) == mis
    assert both(B=0) == both(S=0) == M.ATTN_OK
    assert M.attn_cache_q4_bytes(10, 4, 64, 128) == 10 * 4 * q4_bytes(64, 128)
    assert M.attn_cache_q4_bytes(10, 4, 24, 128) == M.attn_cache_q4_bytes(0, 4, 16, 64) == 0
    t = torch.zeros(1, 2, 3, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        M.attn_cache_store_q4(t, t, torch.zeros(1, 3, dtype=torch.int64),
                              torch.zeros(1, 2, q4_bytes(16, 64), dtype=torch.uint8), page_size=16)


@pytest.mark.gpu
@pytest.mark.parametrize("B,H,S,D", [(3, 8, 4001, 128), (1, 16, 12007, 64), (2, 40, 1301, 128),
                                     (2, 3, 15001, 128), (7, 1, 25003, 64), (3001, 5, 11, 128),
                                     (3201, 19, 3, 64), (14003, 8, 1, 128), (90001, 2, 1, 64),
                                     (2, 7, 6001, 128)])
def test_warps_with_many_batches(B, H, S, D):
    """Enough tokens that every warp goes through three batches of rows and more, whole
    tokens' and packed ones, over the sequences' ends, with skipped places on its way."""
    import masked_attention_gb300 as M
    page, T = 32, B * S
    pages = T // page + 3
    g = torch.Generator().manual_seed(T)
    k, v = (torch.randn(B, H, S, D, generator=g).to(torch.bfloat16) for _ in (0, 1))
    slots = torch.randperm(pages * page, generator=g)[:T]
    slots[torch.randperm(T, generator=g)[:T // 11]] = -1
    slots[torch.randperm(T, generator=g)[:T // 50]] = pages * page + 4
    there = ((slots >= 0) & (slots < pages * page)).numpy()
    at = slots.numpy()[there]
    ref = np.full((pages, H, q4_bytes(page, D)), 0xCC, np.uint8)
    codes = ref[:, :, :page * D].reshape(pages, H, 2, page, D // 2)
    scales = ref[:, :, page * D:].reshape(pages, H, 2, page, D // 16)
    rows, values = [], []
    for i, x in enumerate((k, v)):
        n, bits = q4_quantise(x.transpose(1, 2).reshape(T, H, D).double().numpy())
        values.append((n.astype(np.float32) - 8) * np.repeat(bf16_value(bits), 32, -1).astype(np.float32))
        codes[at // page, :, i, at % page] = (n[..., 0::2] | (n[..., 1::2] << 4))[there]
        scales[at // page, :, i, at % page] = bits.view(np.uint8).reshape(T, H, D // 16)[there]
    ref[:, :, :page * D] = codes.reshape(pages, H, -1)
    ref[:, :, page * D:] = scales.reshape(pages, H, -1)
    ds = slots.view(B, S).cuda()
    pool = store(k, v, slots.view(B, S), pages, page, strided=B % 2 == 1)
    assert np.array_equal(pool.cpu().numpy(), ref)
    out = [guarded_empty((B, S, H, D), torch.bfloat16).transpose(1, 2) for _ in (0, 1)]
    M.attn_cache_load_q4(pool, ds, *out, page_size=page)
    check_canaries()
    for o, x in zip(out, values):
        x[~there] = 0.0
        assert torch.equal(o.transpose(1, 2).reshape(T, H, D).cpu(), torch.from_numpy(x).to(torch.bfloat16))
