"""cache_append on every byte of the caches (MI355X): page sizes, strides, padding, both caches
in one buffer, graphs."""
import numpy as np
import pytest
import torch

import bit_quantized_gemm_amd as w4
import oracle.request_ref as ref

from block_helpers import DEV, TORCH, bits_of

pytestmark = pytest.mark.gpu


def case(T, H, D, page, pages, dtype="bf16", seed=0):
    g = torch.Generator().manual_seed(seed + T)
    joint = torch.randn(T, 2 * H + 1, D, generator=g).to(TORCH[dtype]).to(DEV)
    caches = torch.randn(2, pages, page, H, D, generator=g).to(TORCH[dtype]).to(DEV)
    slots = torch.randperm(pages * page, generator=g)[:T]
    return joint[:, :H], joint[:, H:2 * H], caches[0], caches[1], slots


@pytest.mark.parametrize("T,H,D,page,pages,dtype", [
    (1, 1, 8, 1, 1, "bf16"), (1, 8, 128, 16, 3, "f16"), (7, 3, 72, 5, 9, "bf16"), (64, 8, 128, 64, 4, "bf16"), (1001, 2, 64, 48, 40, "f16"),
    (4352, 8, 128, 16, 300, "bf16"), (3, 100, 40, 7, 2, "f16"), (2500, 1, 8, 32, 100, "bf16"),
    (140000, 1, 8, 16, 9000, "f16")])
def test_every_byte(T, H, D, page, pages, dtype):
    print(f"case: {T} {H}x{D} page {page} of {pages} {dtype}", flush=True)
    k, v, kc, vc, slots = case(T, H, D, page, pages, dtype)
    slots[T // 2] = -1
    if T > 5:
        slots[1], slots[4], slots[5] = pages * page, 2**40, -2**62        # out of the cache: left out
    want = ref.cache_append_ref(bits_of(k), bits_of(v), bits_of(kc), bits_of(vc), slots.tolist())
    got = w4.cache_append(k, v, kc, vc, slots.to(DEV))
    assert got[0].data_ptr() == kc.data_ptr() and got[1].data_ptr() == vc.data_ptr()
    assert np.array_equal(bits_of(kc), want[0]) and np.array_equal(bits_of(vc), want[1])


def test_caches_in_one_buffer():
    """Pages of keys and values in turn; keys and values side by side in a head; heads before places."""
    for layout in ("pages", "heads", "transposed"):
        k, v, _, _, slots = case(50, 3, 40, 16, 9, seed=3)
        both = torch.randn({"pages": (9, 2, 16, 3, 40), "heads": (9, 16, 3, 80), "transposed": (9, 2, 3, 16, 40)}[layout], device=DEV).bfloat16()
        kc, vc = {"pages": lambda: (both[:, 0], both[:, 1]), "heads": lambda: (both[..., :40], both[..., 40:]),
                  "transposed": lambda: (both[:, 0].transpose(1, 2), both[:, 1].transpose(1, 2))}[layout]()
        want = ref.cache_append_ref(*(bits_of(t) for t in (k, v, kc, vc)), slots.tolist())
        w4.cache_append(k, v, kc, vc, slots.to(DEV))
        assert np.array_equal(bits_of(kc), want[0]) and np.array_equal(bits_of(vc), want[1])


def test_past_32_bits():
    """A cache of more than 2^32 bytes: places on both sides of every such border."""
    H, D, page = 8, 128, 64
    pages = 2**33 // (2 * H * D * page) + 70
    kc = torch.zeros(pages, page, H, D, dtype=torch.float16, device=DEV)
    vc = torch.zeros_like(kc)
    k, v = (torch.randn(6, H, D, device=DEV).half() for _ in range(2))
    border = 2**32 // (2 * H * D)
    at = torch.tensor([0, border - 1, border, 2 * border - 1, 2 * border, pages * page - 1], device=DEV)
    w4.cache_append(k, v, kc, vc, at)
    for cache, new in ((kc, k), (vc, v)):
        flat = cache.view(-1, H, D)
        assert torch.equal(flat[at], new)
        flat[at] = 0
        assert not cache.any()


def test_nothing_to_do():
    k, v, kc, vc, slots = case(4, 2, 16, 4, 3)
    before = bits_of(kc)
    w4.cache_append(k[:0], v[:0], kc, vc, slots[:0].to(DEV))
    w4.cache_append(k, v, kc, vc, torch.full((4,), -1, device=DEV))
    w4.cache_append(k, v, kc[:0], vc[:0], slots.to(DEV))
    assert np.array_equal(bits_of(kc), before)


def test_streams_and_graph():
    k, v, kc, vc, slots = case(200, 4, 64, 16, 20, seed=9)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    want = ref.cache_append_ref(*(bits_of(t) for t in (k, v, kc, vc)), slots.tolist())
    held = slots.to(DEV)
    w4.cache_append(k, v, kc, vc, held, stream=side)
    side.synchronize()
    assert np.array_equal(bits_of(kc), want[0]) and np.array_equal(bits_of(vc), want[1])
    sk, sv = k.clone(), v.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        w4.cache_append(sk, sv, kc, vc, held)
    for i in range(4):
        order = torch.randperm(320, generator=torch.Generator().manual_seed(i))[:200]
        sk.copy_(k * (i + 2))
        sv.copy_(v * (i + 2))
        held.copy_(order)
        want = ref.cache_append_ref(*(bits_of(t) for t in (sk, sv, kc, vc)), order.tolist())
        g.replay()
        torch.cuda.synchronize()
        assert np.array_equal(bits_of(kc), want[0]) and np.array_equal(bits_of(vc), want[1])
