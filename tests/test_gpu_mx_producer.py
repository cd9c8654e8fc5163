"""Parity of quantize_mxfp4_act with the float64 oracle (MI355X): act and
ascales byte for byte, lora_act_in within 4e-3 T + 1 ulp (the acceptance of the
NVFP4 producer's)."""
import numpy as np
import pytest
import torch

import bit_quantized_gemm_amd as w4
import oracle.block_ref as ref
import oracle.w4a4_ref as gref
import synthetic

from block_helpers import DEV, TORCH, bits_of, half_bits, normal_bits, to_dev

pytestmark = pytest.mark.gpu


def activations(rng, M, K, dtype):
    c = np.exp2(rng.uniform(-3, 3, size=K)) * np.where(rng.random(K) < 0.01, 32, 1)
    return half_bits(rng.standard_normal((M, K)) * c, dtype)


def check(x_bits, down_bits, dtype, what):
    down = None if down_bits is None else to_dev(down_bits, dtype)
    act, asc, la = w4.quantize_mxfp4_act(to_dev(x_bits, dtype), down)
    ract, rasc = ref.quantize_mxfp4_ref(x_bits, dtype)
    assert np.array_equal(asc.cpu().numpy(), rasc), (what, "ascales")
    assert np.array_equal(act.cpu().numpy(), ract), (what, "act")
    if down is None:
        assert la is None
        return
    y, T = ref.lora_down_half(x_bits, down_bits, dtype)
    res = gref.check_output(bits_of(la), y, T, dtype)
    print(f"  {what}: max err/bound {res['max_ratio']:.3g}", flush=True)
    assert res["ok"], (what, res)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("M,K,R", [
    (1, 32, 0), (1, 32, 1), (1, 3072, 32), (4, 3072, 32), (15, 96, 16), (16, 128, 17), (17, 160, 33), (33, 1056, 128),
    (100, 4128, 64), (255, 12288, 128), (256, 3072, 0), (1000, 3072, 16), (1001, 2080, 127), (4096, 64, 8),
    (4352, 480, 32), (4200, 4128, 9), (2100, 1056, 100), (4097, 96, 16), (2049, 8224, 31)])
def test_sizes(M, K, R, dtype):
    print(f"case: {M} x {K} R={R} {dtype}", flush=True)
    rng = np.random.default_rng(M * 31 + K + R)
    check(activations(rng, M, K, dtype), normal_bits(rng, (R, K), dtype, 0.02) if R else None, dtype, f"{M}x{K} R{R} {dtype}")


@pytest.mark.parametrize("M,K,R", [(3, 8224, 128), (16, 12288, 33), (12, 96, 127), (128, 4096, 32), (700, 4128, 31),
                                   (512, 3072, 128), (100, 12288, 60), (70, 160, 128), (300, 1056, 97), (129, 8224, 128)])
def test_rank_tiles_apart(M, K, R):
    """Few rows: the tiles of 16 ranks are dealt to workgroups of their own, K in slices or not."""
    print(f"case: {M} x {K} R={R}", flush=True)
    rng = np.random.default_rng(M + K + R)
    check(activations(rng, M, K, "bf16"), normal_bits(rng, (R, K), "bf16", 0.02), "bf16", f"{M}x{K} R{R}")


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_every_pattern(dtype):
    """All 65536 patterns, 32 to a block in order (special blocks among them),
    and each with one large neighbour, which sets the scale."""
    every = np.arange(65536, dtype=np.uint16).reshape(64, 1024)
    check(every, None, dtype, "all patterns")
    finite = np.where(np.isfinite(gref.half_bits_to_f64(every, dtype)), every, 0)
    for top in (0x0001, 0x0400, 0x3C00, 0x4E00):
        x = finite.copy()
        x[:, ::32] = top
        check(x, None, dtype, f"all patterns beside {top:#x}")


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_special_values(dtype):
    rng = np.random.default_rng(3)
    x = normal_bits(rng, (40, 256), dtype)
    inf, nan = (0x7F80, 0x7FC1) if dtype == "bf16" else (0x7C00, 0x7E01)
    x[3, 40], x[5, 255], x[7, 0], x[9, 64:96], x[11, 32:64], x[13] = inf, nan, inf | 0x8000, 0, 0x8000, 1
    act, asc, _ = w4.quantize_mxfp4_act(to_dev(x, dtype))
    ract, rasc = ref.quantize_mxfp4_ref(x, dtype)
    assert np.array_equal(asc.cpu().numpy(), rasc) and np.array_equal(act.cpu().numpy(), ract)
    assert rasc[1, 3] == 255 and rasc[7, 5] == 255 and rasc[0, 7] == 255 and rasc[2, 9] == 0


def test_lora_tail_holds_nan():
    """A NaN in a row of x reaches that row's LoRA input and no other; one in the
    next rank's row of lora_down (memory past a K that ends inside a span) none."""
    rng = np.random.default_rng(4)
    x, d = normal_bits(rng, (20, 160), "bf16"), normal_bits(rng, (3, 160), "bf16")
    x[4, 100] = 0x7FC0
    d[2, 0] = 0x7FC0
    la = w4.quantize_mxfp4_act(to_dev(x, "bf16"), to_dev(d, "bf16"))[2].float().cpu().numpy()
    want = np.zeros((20, 3), bool)
    want[4], want[:, 2] = True, True
    assert np.array_equal(np.isnan(la), want)


@pytest.mark.parametrize("K", [3072, 12288])
def test_given_outputs_guarded_and_repeatable(K):
    """Outputs in the middle of larger buffers: nothing outside them changes, and a
    second call gives the same bytes whatever the workspace held."""
    rng = np.random.default_rng(5)
    M, R = 37, 24
    x, d = to_dev(activations(rng, M, K, "bf16"), "bf16"), to_dev(normal_bits(rng, (R, K), "bf16", 0.02), "bf16")
    assert w4.quantize_mxfp4_workspace(M, 12288, R) > 0       # K in slices there

    def guarded(n):
        t = torch.full((n + 512,), 0xA5, dtype=torch.uint8, device=DEV)
        return t, t[256:256 + n]

    ba, act = guarded(M * K // 2)
    bs, asc = guarded(K // 32 * M)
    bl, la = guarded(M * R * 2)
    out = (act.view(M, K // 2), asc.view(K // 32, M), la.view(torch.bfloat16).view(M, R))
    first = None
    for i in range(3):
        torch.empty(1 << 20, dtype=torch.uint8, device=DEV).fill_(255 * (i % 2))
        w4.quantize_mxfp4_act(x, d, *out)
        got = [t.clone() for t in out]
        for b, n in ((ba, M * K // 2), (bs, K // 32 * M), (bl, M * R * 2)):
            assert (b[:256] == 0xA5).all() and (b[256 + n:] == 0xA5).all()
        assert first is None or all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(first, got))
        first = got


def test_feeds_the_products():
    """x -> codes -> gemm_mxfp4 and gemm_mxfp4_few: both within the oracle's bound of
    the chained references."""
    rng = np.random.default_rng(6)
    M, N, K, R = 48, 200, 512, 32
    x, w = activations(rng, M, K, "bf16"), normal_bits(rng, (N, K), "bf16", 0.05)
    down, up = normal_bits(rng, (R, K), "bf16", 0.02), normal_bits(rng, (R, N), "bf16", 0.1)
    wc, bias = rng.uniform(0.5, 1.5, N).astype(np.float32), rng.standard_normal(N).astype(np.float32)
    act, asc, la = w4.quantize_mxfp4_act(to_dev(x, "bf16"), to_dev(down, "bf16"))
    wgt, wsc, _ = w4.quantize_mxfp4_act(to_dev(w, "bf16"))
    host = [t.cpu().numpy() for t in (act, asc, wgt, wsc)] + [wc, bias, bits_of(la), up]
    y, T = gref.gemm_mxfp4_ref(*host), gref.term_magnitude_mx(*host)
    args = (act, asc, wgt, wsc, torch.from_numpy(wc).to(DEV), torch.from_numpy(bias).to(DEV), la, to_dev(up, "bf16"))
    for fn in (w4.gemm_mxfp4, w4.gemm_mxfp4_few):
        res = gref.check_output(bits_of(fn(*args)), y, T)
        assert res["ok"], (fn.__name__, res)


def test_other_stream_and_graph():
    rng = np.random.default_rng(7)
    x = to_dev(activations(rng, 64, 12288, "f16"), "f16")
    d = to_dev(normal_bits(rng, (100, 12288), "f16", 0.02), "f16")
    want = w4.quantize_mxfp4_act(x, d)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = w4.quantize_mxfp4_act(x, d, stream=side)
    side.synchronize()
    assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(want, got))
    static = x.clone()
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        kept = w4.quantize_mxfp4_act(static, d)
    for i in range(4):
        static.copy_(x * (i + 1))
        g.replay()
        eager = w4.quantize_mxfp4_act(x * (i + 1), d)
        torch.cuda.synchronize()
        assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(kept, eager))
