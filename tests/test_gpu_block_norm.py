"""block_norm against the float64 oracle, on every element (MI355X): widths from 1 on, odd
ones, both norms, every combination of what may be left out, strides and broadcast vectors,
in place, and rows at the ends of the number range."""
import itertools

import numpy as np
import pytest
import torch

import bit_quantized_gemm_amd as w4
import oracle.request_ref as ref

from block_helpers import DEV, TORCH, assert_within, values_of

pytestmark = pytest.mark.gpu
VECTORS = ("gate", "scale", "shift", "weight", "bias", "post_weight")


def tensors(seed, B, L, C, dtype, have, mod="batch", std=1.0):
    g = torch.Generator().manual_seed(seed)

    def normal(*shape, scale=1.0, mean=0.0):
        return (torch.randn(*shape, generator=g) * scale + mean).to(TORCH[dtype]).to(DEV)
    t = dict(x=normal(B, L, C, scale=std, mean=0.25))
    rows = {"batch": (B, 1, C), "token": (B, L, C), "one": (C,)}[mod]
    for name in have:
        t[name] = normal(B, L, C) if name == "y" else \
            normal(*(rows if name in ("gate", "scale", "shift") else (C,)), scale=0.5, mean=0.0 if name in ("bias", "shift", "gate") else 1.0)
    return t


def check(t, what, kind="layer", **kw):
    got, res = w4.block_norm(kind=kind, post_norm="post_weight" in t or kw.pop("post_norm", False), **t, **kw)
    v = {k: values_of(a) for k, a in t.items()}
    dtype = "f16" if t["x"].dtype == torch.float16 else "bf16"
    kw.pop("out", None), kw.pop("residual", None)
    out, r, bo, br = ref.block_norm_ref(**v, layer=kind == "layer", post_norm="post_weight" in t, dtype=dtype, **kw)
    assert_within(values_of(got), out, bo, what)
    if "y" in t:
        assert_within(values_of(res), r, br, what + " residual")
    else:
        assert res is None
    return got, res


@pytest.mark.parametrize("kind", ["layer", "rms"])
@pytest.mark.parametrize("width", [1, 2, 5, 7, 8, 9, 16, 63, 72, 511, 512, 513, 1001, 1024, 1030, 2048, 2056, 3072, 4095, 4096, 4097, 8200, 12288,
                                   16381, 16384])
def test_widths(width, kind):
    """Few rows and many (one wave and four a row)."""
    for B, L, dtype in ((1, 1, "bf16"), (3, 5, "f16"), (2, 520, "bf16")):
        if B * L * width > 6e6:
            continue
        print(f"case: {B}x{L}x{width} {kind} {dtype}", flush=True)
        check(tensors(width, B, L, width, dtype, ("y", "gate", "scale", "shift")), f"{B}x{L}x{width}", kind)
        check(tensors(width, B, L, width, dtype, ("weight",)), f"{B}x{L}x{width} plain", kind)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("have", [h for n in range(7) for h in itertools.combinations(VECTORS, n)],
                         ids=lambda h: "-".join(h) or "none")
def test_what_may_be_left_out(have, dtype):
    for kind, mod, width in (("layer", "token", 203), ("rms", "one", 264)):
        t = tensors(len(have), 2, 9, width, dtype, ("y",) + have, mod)
        check(t, f"{have} {kind}", kind, residual_scale=0.75, eps=1e-5)


@pytest.mark.parametrize("width", [24, 1000, 1001, 5000])
def test_strides_and_slices(width):
    """Rows of wider tensors, gate, scale and shift as slices of one, results into strided tensors."""
    B, L = 3, 37
    g = torch.Generator(device=DEV).manual_seed(width)
    wide = torch.randn(L, B, 2 * width + 3, generator=g, device=DEV).bfloat16()
    x, y = wide[..., 1:1 + width].transpose(0, 1), wide[..., 2 + width:2 + 2 * width].transpose(0, 1)
    scale, gate, shift = torch.randn(B, 1, 3 * width, generator=g, device=DEV).bfloat16().chunk(3, -1)
    outs = torch.full((2, B, L, width + 5), 7.0, dtype=torch.bfloat16, device=DEV)
    out, residual = outs[0, :, :, 3:3 + width], outs[1, :, :, 5:]
    t = dict(x=x, y=y, gate=gate, scale=scale, shift=shift)
    got, res = check(t, f"strided {width}", out=out, residual=residual)
    assert got.data_ptr() == out.data_ptr() and res.data_ptr() == residual.data_ptr()
    out.fill_(7.0)
    residual.fill_(7.0)
    assert (outs == 7.0).all()                             # nothing beside the rows was written
    check({"x": x[0], "y": y[0], "gate": gate[0], "scale": scale[1], "shift": shift[2, 0]}, "two dimensions", "rms")


@pytest.mark.parametrize("width,rows", [(72, 3), (1001, 2000), (3072, 40), (9001, 300), (4, 11)])
def test_in_place(width, rows):
    for res_on, out_on in (("x", "y"), ("y", "x"), ("x", None), (None, "x"), (None, "y")):
        t = tensors(rows, 1, rows, width, "f16", ("y", "gate", "weight"))
        want = w4.block_norm(**t)
        kw = {k: t[on] for k, on in (("residual", res_on), ("out", out_on)) if on}
        got = w4.block_norm(**t, **kw)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        assert all(got[i].data_ptr() == kw[k].data_ptr() for i, k in enumerate(("out", "residual")) if k in kw)
    x = tensors(rows, 1, rows, width, "bf16", ())["x"]
    want = w4.block_norm(x)[0]
    assert torch.equal(w4.block_norm(x, out=x)[0], want) and torch.equal(x, want)


@pytest.mark.parametrize("kind", ["layer", "rms"])
@pytest.mark.parametrize("width", [40, 1024, 3072, 7001])
def test_ends_of_the_range(width, kind):
    """Rows of zeros, of one value, of tiny and of the largest values, and the widest spread."""
    rng = np.random.default_rng(width)
    for dtype, top in (("bf16", 3e38), ("f16", 65504.0)):
        rows = np.stack([np.zeros(width), np.full(width, 1000.0), np.full(width, -0.3), rng.standard_normal(width) * 1e-30,
                         rng.uniform(-1, 1, width) * top, np.where(np.arange(width) % 2 == 0, top, -top), np.full(width, top),
                         np.where(np.arange(width) == width // 2, top, 1.0), rng.standard_normal(width) + 4000.0])
        x = torch.from_numpy(rows).to(TORCH[dtype]).to(DEV)
        for n in (1, 200):
            check({"x": x.repeat(n, 1)}, f"{dtype} {n}", kind)
        check({"x": torch.zeros_like(x), "y": x, "post_weight": x.new_ones(width)}, f"{dtype} after", kind)


def test_infinities_and_nan_stay_in_their_rows():
    for width, rows in ((264, 6), (3072, 1500), (1001, 8)):
        t = tensors(1, 1, rows, width, "bf16", ("y", "gate", "scale", "shift"))
        want = w4.block_norm(**t)
        t["x"][0, 2, width - 1], t["y"][0, 4, 3] = float("inf"), float("nan")
        for kind in ("layer", "rms"):
            got = w4.block_norm(kind=kind, **t)
            assert got[0][0, 4].isnan().all() and not torch.isfinite(got[0][0, 2, width - 1])
            assert got[1][0, 2, width - 1] == float("inf") and got[1][0, 4, 3].isnan() and got[1][0, 4].isnan().sum() == 1
            clean = [i for i in range(rows) if i not in (2, 4)]
            if kind == "layer":
                assert got[0][0, 2].isnan().all()
                assert torch.equal(got[0][0, clean], want[0][0, clean]) and torch.equal(got[1][0, clean], want[1][0, clean])


def test_same_rows_same_bytes():
    """A row's result does not depend on the rows beside it, on repetition, or on a stream."""
    t = tensors(5, 1, 1500, 3072, "bf16", ("y", "gate", "scale", "shift"), "one")
    a = w4.block_norm(**t)
    b = w4.block_norm(**t)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    c = w4.block_norm(**t, stream=side)
    side.synchronize()
    assert all(torch.equal(p, q) and torch.equal(p, r) for p, q, r in zip(a, b, c))


def test_in_a_graph():
    t = tensors(6, 2, 33, 1001, "f16", ("y", "gate", "scale", "shift", "post_weight"))
    held = {k: v.clone() for k, v in t.items()}
    w4.block_norm(post_norm=True, **held)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        kept = w4.block_norm(post_norm=True, residual=held["x"], **held)
    for i in range(4):
        for k in held:
            held[k].copy_(t[k] * (1 + i))
        g.replay()
        eager = w4.block_norm(post_norm=True, **{k: v * (1 + i) for k, v in t.items()})
        torch.cuda.synchronize()
        assert torch.equal(kept[0], eager[0]) and torch.equal(kept[1], eager[1]) and torch.equal(held["x"], eager[1])


def test_more_rows_than_a_launch_dimension():
    """17 million short rows: what each gives does not depend on where it lies."""
    rows, width = 17_000_005, 8
    some = torch.randn(1009, width, device=DEV).bfloat16()
    x = some[torch.arange(rows, device=DEV) % 1009]
    want = w4.block_norm(some, kind="rms")[0]
    got = w4.block_norm(x, kind="rms")[0]
    for at in range(0, rows, 2_000_000):
        n = min(2_000_000, rows - at)
        assert torch.equal(got[at:at + n], want[torch.arange(at, at + n, device=DEV) % 1009])
